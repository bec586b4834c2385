"""The rule that finds a tile's sequence from its slot, and the check of every sequence's offsets:
the kernels' own functions, compiled for the host and compared with the offsets themselves."""
import random
import subprocess

import pytest

from deepseek_sparse_attention_gb300 import build as dsa_build

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "expanded_mla.cuh"

// Batches from stdin: n_seq n_q max_q max_kv rows bq, q_off, row_off.  For each a line of
// "sequence:first query:queries:first row:rows the first sees" of every slot with a tile, then
// the sequences refused, and whether the ends are.
int main() {
    long n_seq, n_q, max_q, max_kv, rows, bq;
    while (scanf("%ld %ld %ld %ld %ld %ld", &n_seq, &n_q, &max_q, &max_kv, &rows, &bq) == 6) {
        std::vector<int64_t> q(n_seq + 1), r(n_seq + 1);
        for (auto* v : {&q, &r})
            for (auto& x : *v) {
                long y;
                if (scanf("%ld", &y) != 1) return 1;
                x = y;
            }
        dsa::BatchDev b{};
        b.row_off = r.data(); b.q_off = q.data();
        b.n_seq = (int32_t)n_seq; b.n_q = (int32_t)n_q; b.max_q_len = (int32_t)max_q;
        b.max_kv_len = max_kv; b.total_rows = rows;
        for (int64_t slot = 0; slot < dsa::expanded_slots(n_q, n_seq, (int)bq); ++slot) {
            dsa::ExpandedTile t;
            if (dsa::expanded_tile(b, slot, 0, 1, (int)bq, 32, t))
                printf("%ld:%d:%ld:%ld ", (long)t.q0, t.n_q, (long)t.row0, (long)t.first);
        }
        printf("|");
        for (int32_t s = 0; s < n_seq; ++s)
            if (!dsa::expanded_sound(b, s)) printf("%d ", s);
        printf("|%d\n", (int)dsa::expanded_ends_sound(b));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("slots")
    (d / "slots.cu").write_text(SOURCE)
    subprocess.run([dsa_build._nvcc()] + dsa_build.ARCH + ["-std=c++17", "--expt-relaxed-constexpr", "-I", dsa_build.INCLUDE,
                   "-I", dsa_build.CSRC, "-o", str(d / "slots"), str(d / "slots.cu")], check=True, capture_output=True)

    def run(batches):
        text = "\n".join(" ".join(map(str, list(head) + list(q) + list(r))) for head, q, r in batches)
        out = subprocess.run([str(d / "slots")], input=text, text=True, check=True, capture_output=True).stdout
        result = []
        for line in out.splitlines():
            tiles, bad, ends = line.split("|")
            result.append(([tuple(map(int, t.split(":"))) for t in tiles.split()], list(map(int, bad.split())), ends == "1"))
        assert len(result) == len(batches)
        return result

    return run


def _prefix(lengths):
    off = [0]
    for x in lengths:
        off.append(off[-1] + x)
    return off


@pytest.mark.parametrize("bq", [16, 32, 64, 256])
def test_every_tile_has_its_slot(program, bq):
    """Batches with idle sequences: each sequence's tiles once, and nothing refused."""
    rng = random.Random(bq)
    batches, want = [], []
    for _ in range(300):
        n = rng.choice([1, 2, 7, 60])
        q = [rng.choice([0, 0, 1, bq - 1, bq, bq + 1, rng.randrange(3 * bq)]) for _ in range(n)]
        if sum(q) == 0:
            q[rng.randrange(n)] = 1
        kv = [x + rng.choice([0, 0, 1, 500]) for x in q]
        q_off, r_off = _prefix(q), _prefix(kv)
        batches.append(((n, sum(q), max(q), max(kv), sum(kv), bq), q_off, r_off))
        want.append(sorted((q_off[s] + t, min(bq, x - t), r_off[s], kv[s] - x + 1 + t)
                           for s, x in enumerate(q) for t in range(0, x, bq)))
    for (tiles, bad, ends), w in zip(program(batches), want):
        assert sorted(tiles) == w and bad == [] and ends


def test_broken_sequences_are_refused_wherever_they_stand(program):
    """A sequence is sound if its queries lie in the batch, its rows in the cache, and both within
    the bounds; no slot gives a tile of another."""
    rng = random.Random(5)
    batches = []
    for _ in range(500):
        n = rng.choice([1, 2, 3, 9])
        q_off, r_off = _prefix([rng.choice([0, 1, 5, 40]) for _ in range(n)]), _prefix([rng.randrange(40, 90) for _ in range(n)])
        n_q, rows = max(q_off[-1], 1), r_off[-1]
        for off in (q_off, r_off):
            if rng.random() < 0.6:
                off[rng.randrange(n + 1)] = rng.choice([-3, 0, 1, 17, n_q, n_q + 1, rows, rows + 1, 1 << 40, -(1 << 40)])
        batches.append(((n, n_q, min(n_q, 40), 89, rows, rng.choice([16, 64])), q_off, r_off))
    refused = 0
    for ((n, n_q, max_q, max_kv, rows, bq), q, r), (tiles, bad, ends) in zip(batches, program(batches)):
        sound = [s for s in range(n) if 0 <= q[s] <= q[s + 1] <= n_q and q[s + 1] - q[s] <= max_q and r[s] >= 0 and
                 r[s + 1] <= rows and q[s + 1] - q[s] <= r[s + 1] - r[s] <= max_kv]
        assert bad == [s for s in range(n) if s not in sound]
        assert ends == (q[0] == 0 and q[n] == n_q)
        for q0, m, row0, first in tiles:
            assert any(r[s] == row0 and q[s] <= q0 and q0 + m <= q[s + 1] and
                       first == r[s + 1] - r[s] - (q[s + 1] - q[s]) + 1 + q0 - q[s] for s in sound)
        refused += bool(bad)
    assert 100 < refused < 500


def test_a_sequence_that_runs_backwards(program):
    """The ends in order, the search past it: refused all the same."""
    heads = (3, 20, 20, 50, 150, 16)
    (_, bad, ends), = program([(heads, [0, 20, 0, 20], [0, 50, 100, 150])])
    assert bad == [1] and ends
