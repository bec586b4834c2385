"""Whether tensors of rows, or of heads of tokens, share memory: the host's rule, compiled
by itself, against the bytes."""
import random
import subprocess

import pytest

from deepseek_sparse_attention_gb300 import build as dsa_build

SOURCE = r"""
#include <cstdio>
#include <initializer_list>
#include "extents.h"

int main() {
    char kind;
    long a[6] = {}, b[6] = {};
    while (scanf(" %c", &kind) == 1) {
        for (long* t : {a, b})
            for (int i = 0; i < 6; ++i)
                if (scanf("%ld", t + i) != 1) return 1;
        auto p = [](long at) { return reinterpret_cast<const void*>(at); };
        if (kind == 'r')
            printf("%d\n", (int)dsa::rows_meet(dsa::make_rows(p(a[0]), a[1], a[2], a[3]), dsa::make_rows(p(b[0]), b[1], b[2], b[3])));
        else
            printf("%d\n", (int)dsa::heads_meet(dsa::make_heads(p(a[0]), a[1], a[2], a[3], a[4], a[5]),
                                                dsa::make_heads(p(b[0]), b[1], b[2], b[3], b[4], b[5])));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("extents")
    (d / "meet.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", dsa_build.CSRC, "-o", str(d / "meet"),
                    str(d / "meet.cpp")], check=True, capture_output=True)

    def run(cases):
        text = "\n".join(f"{k} " + " ".join(str(x) for t in (a, b) for x in list(t) + [0] * (6 - len(t))) for k, a, b in cases)
        out = subprocess.run([str(d / "meet")], input=text, text=True, check=True, capture_output=True).stdout.split()
        assert len(out) == len(cases)
        return [x == "1" for x in out]

    return run


def _row_bytes(at, n, stride, width):
    return {at + i * stride + j for i in range(n) for j in range(width)}


def test_rows_meet_where_their_bytes_do(meet):
    rng = random.Random(1)
    cases = []
    for _ in range(20000):
        width = [rng.choice([1, 2, 3, 5, 8]) for _ in range(2)]
        stride = [w + rng.choice([0, 1, 2, 7, rng.randrange(40)]) for w in width]
        if rng.random() < 0.3:
            stride[1] = max(stride[0], width[1])
        n = [rng.choice([1, 2, 3, 10, 25]) for _ in range(2)]
        at = [1000, 1000 + rng.randrange(-300, 300)]
        cases.append(("r", *[(at[i], n[i], stride[i], width[i]) for i in range(2)]))
    want = [bool(_row_bytes(*a) & _row_bytes(*b)) for _, a, b in cases]
    assert meet(cases) == want and 2000 < sum(want) < 18000


def test_rows_of_large_tensors(meet):
    """Counts and strides of a real call's, and past any memory's."""
    n, base = 1 << 31, 1 << 40
    cases = [("r", (base, n, 4096, 2048), (base + 2048, n, 4096, 2048)),       # columns beside each other
             ("r", (base, n, 4096, 2049), (base + 2048, n, 4096, 2048)),
             ("r", (base, n, 4096, 2048), (base + 4096 * n, n, 4096, 4096)),     # behind it
             ("r", (base, n, 4096, 2048), (base + 4096 * (n - 1) + 2047, n, 4096, 4096)),
             ("r", (base, n, 4096, 8), (base + 16, n, 6144, 8)),                 # 0 mod 2048 and 16 mod 2048
             ("r", (base, n, 4096, 8), (base + 16, n, 6145, 8)),                 # sooner or later
             ("r", (base, n, 1 << 62, 8), (base + 16, n, 4096, 8))]
    assert meet(cases) == [False, True, False, True, False, True, True]


def _head_bytes(at, tok, n_tok, head, heads, width):
    return {at + t * tok + h * head + j for t in range(n_tok) for h in range(heads) for j in range(width)}


def test_heads_meet_where_their_bytes_do(meet):
    """Exact for the same strides, and for others whose whole spans are apart; never apart where bytes meet."""
    rng = random.Random(2)
    cases = []
    for _ in range(20000):
        width, heads, n_tok = rng.choice([2, 4, 8]), rng.choice([1, 2, 5]), rng.choice([1, 2, 7])
        layouts = []
        for _ in range(2):
            head = width + rng.choice([0, 1, 8, 16, 24])
            tok = (heads - 1) * head + width + rng.choice([0, 3, 40, 100])
            if rng.random() < 0.2:                            # heads before tokens
                tok, head = width + rng.choice([0, 8]), (n_tok - 1) * (width + 8) + width + rng.choice([0, 40])
            layouts.append((tok, head))
        if rng.random() < 0.5:
            layouts[1] = layouts[0]
        if rng.random() < 0.1:                                # tokens, or heads, that share their input
            layouts[0] = rng.choice([(0, layouts[0][1]), (layouts[0][0], 0)])
        at = [1000, 1000 + rng.randrange(-400, 400)]
        cases.append(("h", *[(at[i], layouts[i][0], n_tok, layouts[i][1], heads, width) for i in range(2)]))
    alike = 0
    for (_, a, b), got in zip(cases, meet(cases)):
        want = bool(_head_bytes(*a) & _head_bytes(*b))
        same = (a[1] == b[1] or a[2] == 1) and (a[3] == b[3] or a[4] == 1)
        alike += same
        assert got == want if same else got or not want
    assert alike > 5000


def test_heads_apart_in_one_tensor(meet):
    """Columns of each head, and a part of the row behind the heads with strides of its own."""
    x = (4096, 64 * 256 * 2 + 8192, 4000, 512, 64, 128)
    cases = [("h", x, (4096 + 128, *x[1:])), ("h", x, (4096 + 64 * 512, x[1], 4000, 128, 64, 128)),
             ("h", x, (4096 + 64, *x[1:])), ("h", x, (4096 + x[1], *x[1:]))]
    assert meet(cases) == [False, False, True, True]
