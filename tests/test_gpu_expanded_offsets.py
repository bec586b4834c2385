"""The expanded attention under offsets that break the batch's bounds, and what it leaves alone."""
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_gpu_expanded import HEADS, SCALE, T, check, make_inputs

pytestmark = pytest.mark.gpu
FILL = 77.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _attend(row_off, q_off, n_q, rows, dtype, max_q, max_kv, seed=6):
    """Output, lse and error code; outputs filled, and the workspace holding an earlier call's partial
    sums of queries that all see something."""
    x = make_inputs([n_q], [rows], 192, 64, 256, dtype, seed=seed)
    sh = dsa.make_shape(rope_dim=64, dtype=dtype, scale=SCALE)
    off = [torch.tensor(o, dtype=torch.int64, device="cuda") for o in (row_off, q_off)]
    b = dsa.make_batch(off[0], off[0], off[1], n_q, max_q, max_kv, rows, rows)
    ws = dsa.alloc_workspace(sh, b, dsa.OP_EXPANDED_MLA)
    ws[256:].view(torch.float32).fill_(1.0)
    out = torch.full((n_q, HEADS, 256), FILL, dtype=T[dtype], device="cuda")
    lse = torch.full((n_q, HEADS), FILL, device="cuda")
    dsa.dsa_expanded_mla_attn(sh, b, *x, out, lse, ws)
    code = dsa.dsa_check_device_error(ws)
    return x, out, lse, code, dsa.dsa_plan(sh, b, dsa.OP_EXPANDED_MLA)["attn_splits"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("row_off,q_off,n_q", [
    ([0, 50, 100, 150], [0, 20, 0, 20], 20),           # a sequence backwards, the ends in order
    ([0, 300, 600, 900], [0, 300, 0, 300], 300),
    ([0, 50, 100, 150, 200], [0, 10, 30, 20, 20], 20),
    ([0, 50, 40, 100], [0, 0, 0, 20], 20),             # idle sequences whose rows end before they begin,
    ([0, 5000, 40, 100], [0, 0, 0, 20], 20),           # lie outside the cache,
    ([0, 10, 900, 950], [0, 0, 0, 20], 20),            # are more than the bound,
    ([0, 50, 100, 90], [0, 0, 20, 20], 20),
])
def test_broken_offsets_of_any_sequence_are_recorded(row_off, q_off, n_q, dtype):
    max_kv = 300 if n_q == 300 else 100
    assert _attend(row_off, q_off, n_q, 1000, dtype, n_q, max_kv)[3] == 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seq,q_lens", [(5000, {4999: 20}), (5000, {}), (700, {3: 5, 600: 15})])
def test_one_broken_idle_sequence_among_many(n_seq, q_lens, dtype):
    """Wherever it stands; without it the same batch is in order."""
    q_lens = q_lens or {i: 1 for i in range(0, 5000, 250)}
    q_off, row_off = [0], [0]
    for s in range(n_seq):
        q_off.append(q_off[-1] + q_lens.get(s, 0))
        row_off.append(row_off[-1] + q_lens.get(s, 0))
    n_q = q_off[-1]
    assert _attend(row_off, q_off, n_q, 100, dtype, n_q, 100)[3] == 0
    for s in (0, 1, 255, 256, 640, n_seq - 2):
        if s in q_lens or s + 1 in q_lens:
            continue
        bad = list(row_off)
        bad[s + 1] = 101                               # outside the cache
        assert _attend(bad, q_off, n_q, 100, dtype, n_q, 100)[3] == 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("row_off,q_off,served", [
    ([0, 50, 5000], [0, 10, 20], [(0, 10, 0, 50)]),
    ([0, 50, 40], [0, 10, 20], [(0, 10, 0, 50)]),
    ([0, 5, 100], [0, 10, 20], [(10, 20, 5, 100)]),
    ([0, 50, 100], [0, 10, 19], [(0, 10, 0, 50), (10, 19, 50, 100)]),
    ([0, 50, 100], [4, 10, 20], [(4, 10, 0, 50), (10, 20, 50, 100)]),
])
def test_queries_that_are_skipped_keep_their_outputs(row_off, q_off, served, dtype):
    """Those of refused sequences and of none: not written, split or not."""
    x, out, lse, code, splits = _attend(row_off, q_off, 20, 100, dtype, 20, 100)
    assert code == 2 and (splits > 1) == (dtype == "f32")
    kept = torch.ones(20, dtype=torch.bool, device="cuda")
    for q0, q1, r0, r1 in served:
        kept[q0:q1] = False
        q, k, cache, v = x
        check([q1 - q0], [r1 - r0], q[q0:q1], k[r0:r1], cache[r0:r1], v[r0:r1], out[q0:q1], lse[q0:q1])
    assert kept.any() and (out[kept] == FILL).all() and (lse[kept] == FILL).all()
