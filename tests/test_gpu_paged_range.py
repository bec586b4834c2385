"""GPU tests of the paged attention over the whole range of its values."""
import numpy as np
import pytest
import torch

import paged_util as ref
from test_gpu_paged import SCALE, TDT, AttnCase, _lib  # noqa: F401 (_lib: the module's fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ a sink over a flat tail

def sink_case(n_q, kv, dense, fmt, at_end):
    """Row 0 has no value and a logit 17 (head 0) to 20 (head 63) above those of
    all other rows, which are equal; pages of one scale."""
    c = AttnCase(41, [kv], [n_q], fmt=fmt, dense=dense, top_k=2048)
    c.scales[:, 0], c.scales[:, 1] = 120, 127
    c.codes[:, :, 512:] = 0
    p = int(c.table[0, 0])
    c.codes[p, 0, :512] = 0
    c.codes[p, 0, 512] = 0x38 if fmt == "e4m3" else 1          # 1.0
    q = torch.zeros(n_q, 64, 576)
    q[:, :, 512] = torch.linspace(17, 20, 64) / SCALE
    c.q_abs = q.to(TDT["bf16"])
    for i in range(n_q):
        c.idx[i, 0] = 0
        if at_end:
            c.idx[i, :c.n_sel[i]] = np.roll(c.idx[i, :c.n_sel[i]], -1)
    return c


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
@pytest.mark.parametrize("n_q,kv,dense,at_end", [(160, 2300, False, False), (160, 2300, False, True),
                                                 (70, 2300, False, False), (160, 9000, True, False),
                                                 (2, 9000, True, False)])
def test_rows_far_below_a_sink_without_value_make_the_output(n_q, kv, dense, at_end, fmt):
    c = sink_case(n_q, kv, dense, fmt, at_end)
    out, lse, code = c.call()
    assert code == 0
    for i in (0, n_q - 1):
        (o, l, *_), _ = c.expect(i)
        # A weight is a multiple of f16's 2^-24 where the sink's is at least 2^12: off by up to
        # 2^-37 of the sink's, which is e^17..e^20 of its own -- the same for all of the equal
        # rows, so that much of the output -- beside what float32 leaves.
        tol = 2.0 ** -37 * np.exp(c.q_abs[i, :, 512].double().numpy() * SCALE) + 1e-5
        err = np.sqrt(((out[i] - o) ** 2).sum(1) / (o ** 2).sum(1))
        assert np.all(err <= tol), (i, (err / tol).max())
        assert np.allclose(lse[i], l, rtol=1e-6, atol=0)
