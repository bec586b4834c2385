"""The norm and the rope refuse outputs that share elements with the call's other tensors.  CPU only:
every refusal comes before anything is enqueued."""
import ctypes

import pytest

import deepseek_sparse_attention_gb300 as dsa
from deepseek_sparse_attention_gb300 import build as dsa_build

P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load()


def _norm(lib, **kw):
    # 100 rows of 64 bf16 columns, 72 apart: 14,400 bytes
    d = dict(n_rows=100, width=64, dtype=1, x=MB, x_ld=72, add=2 * MB, add_ld=72, weight=3 * MB, eps=1e-5, total=4 * MB,
             total_ld=72, out=5 * MB, out_ld=72, fmt=0, scales=6 * MB, group=0, stream=None)
    d.update(kw)
    for k in ("x", "add", "weight", "total", "out", "scales"):
        d[k] = None if d[k] is None else P(d[k])
    return lib.dsa_rms_norm(*d.values())


@pytest.mark.parametrize("change", [
    dict(out=MB + 144), dict(out=MB + 2), dict(out=MB - 144), dict(out=MB + 99 * 144),       # a row later, a column, before, the last
    dict(out=2 * MB + 144), dict(total=MB + 144), dict(total=2 * MB - 144), dict(total=2 * MB + 2),
    dict(out=4 * MB + 144), dict(out=4 * MB - 2),                                            # the two outputs
    dict(out=3 * MB + 16), dict(out=3 * MB - 99 * 144), dict(total=3 * MB),                  # the weights
    dict(out=MB + 144, out_ld=144), dict(out=MB + 64, out_ld=73),                            # other strides
    dict(fmt=1, out=MB + 1), dict(fmt=1, out=MB + 144 * 7 + 127), dict(fmt=1, out=MB + 128, out_ld=145),
    dict(fmt=1, scales=MB + 400), dict(fmt=1, scales=2 * MB), dict(fmt=1, scales=3 * MB), dict(fmt=1, scales=4 * MB + 4),
    dict(fmt=1, scales=5 * MB + 72 * 99), dict(fmt=1, scales=5 * MB - 399 + 3, group=0),
    dict(n_rows=1, out=MB + 2), dict(n_rows=1, out=MB - 126),
])
def test_norm_refuses_outputs_over_other_elements(lib, change):
    assert _norm(lib, **change) == 1


def _rope(lib, **kw):
    # 50 tokens of 4 heads, 64 of 256 bf16 columns
    d = dict(dtype=1, n_tok=50, heads=4, x=MB, x_tok=1024, x_head=256, pos=3 * MB, out=2 * MB, out_tok=1024, out_head=256,
             stream=None)
    d.update(kw)
    for k in ("x", "pos", "out"):
        d[k] = P(d[k])
    return lib.dsa_rope(ctypes.byref(dsa.make_rope(64, 8e6)), *d.values())


@pytest.mark.parametrize("change", [
    dict(out=MB + 2048), dict(out=MB - 2048), dict(out=MB + 512), dict(out=MB + 2), dict(out=MB + 126), dict(out=MB - 126),
    dict(out=MB + 49 * 2048), dict(out=MB + 128, out_head=64, out_tok=256),                  # other strides among them
    dict(x=MB, x_tok=0, out=MB + 2), dict(x=MB, x_tok=64, x_head=3200, out=MB + 256, out_tok=1024),
    dict(out=3 * MB), dict(out=3 * MB + 392), dict(out=3 * MB - 2048 * 49),                  # the positions
])
def test_rope_refuses_outputs_over_other_elements(lib, change):
    assert _rope(lib, **change) == 1
