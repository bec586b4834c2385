"""Host side of the paged 8-bit cache: the refusals of its entry points, their
sizes and plans, the binding's checks, and the plain reference of the tests."""
import ctypes
import math

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
import paged_util as ref
from deepseek_sparse_attention_gb300 import build as dsa_build

P = ctypes.c_void_p
GOOD = P(256)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load()


def _batch(n_seq=1, n_q=1, max_q=1, max_kv=4096, flags=0):
    return dsa.Batch(n_seq, n_q, max_q, flags, max_kv, max_kv, max_kv, P(16), P(16), P(16))


def _size(op, shape=None, batch=None):
    return dsa.dsa_workspace_size(shape or dsa.make_shape(), batch or _batch(), op)


BAD_PAGES = [(dict(page_rows=0), 1), (dict(page_rows=-16), 1), (dict(n_pages=0), 1),
             (dict(table_ld=0), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(page_rows=8), 2),
             (dict(page_rows=48), 2), (dict(page_rows=256), 2), (dict(n_pages=1 << 31), 2),
             (dict(table_ld=1 << 27), 2)]


def _pages(page_rows=64, n_pages=100, table_ld=64, fmt=dsa.CACHE_E4M3):
    return dsa.make_pages(page_rows, n_pages, table_ld, fmt)


def _plan(lib, pages, n_seq=2, max_new=4, ptrs=None, ws=GOOD, ws_bytes=1 << 30):
    ptrs = [GOOD] * 10 if ptrs is None else ptrs
    return lib.dsa_page_plan(ctypes.byref(pages) if pages else None, n_seq, max_new, *ptrs, ws,
                             ws_bytes, None)


def _append(lib, sh=None, b=None, pages=None, ptrs=None, ws=GOOD, ws_bytes=256):
    ptrs = [GOOD] * 4 if ptrs is None else ptrs
    return lib.dsa_cache_append(ctypes.byref(sh or dsa.make_shape()), ctypes.byref(b or _batch()),
                                ctypes.byref(pages or _pages()), *ptrs, ws, ws_bytes, None)


def _attn(lib, sh=None, b=None, pages=None, ptrs=None, ws=GOOD, ws_bytes=1 << 30):
    # q_abs, codes, scales, block_table, idx, n_sel, out, lse
    ptrs = [GOOD] * 8 if ptrs is None else ptrs
    return lib.dsa_paged_mla_attn(ctypes.byref(sh or dsa.make_shape()), ctypes.byref(b or _batch()),
                                  ctypes.byref(pages or _pages()), *ptrs, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", BAD_PAGES)
def test_page_geometry_is_checked(lib, change, code):
    bad = _pages(**change)
    assert _plan(lib, bad) == code
    assert _append(lib, pages=bad) == code
    assert _attn(lib, pages=bad) == code


def _without(n, i, value=None):
    return [value if k == i else GOOD for k in range(n)]


def test_page_plan_rejects_before_enqueue(lib):
    assert _plan(lib, None) == 1
    assert _plan(lib, _pages(), n_seq=-1) == 1
    assert _plan(lib, _pages(), max_new=-1) == 1
    assert _plan(lib, _pages(), n_seq=(1 << 20) + 1) == 2
    assert _plan(lib, _pages(), max_new=1 << 31) == 2
    for i in range(10):
        assert _plan(lib, _pages(), ptrs=_without(10, i)) == 1          # missing
        assert _plan(lib, _pages(), ptrs=_without(10, i, P(258))) == 1  # misaligned
    assert _plan(lib, _pages(), ws=None) == 3
    assert _plan(lib, _pages(), ws=P(264)) == 3
    assert _plan(lib, _pages(), ws_bytes=_size(dsa.OP_PAGE_PLAN, batch=_batch(n_seq=2)) - 1) == 3


def test_cache_append_rejects_before_enqueue(lib):
    for i in range(4):
        assert _append(lib, ptrs=_without(4, i)) == 1
    for i, bad in ((0, P(264)), (1, P(260)), (2, P(272))):
        assert _append(lib, ptrs=_without(4, i, bad)) == 1
    assert _append(lib, sh=dsa.make_shape(rope_dim=32)) == 2
    assert _append(lib, b=_batch(max_q=2, max_kv=1)) == 1
    assert _append(lib, b=_batch(n_seq=65536, n_q=65536)) == 2
    assert _append(lib, ws=None) == 3
    assert _append(lib, ws_bytes=16) == 3
    assert _append(lib, b=_batch(n_q=0, max_q=0), ptrs=[None] * 4) == 0      # nothing to do


def test_paged_attention_rejects_before_enqueue(lib):
    for i in range(7):                                                       # lse may be missing
        assert _attn(lib, ptrs=_without(8, i)) == 1
    for i, bad in ((0, P(264)), (1, P(272)), (3, P(258)), (4, P(264)), (5, P(258)), (6, P(264)),
                   (7, P(258))):
        assert _attn(lib, ptrs=_without(8, i, bad)) == 1
    assert _attn(lib, sh=dsa.make_shape(heads=32)) == 2
    assert _attn(lib, b=_batch(max_kv=1 << 31)) == 2
    assert _attn(lib, b=_batch(flags=0x8)) == 1
    assert _attn(lib, b=_batch(n_seq=65536, n_q=65536)) == 2
    assert _attn(lib, ws_bytes=_size(dsa.OP_PAGED_MLA) - 1) == 3
    # the dense switch reads no selection; no query, nothing to do
    dense = _batch(flags=dsa.FLAG_DENSE)
    assert _attn(lib, b=dense, ptrs=[GOOD] * 4 + [None, None, GOOD, None], ws_bytes=16) == 3
    assert _attn(lib, b=_batch(n_q=0, max_q=0), ptrs=[None] * 8) == 0


def test_sizes_and_plans(lib):
    assert _size(dsa.OP_CACHE_APPEND) == 256
    assert _size(dsa.OP_PAGE_PLAN, batch=_batch(n_seq=1000)) % 256 == 0
    big = _size(dsa.OP_PAGE_PLAN, batch=_batch(n_seq=100000, n_q=1 << 20))
    assert big >= _size(dsa.OP_PAGE_PLAN)
    assert _size(dsa.OP_CACHE_APPEND, batch=_batch(n_q=1 << 20)) == 256      # tokens, not queries
    n = ctypes.c_size_t(0)
    for op in (8, 15, 19):
        assert lib.dsa_workspace_size(ctypes.byref(dsa.make_shape()), ctypes.byref(_batch()), op,
                                      ctypes.byref(n)) == 1
    assert lib.dsa_workspace_size(ctypes.byref(dsa.make_shape()), ctypes.byref(_batch(n_seq=-1)),
                                  dsa.OP_PAGE_PLAN, ctypes.byref(n)) == 1
    for sh in (dsa.make_shape(), dsa.make_shape(dtype="f32")):
        for b in (_batch(max_kv=131072), _batch(64, 64, 1, 131072), _batch(1, 500, 500, 9000),
                  _batch(4, 4, 1, 100000, dsa.FLAG_DENSE)):
            info = dsa.dsa_plan(sh, b, dsa.OP_PAGED_MLA)
            rows = 131072 if b.flags else 2048
            assert info["attn_splits"] * info["attn_rows_per_split"] >= min(rows, b.max_kv_len)
            assert info["kernel_launches"] in (1, 2)
            assert _size(dsa.OP_PAGED_MLA, sh, b) % 256 == 0
    assert dsa.dsa_plan(dsa.make_shape(), _batch(), dsa.OP_CACHE_APPEND)["kernel_launches"] == 1
    assert dsa.dsa_plan(dsa.make_shape(), _batch(), dsa.OP_PAGE_PLAN)["kernel_launches"] >= 1


def test_binding_checks_types_and_sizes(lib, monkeypatch):
    """The binding refuses tensors whose element type, size or device the call
    fixes, before it touches a device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    sh, b, pg = dsa.make_shape(), _batch(), _pages(64, 2, 4)
    z = torch.zeros
    codes, scales = z(2, 64, 576, dtype=torch.uint8), z(2, 2, dtype=torch.uint8)
    i64, i32 = torch.int64, torch.int32
    with pytest.raises(ValueError, match="rows is torch.bfloat16"):
        dsa.dsa_cache_append(sh, b, pg, z(1, 576), z(1, dtype=i64), codes, scales, None)
    with pytest.raises(ValueError, match="rows holds at least 576"):
        dsa.dsa_cache_append(sh, b, pg, z(1, 512, dtype=torch.bfloat16), z(1, dtype=i64), codes, scales,
                             None)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        dsa.dsa_cache_append(sh, b, pg, z(1, 576, dtype=torch.bfloat16), z(1, dtype=i64), codes, scales,
                             None)
    with pytest.raises(ValueError, match="q_abs is torch.bfloat16"):
        dsa.dsa_paged_mla_attn(sh, b, pg, z(1, 64, 576), codes, scales, z(4, dtype=i32), None, None, None,
                               None, None)
    with pytest.raises(ValueError, match="slots is missing"):
        dsa._at(None, i64, 0, 1, "slots")
    with pytest.raises(ValueError, match="slots holds at least 3"):
        dsa._at(z(2, dtype=i64), i64, 0, 3, "slots")
    with pytest.raises(ValueError, match="codes holds 73728 one-byte"):
        dsa._bytes_at(z(2, 64, 512, dtype=torch.uint8), 0, 73728, "codes")
    with pytest.raises(ValueError, match="scales holds 4 one-byte"):
        dsa._bytes_at(z(4, dtype=torch.int16), 0, 4, "scales")

    class OnAnother:                                  # a tensor of a second GPU
        dtype, is_cuda = i64, True
        numel = staticmethod(lambda: 8)
        get_device = staticmethod(lambda: 1)
        is_contiguous = staticmethod(lambda: True)
    with pytest.raises(ValueError, match="another device"):
        dsa._at(OnAnother(), i64, 0, 4, "kv_len")
    lens = z(3, dtype=i64)
    with pytest.raises(ValueError, match="n_free is torch.int32"):
        dsa.dsa_page_plan(pg, lens, lens, lens, z(2, dtype=i32), z(1, dtype=i64), z(3, 4, dtype=i32),
                          z(4, dtype=i64), z(4, dtype=i64), lens, None)


# ------------------------------------------------------------ the reference itself

def test_reference_codes_round_trip_and_tie_to_even():
    v = ref.e4m3_values()
    assert v[0x7E] == 448.0 and v[0x08] == 2.0 ** -6 and v[1] == 2.0 ** -9 and math.isnan(v[0x7F])
    codes = np.array([c for c in range(256) if (c & 0x7F) != 0x7F], dtype=np.uint8)
    assert np.array_equal(ref.encode(ref.decode(codes, "e4m3"), "e4m3"), codes)
    # halfway between 1 and 1.125 (even mantissa 0), and between 1.125 and 1.25 (even: 1.25)
    assert ref.decode(ref.encode([1.0625, 1.1875, 2.0 ** -10, 1000.0, -449.0], "e4m3"),
                      "e4m3").tolist() == [1.0, 1.25, 0.0, 448.0, -448.0]
    assert ref.decode(ref.encode([0.5, 1.5, -2.5, 300.0], "s8"), "s8").tolist() == [0, 2, -2, 127]
    # the library's torch type agrees on every half step
    x = np.concatenate([(v[:0x7E] + v[1:0x7F]) / 2, -v[:0x7F]])
    t = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(t, ref.encode(x, "e4m3"))


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("s8", 127.0)])
def test_reference_exponent_is_the_least_that_fits(fmt, top):
    for amax in (1e-30, 0.3, 1.0, top, top * (1 + 2.0 ** -23), top / 2, 3.7, 1e30):
        e = ref.exponent(float(np.float32(amax)), fmt)
        assert float(np.float32(amax)) <= top * 2.0 ** e or e == ref.E_MAX
        assert float(np.float32(amax)) > top * 2.0 ** (e - 1) or e == ref.E_MIN
    assert ref.exponent(0.0, fmt) == ref.E_MIN and ref.exponent(3.4e38, fmt) <= ref.E_MAX


def test_reference_attention_reduces_to_closed_forms():
    """One row: that row; equal logits: the mean; no row: zeros and -inf."""
    rng = np.random.default_rng(0)
    rows = rng.normal(size=(5, 576))
    q = rng.normal(size=(64, 576))
    o, l, *_ = ref.attention(q, rows, [3], 0.25)
    assert np.allclose(o, rows[3, :512]) and np.allclose(l, 0.25 * q @ rows[3])
    o, l, *_ = ref.attention(np.zeros_like(q), rows, [0, 1, 4], 1.0)
    assert np.allclose(o, rows[[0, 1, 4], :512].mean(0)) and np.allclose(l, math.log(3))
    o, l, *_ = ref.attention(q, rows, [], 1.0)
    assert not o.any() and np.isneginf(l).all()
