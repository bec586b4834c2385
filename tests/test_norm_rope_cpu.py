"""What the norm, the rope, the latent expansion and the expanded attention refuse,
and the rope's rates.  CPU only: every refusal comes before anything is enqueued."""
import ctypes
import math
import random

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from deepseek_sparse_attention_gb300 import build as dsa_build

A = ctypes.c_void_p(4096)                     # an aligned address that no refused call reads
OFF = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load()


def _norm(lib, **kw):
    d = dict(n_rows=2, width=64, dtype=1, x=A, x_ld=64, add=A, add_ld=64, weight=A, eps=1e-5, total=A, total_ld=64,
             out=A, out_ld=64, fmt=0, scales=None, group=0, stream=None)
    d.update(kw)
    return lib.dsa_rms_norm(*d.values())


@pytest.mark.parametrize("change,code", [
    (dict(n_rows=-1), 1), (dict(width=0), 1), (dict(width=-3), 1), (dict(dtype=2), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(x_ld=63), 1), (dict(add_ld=63), 1), (dict(total_ld=1), 1), (dict(out_ld=0), 1),
    (dict(eps=0.0), 1), (dict(eps=-1e-5), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(fmt=2), 1), (dict(fmt=1), 1), (dict(fmt=1, scales=A, group=16), 1), (dict(fmt=1, scales=A, group=-32), 1),
    (dict(group=32), 1), (dict(x=OFF), 1), (dict(out=OFF), 1), (dict(weight=OFF), 1), (dict(fmt=1, scales=OFF), 1),
    (dict(width=16385, x_ld=20000, add_ld=20000, total_ld=20000, out_ld=20000), 2), (dict(n_rows=1 << 31), 2),
    (dict(n_rows=0, x=None, out=None), 0),
])
def test_norm_refuses(lib, change, code):
    assert _norm(lib, **change) == code


B, C, D = (ctypes.c_void_p(4096 * i) for i in (2, 3, 4))


@pytest.mark.parametrize("change", [
    dict(out=A, out_ld=72), dict(out=B, out_ld=72), dict(total=A, total_ld=72), dict(total=B, total_ld=72),
    dict(total=D), dict(total=D, n_rows=1),
    dict(fmt=1, scales=A, out=A), dict(fmt=1, scales=A, out=B), dict(fmt=1, scales=A, out=C),
    dict(fmt=1, scales=A, out=A, n_rows=1),
])
def test_norm_refuses_outputs_over_other_rows(lib, change):
    assert _norm(lib, **{**dict(x=A, add=B, total=C, out=D), **change}) == 1


def _init(lib, plan, **kw):
    d = dict(dims=64, layout=0, inverse=0, base=8e6, factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0,
             magnitude=1.0)
    d.update(kw)
    return lib.dsa_rope_init(plan, *d.values())


@pytest.mark.parametrize("change,code", [
    (dict(dims=0), 1), (dict(dims=3), 1), (dict(dims=258), 2), (dict(layout=2), 1), (dict(inverse=2), 1),
    (dict(base=1.0), 1), (dict(base=math.nan), 1), (dict(base=math.inf), 1), (dict(factor=0.5), 1), (dict(factor=math.inf), 1),
    (dict(magnitude=math.nan), 1), (dict(factor=4.0), 1), (dict(factor=4.0, original_len=-1.0), 1),
    (dict(factor=4.0, original_len=4096.0, beta_slow=0.0), 1), (dict(factor=4.0, original_len=4096.0, beta_fast=0.5), 1),
    (dict(factor=4.0, beta_fast=0.0, beta_slow=0.0), 0), (dict(factor=4.0, original_len=4096.0), 0), (dict(), 0),
])
def test_rope_init_refuses(lib, change, code):
    assert _init(lib, ctypes.byref(dsa.RopePlan()), **change) == code


def test_rope_init_without_a_plan(lib):
    assert _init(lib, None) == 1


@pytest.mark.parametrize("factor,fast,slow", [(1.0, 32.0, 1.0), (8.0, 32.0, 1.0), (4.0, 0.0, 0.0), (40.0, 32.0, 1.0),
                                              (2.0, 1.0, 1.0)])
@pytest.mark.parametrize("dims,base,trained", [(64, 8e6, 131072.0), (128, 1e4, 4096.0), (2, 1e4, 100.0)])
def test_rope_rates(lib, dims, base, trained, factor, fast, slow):
    """The turns a position against the formula: within a rounding of each step in
    double precision (16 of 2^-53) and half of the last place of 64 bits."""
    plan = dsa.make_rope(dims, base, factor=factor, original_len=trained, beta_fast=fast, beta_slow=slow)
    place = lambda n: dims * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))   # noqa: E731
    for i in range(dims // 2):
        g = 0.0 if factor == 1.0 else 1.0
        if factor != 1.0 and fast:
            low, high = max(math.floor(place(fast)), 0), min(math.ceil(place(slow)), dims - 1)
            g = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        want = base ** (-2.0 * i / dims) * ((1 - g) + g / factor) / (2 * math.pi)
        got = plan.turns[i] / 2.0 ** 64
        assert abs(got - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -65
    assert all(plan.turns[i] == 0 for i in range(dims // 2, 128))


def _rope(lib, plan=None, **kw):
    if plan is None:
        plan = dsa.make_rope(64, 8e6)
    d = dict(dtype=1, n_tok=4, heads=3, x=A, x_tok=300, x_head=100, pos=A, out=ctypes.c_void_p(1 << 20), out_tok=300,
             out_head=100, stream=None)
    d.update(kw)
    return lib.dsa_rope(ctypes.byref(plan), *d.values())


@pytest.mark.parametrize("change,code", [
    (dict(dtype=5), 1), (dict(n_tok=-1), 1), (dict(heads=-1), 1), (dict(x=None), 1), (dict(pos=None), 1), (dict(out=None), 1),
    (dict(x=OFF), 1), (dict(out=OFF), 1), (dict(pos=OFF), 1), (dict(out_head=63), 1), (dict(out_tok=0), 1),
    (dict(out_tok=200), 1), (dict(out_tok=1000, out_head=256, heads=65), 1), (dict(out_tok=1 << 62, out_head=1 << 62), 1),
    (dict(x_tok=-300), 1), (dict(out=A, out_tok=400), 1), (dict(out=A, out_head=64), 1),
    (dict(n_tok=1 << 31), 2), (dict(heads=65537, out_tok=65537 * 100), 2),
    (dict(n_tok=0, x=None, out=None, pos=None), 0), (dict(heads=0, x=None, out=None, pos=None), 0),
])
def test_rope_refuses(lib, change, code):
    assert _rope(lib, **change) == code


def test_rope_refuses_an_unfilled_plan(lib):
    assert _rope(lib, dsa.RopePlan()) == 1


def _batch(**kw):
    d = dict(n_seq=1, n_q=4, max_q=4, flags=0, max_kv=64, rows=64, keys=64)
    d.update(kw)
    return dsa.Batch(*d.values(), A, A, A)


def _expand(lib, shape=None, **kw):
    d = dict(n_rows=5, nope=192, v_dim=256, cache=A, w_uk=A, w_uv=A, k=A, v=A, ws=A, n=256, stream=None)
    d.update(kw)
    return lib.dsa_expand_kv(ctypes.byref(shape or dsa.make_shape()), *d.values())


@pytest.mark.parametrize("change,code", [
    (dict(n_rows=-1), 1), (dict(n_rows=(1 << 24) + 1), 2), (dict(nope=0), 1), (dict(nope=96), 1), (dict(nope=256), 2),
    (dict(v_dim=64), 1), (dict(v_dim=192), 1), (dict(v_dim=384), 2), (dict(cache=None), 1), (dict(w_uk=None), 1),
    (dict(w_uv=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cache=OFF), 1), (dict(v=OFF), 1),
    (dict(ws=None), 3), (dict(n=128), 3), (dict(ws=ctypes.c_void_p(4096 + 16)), 3),
])
def test_expand_refuses(lib, change, code):
    assert _expand(lib, **change) == code


def test_expand_of_heads_without_rope_may_be_256_wide(lib):
    assert _expand(lib, dsa.make_shape(rope_dim=0), nope=256, n_rows=-1) == 1
    assert _expand(lib, dsa.make_shape(rope_dim=0), nope=256, ws=None) == 3      # the next check


def _attn(lib, shape=None, batch=None, **kw):
    d = dict(nope=192, v_dim=256, q=A, k=A, cache=A, v=A, out=A, lse=A, ws=A, n=1 << 40, stream=None)
    d.update(kw)
    return lib.dsa_expanded_mla_attn(ctypes.byref(shape or dsa.make_shape()), ctypes.byref(batch or _batch()),
                                     *d.values())


@pytest.mark.parametrize("change,code", [
    (dict(nope=0), 1), (dict(nope=256), 2), (dict(v_dim=192), 1), (dict(v_dim=512), 2), (dict(q=None), 1),
    (dict(k=None), 1), (dict(cache=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(q=OFF), 1), (dict(lse=OFF), 1),
    (dict(ws=None), 3), (dict(n=4096), 3),
])
def test_attention_refuses(lib, change, code):
    assert _attn(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(n_seq=0), 1), (dict(max_q=5), 1), (dict(max_kv=3), 1), (dict(rows=0), 1), (dict(flags=64), 1),
    (dict(n_seq=(1 << 20) + 1), 2), (dict(rows=1 << 31), 2), (dict(n_q=(1 << 24) + 1), 2), (dict(max_kv=1 << 31), 2),
])
def test_attention_refuses_batches(lib, change, code):
    assert _attn(lib, batch=_batch(**change)) == code


def test_attention_workspace_grows_with_the_batch():
    """A workspace of a batch serves those of fewer queries and shorter sequences."""
    size = lambda **kw: dsa.dsa_workspace_size(dsa.make_shape(), _batch(**kw), dsa.OP_EXPANDED_MLA)   # noqa: E731
    last = 0
    for n_q in (0, 1, 5, 64, 300, 4096, 65536, 1 << 24):
        n = [size(n_q=n_q, max_q=n_q, max_kv=kv, rows=max(1, kv)) for kv in (n_q, n_q + 100, n_q + 5000)]
        assert n == sorted(n) and n[0] >= 0 and n[-1] >= last
        last = n[-1]
    assert last < 256 << 20


@pytest.mark.parametrize("bq", [16, 64, 256])
def test_slots_hold_every_tile(bq):
    """The rule that finds a tile's sequence from its slot, for batches with idle sequences: every
    sequence's tiles have slots of their own within the bound, and the search finds them."""
    rng = random.Random(bq)
    for _ in range(300):
        n = rng.choice([1, 2, 7, 60])
        lens = [rng.choice([0, 0, 1, bq - 1, bq, bq + 1, rng.randrange(3 * bq)]) for _ in range(n)]
        off = [0]
        for x in lens:
            off.append(off[-1] + x)
        start = [q // bq + min(s, q) for s, q in enumerate(off)]
        slots = off[-1] // bq + min(n, off[-1])
        found = set()
        for slot in range(slots):
            lo, hi = 0, n - 1
            while lo < hi:
                mid = lo + (hi - lo + 1) // 2
                lo, hi = (mid, hi) if start[mid] <= slot else (lo, mid - 1)
            at = slot - start[lo]
            if 0 <= at and at * bq < lens[lo]:
                found.add((lo, at))
        assert found == {(s, t) for s, x in enumerate(lens) for t in range(-(-x // bq))}


def test_binding_refuses():
    """The binding's own checks, before the library is called."""
    x = torch.zeros(4, 64)
    w = torch.zeros(64)
    with pytest.raises(Exception):
        dsa.dsa_rms_norm(x, w, 1e-5, x.clone())
    with pytest.raises(Exception):
        dsa.dsa_rope(dsa.make_rope(64, 8e6), x, torch.zeros(4, dtype=torch.int64), x.clone())
    with pytest.raises(KeyError):
        dsa.make_shape(dtype="f16")
