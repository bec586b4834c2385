"""Tensors of more than 2^31 elements: the rows behind that border against the formulas."""
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_gpu_expanded import HEADS, LATENT, SCALE, T, U, attend, check
from test_gpu_norm_rope import check_codes, check_norm, check_rope, norm_formula

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    dsa.load()
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _bf16(g, *shape):
    """Values of a few distinct rows: making them all anew takes longer than the call."""
    n = shape[0]
    part = torch.randn((min(n, 509), *shape[1:]), generator=g, device="cuda").bfloat16()
    return part.repeat(-(-n // len(part)), *[1] * (len(shape) - 1))[:n]


@pytest.mark.parametrize("ld", [16384, 16387])
def test_norm_behind_32_bits(ld):
    rows, width = 140001, 16384
    x = _bf16(_gen(1), rows, ld)[:, :width]
    w, at = torch.randn(width, generator=_gen(2), device="cuda"), torch.tensor([0, 131055, 131072, rows - 1], device="cuda")
    y = torch.zeros_like(x)
    dsa.dsa_rms_norm(x, w, 1e-5, y)
    check_norm(y[at], None, x[at], None, w, 1e-5)
    assert torch.equal(y[rows - 509:rows - 1], y[rows - 1018:rows - 510])
    codes, scales = torch.zeros((rows, width), dtype=torch.uint8, device="cuda"), torch.zeros((rows, 128), device="cuda")
    dsa.dsa_rms_norm(x, w, 1e-5, codes, scales=scales, group=128)
    check_codes(codes[at], scales[at], norm_formula(x[at], None, w, 1e-5)[1], 128)


def test_rope_behind_32_bits():
    tokens, plan = 140003, dsa.make_rope(64, 8e6)
    x = _bf16(_gen(3), tokens, HEADS, 256)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=_gen(4), device="cuda", dtype=torch.int64)
    at = torch.tensor([0, 131071, 131072, tokens - 1], device="cuda")
    before = x[at].clone()
    dsa.dsa_rope(plan, x[..., 192:], pos, x[..., 192:])
    check_rope(x[at][..., 192:], plan, before[..., 192:], pos[at], False)
    assert torch.equal(x[at][..., :192], before[..., :192])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expansion_and_attention_behind_32_bits(dtype):
    """Sequences in front of the border, over it and behind it, in one long cache."""
    g, kv_lens, q_lens = _gen(5), [180000, 700, 300], [1, 260, 3]
    rows = sum(kv_lens)
    cache = _bf16(g, rows, 576).to(T[dtype])
    w_uk, w_uv = ((torch.randn((HEADS, n, LATENT), generator=g, device="cuda") / 23).to(T[dtype]) for n in (192, 256))
    k, v = (torch.zeros((rows, HEADS, n), dtype=T[dtype], device="cuda") for n in (192, 256))
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:256]
    dsa.dsa_expand_kv(dsa.make_shape(dtype=dtype), cache, w_uk, w_uv, k, v, ws)
    assert dsa.dsa_check_device_error(ws) == 0
    at = torch.tensor([0, 131071, 131072, 174762, 174763, rows - 1], device="cuda")
    c = cache[at, :LATENT].double()
    for got, w in ((k[at], w_uk), (v[at], w_uv)):
        want, size = torch.einsum("ri,hdi->rhd", c, w.double()), torch.einsum("ri,hdi->rhd", c.abs(), w.abs().double())
        tol = (1024 * U * size + 2.0 ** -8 * want.abs()) if dtype == "bf16" else 513 * U * size
        assert (got.double() - want).abs().le(tol).all()
    q = torch.randn((sum(q_lens), HEADS, 256), generator=g, device="cuda").to(T[dtype])
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    assert SCALE == 1.0 / 16
    check(q_lens, kv_lens, q, k, cache, v, out, lse, heads=(0, 63))
