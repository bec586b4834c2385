"""The norm's codes against the quotients they stand for."""
import math

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_gpu_norm_range import _run
from test_gpu_norm_rope import T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _code_values():
    c = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return c, (c[1:] + c[:-1]) / 2                       # values, and the middles between them


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128, 0])
@pytest.mark.parametrize("size", [0, 40, -60, -100, -113, -120])
def test_codes_are_the_rounded_quotients(size, group, pad, dtype):
    """Rows of +-1 (mean 1, eps lost beside it) have the weights as their norm: a scale is exactly
    the largest of a group / 448 and a code exactly y / scale, both in float32, to nearest even
    -- at, and next to, the middles between two codes as well.  Sizes are powers of two of the weights.
    Scales below 2^-92 have quotients within 2^-22: 1 / s is within 2^-23 and the product within
    2^-24; the step's difference, rounded to a multiple of 2^-149, is at most twice the true one (or zero), so
    that the step leaves no larger error than it found."""
    width = 1024
    g = torch.Generator().manual_seed(group + 7)
    middles = _code_values()[1]
    n = group or width
    w = torch.empty(width)
    for at in range(0, width, n):
        top = float(1 + torch.rand(1, generator=g)) * 2.0 ** size
        top = torch.tensor(top, dtype=torch.float32)
        scale = torch.clamp(top / 448, min=2.0 ** -126)
        pick = middles[torch.randint(0, len(middles), (n,), generator=g)]
        y = (pick * scale.double()).float()
        y = torch.where(torch.arange(n) % 3 == 0, torch.nextafter(y, torch.tensor(0.0)), y)
        y = torch.where(torch.arange(n) % 3 == 1, torch.nextafter(y, torch.tensor(math.inf)), y)
        y = torch.minimum(y, top)
        y[int(torch.randint(0, n, (1,), generator=g))] = top
        w[at:at + n] = y
    w = w.cuda()
    x = torch.ones((3, width), device="cuda")
    x[1] = -1
    x[2, ::2] = -1
    y = _run(x, w, 1e-30, pad=pad)
    assert torch.equal(y, x * w)                         # the premise
    codes, scales = _run(x.to(T[dtype]), w, 1e-30, group=group, pad=pad)
    # in 64 bits: a quotient of two float32 lies no nearer to the middle of two others than 2^-49 of itself
    want = (y.abs().view(3, -1, n).amax(2).double() / 448).float().clamp(min=2.0 ** -126)
    assert torch.equal(scales, want)
    q, got = y.double() / want.double().repeat_interleave(n, 1), codes.view(torch.float8_e4m3fn).float()
    code = lambda t: t.float().clamp(-448, 448).to(torch.float8_e4m3fn).float()                  # noqa: E731
    if -126 < size - 9 < -92:
        assert got.abs().ge(code(q * (1 - 2.0 ** -22)).abs()).all() and got.abs().le(code(q * (1 + 2.0 ** -22)).abs()).all()
        assert (got * y >= 0).all()
    else:
        assert torch.equal(got, code(q))


@pytest.mark.parametrize("pad", [0, 1])
def test_codes_of_an_infinite_weight(pad):
    """A group with an infinite y has an infinite scale: NaN there, zeros elsewhere in it."""
    w = torch.ones(256, device="cuda")
    w[70] = math.inf
    codes, scales = _run(torch.ones((2, 256), device="cuda"), w, 1e-30, group=64, pad=pad)
    one = float(torch.tensor(1.0 / 448, dtype=torch.float32))
    assert scales[0].tolist() == [one, math.inf, one, one]
    c = codes.view(torch.float8_e4m3fn).float()
    assert c[:, 70].isnan().all() and (c[:, 64:70] == 0).all() and (c[:, 71:128] == 0).all()
    assert (c[:, :64] == 448).all() and (c[:, 128:] == 448).all()


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [-79, -40, -9, 0, 40])
def test_codes_of_scales_of_ones(size, group, pad):
    """Scales with a mantissa of ones, and the ones beside it, at middles of one bit and of five."""
    tops = []
    for near in range(-3, 4):                            # a group each
        s = (2 - 2.0 ** -23 * (1 - near if near <= 0 else 1 - 2 * near)) * 2.0 ** size
        tops.append(float(torch.tensor(s * 448, dtype=torch.float32)))
    width = 8 * group
    w = torch.zeros(width)
    for i, top in enumerate(tops):
        scale = torch.tensor(top / 448, dtype=torch.float32)
        part = torch.cat([(m * scale.double()).float().view(1) for m in _code_values()[1]])[:group // 3]
        part = torch.cat([part, torch.nextafter(part, torch.tensor(0.0)), torch.nextafter(part, torch.tensor(math.inf))])
        w[i * group:i * group + len(part)] = part
        w[i * group + len(part)] = top
    w = w.cuda()
    x = torch.ones((2, width), device="cuda")
    codes, scales = _run(x, w, 1e-30, group=group, pad=pad)
    want = (w.view(-1, group).amax(1).double() / 448).float().clamp(min=2.0 ** -126)
    assert torch.equal(scales[0], want)
    q = (w.double() / want.double().repeat_interleave(group)).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(codes[1], q.view(torch.uint8)) and torch.equal(codes[0], codes[1])
