"""bf16's rope against the bound of its own arithmetic.

With u = 2^-24 and angles within [-pi, pi]: the turns are cut at 2^-32 (1.5e-9 in radians); their
conversion to float32, the constant 2 pi / 2^32 and the product with it are each within u of at most
pi (3 x 1.9e-7); the fast sine is within 2^-21.41 and the fast cosine within 2^-21.19 on that
interval (CUDA's documentation); the magnitude's product rounds once (u), the two products
and their sum three times (2 u of |a| + |b|, since a sum's terms share it).  Together
3 pi u + 2^-21.19 + 3 u + 1.5e-9 of |a| + |b|, times the magnitude, and the output's rounding.
"""
import math

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SLACK = 3 * math.pi * U + 2.0 ** -21.19 + 3 * U + 1.5e-9


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("before", [0, 1])
@pytest.mark.parametrize("magnitude", [1.0, 0.7])
def test_rope_in_bf16_over_the_whole_turn(magnitude, before, halves):
    """Every angle of a turn (positions of the slowest pairs among them), values that cancel."""
    dsa.load()
    n, dims = 20000, 64
    g = torch.Generator(device="cuda").manual_seed(before)
    x = torch.randn((n, 2, before + dims), generator=g, device="cuda").bfloat16()[..., before:]
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int64)
    plan = dsa.make_rope(dims, 8e6, layout="halves" if halves else "pairs", magnitude=magnitude)
    # turns modulo one in 64 bits: exact up to the fractions' own last place
    turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in list(plan.turns)[:dims // 2]], dtype=torch.int64,
                         device="cuda")
    angle = (pos[:, None] * turns).double() * (2 * math.pi * 2.0 ** -64)
    a, b = x.double().chunk(2, -1) if halves else (x.double()[..., 0::2], x.double()[..., 1::2])
    m = float(torch.tensor(magnitude, dtype=torch.float32))
    c, s = torch.cos(angle)[:, None] * m, torch.sin(angle)[:, None] * m
    join = (lambda p, q: torch.cat([p, q], -1)) if halves else (lambda p, q: torch.stack([p, q], -1).flatten(-2))
    want = join(a * c - b * s, a * s + b * c)
    size = join(a.abs() + b.abs(), a.abs() + b.abs()) * m
    y = torch.empty_like(x)
    dsa.dsa_rope(plan, x, pos, y)
    # the slack reaches into the rounding too
    assert (y.double() - want).abs().le(SLACK * (1 + 2.0 ** -8) * size + 2.0 ** -8 * want.abs()).all()
