"""The norm at the upper end of float32's range.

Bars: those of test_gpu_norm_rope, whose docstring derives them: 35 u of 40.  A row whose squares
pass float32 takes the same steps, with exact powers of two, and one more rounding where the root is
above 2^126: its inverse, below float32's normal numbers, is within 2^-150 of 2^-128: 4 u.
"""
import math

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_gpu_norm_rope import T, check_codes, check_norm, norm_formula

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _placed(t, pad):
    """The same rows, ``pad`` elements further apart."""
    return torch.nn.functional.pad(t, (0, pad))[:, :t.shape[1]]


def _run(x, w, eps, add=None, group=None, pad=0):
    """Output (and codes) of rows ``pad`` elements further apart."""
    x, add = _placed(x, pad), None if add is None else _placed(add, pad)
    rows, width = x.shape
    if group is None:
        y = torch.full((rows, width + pad), math.nan, dtype=x.dtype, device="cuda")[:, :width]
        dsa.dsa_rms_norm(x, w, eps, y, add=add)
        return y
    codes = torch.zeros((rows, width + pad), dtype=torch.uint8, device="cuda")[:, :width]
    scales = torch.zeros((rows, -(-width // (group or width))), device="cuda")
    dsa.dsa_rms_norm(x, w, eps, codes, add=add, scales=scales, group=group)
    return codes, scales


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("width", [1, 64, 4104, 5000, 8192, 16384])
@pytest.mark.parametrize("low,high", [(3.3e38, 3.38e38), (2e38, 3.3e38), (1e38, 1.2e38)])
def test_norm_of_the_largest_values(width, low, high, pad, dtype):
    """Rows whose squares pass float32 many times over are normed like any others."""
    g = _gen(width)
    size = low + (high - low) * torch.rand((3, width), generator=g, device="cuda")
    x = torch.where(torch.rand((3, width), generator=g, device="cuda") < 0.5, size, -size).to(T[dtype])
    w = torch.randn(width, generator=g, device="cuda")
    check_norm(_run(x, w, 1e-5, pad=pad), None, x, None, w, 1e-5)
    # a sum of two, and codes
    add = (-0.25 * x.float()).to(T[dtype])
    check_norm(_run(x, w, 1e-5, add=add, pad=pad), None, x, add, w, 1e-5)
    for group in (0, 128):
        check_codes(*_run(x, w, 1e-5, group=group, pad=pad), norm_formula(x, None, w, 1e-5)[1], group)


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("width", [64, 16384])
def test_norm_of_small_values_beside_the_largest(width, pad):
    """Elements of every size in a row whose squares pass float32: each keeps its own bits."""
    g = _gen(width + 2)
    x = torch.randn((4, width), generator=g, device="cuda") * torch.exp2(
        torch.randint(-140, 60, (4, width), generator=g, device="cuda").float())
    for row, top in enumerate((3.4e38, 1e30, 2.0 ** 66, 2.0 ** 64)):
        x[row, 3:6] = top
    check_norm(_run(x, None, 1e-5, pad=pad), None, x, None, None, 1e-5)


@pytest.mark.parametrize("x,eps", [(1.8e19, 3e38), (1e19, 3.4e38), (3e38, 3e38), (1.0, 3e38), (1e-30, 3e38)])
def test_norm_with_an_eps_near_the_largest_value(x, eps):
    """The mean and eps may pass float32 together."""
    eps = float(torch.tensor(eps, dtype=torch.float32))
    for width in (1, 8, 16384):
        t = torch.full((2, width), x, device="cuda")
        check_norm(_run(t, None, eps), None, t, None, None, eps)
