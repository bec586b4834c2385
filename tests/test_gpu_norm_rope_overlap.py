"""Outputs among the rows of their inputs, where no element is shared."""
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_gpu_norm_rope import check_codes, check_norm, check_rope, norm_formula

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _randn(*shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()


def test_norm_into_other_columns_of_its_rows():
    wide = _randn(300, 2048)
    before, w = wide.clone(), torch.ones(512, device="cuda")
    dsa.dsa_rms_norm(wide[:, :512], w, 1e-5, wide[:, 1024:1536], add=wide[:, 512:1024], total=wide[:, 1536:])
    check_norm(wide[:, 1024:1536], wide[:, 1536:], before[:, :512], before[:, 512:1024], w, 1e-5)
    assert torch.equal(wide[:, :1024], before[:, :1024])


def test_norm_codes_behind_each_row():
    """Codes in the bytes behind each row's columns."""
    wide = torch.zeros((200, 2 * 512 + 512), dtype=torch.uint8, device="cuda")
    x = torch.as_strided(wide.view(torch.bfloat16), (200, 512), (768, 1))
    x.copy_(_randn(200, 512))
    kept, scales = x.clone(), torch.zeros((200, 4), device="cuda")
    dsa.dsa_rms_norm(x, None, 1e-5, wide[:, 1024:], scales=scales, group=128)
    check_codes(wide[:, 1024:].contiguous(), scales, norm_formula(kept, None, None, 1e-5)[1], 128)
    assert torch.equal(x, kept)


def test_norm_of_every_other_row():
    """Rows of one tensor in turn: the same elements of none."""
    both = _randn(400, 256)
    before = both.clone()
    dsa.dsa_rms_norm(both[0::2], None, 1e-5, both[1::2])
    check_norm(both[1::2], None, before[0::2], None, None, 1e-5)
    assert torch.equal(both[0::2], before[0::2])


def test_rope_into_other_columns_of_its_heads():
    x = _randn(70, 5, 256)
    before, plan, pos = x.clone(), dsa.make_rope(64, 1e4), torch.arange(70, device="cuda")
    dsa.dsa_rope(plan, x[..., 192:], pos, x[..., 64:128])
    check_rope(x[..., 64:128], plan, before[..., 192:], pos, False)
    assert torch.equal(x[..., 128:], before[..., 128:]) and torch.equal(x[..., :64], before[..., :64])


def test_rope_into_the_end_of_its_tokens():
    """Heads of other strides behind those of the input in each token's row."""
    wide = _randn(70, 5 * 256 + 5 * 64)
    before, plan, pos = wide.clone(), dsa.make_rope(64, 1e4), torch.arange(70, device="cuda")
    x = torch.as_strided(wide, (70, 5, 64), (1600, 256, 1), 192)
    out = torch.as_strided(wide, (70, 5, 64), (1600, 64, 1), 1280)
    dsa.dsa_rope(plan, x, pos, out)
    check_rope(out, plan, torch.as_strided(before, (70, 5, 64), (1600, 256, 1), 192), pos, False)
    assert torch.equal(wide[:, :1280], before[:, :1280])


def test_rope_of_one_head_for_all():
    """Heads that share their input, behind which the output lies."""
    room = _randn(30 * 64 + 30 * 4 * 64)
    x = torch.as_strided(room, (30, 4, 64), (64, 0, 1))
    out = torch.as_strided(room, (30, 4, 64), (256, 64, 1), 30 * 64)
    plan, pos = dsa.make_rope(64, 1e4), torch.arange(30, device="cuda")
    dsa.dsa_rope(plan, x, pos, out)
    check_rope(out, plan, x, pos, False)
