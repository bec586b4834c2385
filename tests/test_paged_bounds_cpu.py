"""Host side of the paged 8-bit cache at the ends of its bounds."""
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
from test_paged_cpu import _batch, _pages, lib  # noqa: F401 (lib: the module's fixture)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 114, 153, 2000, 65535])
@pytest.mark.parametrize("max_kv", [(1 << 31) - 1, (1 << 31) - 63, (1 << 31) - 64, (1 << 31) - 65, 1 << 30])
def test_splits_cover_every_row_of_the_longest_bound(lib, max_kv, n_q, dtype):
    info = dsa.dsa_plan(dsa.make_shape(dtype=dtype), _batch(1, n_q, n_q, max_kv, dsa.FLAG_DENSE),
                        dsa.OP_PAGED_MLA)
    assert info["attn_rows_per_split"] > 0
    assert info["attn_splits"] * info["attn_rows_per_split"] >= max_kv


def _rows_batch(n_seq, max_kv, total, flags):
    b = _batch(n_seq, n_seq, 1, max_kv, flags)
    b.total_rows = total
    return b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top_k,kpool", [(2048, 1), (2048, 4), (64, 4), (128, 4), (320, 1)])
@pytest.mark.parametrize("flags", [0, dsa.FLAG_DENSE])
@pytest.mark.parametrize("n_seq", [1, 2, 3, 8, 40, 76, 77, 152, 153, 400])
def test_a_workspace_serves_every_batch_of_fewer_rows(lib, n_seq, flags, top_k, kpool, dtype):
    """A program sizes its workspace once, for the longest sequences and the most
    rows it will ever have."""
    sh = dsa.make_shape(dtype=dtype, top_k=top_k, kpool=kpool)
    lengths = [1, 63, 64, 65, 66, 67, 68, 127, 128, 130, 131, 132, 200, 320, 1000, 2048, 2050, 2051, 2052,
               3000, 9000, 20011, 100003, 131072, 1 << 20, 1 << 30, (1 << 31) - 1]
    largest = 0
    for max_kv in lengths:
        size = dsa.dsa_workspace_size(sh, _rows_batch(n_seq, max_kv, n_seq * max_kv, flags),
                                      dsa.OP_PAGED_MLA)
        for part in (1, 2, 3, 5, 9, 20, 100, 5000):
            b = _rows_batch(n_seq, max_kv, max(n_seq * max_kv // part, 1), flags)
            assert dsa.dsa_workspace_size(sh, b, dsa.OP_PAGED_MLA) == size
            splits = dsa.dsa_plan(sh, b, dsa.OP_PAGED_MLA)["attn_splits"]
            assert splits == 1 or n_seq * splits * 64 * 514 * 4 < size
        assert size >= largest
        largest = size


def test_binding_names_a_missing_tensor(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    sh, b, pg = dsa.make_shape(), _batch(), _pages(64, 2, 4)
    i64, i32 = torch.int64, torch.int32

    class Fine:                                       # a tensor of the current device
        is_cuda = True

        def __init__(self, dtype):
            self.dtype = dtype

        def numel(self): return 1 << 20
        def get_device(self): return 0
        def is_contiguous(self): return True
        def data_ptr(self): return 256

    bf16 = Fine(torch.bfloat16)
    with pytest.raises(ValueError, match="codes is missing"):
        dsa.dsa_cache_append(sh, b, pg, bf16, Fine(i64), None, None, None)
    with pytest.raises(ValueError, match="codes is missing"):
        dsa.dsa_paged_mla_attn(sh, b, pg, bf16, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="held_len is missing"):
        dsa.dsa_page_plan(pg, None, None, None, Fine(i32), Fine(i32), Fine(i32), Fine(i64), Fine(i64),
                          Fine(i64), None)
    with pytest.raises(ValueError, match="slots is missing"):
        dsa.dsa_page_plan(pg, Fine(i64), Fine(i64), Fine(i64), Fine(i32), Fine(i32), Fine(i32), Fine(i64),
                          Fine(i64), None, None)
