"""Host side of the paged 8-bit cache at the ends of its bounds."""
import pytest

import deepseek_sparse_attention_gb300 as dsa
from test_paged_cpu import _batch, lib  # noqa: F401 (lib: the module's fixture)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 114, 153, 2000, 65535])
@pytest.mark.parametrize("max_kv", [(1 << 31) - 1, (1 << 31) - 63, (1 << 31) - 64, (1 << 31) - 65, 1 << 30])
def test_splits_cover_every_row_of_the_longest_bound(lib, max_kv, n_q, dtype):
    info = dsa.dsa_plan(dsa.make_shape(dtype=dtype), _batch(1, n_q, n_q, max_kv, dsa.FLAG_DENSE),
                        dsa.OP_PAGED_MLA)
    assert info["attn_rows_per_split"] > 0
    assert info["attn_splits"] * info["attn_rows_per_split"] >= max_kv
