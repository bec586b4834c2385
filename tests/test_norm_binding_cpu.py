"""What the binding of the norm takes and refuses, with the library's call replaced: CPU only."""
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded; tensors of host memory pass for the current device's."""
    made = []
    monkeypatch.setattr(dsa, "_device", lambda: -1)
    monkeypatch.setattr(dsa, "_stream_at", lambda stream, device: 0)
    monkeypatch.setattr(dsa, "_call", lambda name, *args: made.append((name, *args)))
    return made


X, W = torch.zeros(4, 64), torch.ones(64)


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz])
def test_codes_of_another_type_are_refused(calls, dtype):
    """They would be read as other numbers than those written."""
    with pytest.raises(ValueError, match="out is torch.float32, not torch"):
        dsa.dsa_rms_norm(X, W, 1e-5, torch.zeros(4, 64, dtype=dtype), scales=torch.zeros(4, 2), group=32)
    assert calls == []


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.uint8])
def test_codes_of_the_right_types_are_taken(calls, dtype):
    out, scales = torch.zeros(4, 64, dtype=dtype), torch.zeros(4, 2)
    dsa.dsa_rms_norm(X, W, 1e-5, out, scales=scales, group=32)
    (name, rows, width, kind, x, x_ld, add, add_ld, w, eps, total, total_ld, y, y_ld, fmt, s, group, _), = calls
    assert (name, rows, width, kind, x, x_ld) == ("dsa_rms_norm", 4, 64, dsa.DSA_F32, X.data_ptr(), 64)
    assert (y, y_ld, fmt, s, group) == (out.data_ptr(), 64, dsa.NORM_E4M3, scales.data_ptr(), 32)
    assert add is None and total is None and w == W.data_ptr()
