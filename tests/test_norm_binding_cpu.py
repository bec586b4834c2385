"""What the binding of the norm, the rope and the expanded form takes and refuses, with the library's call replaced: CPU only."""
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


NORM_REFUSALS = [
    (dict(x=None), "x is missing"), (dict(x=X.half()), "x is float32 or bfloat16"), (dict(x=X[0]), "x is a matrix of rows"),
    (dict(x=X.t()), "x's rows are contiguous"), (dict(x=torch.zeros(4, 128)[:, ::2]), "x's rows are contiguous"),
    (dict(w=W[:63]), "weight holds at least 64 elements"), (dict(w=W.double()), "weight is torch.float32, not torch.float64"),
    (dict(out=None), "out is missing"), (dict(out=X[:3]), r"out has the shape \(4, 64\)"),
    (dict(out=X.bfloat16()), "out is torch.float32, not torch.bfloat16"),
    (dict(add=X[:, :60]), "add has the shape"), (dict(add=X.bfloat16()), "add is torch.float32"),
    (dict(total=X.double()), "total is torch.float32"), (dict(total=torch.zeros(4, 128)[:, ::2]), "total's rows are contiguous"),
    (dict(scales=W), "scales go with an out of"), (dict(out=X.to(torch.uint8)), "scales is missing"),
    (dict(out=X.to(torch.uint8), scales=torch.zeros(7), group=32), "scales holds at least 8 elements"),
    (dict(out=X.to(torch.uint8), scales=torch.zeros(3)), "scales holds at least 4 elements"),
]


@pytest.mark.parametrize("change,message", NORM_REFUSALS)
def test_norm_names_what_it_refuses(calls, change, message):
    d = dict(x=X, w=W, out=torch.zeros(4, 64), add=None, total=None, scales=None, group=0)
    d.update(change)
    with pytest.raises(ValueError, match=message):
        dsa.dsa_rms_norm(d["x"], d["w"], 1e-5, d["out"], add=d["add"], total=d["total"], scales=d["scales"], group=d["group"])
    assert calls == []


class Here:
    """A tensor of the current device."""
    is_cuda, dtype, shape = True, torch.float32, torch.Size((4, 64))

    def __init__(self, dense=True, device=0):
        self.dense, self.device = dense, device

    def get_device(self): return self.device
    def stride(self): return (64, 1)
    def numel(self): return 256
    def is_contiguous(self): return self.dense
    def data_ptr(self): return 4096


def test_norm_refuses_weights_of_a_stride_or_of_another_gpu(calls, monkeypatch):
    monkeypatch.setattr(dsa, "_device", lambda: 0)
    for weight, message in ((Here(dense=False), "contiguous tensors only"), (Here(device=1), "weight is on another device")):
        with pytest.raises(ValueError, match=message):
            dsa.dsa_rms_norm(Here(), weight, 1e-5, Here())
    assert calls == []


@pytest.mark.parametrize("which", ["x", "w", "out", "add", "total"])
def test_norm_refuses_tensors_of_another_device(calls, monkeypatch, which):
    monkeypatch.setattr(dsa, "_device", lambda: 0)       # of the others, which say that they are there
    d = {k: Here() for k in ("x", "w", "out", "add", "total")}
    dsa.dsa_rms_norm(d["x"], d["w"], 1e-5, d["out"], add=d["add"], total=d["total"])
    assert len(calls) == 1
    d[which] = X if which != "w" else W
    with pytest.raises(ValueError, match="CUDA tensors only"):
        dsa.dsa_rms_norm(d["x"], d["w"], 1e-5, d["out"], add=d["add"], total=d["total"])
    assert len(calls) == 1


H, POS = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int64)
ROPE_REFUSALS = [
    (dict(x=None), "x is missing"), (dict(x=H.half()), "x is float32 or bfloat16"), (dict(x=H[..., :62]), r"x is \[tokens, heads, 64\]"),
    (dict(x=H[0, 0]), r"x is \[tokens, heads, 64\]"), (dict(x=torch.zeros(4, 2, 128)[..., ::2]), "x's heads are contiguous"),
    (dict(pos=None), "pos is missing"), (dict(pos=POS.int()), "pos is torch.int64"), (dict(pos=POS[:3]), "pos holds at least 4"),
    (dict(out=None), "out is missing"), (dict(out=H[:3]), "out has the shape"), (dict(out=H.bfloat16()), "out is torch.float32"),
    (dict(out=torch.zeros(4, 2, 128)[..., ::2]), "out's heads are contiguous"),
]


@pytest.mark.parametrize("change,message", ROPE_REFUSALS)
def test_rope_names_what_it_refuses(calls, change, message):
    plan = dsa.RopePlan(dims=64)
    d = dict(x=H, pos=POS, out=torch.zeros(4, 2, 64))
    dsa.dsa_rope(plan, *d.values())
    assert [c[0] for c in calls] == ["dsa_rope"]
    d.update(change)
    with pytest.raises(ValueError, match=message):
        dsa.dsa_rope(plan, *d.values())
    assert len(calls) == 1


def _expanded():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)                                          # noqa: E731
    return dict(cache=z(3, 576), w_uk=z(64, 128, 512), w_uv=z(64, 128, 512), k=z(3, 64, 128), v=z(3, 64, 128),
                q=z(2, 64, 192), out=z(2, 64, 128), lse=torch.zeros(2, 64), ws=torch.zeros(256, dtype=torch.uint8))


def _call_expand(d):
    dsa.dsa_expand_kv(dsa.make_shape(), d["cache"], d["w_uk"], d["w_uv"], d["k"], d["v"], d["ws"])


def _call_attn(d):
    batch = dsa.Batch(1, 2, 2, 0, 3, 3, 3, None, None, None)
    dsa.dsa_expanded_mla_attn(dsa.make_shape(), batch, d["q"], d["k"], d["cache"], d["v"], d["out"], d["lse"], d["ws"])


EXPANDED_REFUSALS = [
    (_call_expand, "cache", lambda t: None, "cache is"), (_call_expand, "cache", lambda t: t[:, :512], "cache is"),
    (_call_expand, "cache", lambda t: t.float(), "cache is torch.bfloat16"), (_call_expand, "w_uk", lambda t: None, "w_uk is missing"),
    (_call_expand, "w_uk", lambda t: t[:32], "w_uk is"), (_call_expand, "w_uv", lambda t: t[..., :500], "w_uv is"),
    (_call_expand, "k", lambda t: t[:2], "k_nope holds at least"), (_call_expand, "v", lambda t: t.float(), "v is torch.bfloat16"),
    (_call_expand, "ws", lambda t: None, "ws is missing"), (_call_expand, "ws", lambda t: t.float(), "ws is torch.uint8"),
    (_call_attn, "q", lambda t: t[:1], "q holds at least"), (_call_attn, "q", lambda t: t.float(), "q is torch.bfloat16"),
    (_call_attn, "k", lambda t: t.view(3, 128, 64), "k_nope and v are"), (_call_attn, "k", lambda t: None, "k_nope and v are"),
    (_call_attn, "k", lambda t: t[:2], "k_nope holds at least"), (_call_attn, "v", lambda t: t[:2], "v holds at least"),
    (_call_attn, "cache", lambda t: t[:2], "cache holds at least"), (_call_attn, "cache", lambda t: None, "cache is missing"),
    (_call_attn, "out", lambda t: t.float(), "out is torch.bfloat16"), (_call_attn, "out", lambda t: t[:1], "out holds at least"),
    (_call_attn, "lse", lambda t: t.bfloat16(), "lse is torch.float32"), (_call_attn, "lse", lambda t: t[:1], "lse holds at least"),
    (_call_attn, "ws", lambda t: None, "ws is missing"),
]


@pytest.mark.parametrize("call,which,change,message", EXPANDED_REFUSALS)
def test_expanded_form_names_what_it_refuses(calls, call, which, change, message):
    d = _expanded()
    call(d)
    assert len(calls) == 1
    d[which] = change(d[which])
    with pytest.raises(ValueError, match=message):
        call(d)
    assert len(calls) == 1
