"""The norm and the rope on the GPU against their formulas in 64 bits.

Bars, from the arithmetic (u = 2^-24, float32's half step):
* norm: a row's sum of squares is 32 fused additions in a lane, five shuffles and
  up to 16 warps' sums, each within u of a sum of positive terms, so the root is
  within 27 u; x + add rounds once (u of h, and 2 u of its square, u of the root); the mean, eps,
  the root, the division and the two products are six more: 40 u in all.  The output's
  rounding adds half a step: 2^-8 of a bf16 value.
* codes: half a step is 2^-4 of a value, or 2^-10 of the scale below e4m3's
  normal numbers (2^-6 of the scale); a scale is within 42 u.
* rope: the turns are cut at 2^-32 and rounded to float32 within 2^-24 of half a
  turn (1.9e-7 in radians), the rate is within 2^-53 of itself; sine and cosine are within two
  units in the last place (2.4e-7; bf16: 2^-21.4 = 3.6e-7), the magnitude rounds once and the products and
  their sum three times (2.4e-7): 8e-7 + 2^-52 pos rate of |a| + |b|, times the magnitude.
"""
import math

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def norm_formula(x, add, weight, eps):
    h = x.double() + (0 if add is None else add.double())
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h, y if weight is None else y * weight.double()


def check_norm(y, total, x, add, weight, eps):
    h, want = norm_formula(x, add, weight, eps)
    dt = "bf16" if x.dtype == torch.bfloat16 else "f32"
    tiny = 2.0 ** -149 if dt == "f32" else 2.0 ** -133     # half a step below the normal numbers, or more
    assert (y.double() - want).abs().le((40 * U + HALF[dt]) * want.abs() + tiny).all()
    if total is not None:
        assert (total.double() - h).abs().le((U + HALF[dt]) * h.abs() + tiny).all()


def widen_codes(codes, scales, group):
    rows, width = codes.shape
    c = codes.view(torch.float8_e4m3fn).float().double()
    at = torch.arange(width, device=codes.device) // (group or width)
    return c, scales.double()[:, at]


def check_codes(codes, scales, want, group):
    rows, width = want.shape
    c, s = widen_codes(codes, scales, group)
    g, n = group or width, scales.shape[1]
    padded = torch.nn.functional.pad(want.abs(), (0, n * g - width)).view(rows, n, g)
    top = (padded.amax(2) / 448).clamp(min=2.0 ** -126)
    assert (scales.double() - top).abs().le(42 * U * top).all()
    assert (c * s - want).abs().le((2.0 ** -4 + 100 * U) * want.abs() + 2.0 ** -10 * s).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 7, 8, 512, 1000, 1024, 1032, 4096, 4097, 8192, 16384])
def test_norm_widths(width, dtype):
    """Every count of threads to a row, and both forms of access."""
    g = _gen(width)
    for rows in (1, 13):
        x = torch.randn((rows, width), generator=g, device="cuda").to(T[dtype])
        add = (3 * torch.randn((rows, width), generator=g, device="cuda")).to(T[dtype])
        w = torch.randn(width, generator=g, device="cuda")
        y, total = torch.full_like(x, math.nan), torch.full_like(x, math.nan)
        dsa.dsa_rms_norm(x, w, 1e-5, y)
        check_norm(y, None, x, None, w, 1e-5)
        dsa.dsa_rms_norm(x, None, 1e-6, y, add=add, total=total)
        check_norm(y, total, x, add, None, 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("width,ld,out_ld", [(512, 512, 512), (512, 576, 520), (1001, 1003, 1001), (96, 97, 97), (40, 40, 40),
                                             (4104, 4104, 4104), (8192, 8192, 8192), (16383, 16384, 16383)])
def test_norm_codes(width, ld, out_ld, group, dtype):
    g = _gen(width + group)
    rows = 9
    x = (torch.randn((rows, ld), generator=g, device="cuda") * torch.exp(
        2 * torch.randn((rows, ld), generator=g, device="cuda"))).to(T[dtype])[:, :width]
    w = torch.randn(width, generator=g, device="cuda")
    codes = torch.full((rows, out_ld), 0x55, dtype=torch.uint8, device="cuda")
    n = -(-width // (group or width))
    scales = torch.full((rows * n + 1,), 7.0, device="cuda")
    dsa.dsa_rms_norm(x, w, 1e-5, codes[:, :width], scales=scales[:-1].view(rows, n), group=group)
    check_codes(codes[:, :width], scales[:-1].view(rows, n), norm_formula(x, None, w, 1e-5)[1], group)
    assert (codes[:, width:] == 0x55).all() and scales[-1] == 7.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [8, 512, 520, 1024, 2048, 2056, 4096, 8192, 16384])
def test_norm_of_inputs_at_any_place(width, dtype):
    """Rows that begin at any element, x's and the residual's at different ones, between NaN.  As
    codes the same bits as of aligned copies, whose sums have the same order."""
    g = _gen(width + 1)
    rows = 11
    x = torch.randn((rows, width), generator=g, device="cuda").to(T[dtype])
    add = torch.randn((rows, width), generator=g, device="cuda").to(T[dtype])
    w = torch.randn(width, generator=g, device="cuda")

    def placed(t, at, ld):
        room = torch.full((at + (rows - 1) * ld + width,), math.nan, dtype=t.dtype, device="cuda")
        view = torch.as_strided(room, (rows, width), (ld, 1), at)
        view.copy_(t)
        return view

    def run(x, add, codes):
        y = torch.full((rows, width), math.nan, dtype=T[dtype], device="cuda") if not codes else \
            torch.full((rows, width), 0x55, dtype=torch.uint8, device="cuda")
        total = torch.full((rows, width), math.nan, dtype=T[dtype], device="cuda")
        scales = torch.full((rows, -(-width // 64)), 7.0, device="cuda") if codes else None
        dsa.dsa_rms_norm(x, w, 1e-5, y, add=add, total=None if add is None else total, scales=scales,
                         group=64 if codes else 0)
        return [y] + ([] if add is None else [total]) + ([scales] if codes else [])

    for codes in (False, True):
        for with_add in (False, True):
            want = run(x, add if with_add else None, codes)
            for at, ld in [(0, width + 1), (1, width), (1, width + 3), (2, width + 8), (3, width + 5), (5, width + 7),
                           (7, width + 2), (4, width + 4)]:
                got = run(placed(x, at, ld), placed(add, 8 - at, ld + at) if with_add else None, codes)
                if codes:
                    assert all(torch.equal(p, q) for p, q in zip(got, want))
                else:
                    check_norm(got[0], got[1] if with_add else None, x, add if with_add else None, w, 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_part_of_a_row(dtype):
    """The latent columns of cache rows, in place; the rope columns stay as they are."""
    g = _gen(3)
    cache = torch.randn((77, 576), generator=g, device="cuda").to(T[dtype])
    w = torch.randn(512, generator=g, device="cuda")
    before = cache.clone()
    dsa.dsa_rms_norm(cache[:, :512], w, 1e-5, cache[:, :512])
    check_norm(cache[:, :512], None, before[:, :512], None, w, 1e-5)
    assert torch.equal(cache[:, 512:], before[:, 512:])


@pytest.mark.parametrize("width", [512, 515, 5000])
def test_norm_writes_over_its_inputs(width):
    """out may be x, and total the residual itself."""
    g = _gen(width)
    x = torch.randn((33, width), generator=g, device="cuda").bfloat16()
    add = torch.randn((33, width), generator=g, device="cuda").bfloat16()
    x0, add0 = x.clone(), add.clone()
    dsa.dsa_rms_norm(x, None, 1e-5, x, add=add, total=add)
    check_norm(x, add, x0, add0, None, 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(6001, 512), (6001, 1000), (2503, 2048), (1300, 4096), (701, 8192), (400, 16384)])
def test_norm_of_more_rows_than_a_wave(rows, width, dtype):
    """Rows one after the other in a CTA, over the inputs themselves, and with codes."""
    g = _gen(rows)
    x = torch.randn((rows, width), generator=g, device="cuda").to(T[dtype])
    add = torch.randn((rows, width), generator=g, device="cuda").to(T[dtype])
    w = torch.randn(width, generator=g, device="cuda")
    codes = torch.empty((rows, width), dtype=torch.uint8, device="cuda")
    for group in (0, 128):
        scales = torch.empty((rows, -(-width // (group or width))), device="cuda")
        dsa.dsa_rms_norm(x, w, 1e-5, codes, add=add, scales=scales, group=group)
        check_codes(codes, scales, norm_formula(x, add, w, 1e-5)[1], group)
    x0, add0 = x.clone(), add.clone()
    dsa.dsa_rms_norm(x, w, 1e-5, x, add=add, total=add)
    check_norm(x, add, x0, add0, w, 1e-5)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-22, 1e-12, 1e12, 1e19, 1e25, 1e37])
@pytest.mark.parametrize("width,eps", [(64, 1e-5), (64, 1e-30), (3000, 1e-30), (3000, 1e-38), (9000, 1e-5)])
def test_norm_over_float32s_range(size, width, eps):
    x = torch.randn((3, width), generator=_gen(1), device="cuda") * size
    y = torch.empty_like(x)
    dsa.dsa_rms_norm(x, None, eps, y)
    # inputs and eps below float32's normal numbers are what they are there
    check_norm(y, None, x, None, None, float(torch.tensor(eps, dtype=torch.float32)))


def test_norm_of_zeros_infinities_and_nans():
    x = torch.randn((5, 300), generator=_gen(2), device="cuda")
    x[0] = 0
    x[1, 7] = math.inf
    x[2, 9] = math.nan
    y = torch.empty_like(x)
    dsa.dsa_rms_norm(x, None, 1e-5, y)
    assert (y[0] == 0).all() and y[1, 7].isnan() and (y[1, :7] == 0).all() and y[2].isnan().all()
    check_norm(y[3:], None, x[3:], None, None, 1e-5)
    for pad in (0, 1):                                     # both forms of access
        codes = torch.zeros((5, 300 + pad), dtype=torch.uint8, device="cuda")[:, :300]
        scales = torch.zeros((5, 10), device="cuda")
        xs = torch.zeros((5, 304 + pad), device="cuda")[:, :300]
        xs.copy_(x)
        dsa.dsa_rms_norm(xs, None, 1e-5, codes, scales=scales, group=32)
        c = codes.view(torch.uint8)
        assert (c[0] == 0).all() and (scales[0] == 2.0 ** -126).all()
        assert scales[1, 0].isnan() and (c[1, :32] & 0x7f == 0x7f).all() and (scales[1, 1:] == 2.0 ** -126).all()
        assert scales[2].isnan().all() and (c[2] & 0x7f == 0x7f).all()
        check_codes(codes[3:], scales[3:], norm_formula(x[3:], None, None, 1e-5)[1], 32)


def test_norm_refuses_tensors():
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    ok = torch.empty_like(x)
    bad = [dict(x=x.half()), dict(x=x.t()), dict(x=x[0]), dict(w=w[:63]), dict(w=w.double()), dict(w=w.cpu()),
           dict(out=ok[:3]), dict(out=ok.bfloat16()), dict(out=None), dict(add=x[:, :60]), dict(add=x.bfloat16()),
           dict(total=x.double()), dict(scales=w), dict(out=torch.empty((4, 64), dtype=torch.uint8, device="cuda")),
           dict(x=torch.zeros((4, 128), device="cuda")[:, ::2])]
    for b in bad:
        with pytest.raises(ValueError):
            dsa.dsa_rms_norm(b.get("x", x), b.get("w", w), 1e-5, b.get("out", ok), add=b.get("add"),
                             total=b.get("total"), scales=b.get("scales"))
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rms_norm(x, w, 0.0, ok)


def test_norm_on_no_rows():
    x = torch.zeros((0, 64), device="cuda")
    dsa.dsa_rms_norm(x, None, 1e-5, torch.empty_like(x))


# ------------------------------------------------------------------ rope

def rope_formula(plan, x, pos, halves, rates):
    """In 64 bits: the result and the bound's |a| + |b| of each column."""
    t = pos.double()[:, None, None] * rates
    c, s = torch.cos(t) * plan.magnitude, torch.sin(t) * plan.magnitude * (-1 if plan.inverse else 1)
    x = x.double()
    a, b = x.chunk(2, -1) if halves else (x[..., 0::2], x[..., 1::2])
    ya, yb, m = a * c - b * s, a * s + b * c, (a.abs() + b.abs()).expand_as(a)
    join = (lambda p, q: torch.cat([p, q], -1)) if halves else (lambda p, q: torch.stack([p, q], -1).flatten(-2))
    slack = (8e-7 + 2.0 ** -52 * t.abs()) * m * abs(plan.magnitude)
    return join(ya, yb), join(slack, slack)


def rope_rates(plan):
    return torch.tensor([plan.turns[i] * 2.0 ** -64 * 2 * math.pi for i in range(plan.dims // 2)], dtype=torch.float64,
                        device="cuda")


def check_rope(y, plan, x, pos, halves):
    want, slack = rope_formula(plan, x, pos, halves, rope_rates(plan))
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0      # float32's own is among the slack's
    assert (y.double() - want).abs().le(slack + half * want.abs() + 2.0 ** -133).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dims,before,after", [(2, 0, 0), (6, 1, 2), (64, 192, 0), (64, 512, 0), (64, 0, 64), (128, 3, 1),
                                               (256, 0, 0), (24, 8, 0)])
def test_rope_layouts(dims, before, after, halves, dtype):
    g = _gen(dims + before)
    for tok, heads in ((1, 1), (5, 64), (77, 3), (1000, 1)):
        wide = torch.randn((tok, heads, before + dims + after), generator=g, device="cuda").to(T[dtype])
        pos = torch.randint(0, 1 << 20, (tok,), generator=g, device="cuda", dtype=torch.int64)
        plan = dsa.make_rope(dims, 1e4, layout="halves" if halves else "pairs")
        x, out = wide[..., before:before + dims], torch.full((tok, heads, dims + 8), 9.0, dtype=T[dtype], device="cuda")
        dsa.dsa_rope(plan, x, pos, out[..., :dims])
        check_rope(out[..., :dims], plan, x, pos, halves)
        assert (out[..., dims:] == 9.0).all()
        kept = wide.clone()
        dsa.dsa_rope(plan, x, pos, x)                          # in place: the same values, the rest as it was
        assert torch.equal(x, out[..., :dims])
        wide[..., before:before + dims] = 0
        kept[..., before:before + dims] = 0
        assert torch.equal(wide, kept)


@pytest.mark.parametrize("tok,heads", [(5000, 64), (40000, 5), (3001, 7)])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("before", [0, 1])
def test_rope_of_many_heads(tok, heads, halves, before):
    """Several heads to a thread, a count that no thread's share divides, both forms of access."""
    g = _gen(tok)
    x = torch.randn((tok, heads, before + 64), generator=g, device="cuda").bfloat16()[..., before:]
    pos = torch.randint(0, 4096, (tok,), generator=g, device="cuda", dtype=torch.int64)
    plan = dsa.make_rope(64, 8e6, layout="halves" if halves else "pairs", magnitude=1.25)
    y = torch.empty_like(x)
    dsa.dsa_rope(plan, x, pos, y)
    check_rope(y, plan, x, pos, halves)


@pytest.mark.parametrize("pos", [0, 1, -1, -4096, (1 << 31) - 1, 1 << 31, (1 << 40) + 12345, -(1 << 62)])
def test_rope_at_any_position(pos):
    """Angles of whole turns wrap exactly: compared with the 64-bit fractions' own angle."""
    plan = dsa.make_rope(64, 8e6)
    x = torch.randn((1, 3, 64), generator=_gen(4), device="cuda")
    y = torch.empty_like(x)
    dsa.dsa_rope(plan, x, torch.tensor([pos], device="cuda"), y)
    turns = [(pos * plan.turns[i]) % (1 << 64) * 2.0 ** -64 for i in range(32)]
    angle = torch.tensor(turns, dtype=torch.float64, device="cuda") * 2 * math.pi
    want, slack = rope_formula(plan, x, torch.ones(1, device="cuda"), False, angle)
    assert (y.double() - want).abs().le(slack).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_inverse_turns_back(dtype):
    g = _gen(5)
    x = torch.randn((50, 4, 128), generator=g, device="cuda").to(T[dtype])
    pos = torch.randint(0, 1 << 20, (50,), generator=g, device="cuda", dtype=torch.int64)
    y, z = torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rope(dsa.make_rope(128, 1e4), x, pos, y)
    back = dsa.make_rope(128, 1e4, inverse=True)
    dsa.dsa_rope(back, y, pos, z)
    check_rope(z, back, y, pos, False)


def test_rope_strides_of_heads_before_tokens():
    """A tensor kept as [heads, tokens, dims], and tokens that share their input."""
    g = _gen(6)
    x = torch.randn((4, 30, 64), generator=g, device="cuda").transpose(0, 1)
    pos = torch.arange(30, device="cuda")
    plan = dsa.make_rope(64, 1e4)
    y = torch.empty((4, 30, 64), device="cuda").transpose(0, 1)
    dsa.dsa_rope(plan, x, pos, y)
    check_rope(y, plan, x, pos, False)
    shared = x[:1].expand(30, 4, 64)
    dsa.dsa_rope(plan, shared, pos, y)
    check_rope(y, plan, shared, pos, False)


def test_rope_refuses_tensors():
    plan = dsa.make_rope(64, 1e4)
    x, pos = torch.zeros((4, 2, 64), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    ok = torch.empty_like(x)
    for b in (dict(x=x[..., :62]), dict(x=x.half()), dict(x=x[0, 0]), dict(pos=pos[:3]), dict(pos=pos.int()),
              dict(pos=pos.cpu()), dict(out=ok[:3]), dict(out=ok.bfloat16()), dict(out=None), dict(pos=None),
              dict(x=torch.zeros((4, 2, 128), device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            dsa.dsa_rope(plan, b.get("x", x), b.get("pos", pos), b.get("out", ok))
    with pytest.raises(dsa.DsaError):                          # heads of the output that share columns
        dsa.dsa_rope(plan, x, pos, ok[:, :1].expand(4, 2, 64))


def test_norm_and_rope_in_a_captured_graph():
    """A cache row's chain, captured and replayed on other inputs, on a stream of its own."""
    g = _gen(7)
    src = torch.randn((64, 576), generator=g, device="cuda").bfloat16()
    rows, pos = src.clone(), torch.arange(64, device="cuda") * 1000
    w, plan = torch.ones(512, device="cuda"), dsa.make_rope(64, 8e6)
    stream = torch.cuda.Stream()
    step = lambda: (dsa.dsa_rms_norm(rows[:, :512], w, 1e-5, rows[:, :512]),           # noqa: E731
                    dsa.dsa_rope(plan, rows[:, 512:], pos, rows[:, 512:]))
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.synchronize()
    for seed in (8, 9):
        fresh = torch.randn((64, 576), generator=_gen(seed), device="cuda").bfloat16()
        rows.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        check_norm(rows[:, :512], None, fresh[:, :512], None, w, 1e-5)
        check_rope(rows[:, None, 512:], plan, fresh[:, None, 512:], pos, False)
