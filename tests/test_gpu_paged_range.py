"""GPU tests of the paged attention over the whole range of its values."""
import numpy as np
import pytest
import torch

import paged_util as ref
from test_gpu_paged import SCALE, TDT, AttnCase, _lib  # noqa: F401 (_lib: the module's fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ a sink over a flat tail

def sink_case(n_q, kv, dense, fmt, at_end):
    """Row 0 has no value and a logit 17 (head 0) to 20 (head 63) above those of
    all other rows, which are equal; pages of one scale."""
    c = AttnCase(41, [kv], [n_q], fmt=fmt, dense=dense, top_k=2048)
    c.scales[:, 0], c.scales[:, 1] = 120, 127
    c.codes[:, :, 512:] = 0
    p = int(c.table[0, 0])
    c.codes[p, 0, :512] = 0
    c.codes[p, 0, 512] = 0x38 if fmt == "e4m3" else 1          # 1.0
    q = torch.zeros(n_q, 64, 576)
    q[:, :, 512] = torch.linspace(17, 20, 64) / SCALE
    c.q_abs = q.to(TDT["bf16"])
    for i in range(n_q):
        c.idx[i, 0] = 0
        if at_end:
            c.idx[i, :c.n_sel[i]] = np.roll(c.idx[i, :c.n_sel[i]], -1)
    return c


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
@pytest.mark.parametrize("n_q,kv,dense,at_end", [(160, 2300, False, False), (160, 2300, False, True),
                                                 (70, 2300, False, False), (160, 9000, True, False),
                                                 (2, 9000, True, False)])
def test_rows_far_below_a_sink_without_value_make_the_output(n_q, kv, dense, at_end, fmt):
    c = sink_case(n_q, kv, dense, fmt, at_end)
    out, lse, code = c.call()
    assert code == 0
    for i in (0, n_q - 1):
        (o, l, *_), _ = c.expect(i)
        # A weight is a multiple of f16's 2^-24 where the sink's is at least 2^12: off by up to
        # 2^-37 of the sink's, which is e^17..e^20 of its own -- the same for all of the equal
        # rows, so that much of the output -- beside what float32 leaves.
        tol = 2.0 ** -37 * np.exp(c.q_abs[i, :, 512].double().numpy() * SCALE) + 1e-5
        err = np.sqrt(((out[i] - o) ** 2).sum(1) / (o ** 2).sum(1))
        assert np.all(err <= tol), (i, (err / tol).max())
        assert np.allclose(lse[i], l, rtol=1e-6, atol=0)


# ------------------------------------------------------------------ large logits

@pytest.mark.parametrize("n_q", [160, 70, 2])
@pytest.mark.parametrize("size", [22.2, 23.3, 24.4, 26.5, 27.5, 31.5, 60.5, 100.5])
def test_finite_logits_of_any_size_give_finite_outputs(size, n_q):
    """Rows whose logits, about 2^size in log2 units, differ by up to 32 of them:
    float32 tells them apart to 2^(size - 24) only, but an output is a mean of rows,
    and the sum of weights lies between one and the number of rows."""
    c = AttnCase(43, [400], [n_q], page=16, fmt="s8", top_k=300)
    rng = np.random.default_rng(1)
    c.scales[:] = 127
    c.codes[:, :, 512:] = 0
    c.codes[:, :, 512] = 64
    c.codes[:, :, 513] = rng.integers(0, 128, c.codes.shape[:2])
    c.codes[c.table[0, :6], :, 513] //= 4                # the first rows are the lowest
    q = torch.zeros(n_q, 64, 576)
    sign = torch.tensor(np.where(rng.random((n_q, 64)) < 0.5, 1.0, -1.0))
    q[:, :, 512] = (sign * 2.0 ** size / 64 / SCALE / 1.4427).float()
    q[:, :, 513] = torch.tensor(rng.uniform(0.5, 1.0, (n_q, 64)) * 0.25 / SCALE / 1.4427).float()
    c.q_abs = q.to(TDT["bf16"])
    out, lse, code = c.call()
    assert code == 0
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    assert np.abs(out).max() <= 128.0
    z = c.q_abs[:, :, 512].double().numpy() * 64 * SCALE
    assert np.all(np.abs(lse - z) <= 2.0 ** -20 * np.abs(z) + 40)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [160, 70, 2])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("every", [1, 2])
def test_logits_beyond_float32_take_no_weight_beside_finite_ones(every, first, n_q, dtype):
    """Half of the list, whole tiles and splits of it, at about -1e42 for every
    head, or for every other one."""
    if dtype == "f32" and n_q == 160:
        n_q = 40
    c = AttnCase(49, [640], [n_q], page=16, top_k=480, dtype=dtype, fmt="s8")
    c.q_abs[:, ::every, 512] = 2.0 ** 20
    c.q_abs[:, 1::2, 512] = 2.0 ** 20 if every == 1 else 0
    c.scales[:, 1] = ref.E_MAX + 127
    c.codes[:, :, 512:] = 0
    low = np.arange(c.ld) < 20 if first else np.arange(c.ld) >= 20
    c.codes[c.table[0, :c.ld][low], :, 512] = np.uint8(256 - 100)
    out, lse, code = c.call()
    assert code == 0
    for i in (0, n_q - 1):
        at = c.idx[i, :c.n_sel[i]]
        drop = {int(j) for j in at if low[j // 16]}
        (o, l, weight, reach, floor), n = c.expect(i, drop)
        tol, tol_lse = ref.attention_bounds(dtype, c.width, n, weight, reach, l, floor)
        heads = slice(None, None, every)                 # those that give the low rows no weight
        assert (np.abs(out[i] - o) <= tol)[heads].all() and (np.abs(lse[i] - l) <= tol_lse)[heads].all()
        if every == 2:
            (o, l, weight, reach, floor), n = c.expect(i)
            clean = c.q_abs[i].double().numpy()[1::2]
            rows, unit = c.rows_of(i)
            o, l, weight, reach, floor = ref.attention(clean, rows, at, SCALE, unit)
            tol, tol_lse = ref.attention_bounds(dtype, c.width, n, weight, reach, l, floor)
            assert (np.abs(out[i, 1::2] - o) <= tol).all() and (np.abs(lse[i, 1::2] - l) <= tol_lse).all()


# ------------------------------------------------------------------ scales far apart

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [160, 3])
@pytest.mark.parametrize("order", ["rising", "falling", "any", "low first", "high first", "lowest", "highest"])
def test_scales_of_any_distance(order, n_q, dtype):
    """Every exponent the append writes, in one list; the logits come from the
    rope columns, whose scales are ordinary."""
    if dtype == "f32" and n_q == 160:
        n_q = 40
    c = AttnCase(45, [1800], [n_q], page=16, fmt="s8", dtype=dtype, top_k=1500, spread=4.0)
    rng = np.random.default_rng(2)
    pages = c.table[0, :ref.pages_for(1800, 16)]
    n = len(pages)
    top = ref.E_MAX if dtype == "bf16" else ref.E_MAX - 14      # the float32 path sums widened rows
    e = np.rint(np.linspace(ref.E_MIN, top, n)).astype(int)
    if order == "falling": e = e[::-1]
    if order == "any": e = rng.permutation(e)
    if order == "low first": e = np.where(np.arange(n) < n // 2, -105, top - 4)
    if order == "high first": e = np.where(np.arange(n) < n // 2, top - 4, -105)
    if order == "lowest": e = np.full(n, ref.E_MIN)
    if order == "highest": e = np.full(n, top)
    c.scales[pages, 0] = e + 127
    c.codes[:, :, :512] = rng.integers(-127, 128, c.codes[:, :, :512].shape).astype(np.int8).view(np.uint8)
    q = c.q_abs.float()
    q[:, :, :512] = 0
    # rows of small pages above those of large ones in the first half of the heads, 40 at most
    q[:, :, 512] = 0
    c.codes[:, :, 512] = 0
    c.codes[pages, :, 512] = np.rint(np.linspace(-100, 100, n)).astype(np.int8).view(np.uint8)[:, None]
    unit = np.exp2(c.scales[pages[0], 1].astype(float) - 127)
    c.scales[pages, 1] = c.scales[pages[0], 1]
    q[:, :, 512] = torch.linspace(-40, 40, 64) / SCALE / 100 / float(unit)
    c.q_abs = q.to(TDT[dtype])
    out, lse, code = c.call()
    assert code == 0
    some = [0, n_q // 2, n_q - 1]
    c.check(out, lse, some)
    # head by head and column by column as close as float32 sums of rows of one sign pattern are:
    # attention_bounds' relative part, doubled, against the rows' weighted magnitudes
    for i in some:
        (o, l, weight, reach, floor), m = c.expect(i)
        logit = c.width * 2.0 ** -23 * reach
        rel = 4 * (logit + 2.0 ** -21 + 2.0 ** -23 * reach + 2.0 ** -22) + 2 * (m + 2) * 2.0 ** -23
        largest = 2.0 ** -36 * floor if dtype == "bf16" else 0.0
        assert np.all(np.abs(out[i] - o) <= rel * weight + largest + 1e-37)


# ------------------------------------------------------------------ infinite queries

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,top_k,n_sel", [(160, 128, 1), (160, 128, 128), (70, 512, 512), (70, 512, 1),
                                             (2, 512, 512), (2, 512, 1)])
@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
def test_an_infinite_query_element_gives_nan_whatever_the_signs(inf, n_q, top_k, n_sel, dtype):
    """Columns 3 (latent) and 520 (rope) hold codes of one sign in every row:
    the logits are all +inf or all -inf."""
    c = AttnCase(47, [700], [n_q], page=16, top_k=top_k, dtype=dtype, n_sel=[n_sel] * n_q)
    for col, sign in ((3, 0x00), (4, 0x80), (520, 0x00), (521, 0x80)):
        c.codes[:, :, col] = 0x30 | sign
    heads = {5: 3, 9: 4, 20: 520, 40: 521}
    clean = c.q_abs.clone()
    for h, col in heads.items():
        c.q_abs[:, h, col] = inf
        clean[:, h] = 0
    out, lse, code = c.call()
    assert code == 0
    bad = sorted(heads)
    assert np.isnan(out[:, bad]).all() and np.isnan(lse[:, bad]).all()
    fine = [h for h in range(64) if h not in heads]
    c.q_abs = clean
    for i in (0, n_q - 1):
        (o, l, weight, reach, floor), n = c.expect(i)
        tol, tol_lse = ref.attention_bounds(dtype, c.width, n, weight, reach, l, floor)
        assert (np.abs(out[i] - o) <= tol)[fine].all() and (np.abs(lse[i] - l) <= tol_lse)[fine].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinite_query_without_rows_is_an_empty_selection(dtype):
    c = AttnCase(48, [700] * 3, top_k=512, dtype=dtype, n_sel=[0, 40, 512])
    c.q_abs[0, 5, 3] = float("inf")
    out, lse, code = c.call()
    assert code == 0 and not out[0].any() and np.isneginf(lse[0]).all()
    c.check(out, lse, [1, 2])


# ------------------------------------------------------------------ queries of any size

@pytest.mark.parametrize("n_q", [160, 2])
@pytest.mark.parametrize("size", [-133, -125, -110, -90, 0, 90])
def test_queries_of_any_size_keep_their_logits(size, n_q):
    """Elements around 2^size, rows as large as it takes for logits of order one
    (2^110 at most)."""
    c = AttnCase(51, [300], [n_q], page=16, top_k=256)
    c.q_abs = (c.q_abs.double() * 2.0 ** size).to(TDT["bf16"])
    c.scales = (c.scales.astype(int) + np.clip(-size, -90, 110)).astype(np.uint8)
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse, [0, n_q - 1])


@pytest.mark.parametrize("n_q", [160, 2])
@pytest.mark.parametrize("largest", [1.0, 1.9921875])
def test_elements_down_to_2_to_the_minus_31_of_the_largest_count(largest, n_q):
    """One element decides each logit: a large one, which meets zeros, lies 2^31
    above it."""
    c = AttnCase(53, [300], [n_q], page=16, top_k=256, fmt="s8")
    rng = np.random.default_rng(4)
    c.codes[:, :, 512:] = 0
    c.codes[:, :, 513] = rng.integers(0, 128, c.codes.shape[:2])
    c.scales[:, 1] = 127
    q = torch.zeros(n_q, 64, 576, dtype=torch.float64)
    q[:, :, 513] = 1.9921875                             # 8 significant bits
    q[:, :, 514] = 2.0 ** 31 * largest
    c.q_abs = q.to(TDT["bf16"])
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse, [0, n_q - 1])
    # as good as if the element were alone
    c.q_abs[:, :, 514] = 0
    alone = c.call()
    assert np.array_equal(out, alone[0]) and np.array_equal(lse, alone[1])


# ------------------------------------------------------------------ sums of long lists

@pytest.mark.parametrize("rope_fmt", ["s8", "e4m3"])
@pytest.mark.parametrize("n_q", [160, 70])
@pytest.mark.parametrize("steps", [(0, 40, 44, 44, 44), (0, 36, 44, 44, 40), (0, 20, 36, 44, 44), (0, 0, 40, 44, 48),
                                   (0, 44, 44, 44, 44), (0, 36, 44, 72, 80), (80, 44, 0, 40, 80), (0, 120, 112, 120, 120)])
def test_logits_that_climb_by_hundreds_of_binades(steps, n_q, rope_fmt):
    """Five stretches of some 700 rows whose logits are 2 steps[k] in log2 units,
    each with values in columns of its own: every column is one stretch's output.
    A stretch ends with the tile in which sums leave the accumulators."""
    kv = 3500
    c = AttnCase(55, [kv], [n_q], page=16, fmt="s8", dense=True)
    pos = np.arange(c.ld * 16)
    part = np.searchsorted([768, 1472, 2176, 2880], pos, side="right")
    page, row = c.table[0][pos // 16], pos % 16
    codes = np.zeros((len(pos), 576), dtype=np.int8)
    rng = np.random.default_rng(5)
    for k in range(5):
        codes[part == k, 100 * k:100 * k + 100] = rng.integers(1, 128, ((part == k).sum(), 100))
    codes[:, 512] = np.array(steps)[part]
    c.codes[page, row] = codes.view(np.uint8)
    c.scales[:] = 127
    if rope_fmt == "e4m3":                               # the same in the other format
        c.fmt = "e4m3"
        c.codes[page, row] = ref.encode(codes.astype(float), "e4m3")
    q = torch.zeros(n_q, 64, 576)
    q[:, :, 512] = 22.125
    c.q_abs = q.to(TDT["bf16"])
    out, lse, code = c.call()
    assert code == 0
    for i in (0, n_q - 1):
        (o, l, weight, reach, floor), n = c.expect(i)
        # a logit is one product here, exact in float32 but for its rounding, twice: 2^-22 of it, as
        # much of a weight; sums of 700 rows and more, cut off: (n + 2) 2^-23; a weight to 2^-21; and
        # 2^-37 of the largest weight for each of a stretch's rows
        rel = 2 * (2.0 ** -22 * reach + 2.0 ** -21) + (n + 2) * 2.0 ** -23
        assert np.all(np.abs(out[i] - o) <= rel * np.abs(o) + 2.0 ** -37 * floor + 1e-37), i
        assert np.all(np.abs(lse[i] - l) <= 2.0 ** -21 * np.abs(l) + n * 2.0 ** -23)
