"""The latent expansion and the expanded attention on the GPU, against the formulas in
64 bits and against the absorbed path.

Bars, from the arithmetic (u = 2^-24; sums on the tensor cores cut instead of
rounding, 2 u a step):
* expansion: 512 exact products of bf16 (or rounded ones of float32): 1024 u (bf16) or
  513 u of the sum of their sizes; bf16's rounding is 2^-8 of the value.
* a logit: d <= 256 products likewise, then the scale's and log2 e's product (2 u):
  dz = (2 d u + 3 u) times scale sum |q k|, and 3 u of the largest |z| for its difference from the
  maximum; a weight's exponential is within 4 u.  A weight is within w = 2 dz + 8 u of
  itself; for bf16 its rounding is 2^-8 more.  Sums and value products over n rows: 2 n u.
  The output is then within (2 w + 2^-8 + 4 n u) sum_j p_j |v_j|, and its rounding.
* lse: dz + 8 u, n u for the sum, and 4 u of itself.
"""
import math

import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "f32": torch.float32}
HEADS, LATENT, SCALE = 64, 512, 1.0 / 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype="bf16"):
    return torch.randn(shape, generator=g, device="cuda").to(T[dtype])


def offsets(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int64, device="cuda")


def make_batch(q_lens, kv_lens, rows=None):
    q_off, row_off = offsets(q_lens), offsets(kv_lens)
    return dsa.make_batch(row_off, row_off, q_off, sum(q_lens), max(q_lens), max(kv_lens),
                          sum(kv_lens) if rows is None else rows, 0)


def workspace(shape, batch):
    return dsa.alloc_workspace(shape, batch, dsa.OP_EXPANDED_MLA)


def make_inputs(q_lens, kv_lens, nope, rope, v_dim, dtype, seed, extra=0):
    g, n_q, rows = _gen(seed), sum(q_lens), sum(kv_lens) + extra
    return (_randn(g, n_q, HEADS, nope + rope, dtype=dtype), _randn(g, rows, HEADS, nope, dtype=dtype),
            _randn(g, rows, LATENT + rope, dtype=dtype), _randn(g, rows, HEADS, v_dim, dtype=dtype))


def attend(q_lens, kv_lens, q, k, cache, v, dtype, ws=None, want_lse=True):
    rope = cache.shape[1] - LATENT
    sh, b = dsa.make_shape(rope_dim=rope, dtype=dtype, scale=SCALE), make_batch(q_lens, kv_lens, k.shape[0])
    ws = workspace(sh, b) if ws is None else ws
    out = torch.full((b.n_q, HEADS, v.shape[2]), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((b.n_q, HEADS), 77.0, device="cuda") if want_lse else None
    dsa.dsa_expanded_mla_attn(sh, b, q, k, cache, v, out, lse, ws)
    assert dsa.dsa_check_device_error(ws) == 0
    return out, lse


def check(q_lens, kv_lens, q, k, cache, v, out, lse, heads=(0, 1, 37, 63)):
    """Some heads of every sequence against the formula."""
    bf16 = q.dtype == torch.bfloat16
    q0 = r0 = 0
    for nq, nk in zip(q_lens, kv_lens):
        if nq == 0:                                        # an idle sequence
            r0 += nk
            continue
        hidden = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in heads:
            qh = q[q0:q0 + nq, h].double()
            kh = torch.cat([k[r0:r0 + nk, h], cache[r0:r0 + nk, LATENT:]], 1).double()
            vh = v[r0:r0 + nk, h].double()
            z = (qh @ kh.T * SCALE).masked_fill(hidden, -math.inf)
            size = (qh.abs() @ kh.abs().T * SCALE).masked_fill(hidden, 0).amax(1, keepdim=True)
            p, want_lse = torch.softmax(z, 1), torch.logsumexp(z, 1, keepdim=True)
            want, weight = p @ vh, p @ vh.abs()
            big = z.masked_fill(hidden, 0).abs().amax(1, keepdim=True)
            dz = (2 * qh.shape[1] + 3) * U * size + 3 * U * big
            w = 2 * dz + 8 * U
            tol = (2 * w + (2.0 ** -8 if bf16 else 0) + 4 * nk * U) * weight + (2.0 ** -8 if bf16 else U) * want.abs()
            assert (out[q0:q0 + nq, h].double() - want).abs().le(tol).all()
            if lse is not None:
                tol = dz + (8 + nk) * U + 4 * U * want_lse.abs()
                assert (lse[q0:q0 + nq, h, None].double() - want_lse).abs().le(tol).all()
        q0, r0 = q0 + nq, r0 + nk


BATCHES = {
    "one_row": ([1], [1]),
    "one_query": ([1], [333]),
    "tile": ([128], [128]),
    "odd": ([129], [131]),
    "behind_a_prefix": ([70], [1000]),
    "ragged": ([64, 0, 1, 200, 17, 1], [64, 5, 129, 333, 17, 1]),
    "decode": ([1] * 9, [1, 31, 32, 33, 127, 128, 129, 500, 64]),
    "long_split": ([3], [5003]),
    "few_of_many": ([16, 1, 2], [300, 2000, 2]),
    "idle": ([0, 0, 1, 0, 300, 0, 0, 0, 1, 0], [0, 9, 700, 0, 300, 64, 0, 0, 65, 0]),
    "many_tiles": ([1000, 513], [1000, 1500]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", BATCHES)
def test_attention_batches(name, dtype):
    q_lens, kv_lens = BATCHES[name]
    x = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=len(name))
    out, lse = attend(q_lens, kv_lens, *x, dtype)
    check(q_lens, kv_lens, *x, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nope,rope,v_dim", [(64, 0, 128), (64, 64, 256), (128, 64, 128), (192, 0, 256), (256, 0, 256),
                                             (192, 64, 128), (128, 0, 128)])
def test_attention_head_widths(nope, rope, v_dim, dtype):
    q_lens, kv_lens = [150, 3], [290, 700]
    x = make_inputs(q_lens, kv_lens, nope, rope, v_dim, dtype, seed=nope + rope)
    out, lse = attend(q_lens, kv_lens, *x, dtype)
    check(q_lens, kv_lens, *x, out, lse)


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([17], [17]), ([32, 1], [40, 700]), ([20, 31, 2, 32], [500, 31, 2, 65]), ([33, 16], [33, 300]),
    ([64, 65, 16, 80, 1], [64, 100, 16, 3000, 129]), ([25] * 3, [25, 5000, 64]),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_few_queries(q_lens, kv_lens, dtype):
    """Tiles of 16, 32 and 64 queries and nearly empty ones, in a workspace for more queries."""
    sh = dsa.make_shape(rope_dim=64, dtype=dtype, scale=SCALE)
    ws = workspace(sh, make_batch(q_lens + [40], kv_lens + [40]))
    q, k, cache, v = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=14)
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype, ws=ws)
    check(q_lens, kv_lens, q, k, cache, v, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_without_lse_and_past_its_sequences(dtype):
    """No lse, a cache with rows behind the last sequence, of NaN."""
    q_lens, kv_lens = [40, 90], [100, 90]
    q, k, cache, v = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=1, extra=200)
    for t in (k, cache, v):
        t[190:] = math.nan
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype, want_lse=False)
    check(q_lens, kv_lens, q, k, cache, v, out, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "rope", "v"])
def test_attention_hidden_rows_may_hold_anything(where, bad, dtype):
    """A bad row of one sequence reaches its own later queries alone: not the earlier ones of
    its tile, nor the sequences beside it."""
    q_lens, kv_lens, at = [200, 130, 50], [260, 130, 50], 170           # row 110 of 260 in positions 60..
    q, k, cache, v = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=2)
    clean = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    check(q_lens, kv_lens, q, k, cache, v, *clean)
    k, cache, v = k.clone(), cache.clone(), v.clone()
    {"k": k[at, :, 5], "rope": cache[at, LATENT + 3:LATENT + 4], "v": v[at, :, 9]}[where].fill_(bad)
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    sees = at - (260 - 200)                                             # the first query that sees the row
    assert torch.equal(out[:sees], clean[0][:sees]) and torch.equal(lse[:sees], clean[1][:sees])
    assert torch.equal(out[200:], clean[0][200:]) and torch.equal(lse[200:], clean[1][200:])
    if where == "v":
        assert torch.equal(lse, clean[1])
        assert not out[sees:200, :, 9].isfinite().any()
        assert torch.equal(out[sees:200, :, :9], clean[0][sees:200, :, :9])
        if not math.isnan(bad):
            assert (out[sees:200, :, 9].float() == bad).all()
    elif math.isnan(bad):
        assert out[sees:200].isnan().all() and lse[sees:200].isnan().all()
    else:
        # the sign of q decides: +inf is NaN, -inf leaves the row out
        up = (q[sees:200, :, 5] if where == "k" else q[sees:200, :, 195]).float() * (1 if bad > 0 else -1) > 0
        assert out[sees:200][up].isnan().all() and out[sees:200][~up].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length,spare", [(100, 0), (40, 3), (200, 1)])
def test_attention_of_many_sequences_with_a_bad_value_each(length, spare, dtype):
    """Short units one after the other on each pair of CTAs, all of them with an infinity that
    later queries see: none takes another's for its own, none loses it."""
    n = 61
    q_lens, kv_lens = [length] * n, [length + (i * spare) % 7 for i in range(n)]
    q, k, cache, v = make_inputs(q_lens, kv_lens, 64, 64, 128, dtype, seed=7)
    clean = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    bad = torch.zeros((n * length,), dtype=torch.bool, device="cuda")
    for i in range(n):
        at = (i * 13) % length                                  # the new row that is bad
        v[sum(kv_lens[:i]) + kv_lens[i] - length + at, :, i] = math.inf
        bad[i * length + at:(i + 1) * length] = True
    column = torch.arange(n, device="cuda").repeat_interleave(length)
    for _ in range(3):
        out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype)
        assert torch.equal(lse, clean[1])
        hit = torch.zeros((n * length, 128), dtype=torch.bool, device="cuda")
        hit[torch.arange(n * length, device="cuda"), column] = bad
        hit = hit[:, None].expand(-1, HEADS, -1)
        assert (out[hit].float() == math.inf).all()
        assert torch.equal(out[~hit], clean[0][~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_infinite_queries(dtype):
    """A query of NaN or infinity is NaN by itself."""
    q, k, cache, v = make_inputs([140], [140], 192, 64, 256, dtype, seed=3)
    clean = attend([140], [140], q, k, cache, v, dtype)
    q = q.clone()
    q[7, 3, 0], q[100, 5, 250] = math.nan, math.inf
    out, lse = attend([140], [140], q, k, cache, v, dtype)
    assert out[7, 3].isnan().all() and lse[7, 3].isnan() and out[100, 5].isnan().all()
    keep = torch.ones((140, HEADS), dtype=torch.bool, device="cuda")
    keep[7, 3] = keep[100, 5] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_logits_at_minus_infinity(dtype):
    """Rows of -inf alone give NaN; one finite logit is all of the softmax."""
    q, k, cache, v = make_inputs([2], [300], 192, 64, 256, dtype, seed=4)
    q = q.abs() + 0.5
    k[:, :, 0] = -math.inf
    out, lse = attend([2], [300], q, k, cache, v, dtype)
    assert out.isnan().all() and lse.isnan().all()
    k[5, :, 0] = 1.0
    out, lse = attend([2], [300], q, k, cache, v, dtype)
    assert torch.equal(out[0], v[5]) and torch.equal(out[1], v[5]) and lse.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_one_logit_at_minus_infinity(dtype):
    """Among others it has the weight zero: the result is that of a key with a very low logit."""
    q_lens, kv_lens = [150, 3], [170, 90]
    q, k, cache, v = make_inputs(q_lens, kv_lens, 64, 64, 128, dtype, seed=12)
    q[..., 5] = 2.0 ** 70
    k[..., 5] = 0
    for row in (9, 169, 171):
        k[row, :, 5] = -1
    low = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    for row in (9, 169, 171):
        k[row, :, 5] = -2.0 ** 70
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    assert torch.isfinite(lse).all() and torch.equal(lse, low[1]) and torch.equal(out, low[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [30.0, 1000.0])
def test_attention_of_large_logits(size, dtype):
    """Maxima that rise through the whole list, by up to thousands, and fall again."""
    q_lens, kv_lens = [130, 1], [700, 900]
    q, k, cache, v = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=5)
    ramp = torch.linspace(-1, 1, sum(kv_lens), device="cuda")[:, None]
    k[:, :, 0] = (ramp * size).to(k.dtype)
    q[:, 0::2, 0], q[:, 1::2, 0] = 16.0, -16.0
    out, lse = attend(q_lens, kv_lens, q, k, cache, v, dtype)
    check(q_lens, kv_lens, q, k, cache, v, out, lse, heads=(0, 1))


def test_attention_refuses_keys_of_other_heads():
    """Large enough, but not of the shape's 64 heads."""
    q, k, cache, v = make_inputs([2], [8], 128, 64, 128, "bf16", seed=13)
    for bad_k, bad_v in ((k.view(16, 32, 128), v), (k, v.view(4, 128, 128))):
        with pytest.raises(ValueError, match="64"):
            attend([2], [8], q, bad_k, cache, bad_v, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_workspace_of_a_larger_batch(dtype):
    """One workspace, never cleared, for smaller batches of every kind, in turn."""
    sh = dsa.make_shape(rope_dim=64, dtype=dtype, scale=SCALE)
    ws = workspace(sh, make_batch([300, 200], [3000, 200]))
    for i, (q_lens, kv_lens) in enumerate([([300, 200], [3000, 200]), ([1], [3000]), ([1, 1], [2999, 3]), ([500], [500]),
                                           ([5] * 20, [100] * 20)]):
        x = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=20 + i)
        out, lse = attend(q_lens, kv_lens, *x, dtype, ws=ws)
        check(q_lens, kv_lens, *x, out, lse, heads=(0, 50))


@pytest.mark.parametrize("row_off,q_off", [
    ([0, 50, 40], [0, 10, 20]),            # rows that end before they begin
    ([0, 50, 5000], [0, 10, 20]),          # rows outside the cache
    ([0, 5, 100], [0, 10, 20]),            # more queries than rows
    ([-8, 50, 100], [0, 10, 20]),
    ([0, 50, 100], [0, 30, 20]),           # queries past the batch, and before
    ([0, 50, 100], [0, 10, 19]),           # a query that no sequence has
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_bad_offsets(row_off, q_off, dtype):
    """The error word is set, nothing outside the tensors is touched, and sequences in order are served."""
    x = make_inputs([10, 10], [50, 50], 192, 64, 256, dtype, seed=6)
    sh = dsa.make_shape(rope_dim=64, dtype=dtype, scale=SCALE)
    off = [torch.tensor(o, dtype=torch.int64, device="cuda") for o in (row_off, q_off)]
    b = dsa.make_batch(off[0], off[0], off[1], 20, 20, 100, 100, 100)
    ws = workspace(sh, b)
    out = torch.zeros((20, HEADS, 256), dtype=T[dtype], device="cuda")
    dsa.dsa_expanded_mla_attn(sh, b, *x, out, None, ws)
    assert dsa.dsa_check_device_error(ws) == 2
    if row_off[:2] == [0, 50] and q_off[:2] == [0, 10]:
        check([10], [50], x[0][:10], *x[1:], out, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_follows_and_precedes_other_kernels(dtype):
    """Inputs written by the kernels just before and outputs read by those just after, over and
    over, on a stream of its own."""
    q_lens, kv_lens = [3, 60], [400, 300]
    x = make_inputs(q_lens, kv_lens, 192, 64, 256, dtype, seed=40)
    sh, b = dsa.make_shape(dtype=dtype, scale=SCALE), make_batch(q_lens, kv_lens)
    ws, want = workspace(sh, b), attend(q_lens, kv_lens, *x, dtype)[0]
    now = [torch.zeros_like(t) for t in x]
    out = torch.empty_like(want)
    stream, kept = torch.cuda.Stream(), []
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(5):
            for t, src in zip(now, x):
                t.copy_(src)
            dsa.dsa_expanded_mla_attn(sh, b, *now, out, None, ws)
            kept.append(out.clone())
            for t in now:
                t.zero_()
            out.zero_()
    stream.synchronize()
    assert all(torch.equal(k, want) for k in kept) and dsa.dsa_check_device_error(ws) == 0


def test_attention_in_captured_graphs_on_two_streams():
    """Two captured graphs with workspaces of their own, replayed at once on two streams; the
    results are those of calls one after another, bit for bit."""
    cases = [([3], [4000]), ([200, 1], [200, 900])]
    runs = []
    for i, (q_lens, kv_lens) in enumerate(cases):
        x = make_inputs(q_lens, kv_lens, 192, 64, 256, "bf16", seed=30 + i)
        sh, b = dsa.make_shape(), make_batch(q_lens, kv_lens)
        ws, out = workspace(sh, b), torch.empty((b.n_q, HEADS, 256), dtype=torch.bfloat16, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        call = lambda: dsa.dsa_expanded_mla_attn(sh, b, *x, out, None, ws)          # noqa: E731
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
        runs.append((q_lens, kv_lens, x, out, out.clone(), stream, graph, ws, b))   # b keeps the offsets
    for _ in range(5):
        for r in runs:
            r[3].zero_()
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r[5]):
                r[6].replay()
        torch.cuda.synchronize()
        for q_lens, kv_lens, x, out, first, _, _, ws, _ in runs:
            assert torch.equal(out, first) and dsa.dsa_check_device_error(ws) == 0
            check(q_lens, kv_lens, *x, out, None, heads=(2,))


@pytest.mark.parametrize("rows", [0, 1, 127, 300, 513])
@pytest.mark.parametrize("dtype,nope,rope,v_dim", [("bf16", 192, 64, 256), ("f32", 192, 64, 256), ("bf16", 64, 0, 128),
                                                   ("bf16", 256, 0, 256), ("f32", 128, 64, 128)])
def test_expansion(rows, dtype, nope, rope, v_dim):
    g = _gen(rows + nope)
    cache = _randn(g, rows, LATENT + rope, dtype=dtype)
    w_uk, w_uv = _randn(g, HEADS, nope, LATENT, dtype=dtype), _randn(g, HEADS, v_dim, LATENT, dtype=dtype)
    sh = dsa.make_shape(rope_dim=rope, dtype=dtype)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:256]
    k = torch.full((rows + 1, HEADS, nope), 5.0, dtype=T[dtype], device="cuda")
    v = torch.full((rows + 1, HEADS, v_dim), 5.0, dtype=T[dtype], device="cuda")
    dsa.dsa_expand_kv(sh, cache, w_uk, w_uv, k[:rows], v[:rows], ws)
    assert dsa.dsa_check_device_error(ws) == 0
    assert (k[rows:] == 5.0).all() and (v[rows:] == 5.0).all()
    c = cache[:, :LATENT].double()
    for got, w in ((k[:rows], w_uk), (v[:rows], w_uv)):
        w = w.double()
        want, size = torch.einsum("ri,hdi->rhd", c, w), torch.einsum("ri,hdi->rhd", c.abs(), w.abs())
        tol = (1024 * U * size + 2.0 ** -8 * want.abs()) if dtype == "bf16" else 513 * U * size
        assert (got.double() - want).abs().le(tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expansion_of_bad_rows(dtype):
    """A NaN row is NaN by itself, and the rope columns do not matter."""
    g = _gen(9)
    cache = _randn(g, 140, 576, dtype=dtype)
    w_uk, w_uv = _randn(g, HEADS, 64, LATENT, dtype=dtype), _randn(g, HEADS, 128, LATENT, dtype=dtype)
    sh, ws = dsa.make_shape(dtype=dtype), torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:256]
    outs = []
    for bad in (False, True):
        c = cache.clone()
        if bad:
            c[:, LATENT:] = math.nan
            c[130, 100] = math.nan
        k, v = (torch.empty((140, HEADS, n), dtype=T[dtype], device="cuda") for n in (64, 128))
        dsa.dsa_expand_kv(sh, c, w_uk, w_uv, k, v, ws)
        outs.append((k, v))
    for a, b in zip(*outs):
        assert torch.equal(a[:130], b[:130]) and torch.equal(a[131:], b[131:]) and b[130].isnan().all()


def test_prompt_through_both_forms():
    """A prompt's chain as a layer runs it -- norm of the latent columns, rope of the tails,
    expansion, attention -- against the absorbed path over the same cache rows (absorbed
    queries, dense attention, up-projection).  The two forms round at other places: keys, values and
    absorbed queries to bf16 (2^-8 each, of sums of 512 terms), so outputs are compared in the
    norm: both within 2^-6 of the formula's in 64 bits over the unrounded expansion."""
    g = _gen(11)
    q_lens = kv_lens = [150, 77, 1]
    n, sh = sum(kv_lens), dsa.make_shape(scale=SCALE)
    raw, q = _randn(g, n, 576), _randn(g, n, HEADS, 256)
    w_uk = _randn(g, HEADS, 192, LATENT) / math.sqrt(LATENT)
    w_uv = _randn(g, HEADS, 256, LATENT) / math.sqrt(LATENT)
    weight, plan = 1 + 0.1 * torch.randn(512, generator=g, device="cuda"), dsa.make_rope(64, 8e6)
    pos = torch.cat([torch.arange(m, device="cuda") for m in kv_lens])
    b = make_batch(q_lens, kv_lens)
    ws = workspace(sh, b)

    cache = torch.empty_like(raw)
    dsa.dsa_rms_norm(raw[:, :LATENT], weight, 1e-5, cache[:, :LATENT])
    dsa.dsa_rope(plan, raw[:, LATENT:], pos, cache[:, LATENT:])
    dsa.dsa_rope(plan, q[..., 192:], pos, q[..., 192:])
    k = torch.empty((n, HEADS, 192), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((n, HEADS, 256), dtype=torch.bfloat16, device="cuda")
    dsa.dsa_expand_kv(sh, cache, w_uk, w_uv, k, v, ws)
    out = torch.empty((n, HEADS, 256), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, HEADS), device="cuda")
    dsa.dsa_expanded_mla_attn(sh, b, q, k, cache, v, out, lse, ws)
    assert dsa.dsa_check_device_error(ws) == 0
    check(q_lens, kv_lens, q, k, cache, v, out, lse)

    off = offsets(kv_lens)
    dense = dsa.make_batch(off, off, off, n, max(q_lens), max(kv_lens), n, n, dsa.FLAG_DENSE)
    ws2 = dsa.alloc_workspace(sh, dense, dsa.OP_SPARSE_MLA)
    q_abs = torch.empty((n, HEADS, 576), dtype=torch.bfloat16, device="cuda")
    latent, lse2 = torch.empty((n, HEADS, 512), device="cuda"), torch.empty((n, HEADS), device="cuda")
    up = torch.empty((n, HEADS, 256), device="cuda")
    dsa.dsa_absorb_q(sh, q, w_uk, q_abs, ws2)
    dsa.dsa_sparse_mla_attn(sh, dense, q_abs, cache, None, None, latent, lse2, ws2)
    dsa.dsa_up_project(sh, latent, w_uv, up, ws2)
    assert dsa.dsa_check_device_error(ws2) == 0

    at = 0
    want = torch.empty((n, HEADS, 256), dtype=torch.float64, device="cuda")
    for m in kv_lens:
        c = cache[at:at + m].double()
        kk = torch.cat([torch.einsum("ri,hdi->hrd", c[:, :LATENT], w_uk.double()),
                        c[:, LATENT:].expand(HEADS, m, 64)], 2)
        z = q[at:at + m].double().transpose(0, 1) @ kk.transpose(1, 2) * SCALE
        z.masked_fill_(torch.ones((m, m), dtype=torch.bool, device="cuda").triu(1), -math.inf)
        vv = torch.einsum("ri,hdi->hrd", c[:, :LATENT], w_uv.double())
        want[at:at + m] = (torch.softmax(z, 2) @ vv).transpose(0, 1)
        at += m
    for got in (out.double(), up.double()):
        assert float((got - want).norm() / want.norm()) < 2.0 ** -6
