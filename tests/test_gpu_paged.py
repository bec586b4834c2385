"""GPU tests of the paged 8-bit cache (dsa_page_plan, dsa_cache_append,
dsa_paged_mla_attn) against a plain 64-bit reference, through the binding."""
import numpy as np
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
import paged_util as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALE = 1.0 / 16.0
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa.load()


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to(DEV)


def i64(x):
    return dev(np.asarray(x, dtype=np.int64))


def host(t):
    return t.detach().cpu().numpy()


def prefix(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int64)


# ------------------------------------------------------------------ page plan

def plan_batch(n_seq):
    return dsa.Batch(n_seq, 1, 1, 0, 1, 1, 1, None, None, None)


class PlanCase:
    """Tables of a running server: rows with held pages, the rest on the stack."""

    def __init__(self, rng, n, page, ld, spare):
        self.page, self.ld, self.n = page, ld, n
        self.held = rng.integers(0, ld * page + 1, n)
        self.held[rng.random(n) < 0.2] = 0
        need = ref.pages_for(self.held, page)
        self.n_pages = int(need.sum()) + spare
        perm = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((n, ld), -7, dtype=np.int32)
        at = 0
        for s in range(n):
            self.table[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
        self.free = np.full(self.n_pages, -9, dtype=np.int32)
        self.n_free = self.n_pages - at
        self.free[:self.n_free] = perm[at:]

    def call(self, kv, q, max_new, in_place=True):
        pages = dsa.make_pages(self.page, self.n_pages, self.ld)
        t = dict(table=dev(self.table), free=dev(self.free),
                 n_free=dev(np.array([self.n_free], dtype=np.int32)),
                 row_off=torch.full((self.n + 1,), -5, dtype=torch.int64, device=DEV),
                 q_off=torch.full((self.n + 1,), -5, dtype=torch.int64, device=DEV),
                 slots=torch.full((max_new,), -5, dtype=torch.int64, device=DEV))
        out = None if in_place else torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = dsa.alloc_workspace(dsa.make_shape(), plan_batch(self.n), dsa.OP_PAGE_PLAN)
        dsa.dsa_page_plan(pages, i64(self.held), i64(kv), i64(q), t["free"], t["n_free"],
                          t["table"], t["row_off"], t["q_off"], t["slots"], ws, n_free_out=out)
        code = dsa.dsa_check_device_error(ws)
        got = {k: host(v) for k, v in t.items()}
        got["n_free"] = int((got["n_free"] if in_place else host(out))[0])
        return got, code

    def check(self, kv, q, max_new, **kw):
        got, code = self.call(kv, q, max_new, **kw)
        names = ("table", "free", "n_free", "row_off", "q_off", "slots")
        want = ref.plan(self.page, self.held, kv, q, self.free, self.n_free, self.table, max_new)
        for name, w in zip(names, want):
            assert np.array_equal(got[name], w), name
        return want[-1], code


def lengths(rng, case, mode):
    n, cap = case.n, case.ld * case.page
    if mode == "decode":
        q = np.minimum(1, cap - case.held)
        return case.held + q, q
    kv = rng.integers(0, cap + 1, n)                    # some grow, some shrink, some end
    kv[rng.random(n) < 0.2] = 0
    q = np.minimum(kv, rng.integers(0, 2 * case.page, n))
    return kv, q


@pytest.mark.parametrize("mode", ["decode", "mixed"])
@pytest.mark.parametrize("n,page,ld", [(1, 16, 1), (1, 64, 40), (2, 128, 3), (33, 16, 7),
                                       (1000, 32, 9), (1024, 64, 2), (1025, 16, 3), (3001, 32, 2)])
def test_page_plan_matches_the_reference(n, page, ld, mode):
    rng = np.random.default_rng(n * page + ld)
    case = PlanCase(rng, n, page, ld, spare=n * ld)
    kv, q = lengths(rng, case, mode)
    enough, code = case.check(kv, q, int(q.sum()) + 5)
    assert enough and code == 0
    case.check(kv, q, int(q.sum()), in_place=False)


def test_page_plan_gives_back_before_it_takes():
    """With nothing free, a finished row's pages serve the rows that grow."""
    case = PlanCase(np.random.default_rng(1), 3, 16, 8, spare=0)
    case.held = np.array([64, 16, 16])
    case.table[:, :] = -7
    case.table[0, :4], case.table[1, 0], case.table[2, 0] = [3, 1, 5, 0], 4, 2
    case.n_pages, case.n_free = 6, 0
    case.free = np.full(6, -9, dtype=np.int32)
    enough, code = case.check(np.array([0, 49, 17]), np.array([0, 33, 1]), 34)
    assert enough and code == 0
    # five wanted, four given back: nothing moves
    enough, code = case.check(np.array([0, 64, 33]), np.array([0, 33, 1]), 34)
    assert not enough and code == 4


def test_page_plan_without_sequences_or_tokens():
    case = PlanCase(np.random.default_rng(1), 2, 16, 8, spare=3)
    enough, code = case.check(np.array([0, 0]), np.array([0, 0]), 0)
    assert enough and code == 0
    pages = dsa.make_pages(16, 4, 2)
    z = torch.zeros(0, dtype=torch.int64, device=DEV)
    off = [torch.full((1,), -5, dtype=torch.int64, device=DEV) for _ in range(2)]
    n_free = torch.tensor([3], dtype=torch.int32, device=DEV)
    ws = dsa.alloc_workspace(dsa.make_shape(), plan_batch(0), dsa.OP_PAGE_PLAN)
    table = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    dsa.dsa_page_plan(pages, z, z, z, torch.zeros(4, dtype=torch.int32, device=DEV), n_free, table,
                      off[0], off[1], slots, ws)
    assert dsa.dsa_check_device_error(ws) == 0
    assert off[0].item() == 0 and off[1].item() == 0 and n_free.item() == 3 and slots.item() == -1


@pytest.mark.parametrize("bad", ["negative kv", "q over kv", "held over table", "kv over table",
                                 "negative q", "negative held"])
def test_page_plan_counts_a_bad_row_as_empty(bad):
    case = PlanCase(np.random.default_rng(5), 40, 16, 6, spare=200)
    kv, q = lengths(np.random.default_rng(6), case, "mixed")
    kv[17], q[17], case.held[17] = 20, 3, 0
    kv0, q0, held0 = kv.copy(), q.copy(), case.held.copy()
    cap = case.ld * case.page
    if bad == "negative kv": kv[17], q[17] = -1, 0
    if bad == "q over kv": q[17] = 21
    if bad == "negative q": q[17] = -2
    if bad == "held over table": case.held[17] = cap + 1
    if bad == "negative held": case.held[17] = -3
    if bad == "kv over table": kv[17] = cap + 1
    got, code = case.call(kv, q, 4000)
    assert code == 2
    kv0[17] = q0[17] = held0[17] = 0
    want = ref.plan(case.page, held0, kv0, q0, case.free, case.n_free, case.table, 4000)
    for name, w in zip(("table", "free", "n_free", "row_off", "q_off", "slots"), want):
        assert np.array_equal(got[name], w), name


def test_page_plan_reports_a_short_slot_map_and_a_bad_stack():
    case = PlanCase(np.random.default_rng(8), 10, 16, 6, spare=60)
    kv, q = lengths(np.random.default_rng(9), case, "decode")
    total = int(q.sum())
    got, code = case.call(kv, q, total - 2)
    want = ref.plan(case.page, case.held, kv, q, case.free, case.n_free, case.table, total - 2)
    assert code == 2 and np.array_equal(got["slots"], want[5]) and np.array_equal(got["table"], want[0])
    for n_free in (-1, case.n_pages + 1):
        case.n_free = n_free
        _, code = case.call(case.held, np.zeros_like(q), 0)
        assert code == 2


def test_page_plan_over_many_steps_keeps_every_page_once():
    """A small server: requests arrive, decode, are rolled back and finish; at
    every step each page is held by exactly one row or free."""
    rng = np.random.default_rng(11)
    n, page, ld, n_pages = 9, 16, 12, 108
    pages = dsa.make_pages(page, n_pages, ld)
    table = torch.full((n, ld), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    n_free = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    off = [torch.zeros(n + 1, dtype=torch.int64, device=DEV) for _ in range(2)]
    slots = torch.zeros(1200, dtype=torch.int64, device=DEV)
    ws = dsa.alloc_workspace(dsa.make_shape(), plan_batch(n), dsa.OP_PAGE_PLAN)
    held = np.zeros(n, dtype=np.int64)
    for _ in range(60):
        q = np.where(held == 0, rng.integers(0, 120, n), 1)
        back = np.where(rng.random(n) < 0.2, np.minimum(held, rng.integers(0, 20, n)), 0)
        kv = np.minimum(held - back + q, ld * page)
        q = np.minimum(q, kv)
        done = rng.random(n) < 0.1
        kv, q = np.where(done, 0, kv), np.where(done, 0, q)
        dsa.dsa_page_plan(pages, i64(held), i64(kv), i64(q), free, n_free, table, off[0], off[1],
                          slots, ws)
        assert dsa.dsa_check_device_error(ws) == 0
        held = kv
        t, f = host(table), host(free)[:n_free.item()]
        used = [p for s in range(n) for p in t[s, :ref.pages_for(held[s], page)]]
        assert sorted(used + list(f)) == list(range(n_pages))


@pytest.mark.parametrize("n", [7, 1500])
def test_page_plan_captured_and_replayed_in_place(n):
    """One captured plan: the stack, its height and the table carry over from
    replay to replay, and a step that finds too few pages changes nothing."""
    rng = np.random.default_rng(12)
    page, ld = 16, 6
    n_pages = 4 * n
    pages = dsa.make_pages(page, n_pages, ld)
    table = np.full((n, ld), -1, dtype=np.int32)
    free, n_free = np.arange(n_pages, dtype=np.int32), n_pages
    t_table, t_free = dev(table), dev(free)
    t_n = torch.tensor([n_free], dtype=torch.int32, device=DEV)
    held = np.zeros(n, dtype=np.int64)
    lens = [torch.zeros(n, dtype=torch.int64, device=DEV) for _ in range(3)]
    off = [torch.zeros(n + 1, dtype=torch.int64, device=DEV) for _ in range(2)]
    slots = torch.zeros(100 * n, dtype=torch.int64, device=DEV)
    ws = dsa.alloc_workspace(dsa.make_shape(), plan_batch(n), dsa.OP_PAGE_PLAN)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dsa.dsa_page_plan(pages, *lens, t_free, t_n, t_table, off[0], off[1], slots, ws)
    short = 0
    for step in range(12):
        kv = rng.integers(0, ld * page + 1, n)
        if step % 4 == 3:
            kv[:] = ld * page                           # more pages than there are
        q = np.minimum(kv, rng.integers(0, 90, n))
        for x, y in zip(lens, (held, kv, q)):
            x.copy_(i64(y))
        graph.replay()
        code = dsa.dsa_check_device_error(ws)
        want = ref.plan(page, held, kv, q, free, n_free, table, slots.numel())
        table, free, n_free, enough = want[0], want[1], want[2], want[-1]
        assert code == (0 if enough else 4)
        assert np.array_equal(host(t_table), table) and np.array_equal(host(t_free), free)
        assert t_n.item() == n_free and np.array_equal(host(slots), want[5])
        assert np.array_equal(host(off[0]), want[3]) and np.array_equal(host(off[1]), want[4])
        held = kv if enough else held
        short += not enough
    assert short >= 3


# ------------------------------------------------------------------ append

def random_rows(rng, n, width, dtype):
    x = rng.normal(size=(n, width)) * np.exp(rng.normal(size=(n, 1)))
    t = torch.tensor(x, dtype=torch.float32).to(TDT[dtype])
    return t.to(DEV), t.double().numpy()


class AppendCase:
    def __init__(self, rng, kv, q, page, width, fmt, spare=3):
        self.kv, self.q, self.page, self.width, self.fmt = np.array(kv), np.array(q), page, width, fmt
        need = [ref.pages_for(k, page) for k in kv]
        self.n_pages, self.ld = int(sum(need)) + spare, max(max(need), 1)
        perm = rng.permutation(self.n_pages)
        self.table = np.full((len(kv), self.ld), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = perm[at:at + k]
            at += k
        n_parts = len(ref.parts(width))
        self.codes = rng.integers(0, 256, (self.n_pages, page, width)).astype(np.uint8)
        if fmt == "e4m3":
            self.codes[(self.codes & 0x7F) == 0x7F] = 0x30
        else:
            self.codes[self.codes == 0x80] = 0x30
        self.scales = rng.integers(115, 122, (self.n_pages, n_parts)).astype(np.uint8)
        self.slots = np.array([int(self.table[s, p // page]) * page + p % page
                               for s in range(len(kv)) for p in range(kv[s] - q[s], kv[s])],
                              dtype=np.int64)

    def shape(self, dtype):
        return dsa.make_shape(rope_dim=self.width - 512, dtype=dtype)

    def batch(self):
        key = prefix(self.kv)
        return dsa.make_batch(i64(prefix(self.kv)), i64(key), i64(prefix(self.q)),
                              int(self.q.sum()), int(max(self.q.max(), 1)), int(max(self.kv.max(), 1)),
                              max(int(self.kv.sum()), 1), int(self.kv.sum()))

    def call(self, rows, dtype, slots=None):
        sh, b = self.shape(dtype), self.batch()
        codes, scales = dev(self.codes), dev(self.scales)
        ws = dsa.alloc_workspace(sh, b, dsa.OP_CACHE_APPEND)
        dsa.dsa_cache_append(sh, b, dsa.make_pages(self.page, self.n_pages, self.ld, self.fmt), rows,
                             i64(self.slots if slots is None else slots), codes, scales, ws)
        code = dsa.dsa_check_device_error(ws)
        return host(codes), host(scales), code

    def check(self, rows, rows64, dtype, slots=None):
        codes, scales, code = self.call(rows, dtype, slots)
        want = ref.append(self.page, self.kv, self.q, rows64,
                          self.slots if slots is None else slots, self.codes, self.scales, self.fmt)
        assert np.array_equal(scales, want[1])
        assert np.array_equal(codes, want[0])           # untouched rows and pages too
        return code


APPENDS = [
    ([1], [1]), ([64], [1]), ([65], [1]), ([63, 64, 65, 200], [1, 1, 1, 1]),
    ([130], [130]), ([300, 5, 77, 0, 129], [300, 5, 30, 0, 1]), ([1000], [517]),
    ([90, 91, 92], [64, 63, 65]),
]


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [576, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_matches_the_reference(page, width, dtype, fmt):
    for i, (kv, q) in enumerate(APPENDS):
        rng = np.random.default_rng(100 * page + i)
        case = AppendCase(rng, kv, q, page, width, fmt)
        rows, rows64 = random_rows(rng, int(sum(q)), width, dtype)
        assert case.check(rows, rows64, dtype) == 0


def test_append_of_a_long_prompt_beside_single_tokens():
    """More tokens than a grid dimension holds, in one call."""
    kv, q = [70001, 129, 5000], [70001, 1, 4990]
    rng = np.random.default_rng(31)
    case = AppendCase(rng, kv, q, 64, 512, "e4m3")
    rows, rows64 = random_rows(rng, sum(q), 512, "bf16")
    assert case.check(rows, rows64, "bf16") == 0


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
def test_append_row_by_row_and_again(fmt):
    """Rows one at a time through three pages: exponents only rise, earlier rows
    follow them; the same call again changes nothing."""
    rng = np.random.default_rng(3)
    page, n = 16, 40
    whole = AppendCase(rng, [n], [n], page, 576, fmt)
    rows, rows64 = random_rows(rng, n, 576, "bf16")
    codes, scales = whole.codes, whole.scales
    for t in range(n):
        step = AppendCase(rng, [t + 1], [1], page, 576, fmt)
        step.table, step.n_pages, step.ld = whole.table, whole.n_pages, whole.ld
        step.codes, step.scales, step.slots = codes, scales, whole.slots[t:t + 1]
        assert step.check(rows[t:t + 1].contiguous(), rows64[t:t + 1], "bf16") == 0
        codes, scales, _ = step.call(rows[t:t + 1].contiguous(), "bf16")
        step.codes, step.scales = codes, scales
        again = step.call(rows[t:t + 1].contiguous(), "bf16")
        assert np.array_equal(again[0], codes) and np.array_equal(again[1], scales)


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_at_the_borders_of_its_range(dtype, fmt):
    """Zeros, signed zeros, the smallest and largest finite values, ties."""
    rng = np.random.default_rng(4)
    case = AppendCase(rng, [16 * 6], [16 * 6], 16, 576, fmt)
    x = np.zeros((96, 576))
    x[16:32] = rng.normal(size=(16, 576)) * 1e-38
    x[32:48] = 3.3e38 * np.sign(rng.normal(size=(16, 576)))
    x[48:64] = ref.TOP[fmt] * np.where(rng.random((16, 576)) < 0.5, 0.5, -1.0)
    x[64:80] = (rng.integers(-40, 41, (16, 576)) + 0.5) / 4.0
    x[80:96, :512] = -0.0
    x[80:96, 512:] = rng.normal(size=(16, 64)) * 1e-30
    t = torch.tensor(x, dtype=torch.float64).to(torch.float32).to(TDT[dtype])
    assert case.check(t.to(DEV), t.double().numpy(), dtype) == 0


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
def test_append_reports_values_it_cannot_hold(fmt, bad):
    rng = np.random.default_rng(5)
    case = AppendCase(rng, [40, 7], [20, 7], 16, 576, fmt)
    rows, rows64 = random_rows(rng, 27, 576, "bf16")
    rows[4, 100] = bad
    rows64[4, 100] = bad
    codes, scales, code = case.call(rows, "bf16")
    want = ref.append(16, case.kv, case.q, rows64, case.slots, case.codes, case.scales, fmt)
    assert code == 5 and np.array_equal(scales, want[1])
    if np.isnan(bad) and fmt == "e4m3":                  # a NaN of either sign
        p, r = divmod(int(case.slots[4]), 16)
        codes[p, r, 100] &= 0x7F
        want[0][p, r, 100] &= 0x7F
    assert np.array_equal(codes, want[0])


def test_append_refuses_a_page_of_a_scale_it_never_writes():
    rng = np.random.default_rng(5)
    case = AppendCase(rng, [40], [1], 16, 576, "e4m3")
    rows, _ = random_rows(rng, 1, 576, "bf16")
    for b in (247, 255):
        case.scales[:] = b
        codes, scales, code = case.call(rows, "bf16")
        assert code == 5 and np.array_equal(codes, case.codes) and np.array_equal(scales, case.scales)


def test_append_leaves_out_pages_without_slots():
    rng = np.random.default_rng(6)
    case = AppendCase(rng, [40, 33], [40, 10], 16, 576, "e4m3")
    rows, rows64 = random_rows(rng, 50, 576, "bf16")
    slots = case.slots.copy()
    slots[16:32] = -1
    assert case.check(rows, rows64, "bf16", slots) == 0
    slots[:] = -1
    assert case.check(rows, rows64, "bf16", slots) == 0


@pytest.mark.parametrize("kind", ["outside", "far outside", "negative", "wrong row", "gap", "twice"])
def test_append_refuses_bad_slots(kind):
    rng = np.random.default_rng(7)
    case = AppendCase(rng, [40, 33], [40, 10], 16, 576, "e4m3")
    rows, rows64 = random_rows(rng, 50, 576, "bf16")
    slots = case.slots.copy()
    if kind == "outside": slots[:16] += case.n_pages * 16 - slots[0]
    if kind == "far outside": slots[:16] += 1 << 40
    if kind == "negative": slots[:16] -= 16 * case.n_pages + slots[0]
    if kind == "wrong row": slots[:16] += 1
    if kind == "gap": slots[9] += 1
    if kind == "twice": slots[9] = slots[8]
    codes, scales, code = case.call(rows, "bf16", slots)
    assert code == 1
    good = case.slots.copy()
    good[:16] = -1                                        # only that page is left out
    want = ref.append(16, case.kv, case.q, rows64, good, case.codes, case.scales, "e4m3")
    assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])


def test_append_skips_a_sequence_outside_the_host_bounds():
    rng = np.random.default_rng(8)
    case = AppendCase(rng, [40, 33], [40, 10], 16, 576, "e4m3")
    rows, rows64 = random_rows(rng, 50, 576, "bf16")
    sh, b = case.shape("bf16"), case.batch()
    b.max_q_len = 39
    codes, scales = dev(case.codes), dev(case.scales)
    ws = dsa.alloc_workspace(sh, b, dsa.OP_CACHE_APPEND)
    dsa.dsa_cache_append(sh, b, dsa.make_pages(16, case.n_pages, case.ld), rows, i64(case.slots),
                         codes, scales, ws)
    assert dsa.dsa_check_device_error(ws) == 2
    slots = case.slots.copy()
    slots[:40] = -1
    want = ref.append(16, case.kv, case.q, rows64, slots, case.codes, case.scales, "e4m3")
    assert np.array_equal(host(codes), want[0]) and np.array_equal(host(scales), want[1])


# ------------------------------------------------------------------ attention

class AttnCase:
    def __init__(self, seed, kv, q=None, page=64, rope=64, fmt="e4m3", dtype="bf16", top_k=128,
                 kpool=1, dense=False, n_sel=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.kv, self.q = list(kv), list(q or [1] * len(kv))
        self.page, self.rope, self.fmt, self.dtype = page, rope, fmt, dtype
        self.width, self.dense, self.kpool = 512 + rope, dense, kpool
        app = AppendCase(rng, self.kv, [0] * len(kv), page, self.width, fmt, spare=2)
        self.table, self.n_pages, self.ld = app.table, app.n_pages, app.ld
        x = rng.normal(size=(self.n_pages, page, self.width)) * spread * \
            np.exp(0.5 * rng.normal(size=(self.n_pages, 1, 1)))
        self.codes = np.zeros(x.shape, dtype=np.uint8)
        self.scales = np.zeros((self.n_pages, len(ref.parts(self.width))), dtype=np.uint8)
        for p in range(self.n_pages):
            for i, (a, b) in enumerate(ref.parts(self.width)):
                e = ref.exponent(float(np.abs(x[p, :, a:b]).max()), fmt)
                self.scales[p, i] = e + 127
                self.codes[p, :, a:b] = ref.encode(x[p, :, a:b] / 2.0 ** e, fmt)
        self.n_q = sum(self.q)
        qa = torch.tensor(rng.normal(size=(self.n_q, 64, self.width)), dtype=torch.float32)
        self.q_abs = qa.to(TDT[dtype])
        self.seq = np.repeat(np.arange(len(kv)), self.q)
        self.L = np.concatenate([np.arange(k - n + 1, k + 1) for k, n in zip(self.kv, self.q)])
        self.shape = dsa.make_shape(rope_dim=rope, dtype=dtype, top_k=top_k, kpool=kpool, scale=SCALE)
        self.idx_width = top_k + kpool - 1
        self.idx = np.full((self.n_q, self.idx_width), -1, dtype=np.int32)
        self.n_sel = np.zeros(self.n_q, dtype=np.int32)
        for i in range(self.n_q):
            n = min(self.L[i], self.idx_width) if n_sel is None else min(self.L[i], n_sel[i])
            self.idx[i, :n] = np.sort(rng.permutation(self.L[i])[:n])
            self.n_sel[i] = n

    def batch(self):
        keys = prefix([k // self.kpool for k in self.kv])
        return dsa.make_batch(i64(prefix(self.kv)), i64(keys), i64(prefix(self.q)), self.n_q,
                              max(self.q), max(self.kv), sum(self.kv), int(keys[-1]),
                              dsa.FLAG_DENSE if self.dense else 0)

    def tensors(self):
        return dict(q=self.q_abs.to(DEV), codes=dev(self.codes), scales=dev(self.scales),
                    table=dev(self.table), idx=dev(self.idx), n_sel=dev(self.n_sel),
                    out=torch.full((self.n_q, 64, 512), float("nan"), device=DEV),
                    lse=torch.full((self.n_q, 64), float("nan"), device=DEV))

    def launch(self, t, b, ws, stream=None):
        dsa.dsa_paged_mla_attn(self.shape, b, dsa.make_pages(self.page, self.n_pages, self.ld, self.fmt),
                               t["q"], t["codes"], t["scales"], t["table"],
                               None if self.dense else t["idx"], None if self.dense else t["n_sel"],
                               t["out"], t["lse"], ws, stream)

    def call(self, t=None):
        t = t or self.tensors()
        b = self.batch()
        ws = dsa.alloc_workspace(self.shape, b, dsa.OP_PAGED_MLA)
        self.launch(t, b, ws)
        code = dsa.dsa_check_device_error(ws)
        return host(t["out"]), host(t["lse"]), code

    def rows_of(self, i):
        """The rows query i may attend over, float64."""
        pool = ref.widen(self.codes, self.scales, self.fmt)
        pos = np.arange(self.L[i])
        page = self.table[self.seq[i]][pos // self.page]
        return pool[page, pos % self.page], np.exp2(self.scales[page, 0].astype(np.float64) - 127)

    def expect(self, i, drop=()):
        at = np.arange(self.L[i]) if self.dense else self.idx[i, :self.n_sel[i]]
        at = np.array([j for j in at if j not in drop], dtype=np.int64)
        rows, unit = self.rows_of(i)
        return ref.attention(self.q_abs[i].double().numpy(), rows, at, SCALE, unit), len(at)

    def check(self, out, lse, queries=None, drop=(), rms=1e-5):
        num = den = 0.0
        for i in range(self.n_q) if queries is None else queries:
            (o, l, weight, reach, floor), n = self.expect(i, drop)
            tol, tol_lse = ref.attention_bounds(self.dtype, self.width, n, weight, reach, l, floor)
            assert np.all(np.abs(out[i] - o) <= tol), (i, np.abs(out[i] - o).max())
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[i]), empty)
            assert np.all(np.abs(lse[i][~empty] - l[~empty]) <= tol_lse[~empty]), i
            num += ((out[i] - o) ** 2).sum()
            den += (o ** 2).sum()
        # everything to about float32
        # (and, as element by element, 1e-37: float32 ends there -- a row that weighs
        # e^-130 / 236 and holds 1e4 gives 1e-54, which is 0)
        assert num <= rms ** 2 * den + out.size * 1e-37 ** 2


GRID = [(dtype, fmt, rope) for dtype in ("bf16", "f32") for fmt in ("e4m3", "s8") for rope in (64, 0)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,fmt,rope", GRID)
def test_attention_matches_the_reference(dtype, fmt, rope, page):
    """Selections from one row to several tiles, around a tile's and a page's end."""
    case = AttnCase(7 + page, [1, 2, 63, 64, 65, 130, 700, 1001], page=page, rope=rope, fmt=fmt,
                    dtype=dtype, top_k=384)
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_empty_and_short_selections(dtype):
    case = AttnCase(3, [900] * 6, top_k=512, dtype=dtype, n_sel=[0, 1, 0, 64, 511, 512])
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)
    assert not out[0].any() and np.isneginf(lse[0]).all()


@pytest.mark.parametrize("n_q", [1, 3, 40, 170])
def test_attention_plans_of_every_batch_size(n_q):
    """One query (many splits), a few, a pair of splits, one split."""
    case = AttnCase(n_q, [1500] + [300 + 7 * i for i in range(n_q - 1)], top_k=1024, page=32)
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse, range(0, n_q, max(1, n_q // 12)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dense", [False, True])
def test_attention_of_chunks(dense, dtype):
    """Several queries per sequence, each with its own causal length."""
    case = AttnCase(21, [70, 5, 300], q=[9, 5, 33], top_k=128, dense=dense, dtype=dtype, page=16)
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
def test_attention_dense_over_a_long_sequence(fmt):
    case = AttnCase(5, [9000, 1, 4097], dense=True, fmt=fmt, rope=0, kpool=4)
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("dense", [True, False])
def test_attention_of_uneven_lengths(dense):
    """Splits planned for the rows of all sequences together."""
    c = AttnCase(20, [9001, 3, 640, 65, 1, 2100], dense=dense, top_k=900)
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse)


def test_attention_with_the_kpool_tail():
    case = AttnCase(9, [2054, 2052, 40], top_k=2048, kpool=4, rope=0, fmt="s8")
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [1e-30, 3e-3, 40.0])
def test_attention_over_the_scales_range(spread, dtype):
    """Logits near zero (a flat softmax) up to one row taking all the weight."""
    case = AttnCase(13, [500, 77], spread=spread, top_k=256, dtype=dtype)
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("rope", [64, 0])
@pytest.mark.parametrize("n_q", [160, 70])
@pytest.mark.parametrize("spread", [1.0, 40.0])
def test_attention_of_long_lists_whose_logits_climb(spread, n_q, rope):
    """One or two CTAs of many tiles to a query; a head's rows from its lowest
    logit to its highest (with the large spread by far more than 2^80), another
    head's the other way round."""
    c = AttnCase(19, [2100], [n_q], rope=rope, spread=spread, top_k=1990)
    some = [0, n_q // 2, n_q - 1]
    for k, i in enumerate(some):
        rows, _ = c.rows_of(i)
        n = c.n_sel[i]
        z = c.q_abs[i, 7 * k].double().numpy() @ rows[c.idx[i, :n]].T
        c.idx[i, :n] = c.idx[i, :n][np.argsort(z if k < 2 else -z)]
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse, some)


def test_attention_any_order_and_the_same_row_twice():
    case = AttnCase(15, [600, 300], top_k=256)
    rng = np.random.default_rng(1)
    for i in range(2):
        rng.shuffle(case.idx[i, :case.n_sel[i]])
    case.idx[0, 5] = case.idx[0, 4]
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


def test_attention_of_shared_pages():
    """Two sequences whose first pages are the same."""
    case = AttnCase(17, [400, 333], top_k=256, page=32)
    case.table[1, :5] = case.table[0, :5]
    out, lse, code = case.call()
    assert code == 0
    case.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", ["index", "negative", "page", "no page"])
def test_attention_skips_and_reports_bad_rows(bad, dtype):
    case = AttnCase(19, [600, 300], top_k=256, page=16, dtype=dtype)
    t = case.tensors()
    if bad in ("index", "negative"):
        t["idx"][0, 7] = 600 if bad == "index" else -2
        drop = {int(case.idx[0, 7])}
    else:
        c = int(case.idx[0, 7]) // 16
        t["table"][0, c] = case.n_pages if bad == "page" else -1
        drop = set(range(16 * c, 16 * c + 16))
    out, lse, code = case.call(t)
    assert code == 1
    case.check(out, lse, [0], drop)
    case.check(out, lse, [1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_is_not_touched_by_values_it_does_not_attend_over(dtype):
    """NaN codes and NaN scales everywhere but in the selected rows' pages and
    rows; a selection that ends inside a tile."""
    case = AttnCase(23, [640, 200], top_k=64, page=16, dtype=dtype, n_sel=[37, 1])
    clean = case.call()
    codes = case.codes.copy()
    keep = np.zeros(codes.shape[:2], dtype=bool)
    for i in range(2):
        at = case.idx[i, :case.n_sel[i]]
        keep[case.table[i][at // 16], at % 16] = True
    codes[~keep] = 0x7F
    scales = case.scales.copy()
    scales[~keep.any(1)] = 255
    t = case.tensors()
    t["codes"], t["scales"] = dev(codes), dev(scales)
    out, lse, code = case.call(t)
    assert code == 0 and np.array_equal(out, clean[0]) and np.array_equal(lse, clean[1])
    # and a NaN in an attended row does show
    p, r = case.table[0][case.idx[0, 3] // 16], case.idx[0, 3] % 16
    t["codes"][p, r, 11] = 0x7F
    out, _, _ = case.call(t)
    assert np.isnan(out[0]).all() and np.array_equal(out[1], clean[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,top_k", [(160, 100), (70, 300), (2, 300)])
def test_attention_passes_nan_and_inf_on(n_q, top_k, dtype):
    """One CTA to a query, a pair and a merge of several.  A query all of whose
    rows are NaN; one head with an infinity and one with a NaN beside others."""
    c = AttnCase(29, [700], [n_q], page=16, top_k=top_k, dtype=dtype)
    c.q_abs[1, 5, 3] = float("inf")
    c.q_abs[1, 9, 100] = float("nan")
    c.idx[0, :c.n_sel[0]] = np.arange(c.n_sel[0]) % 16
    for i in range(1, n_q):
        c.idx[i] = np.where(c.idx[i] >= 0, np.maximum(c.idx[i], 16), -1)
    t = c.tensors()
    t["scales"][int(c.table[0, 0]), 0] = 255
    out, lse, code = c.call(t)
    assert code == 0 and np.isnan(out[0]).all() and np.isnan(lse[0]).all()
    assert np.isnan(out[1, [5, 9]]).all() and np.isnan(lse[1, [5, 9]]).all()
    fine = [h for h in range(64) if h not in (5, 9)]
    finite = c.q_abs.clone()
    finite[1, [5, 9]] = 0
    c.q_abs = finite
    (o, l, weight, reach, floor), n = c.expect(1)
    tol, tol_lse = ref.attention_bounds(dtype, c.width, n, weight, reach, l, floor)
    assert (np.abs(out[1] - o) <= tol)[fine].all() and (np.abs(lse[1] - l) <= tol_lse)[fine].all()
    if n_q > 2:
        c.check(out, lse, [2, n_q - 1])


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
@pytest.mark.parametrize("kv", [400, 700])
def test_attention_of_pages_of_zeros(kv, fmt):
    """Pages of zeros have the least scale there is: first in the list, and all
    of it, beside large values with small logits."""
    c = AttnCase(30, [kv, 120, 300], top_k=600, fmt=fmt, spread=3000.0)
    c.q_abs = c.q_abs / 1024
    zero = np.concatenate([c.table[0, :2], c.table[1, :2], c.table[2, -1:]])
    c.codes[zero], c.scales[zero] = 0, ref.E_MIN + 127
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("apart", [60.0, 75.0, 90.0, 130.0])
def test_attention_of_zeros_that_outweigh_large_rows(apart, dtype):
    """A page of large rows with logits far below those of pages of zeros."""
    c = AttnCase(32, [300], top_k=300, spread=2e4, dtype=dtype)
    c.codes[c.table[0, 0]] = c.codes[c.table[0, 0], :1]
    c.codes[c.table[0, 1:]], c.scales[c.table[0, 1:]] = 0, ref.E_MIN + 127
    row = c.rows_of(0)[0][0]
    q = -apart / SCALE * row / (row @ row) * (1 + 0.002 * np.arange(64))[:, None]
    c.q_abs = torch.tensor(q[None], dtype=torch.float32).to(TDT[dtype])
    out, lse, code = c.call()
    assert code == 0
    # The whole output is one row times its weight e^(z - lse), z = -apart: a
    # float32 sum of W products of mostly one sign, off by up to W 2^-23 |z|, which
    # is the output's relative error (attention_bounds' first term).  With rounding
    # errors of one size and any sign it would be sqrt(W) 2^-24 |z| = 8.6e-5 at 60.
    c.check(out, lse, rms=c.width * 2.0 ** -23 * apart)


def test_attention_far_into_a_large_pool():
    """Pages behind the first 4 GiB of codes."""
    case = AttnCase(25, [300, 100], top_k=128, page=128)
    n_pages = (5 << 30) // (128 * 576)
    pool = torch.zeros((n_pages, 128, 576), dtype=torch.uint8, device=DEV)
    scales = torch.full((n_pages, 2), 127, dtype=torch.uint8, device=DEV)
    pool[-case.n_pages:] = dev(case.codes)
    scales[-case.n_pages:] = dev(case.scales)
    t = case.tensors()
    t["codes"], t["scales"] = pool, scales
    t["table"] = torch.where(t["table"] >= 0, t["table"] + (n_pages - case.n_pages), -1).int()
    small, case.n_pages = case.n_pages, n_pages
    out, lse, code = case.call(t)
    case.n_pages = small
    assert code == 0
    case.check(out, lse)


def test_attention_twice_the_same_bits_and_captured():
    """Deterministic; a captured graph replayed on new inputs in the same
    buffers, beside calls on another stream with a workspace of their own."""
    a, b = AttnCase(27, [3000, 900, 64], top_k=512), AttnCase(28, [3000, 900, 64], top_k=512)
    want_a, want_b = a.call(), b.call()
    assert all(np.array_equal(x, y) for x, y in zip(want_a[:2], a.call()[:2]))
    ta, tb = a.tensors(), b.tensors()
    ba, bb = a.batch(), b.batch()
    wa, wb = (dsa.alloc_workspace(a.shape, x, dsa.OP_PAGED_MLA) for x in (ba, bb))
    a.launch(ta, ba, wa)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.launch(ta, ba, wa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        src = b if k % 2 == 0 else a
        for name in ("q", "codes", "scales", "table", "idx", "n_sel"):
            ta[name].copy_(src.tensors()[name])
        ta["out"].fill_(float("nan"))
        tb["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            b.launch(tb, bb, wb)
        torch.cuda.synchronize()
        want = want_b if src is b else want_a
        assert np.array_equal(host(ta["out"]), want[0]) and np.array_equal(host(ta["lse"]), want[1])
        assert np.array_equal(host(tb["out"]), want_b[0])
    assert dsa.dsa_check_device_error(wa) == 0 and dsa.dsa_check_device_error(wb) == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
def test_plan_append_select_and_attend(fmt):
    """A few steps of serving -- prompts, then decode with a request ending and
    one arriving: the plan's offsets and slots feed the append, the indexer's
    selection and the attention on one stream without a synchronisation."""
    rng = np.random.default_rng(31)
    page, n, n_pages, ld, top_k = 16, 4, 120, 40, 64
    sh = dsa.make_shape(top_k=top_k, scale=SCALE)
    pages = dsa.make_pages(page, n_pages, ld, fmt)
    codes = torch.zeros((n_pages, page, 576), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n_pages, 2), dtype=torch.uint8, device=DEV)
    table = torch.full((n, ld), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    n_free = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    row_off, q_off = (torch.zeros(n + 1, dtype=torch.int64, device=DEV) for _ in range(2))
    cap = 600                                              # keys reserved per sequence
    key_off = i64(np.arange(n + 1) * cap)
    keys = torch.zeros((n * cap, 128), dtype=torch.bfloat16, device=DEV)
    cache = [np.zeros((0, 576)) for _ in range(n)]         # the rows as given
    held = np.zeros(n, dtype=np.int64)
    steps = [([300, 20, 0, 131], None), ([1, 1, 0, 1], None), ([1, 1, 250, 1], None),
             ([1, 0, 3, 1], 1), ([1, 40, 1, 1], None)]
    for q, done in steps:
        q = np.array(q)
        kv = held + q
        if done is not None:
            cache[done] = np.zeros((0, 576))
            kv[done] = 0
        n_q = int(q.sum())
        rows = torch.tensor(rng.normal(size=(n_q, 576)), dtype=torch.float32).bfloat16()
        q_idx = torch.tensor(rng.normal(size=(n_q, 32, 128)), dtype=torch.float32).bfloat16().to(DEV)
        w = torch.tensor(rng.normal(size=(n_q, 32)), dtype=torch.float32).to(DEV)
        q_abs = torch.tensor(rng.normal(size=(n_q, 64, 576)), dtype=torch.float32).bfloat16()
        new_keys = torch.tensor(rng.normal(size=(n_q, 128)), dtype=torch.float32).bfloat16()
        t = 0
        for s in range(n):
            cache[s] = np.concatenate([cache[s], rows[t:t + q[s]].double().numpy()])
            keys[s * cap + kv[s] - q[s]:s * cap + kv[s]] = new_keys[t:t + q[s]].to(DEV)
            t += q[s]
        slots = torch.zeros(n_q, dtype=torch.int64, device=DEV)
        b = dsa.make_batch(row_off, key_off, q_off, n_q, int(q.max()), int(kv.max()), n * cap, n * cap)
        ws = [dsa.alloc_workspace(sh, b, op) for op in
              (dsa.OP_PAGE_PLAN, dsa.OP_CACHE_APPEND, dsa.OP_INDEX_SELECT, dsa.OP_PAGED_MLA)]
        idx = torch.full((n_q, top_k), -7, dtype=torch.int32, device=DEV)
        n_sel = torch.zeros(n_q, dtype=torch.int32, device=DEV)
        out = torch.full((n_q, 64, 512), float("nan"), device=DEV)
        lse = torch.full((n_q, 64), float("nan"), device=DEV)
        lens = [i64(x) for x in (held, kv, q)]
        rows_d, q_abs_d = rows.to(DEV), q_abs.to(DEV)
        torch.cuda.synchronize()
        dsa.dsa_page_plan(pages, *lens, free, n_free, table, row_off, q_off, slots, ws[0])
        dsa.dsa_cache_append(sh, b, pages, rows_d, slots, codes, scales, ws[1])
        dsa.dsa_index_select(sh, b, q_idx, w, keys, idx, n_sel, ws[2])
        dsa.dsa_paged_mla_attn(sh, b, pages, q_abs_d, codes, scales, table, idx, n_sel, out, lse, ws[3])
        assert [dsa.dsa_check_device_error(x) for x in ws] == [0, 0, 0, 0]
        held = kv
        tab, pool = host(table), ref.widen(host(codes), host(scales), fmt)
        sel, cnt, o, l = host(idx), host(n_sel), host(out), host(lse)
        t = 0
        for s in range(n):
            pos = np.arange(kv[s])
            got = pool[tab[s][pos // page], pos % page] if kv[s] else np.zeros((0, 576))
            # a value is off by half a step (e4m3: 2^-4 of it, or 2^-10 of the scale below the normal
            # codes; integers: half the scale), and once more for each further exponent its page
            # had, each time by half a step of a scale at least twice the last: less than twice the
            # last half step in all.  A scale is at most twice the largest value over 448 or 127.
            if kv[s]:
                big = np.abs(cache[s]).max()
                half = 2.0 ** -4 * np.abs(cache[s]) + 2.0 ** -10 * big / 224 if fmt == "e4m3" \
                    else 0.5 * big / 63.5
                assert np.all(np.abs(got - cache[s]) <= 2 * half + 1e-12)
            for i in range(q[s]):
                L = kv[s] - q[s] + i + 1
                at = sel[t, :cnt[t]]
                assert cnt[t] == min(L, top_k) and (np.diff(at) > 0).all() and at.max() < L
                unit = np.exp2(host(scales)[tab[s][pos // page], 0].astype(np.float64) - 127)
                want, want_l, weight, reach, floor = ref.attention(q_abs[t].double().numpy(), got, at,
                                                                   SCALE, unit)
                tol, tol_l = ref.attention_bounds("bf16", 576, cnt[t], weight, reach, want_l, floor)
                assert np.all(np.abs(o[t] - want) <= tol) and np.all(np.abs(l[t] - want_l) <= tol_l)
                t += 1
