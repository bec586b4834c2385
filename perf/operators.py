"""Cases of the paged 8-bit cache operators: plain forms, calls, sizes and 64-bit values.

Three operators: the page plan (block tables, slot maps and offsets from
request lengths), the cache append (new rows rounded to 8 bits with a
power-of-two scale per page and part of a row) and the absorbed-MLA attention
that reads such a cache through the block table.

A row has W = 512 + rope columns; its parts are the latent (512 columns) and,
with rope, the 64-wide tail.  A page holds ``page`` rows and, per part, one
E8M0 byte b standing for 2^(b - 127).
"""
import math

import torch

own = False

HEADS, LATENT, SCALE = 64, 512, 1.0 / 16.0
E_MIN, E_MAX = -110, 119                      # exponents a page's scale may take
DEV = "cuda"


def listed():
    return [
        # one decode step's tables for the 64 ragged sequences of the decode benchmark
        {"name": "plan_decode_64", "op": "plan", "n_seq": 64, "page": 64, "longest": 131072,
         "chunk": 1, "mix": False},
        # a busy server's step: 1021 requests, most decoding, some with a chunk of prompt,
        # some finished (their pages come back), some rolled back by a few tokens
        {"name": "plan_mixed_1021", "op": "plan", "n_seq": 1021, "page": 32, "longest": 16384,
         "chunk": 512, "mix": True},
        # prompts being admitted: 250 chunks of up to 4096 tokens
        {"name": "plan_prompts_250", "op": "plan", "n_seq": 250, "page": 64, "longest": 8192,
         "chunk": 4096, "mix": False},
        # the rows of one decode step, one per sequence, into partly filled pages
        {"name": "append_decode_64", "op": "append", "n_seq": 64, "page": 64, "longest": 8192,
         "chunk": 1, "rope": 64, "dtype": "bf16", "format": "e4m3"},
        # a prefill chunk of one long sequence
        {"name": "append_chunk_4096", "op": "append", "n_seq": 1, "page": 64, "longest": 65553,
         "chunk": 4096, "rope": 64, "dtype": "bf16", "format": "e4m3"},
        # float32 rows of many ragged prompts at once, no rope tail, 8-bit integers
        {"name": "append_prompts_f32", "op": "append", "n_seq": 61, "page": 32, "longest": 4000,
         "chunk": 4000, "rope": 0, "dtype": "f32", "format": "s8"},
        # the small parity workload: one float32 query, 256 of 4096 rows
        {"name": "attn_tiny_f32", "op": "attn", "n_seq": 1, "page": 16, "shortest": 4096,
         "longest": 4096, "queries": 1, "rope": 64, "top_k": 256, "tail": 0, "dtype": "f32",
         "format": "e4m3", "dense": False},
        # batch-1 decode at 128K: 2048 selected rows
        {"name": "attn_decode_128k", "op": "attn", "n_seq": 1, "page": 64, "shortest": 131072,
         "longest": 131072, "queries": 1, "rope": 64, "top_k": 2048, "tail": 0, "dtype": "bf16",
         "format": "e4m3", "dense": False},
        # 64 ragged decode sequences
        {"name": "attn_ragged_64", "op": "attn", "n_seq": 64, "page": 64, "shortest": 8192,
         "longest": 131072, "queries": 1, "rope": 64, "top_k": 2048, "tail": 0, "dtype": "bf16",
         "format": "e4m3", "dense": False},
        # four 1M-token decodes without rope, 512 pools of 4 rows and a tail of up to 3
        {"name": "attn_nope_1m_s8", "op": "attn", "n_seq": 4, "page": 64, "shortest": 1048573,
         "longest": 1048576, "queries": 1, "rope": 0, "top_k": 2048, "tail": 3, "dtype": "bf16",
         "format": "s8", "dense": False},
        # a prefill chunk: 1024 queries over one 64K sequence
        {"name": "attn_chunk_1024", "op": "attn", "n_seq": 1, "page": 64, "shortest": 65536,
         "longest": 65536, "queries": 1024, "rope": 64, "top_k": 2048, "tail": 0, "dtype": "bf16",
         "format": "e4m3", "dense": False},
        # the dense switch: every visible row of eight long sequences
        {"name": "attn_dense_8", "op": "attn", "n_seq": 8, "page": 64, "shortest": 20000,
         "longest": 100003, "queries": 1, "rope": 64, "top_k": 2048, "tail": 0, "dtype": "bf16",
         "format": "e4m3", "dense": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        n = _log(rng, 1, 1500)
        return {"op": op, "n_seq": n, "page": page, "longest": _log(rng, 64, max(64, min(131072, (1 << 24) // n))),
                "chunk": _log(rng, 1, max(1, min(4096, 500000 // n))), "mix": rng.random() < 0.5}
    kind = {"page": page, "rope": rng.choice([64, 64, 0]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "format": rng.choice(["e4m3", "s8"])}
    if op == "append":
        n = _log(rng, 1, 300)
        chunk = _log(rng, 1, max(1, min(8192, 120000 // n)))
        return {"op": op, "n_seq": n, "longest": chunk + _log(rng, 1, 4000), "chunk": chunk, **kind}
    if kind["dtype"] == "f32":
        n, queries = _log(rng, 1, 12), 1
    else:
        n = _log(rng, 1, 80)
        queries = rng.choice([1, 1, _log(rng, 1, max(1, 700 // n))])
    dense = rng.random() < 0.2
    longest = queries + _log(rng, 1, 8000 if dense else 60000)
    if dense and queries > 4:
        longest = queries + 500
    return {"op": op, "n_seq": n, "shortest": queries + longest // 8, "longest": max(longest, queries + longest // 8),
            "queries": queries, "top_k": rng.choice([64, 256, 1024, 2048]), "tail": rng.choice([0, 3]),
            "dense": dense, **kind}


# ------------------------------------------------------------------ inputs

def _lengths(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int64)


def _prefix(x):
    return torch.cat([x.new_zeros(1), torch.cumsum(x, 0)])


def _parts(rope):
    return [(0, LATENT)] + ([(LATENT, LATENT + rope)] if rope else [])


def _pool(g, n_pages, page, rope, fmt, chunk=1 << 14):
    """A pool of pages filled as the append fills them: normal rows, each page
    of its own spread, rounded with the page's power-of-two scale."""
    W = LATENT + rope
    codes = torch.empty((n_pages, page, W), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n_pages, len(_parts(rope))), dtype=torch.uint8, device=DEV)
    top = 448.0 if fmt == "e4m3" else 127.0
    for p0 in range(0, n_pages, chunk):
        p1 = min(n_pages, p0 + chunk)
        x = torch.randn((p1 - p0, page, W), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((p1 - p0, 1, 1), generator=g, device=DEV))
        if rope:
            x[..., LATENT:] *= 3.0
        for i, (a, b) in enumerate(_parts(rope)):
            m, k = torch.frexp(x[..., a:b].abs().amax((1, 2)) / top)
            e = k - (m == 0.5).int()
            scales[p0:p1, i] = (e + 127).to(torch.uint8)
            y = x[..., a:b] * torch.exp2(-e.float())[:, None, None]
            codes[p0:p1, :, a:b] = _encode(y, fmt)
    return codes, scales


def _encode(y, fmt):
    if fmt == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _decode(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _table(g, need, ld, n_pages):
    """Block table whose row s holds need[s] pages of a shuffled pool, and the
    pages left over."""
    perm = torch.randperm(n_pages, generator=g, device=DEV).int()
    col = torch.arange(ld, device=DEV)
    rank = (_prefix(need)[:-1])[:, None] + col
    table = torch.where(col < need[:, None], perm[rank.clamp(max=n_pages - 1)], -1).int()
    return table, perm[int(need.sum()):]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    n, P = case["n_seq"], case["page"]
    if case["op"] == "plan":
        # the same lengths of new tokens for every seed, in another order: what is put out keeps its size
        order = torch.randperm(n, generator=g, device=DEV)
        q = (1 + torch.arange(n, device=DEV) * (case["chunk"] - 1) // max(n - 1, 1))[order]
        held = _lengths(g, 0, case["longest"], n)
        kv = held + q
        if case["mix"]:
            kind = order * 7 % 16
            q = torch.where(kind < 10, 1, q)                             # decoding
            kv = held + q
            back = torch.clamp(held - 5, min=0)
            kv = torch.where(kind == 14, back + q, kv)                   # rolled back, then more
            q = torch.where(kind == 15, 0, q)                            # finished
            kv = torch.where(kind == 15, 0, kv)
        need_max = (case["longest"] + case["chunk"]) // P + 2
        n_pages = n * need_max
        table, rest = _table(g, (held + P - 1) // P, need_max, n_pages)
        free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        free[:rest.numel()] = rest
        max_new = int(q.sum()) + 3
        s.update(held=held, kv=kv, q=q, table=table, free=free, ld=need_max, n_pages=n_pages,
                 n_free=torch.tensor([rest.numel()], dtype=torch.int32, device=DEV),
                 max_new=max_new, row_off=torch.zeros(n + 1, dtype=torch.int64, device=DEV),
                 q_off=torch.zeros(n + 1, dtype=torch.int64, device=DEV),
                 slots=torch.zeros(max_new, dtype=torch.int64, device=DEV),
                 n_free_out=torch.zeros(1, dtype=torch.int32, device=DEV))
    elif case["op"] == "append":
        q = _lengths(g, max(1, case["chunk"] // 2), case["chunk"], n) if n > 1 else \
            torch.full((1,), case["chunk"], dtype=torch.int64, device=DEV)
        kv = torch.maximum(_lengths(g, (case["longest"] + 1) // 2, case["longest"], n), q) if n > 1 \
            else torch.full((1,), case["longest"], dtype=torch.int64, device=DEV)
        # only the pages that the step touches exist in this pool, and one that no row uses
        first = (kv - q) // P
        need = (kv + P - 1) // P - first
        n_pages = n * ((case["chunk"] + P - 2) // P + 1) + 1
        perm = torch.randperm(n_pages - 1, generator=g, device=DEV)
        row_off, q_off = _prefix(kv), _prefix(q)
        n_tok = int(q_off[-1])
        i = torch.arange(n_tok, device=DEV)
        seq = torch.searchsorted(q_off[1:], i, right=True)
        pos = (kv - q)[seq] + i - q_off[seq]
        slots = perm[_prefix(need)[:-1][seq] + pos // P - first[seq]] * P + pos % P
        W = LATENT + case["rope"]
        rows = torch.randn((n_tok, W), generator=g, device=DEV)
        rows *= torch.exp(0.3 * torch.randn((n_tok, 1), generator=g, device=DEV))
        codes, scales = _pool(g, n_pages, P, case["rope"], case["format"])
        s.update(kv=kv, q=q, row_off=row_off, q_off=q_off, slots=slots, n_pages=n_pages, n_tok=n_tok,
                 max_q=int(q.max()), max_kv=int(kv.max()), codes=codes, scales=scales,
                 rows=rows.bfloat16() if case["dtype"] == "bf16" else rows)
    else:
        ql = case["queries"]
        kv = _lengths(g, case["shortest"], case["longest"], n)
        need = (kv + P - 1) // P
        n_pages, ld = int(need.sum()), int(need.max())
        table, _ = _table(g, need, ld, n_pages)
        codes, scales = _pool(g, n_pages, P, case["rope"], case["format"])
        n_q, W, k = n * ql, LATENT + case["rope"], case["top_k"]
        seq = torch.arange(n_q, device=DEV) // ql
        L = kv[seq] - ql + 1 + torch.arange(n_q, device=DEV) % ql
        qa = torch.randn((n_q, HEADS, W), generator=g, device=DEV)
        s.update(kv=kv, seq=seq, L=L, table=table, codes=codes, scales=scales, n_pages=n_pages, ld=ld,
                 n_q=n_q, q_abs=qa.bfloat16() if case["dtype"] == "bf16" else qa,
                 row_off=_prefix(kv), q_off=torch.arange(n + 1, device=DEV) * ql,
                 rows_in_all=int(kv.sum()), max_kv=int(kv.max()))
        if not case["dense"]:
            # as a selection leaves it: every visible row up to top_k + tail of them, else top_k rows
            # spread over the sequence and the last `tail` rows, ascending, -1 behind
            width = k + case["tail"]
            j = torch.arange(k, device=DEV)
            body = (L - case["tail"])[:, None]
            lo, hi = j * body // k, (j + 1) * body // k
            u = torch.rand((n_q, k), generator=g, device=DEV)
            picked = lo + (u * (hi - lo)).long().clamp(max=(hi - lo - 1).clamp(min=0))
            picked = torch.cat([picked, body + torch.arange(case["tail"], device=DEV)], 1)
            every = torch.arange(width, device=DEV).expand(n_q, width)
            few = (L <= width)[:, None]
            idx = torch.where(few, torch.where(every < L[:, None], every, -1), picked)
            s.update(idx=idx.int().contiguous(), n_sel=torch.where(L <= width, L, width).int())
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the framework keeps beside its tensors: descriptors, workspace, outputs."""
    import deepseek_sparse_attention_gb300 as dsa

    fmt = dsa.CACHE_E4M3 if s.get("format") != "s8" else dsa.CACHE_S8
    kpool = s.get("tail", 0) + 1
    key_off = _prefix(s["kv"] // kpool)
    if s["op"] == "plan":
        sh = dsa.make_shape()
        b = dsa.make_batch(s["row_off"], key_off, s["q_off"], s["max_new"], s["max_new"], 1 << 30, 1 << 30, 0)
        s["pages"] = dsa.make_pages(s["page"], s["n_pages"], s["ld"], fmt)
        s["ws"] = dsa.alloc_workspace(sh, b, dsa.OP_PAGE_PLAN)
        return
    if s["op"] == "append":
        sh = dsa.make_shape(rope_dim=s["rope"], dtype=s["dtype"])
        b = dsa.make_batch(s["row_off"], key_off, s["q_off"], s["n_tok"], s["max_q"], s["max_kv"],
                           int(s["row_off"][-1]), int(key_off[-1]))
        s["pages"] = dsa.make_pages(s["page"], s["n_pages"], 1, fmt)
        s["ws"] = dsa.alloc_workspace(sh, b, dsa.OP_CACHE_APPEND)
    else:
        # a k-pool shape has a selection row of top_k + kpool - 1 entries
        sh = dsa.make_shape(rope_dim=s["rope"], dtype=s["dtype"], top_k=s["top_k"], kpool=kpool,
                            scale=SCALE)
        b = dsa.make_batch(s["row_off"], key_off, s["q_off"], s["n_q"], s["queries"], s["max_kv"],
                           s["rows_in_all"], int(key_off[-1]), dsa.FLAG_DENSE if s["dense"] else 0)
        s["pages"] = dsa.make_pages(s["page"], s["n_pages"], s["ld"], fmt)
        s["ws"] = dsa.alloc_workspace(sh, b, dsa.OP_PAGED_MLA)
        s["out"] = torch.empty((s["n_q"], HEADS, LATENT), device=DEV)
        s["lse"] = torch.empty((s["n_q"], HEADS), device=DEV)
    s["shape"], s["batch"] = sh, b


# ------------------------------------------------------------------ the operators

def run(s):
    if own:
        return {"plan": _own_plan, "append": _own_append, "attn": _own_attn}[s["op"]](s)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)


def _own_plan(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_page_plan(s["pages"], s["held"], s["kv"], s["q"], s["free"], s["n_free"], s["table"],
                      s["row_off"], s["q_off"], s["slots"], s["ws"], n_free_out=s["n_free_out"])
    return {"table": s["table"], "free": s["free"], "n_free": s["n_free_out"], "row_off": s["row_off"],
            "q_off": s["q_off"], "slots": s["slots"]}


def _plain_plan(s):
    P, table, free, F = s["page"], s["table"], s["free"], s["n_free"].long()
    held, need = (s["held"] + P - 1) // P, (s["kv"] + P - 1) // P
    grow, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    A, R = grow.sum(), back.sum()
    enough = A <= F + R                       # else no page moves and no token has a slot
    col = torch.arange(s["ld"], device=DEV)
    # released pages go on the stack in the order of (sequence, column)
    rank = (torch.cumsum(back, 0) - back)[:, None] + col - need[:, None]
    given = (col >= need[:, None]) & (col < held[:, None]) & enough
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(given, F + rank, s["n_pages"]).reshape(-1), table.reshape(-1))
    # then every row that grows takes its pages from the top
    rank = (torch.cumsum(grow, 0) - grow)[:, None] + col - held[:, None]
    taken = (col >= held[:, None]) & (col < need[:, None]) & enough
    table = torch.where(taken, stack[(F + R - 1 - rank).clamp(0, s["n_pages"])], table)
    n_free = torch.where(enough, F + R - A, F)
    k = torch.arange(s["n_pages"], device=DEV)
    free = torch.where((k >= F) & (k < n_free), stack[:-1], free)
    row_off, q_off = _prefix(s["kv"]), _prefix(s["q"])
    i = torch.arange(s["max_new"], device=DEV)
    seq = torch.searchsorted(q_off[1:], i, right=True).clamp(max=s["n_seq"] - 1)
    pos = (s["kv"] - s["q"])[seq] + i - q_off[seq]
    page = table[seq, (pos // P).clamp(0, s["ld"] - 1)].long()
    slots = torch.where((i < q_off[-1]) & (page >= 0) & enough, page * P + pos % P, -1)
    return {"table": table, "free": free, "n_free": n_free.int(), "row_off": row_off, "q_off": q_off,
            "slots": slots}


def _codes_out(s):
    # e4m3 codes are values; s8 codes are whole numbers
    return {"codes": s["codes"].view(torch.float8_e4m3fn if s["format"] == "e4m3" else torch.int8),
            "scales": s["scales"]}


def _own_append(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_cache_append(s["shape"], s["batch"], s["pages"], s["rows"], s["slots"], s["codes"],
                         s["scales"], s["ws"])
    return _codes_out(s)


def _plain_append(s):
    P, fmt, n = s["page"], s["format"], s["n_seq"]
    mant, shift = (0x600000, 8) if fmt == "e4m3" else (0x7E0000, 6)     # 448 = 1.75 2^8, 127 = 1.984375 2^6
    base = s["row_off"][1:] - s["row_off"][:-1] - (s["q_off"][1:] - s["q_off"][:-1])
    kv = s["row_off"][1:] - s["row_off"][:-1]
    pg = (base // P)[:, None] + torch.arange((s["max_q"] + P - 2) // P + 1, device=DEV)   # [n, C]
    lo, hi = torch.maximum(base[:, None], pg * P), torch.minimum(kv[:, None], (pg + 1) * P)
    live = lo < hi
    first = s["slots"][(s["q_off"][:-1, None] + lo - base[:, None]).clamp(0, s["n_tok"] - 1)]
    page = torch.where(live, first // P, s["n_pages"] - 1).reshape(-1)   # no unit: the unused page as it is
    pos = pg[..., None] * P + torch.arange(P, device=DEV)               # [n, C, P]
    new = (live[..., None] & (pos >= lo[..., None]) & (pos < hi[..., None])).reshape(-1, P, 1)
    tok = (s["q_off"][:-1, None, None] + pos - base[:, None, None]).clamp(0, s["n_tok"] - 1)
    x = s["rows"][tok.reshape(-1, P)].float()                           # [n C, P, W]
    old = s["codes"][page]
    fresh = (lo % P == 0).reshape(-1)
    out, sc = old.clone(), s["scales"][page]
    for i, (a, b) in enumerate(_parts(s["rope"])):
        amax = torch.where(new, x[..., a:b].abs(), 0.0).amax((1, 2))
        bits = amax.view(torch.int32)
        e = ((bits >> 23) - 127 - shift + ((bits & 0x7FFFFF) > mant).int()).clamp(E_MIN, E_MAX)
        e_old = sc[:, i].int() - 127
        e = torch.where(fresh, e, torch.maximum(e, e_old))
        e = torch.where(live.reshape(-1), e, e_old)
        moved = _encode(_decode(old[..., a:b], fmt) * torch.exp2((e_old - e).float())[:, None, None], fmt)
        coded = _encode(x[..., a:b] * torch.exp2(-e.float())[:, None, None], fmt)
        behind = (pos >= hi[..., None]).reshape(-1, P, 1)
        out[..., a:b] = torch.where(new, coded, torch.where(behind, old[..., a:b], moved))
        sc[:, i] = (e + 127).to(torch.uint8)
    s["codes"][page] = out
    s["scales"][page] = sc
    return _codes_out(s)


def _own_attn(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_paged_mla_attn(s["shape"], s["batch"], s["pages"], s["q_abs"], s["codes"], s["scales"],
                           s["table"], s.get("idx"), s.get("n_sel"), s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attn(s):
    P = s["page"]
    if s["dense"]:
        pos = torch.arange(s["max_kv"], device=DEV).expand(s["n_q"], s["max_kv"])
        keep = pos < s["L"][:, None]
    else:
        pos = s["idx"].long()
        keep = torch.arange(pos.shape[1], device=DEV) < s["n_sel"][:, None]
    pos = torch.where(keep, pos, 0)
    page = s["table"][s["seq"][:, None], pos // P].long()
    row = _decode(s["codes"][page, pos % P], s["format"])                # [n_q, K, W]
    sc = torch.exp2(s["scales"].float() - 127.0)[page]
    for i, (a, b) in enumerate(_parts(s["rope"])):
        row[..., a:b] *= sc[..., i:i + 1]
    z = torch.matmul(s["q_abs"].float(), row.transpose(1, 2)) * SCALE    # [n_q, 64, K]
    z = torch.where(keep[:, None, :], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, row[..., :LATENT]) / total
    return {"out": out, "lse": (m + torch.log(total))[..., 0]}


# ------------------------------------------------------------------ work and 64-bit values

def _expected(case):
    """Sequence lengths a case has on average, for its bytes."""
    if case["op"] == "attn":
        return (case["shortest"] + case["longest"]) / 2
    return case["longest"] if case["n_seq"] == 1 else case["longest"] * 3 / 4


def work(case):
    n, P = case["n_seq"], case["page"]
    if case["op"] == "plan":
        q = (1 + case["chunk"]) / 2
        if case["mix"]:
            q = 10 / 16 + q * 5 / 16
        pages = n * max(q / P, 1 / P)                      # pages taken, each read and written
        return {"bytes": n * (3 * 8 + 2 * 8) + pages * 8 + n * q * 8 + n * (q / P + 1) * 4, "flops": 0}
    W = LATENT + case["rope"]
    esize = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        tok = case["chunk"] if n == 1 else n * 0.75 * case["chunk"]
        return {"bytes": tok * (W * (esize + 1) + 8) + n * 32, "flops": tok * W * 3}
    n_q, L = n * case["queries"], _expected(case)
    rows = L if case["dense"] else min(L, case["top_k"] + case["tail"])
    # a sequence's queries share its rows: no row need be read more often than once
    unique = n * min(L, rows * case["queries"])
    return {"bytes": unique * W + n_q * HEADS * (W * esize + LATENT * 4 + 4) + (0 if case["dense"] else n_q * rows * 4),
            "flops": n_q * rows * HEADS * 2 * (W + LATENT)}


def exact(case, seed):
    if case["op"] == "plan" or (case["op"] == "append" and case["format"] == "s8"):
        return None                                        # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        return {"codes": _exact_codes(s), "scales": None}
    n_q = s["n_q"]
    out = torch.zeros((n_q, HEADS, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.full((n_q, HEADS), -math.inf, dtype=torch.float64, device=DEV)
    table = s["table"].cpu()
    for i in range(n_q):                                   # one query after the other
        at = torch.arange(int(s["L"][i])) if case["dense"] else s["idx"][i, :int(s["n_sel"][i])].long().cpu()
        page = table[int(s["seq"][i])][at // case["page"]].to(DEV).long()
        c = s["codes"][page, (at % case["page"]).to(DEV)]
        c = c.view(torch.float8_e4m3fn if case["format"] == "e4m3" else torch.int8).to(torch.float32).double()
        f = torch.pow(2.0, s["scales"][page].double() - 127)
        c[:, :LATENT] *= f[:, :1]
        c[:, LATENT:] *= f[:, 1:]                          # no columns without a rope tail
        z = (s["q_abs"][i].double() @ c.T) * SCALE
        lse[i] = torch.logsumexp(z, 1)
        out[i] = torch.exp(z - lse[i][:, None]) @ c[:, :LATENT]
    return {"out": out, "lse": lse}


def _exact_codes(s):
    """The append's codes before their rounding: x / 2^e, sequence by sequence."""
    P, slots = s["page"], s["slots"].cpu()
    q_off, kv, q = s["q_off"].tolist(), s["kv"].tolist(), s["q"].tolist()
    pool = s["codes"].view(torch.float8_e4m3fn).to(torch.float32).double()
    rows, e_byte = s["rows"].double(), s["scales"].double()
    for n in range(s["n_seq"]):
        t = 0
        while t < q[n]:
            pos = kv[n] - q[n] + t
            end = min(q[n], t + P - pos % P)
            page, off = int(slots[q_off[n] + t]) // P, pos % P
            new = rows[q_off[n] + t:q_off[n] + end]
            for i, (a, b) in enumerate(_parts(s["rope"])):
                ratio = float(new[:, a:b].abs().max()) / 448.0
                m, k = math.frexp(ratio)
                e = min(max((k - (m == 0.5)) if ratio > 0 else E_MIN, E_MIN), E_MAX)
                before = float(e_byte[page, i]) - 127
                if off > 0:
                    e = max(e, before)
                    pool[page, :off, a:b] *= 2.0 ** (before - e)
                pool[page, off:off + end - t, a:b] = new[:, a:b] / 2.0 ** e
            t = end
    return pool
