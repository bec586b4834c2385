"""Cases of the operators around the expanded latent attention: plain forms, calls, sizes, 64-bit values.

Four operators: the root-mean-square norm with the residual's addition and an
output in 8 bits with scales, the rotary embedding of part of a head, the
expansion of latent rows into each head's keys and values, and the causal
attention over those expanded keys and values.
"""
import math

import torch

own = False

HEADS, LATENT, NOPE, ROPE, V_DIM, SCALE = 64, 512, 192, 64, 256, 1.0 / 16.0
EPS, TOP, LEAST = 1e-5, 448.0, 2.0 ** -126    # e4m3's largest value, the least scale
DEV = "cuda"


def listed():
    return [
        # one decode step's latent columns of the projected cache rows, 64 sequences
        {"name": "norm_latent_64", "op": "norm", "rows": 64, "width": LATENT, "ld": LATENT + ROPE,
         "dtype": "bf16", "add": False, "out": "same", "group": 0},
        # the hidden states of a prefill chunk and their residual, for an 8-bit product
        {"name": "norm_chunk_e4m3", "op": "norm", "rows": 4096, "width": 8192, "ld": 8192,
         "dtype": "bf16", "add": True, "out": "e4m3", "group": 128},
        # float32 rows of an odd width, as a small model has them
        {"name": "norm_odd_f32", "op": "norm", "rows": 3001, "width": 1001, "ld": 1003,
         "dtype": "f32", "add": True, "out": "same", "group": 0},
        # the queries of 64 decode sequences: the last 64 columns of heads of 256
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "heads": HEADS, "dims": ROPE,
         "before": NOPE, "dtype": "bf16", "halves": False, "factor": 1.0, "longest": 131072},
        # the queries of a prefill chunk, positions stretched to eight times the trained context
        {"name": "rope_chunk_4096", "op": "rope", "tokens": 4096, "heads": HEADS, "dims": ROPE,
         "before": NOPE, "dtype": "bf16", "halves": False, "factor": 8.0, "longest": 1048576},
        # the shared keys of a long prompt: the tail of float32 cache rows, half layout
        {"name": "rope_rows_f32", "op": "rope", "tokens": 131071, "heads": 1, "dims": ROPE,
         "before": LATENT, "dtype": "f32", "halves": True, "factor": 1.0, "longest": 131072},
        # the latent rows of a prefill chunk into every head's keys and values
        {"name": "expand_chunk_4096", "op": "expand", "rows": 4096, "rope": ROPE, "nope": NOPE,
         "v_dim": V_DIM, "dtype": "bf16"},
        # a short prompt of the float32 parity shape
        {"name": "expand_f32_300", "op": "expand", "rows": 300, "rope": ROPE, "nope": NOPE,
         "v_dim": V_DIM, "dtype": "f32"},
        # a prompt of 4096 tokens
        {"name": "attn_prompt_4096", "op": "attn", "n_seq": 1, "queries": 4096, "before": 0,
         "rope": ROPE, "nope": NOPE, "v_dim": V_DIM, "dtype": "bf16"},
        # prompts of all lengths up to 1,100 admitted together
        {"name": "attn_ragged_13", "op": "attn", "n_seq": 13, "queries": 1100, "before": 0,
         "rope": ROPE, "nope": NOPE, "v_dim": V_DIM, "dtype": "bf16"},
        # one more turn of a conversation: 300 new tokens behind 16,000
        {"name": "attn_turn_300", "op": "attn", "n_seq": 1, "queries": 300, "before": 16000,
         "rope": ROPE, "nope": NOPE, "v_dim": V_DIM, "dtype": "bf16"},
        # float32 prompts of the parity shape
        {"name": "attn_f32_3", "op": "attn", "n_seq": 3, "queries": 257, "before": 100,
         "rope": ROPE, "nope": NOPE, "v_dim": V_DIM, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "expand", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        width = rng.choice([LATENT, 1024, 2048, 4096, 8192, 16384, _log(rng, 1, 16384)])
        out, most = rng.choice(["same", "e4m3"]), (28 << 20) if dtype == "bf16" else 14 << 20
        return {"op": op, "rows": _log(rng, 1, max(1, min(131072, most // width))), "width": width,
                "ld": width + rng.choice([0, 0, 3, 64]), "dtype": dtype, "add": rng.random() < 0.5,
                "out": out, "group": rng.choice([0, 32, 64, 128]) if out == "e4m3" else 0}
    if op == "rope":
        heads, dims = rng.choice([1, 1, 3, 32, HEADS]), rng.choice([2, 6, 32, ROPE, ROPE, 128, 256])
        most = ((1 << 24) if dtype == "bf16" else 1 << 23) // (max(heads, 2) * dims)
        return {"op": op, "tokens": _log(rng, 1, max(1, min(300000, most))), "heads": heads, "dims": dims,
                "before": rng.choice([0, 1, NOPE, LATENT]), "dtype": dtype,
                "halves": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 40.0]),
                "longest": rng.choice([4096, 131072, 1048576])}
    kind = {"rope": rng.choice([ROPE, ROPE, 0]), "nope": rng.choice([64, 128, NOPE]),
            "v_dim": rng.choice([128, V_DIM]), "dtype": dtype}
    if op == "expand":
        return {"op": op, "rows": _log(rng, 1, 4096 if dtype == "bf16" else 700), **kind}
    n = _log(rng, 1, 40)
    most = (1 << 24) if dtype == "bf16" else 1 << 20     # of query-key pairs, padded
    queries = rng.choice([1, _log(rng, 1, max(1, min(3000, int(math.sqrt(most // n)))))])
    before = rng.choice([0, _log(rng, 1, max(1, min(32768 // n, most // (n * queries)) - queries))])
    return {"op": op, "n_seq": n, "queries": queries, "before": before, **kind}


# ------------------------------------------------------------------ inputs

def _prefix(x):
    return torch.cat([x.new_zeros(1), torch.cumsum(x, 0)])


def _typed(x, case):
    return x.bfloat16() if case["dtype"] == "bf16" else x


def _lengths(case):
    """New tokens and earlier rows of each sequence: spread from few to the most, the same for every seed."""
    n, q, b = case["n_seq"], case["queries"], case["before"]
    if n == 1:
        return [q], [b]
    return [1 + i * (q - 1) // (n - 1) for i in range(n)], [(n - 1 - i) * b // (n - 1) for i in range(n)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)          # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        rows, width, ld = case["rows"], case["width"], case["ld"]
        x = normal(rows, ld)
        x *= torch.exp(0.5 * normal(rows, 1))                       # rows of different sizes
        s["x"] = _typed(x, case)[:, :width]
        s["weight"] = 1.0 + 0.2 * normal(width)
        if case["add"]:
            s["add_in"] = _typed(2.0 * normal(rows, ld), case)[:, :width]
    elif case["op"] == "rope":
        n, heads, dims, before = case["tokens"], case["heads"], case["dims"], case["before"]
        s["x"] = _typed(normal(n, heads, before + dims), case)[..., before:]
        s["pos"] = torch.randint(0, case["longest"], (n,), generator=g, device=DEV, dtype=torch.int64)
        s["rates"] = torch.tensor(_rates(case), dtype=torch.float64, device=DEV)
    elif case["op"] == "expand":
        s["cache"] = _typed(normal(case["rows"], LATENT + case["rope"]), case)
        s["w_uk"] = _typed(normal(HEADS, case["nope"], LATENT) / math.sqrt(LATENT), case)
        s["w_uv"] = _typed(normal(HEADS, case["v_dim"], LATENT) / math.sqrt(LATENT), case)
    else:
        q_len, before = _lengths(case)
        order = torch.randperm(case["n_seq"], generator=g, device=DEV)
        q_len = torch.tensor(q_len, device=DEV)[order]
        kv_len = q_len + torch.tensor(before, device=DEV)[order]
        s["q_off"], s["row_off"] = _prefix(q_len), _prefix(kv_len)
        s["n_q"], s["rows"] = int(q_len.sum()), int(kv_len.sum())
        s["max_q"], s["max_kv"] = int(q_len.max()), int(kv_len.max())
        s["q"] = _typed(normal(s["n_q"], HEADS, case["nope"] + case["rope"]), case)
        s["k_nope"] = _typed(normal(s["rows"], HEADS, case["nope"]), case)
        s["cache"] = _typed(normal(s["rows"], LATENT + case["rope"]), case)
        s["v"] = _typed(normal(s["rows"], HEADS, case["v_dim"]), case)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the framework keeps beside its tensors: descriptors, workspace, outputs."""
    import deepseek_sparse_attention_gb300 as dsa

    t = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    if s["op"] == "norm":
        rows, width = s["rows"], s["width"]
        if s["out"] == "e4m3":
            s["y"] = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device=DEV)
            s["scales"] = torch.empty((rows, -(-width // (s["group"] or width))), device=DEV)
        else:
            s["y"] = torch.empty((rows, s["ld"]), dtype=t, device=DEV)[:, :width]
        if s["add"]:
            s["total"] = torch.empty((rows, s["ld"]), dtype=t, device=DEV)[:, :width]
    elif s["op"] == "rope":
        s["rope"] = dsa.make_rope(s["dims"], 8e6, layout="halves" if s["halves"] else "pairs",
                                  factor=s["factor"], original_len=s["longest"] / s["factor"])
        whole = torch.empty((s["tokens"], s["heads"], s["before"] + s["dims"]), dtype=t, device=DEV)
        s["y"] = whole[..., s["before"]:]
    elif s["op"] == "expand":
        s["shape"] = dsa.make_shape(rope_dim=s["rope"], dtype=s["dtype"], scale=SCALE)
        zero = torch.zeros(2, dtype=torch.int64, device=DEV)
        batch = dsa.make_batch(zero, zero, zero, 0, 0, 0, s["rows"], s["rows"])
        s["ws"] = dsa.alloc_workspace(s["shape"], batch, dsa.OP_PROJECT)
        s["k_nope"] = torch.empty((s["rows"], HEADS, s["nope"]), dtype=t, device=DEV)
        s["v"] = torch.empty((s["rows"], HEADS, s["v_dim"]), dtype=t, device=DEV)
    else:
        s["shape"] = dsa.make_shape(rope_dim=s["rope"], dtype=s["dtype"], scale=SCALE)
        s["batch"] = dsa.make_batch(s["row_off"], s["row_off"], s["q_off"], s["n_q"], s["max_q"], s["max_kv"],
                                    s["rows"], s["rows"])
        s["ws"] = dsa.alloc_workspace(s["shape"], s["batch"], dsa.OP_EXPANDED_MLA)
        s["out"] = torch.empty((s["n_q"], HEADS, s["v_dim"]), dtype=t, device=DEV)
        s["lse"] = torch.empty((s["n_q"], HEADS), device=DEV)


# ------------------------------------------------------------------ the operators

def run(s):
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "expand": _own_expand, "attn": _own_attn}[s["op"]](s)
    return {"norm": _plain_norm, "rope": _plain_rope, "expand": _plain_expand, "attn": _plain_attn}[s["op"]](s)


def _own_norm(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_rms_norm(s["x"], s["weight"], EPS, s["y"], add=s.get("add_in"), total=s.get("total"),
                     scales=s.get("scales"), group=s["group"])
    return {"y": s["y"], "scales": s.get("scales"), "total": s.get("total")}


def _plain_norm(s):
    h = s["x"].float()
    if s["add"]:
        h = h + s["add_in"].float()
    y = h * torch.rsqrt(torch.mean(h * h, -1, keepdim=True) + EPS) * s["weight"]
    total = h.to(s["x"].dtype) if s["add"] else None
    if s["out"] != "e4m3":
        return {"y": y.to(s["x"].dtype), "scales": None, "total": total}
    rows, width, group = s["rows"], s["width"], s["group"] or s["width"]
    n = -(-width // group)
    y = torch.nn.functional.pad(y, (0, n * group - width)).view(rows, n, group)
    scales = torch.clamp(y.abs().amax(-1) / TOP, min=LEAST)
    codes = (y / scales[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return {"y": codes.view(rows, n * group)[:, :width], "scales": scales, "total": total}


def _own_rope(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_rope(s["rope"], s["x"], s["pos"], s["y"])
    return s["y"]


def _plain_rope(s):
    angle = (s["pos"].double()[:, None] * s["rates"])[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x, half = s["x"].float(), s["dims"] // 2
    if s["halves"]:
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(s["x"].dtype)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(s["x"].dtype)


def _own_expand(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_expand_kv(s["shape"], s["cache"], s["w_uk"], s["w_uv"], s["k_nope"], s["v"], s["ws"])
    return {"k_nope": s["k_nope"], "v": s["v"]}


def _plain_expand(s):
    latent = s["cache"][:, :LATENT].float()
    k = torch.matmul(latent, s["w_uk"].float().view(-1, LATENT).t()).view(-1, HEADS, s["nope"])
    v = torch.matmul(latent, s["w_uv"].float().view(-1, LATENT).t()).view(-1, HEADS, s["v_dim"])
    return {"k_nope": k.to(s["cache"].dtype), "v": v.to(s["cache"].dtype)}


def _own_attn(s):
    import deepseek_sparse_attention_gb300 as dsa

    dsa.dsa_expanded_mla_attn(s["shape"], s["batch"], s["q"], s["k_nope"], s["cache"], s["v"], s["out"],
                              s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attn(s):
    """All sequences at once, padded to the longest."""
    q_off, row_off = s["q_off"], s["row_off"]
    q_len, kv_len = q_off[1:] - q_off[:-1], row_off[1:] - row_off[:-1]
    i = torch.arange(s["max_q"], device=DEV)
    j = torch.arange(s["max_kv"], device=DEV)
    at_q = (q_off[:-1, None] + i).clamp(max=s["n_q"] - 1)                        # [n, Q]
    at_k = (row_off[:-1, None] + j).clamp(max=s["rows"] - 1)                     # [n, K]
    q = s["q"][at_q].float().transpose(1, 2)                                     # [n, 64, Q, d]
    k = s["k_nope"][at_k].float().transpose(1, 2)
    if s["rope"]:
        tail = s["cache"][:, LATENT:][at_k].float()[:, None].expand(-1, HEADS, -1, -1)
        k = torch.cat([k, tail], -1)
    sees = (kv_len - q_len + 1)[:, None] + i                                     # rows that a query sees
    keep = (j < sees[..., None])[:, None]                                        # [n, 1, Q, K]
    z = torch.matmul(q, k.transpose(2, 3)).mul_(SCALE)
    z = z.masked_fill_(~keep, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z.sub_(m))
    total = p.sum(-1, keepdim=True)
    v = s["v"][at_k].float().transpose(1, 2)
    out = (torch.matmul(p, v) / total).transpose(1, 2)                           # [n, Q, 64, v]
    lse = (m + torch.log(total))[..., 0].transpose(1, 2)
    real = i < q_len[:, None]
    return {"out": out[real].to(s["q"].dtype), "lse": lse[real]}


# ------------------------------------------------------------------ work and 64-bit values

def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        each = e + (2 * e if case["add"] else 0)                    # x; the residual and the sum
        if case["out"] == "e4m3":
            scales = case["rows"] * -(-case["width"] // (case["group"] or case["width"])) * 4
            return {"bytes": n * (each + 1) + scales + case["width"] * 4, "flops": n * 6}
        return {"bytes": n * (each + e) + case["width"] * 4, "flops": n * 5}
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dims"]
        return {"bytes": 2 * n * e + case["tokens"] * 8, "flops": 3 * n}
    wide = HEADS * (case["nope"] + case["v_dim"])
    if case["op"] == "expand":
        return {"bytes": (case["rows"] * (LATENT + wide) + wide * LATENT) * e,
                "flops": 2 * case["rows"] * wide * LATENT}
    q_len, before = _lengths(case)
    n_q, rows = sum(q_len), sum(q_len) + sum(before)
    pairs = sum(q * b + q * (q + 1) // 2 for q, b in zip(q_len, before))
    d = case["nope"] + case["rope"]
    return {"bytes": (n_q * HEADS * (d + case["v_dim"]) + rows * (wide + case["rope"])) * e + n_q * HEADS * 4,
            "flops": 2 * pairs * HEADS * (d + case["v_dim"])}


def _rates(case):
    """Radians a position of each pair; stretched contexts turn the slow pairs more slowly (32 turns or more
    over the trained context: as trained; one or fewer: divided by the factor; between: in proportion to the
    pair's place)."""
    dims, base, factor = case["dims"], 8e6, case["factor"]
    rates = [base ** (-2.0 * i / dims) for i in range(dims // 2)]
    if factor == 1.0:
        return rates
    trained = case["longest"] / factor
    place = lambda turns: dims * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))    # noqa: E731
    low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), dims - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(dims // 2)]
    return [r * ((1 - g) + g / factor) for r, g in zip(rates, ramp)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "rope":
        x = torch.complex(*_pairs(s["x"].double(), case["halves"]))
        turned = x * torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None, None] * s["rates"])
        out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
        a, b = _pairs(out, case["halves"])
        a.copy_(turned.real)
        b.copy_(turned.imag)
        return out
    if case["op"] == "expand":
        c = s["cache"][:, :LATENT].double()
        return {"k_nope": torch.einsum("ri,hdi->rhd", c, s["w_uk"].double()),
                "v": torch.einsum("ri,hdi->rhd", c, s["w_uv"].double())}
    out = torch.empty((s["n_q"], HEADS, case["v_dim"]), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["n_q"], HEADS), dtype=torch.float64, device=DEV)
    q_off, row_off = s["q_off"].tolist(), s["row_off"].tolist()
    for n in range(case["n_seq"]):                                  # one sequence and head after the other
        qs, rs = slice(q_off[n], q_off[n + 1]), slice(row_off[n], row_off[n + 1])
        n_q, n_kv = q_off[n + 1] - q_off[n], row_off[n + 1] - row_off[n]
        hidden = torch.ones((n_q, n_kv), dtype=torch.bool, device=DEV).triu_(n_kv - n_q + 1)
        for h in range(HEADS):
            key = torch.cat([s["k_nope"][rs, h], s["cache"][rs, LATENT:]], 1).double()
            z = (s["q"][qs, h].double() @ key.T * SCALE).masked_fill_(hidden, -math.inf)
            lse[qs, h] = torch.logsumexp(z, 1)
            out[qs, h] = torch.softmax(z, 1) @ s["v"][rs, h].double()
    return {"out": out, "lse": lse}


def _pairs(x, halves):
    return x.chunk(2, -1) if halves else (x[..., 0::2], x[..., 1::2])


def _exact_norm(s):
    h = s["x"].double() + (s["add_in"].double() if s["add"] else 0.0)
    y = s["weight"].double() * h / (h.square().mean(1) + EPS).sqrt()[:, None]
    total = h if s["add"] else None
    if s["out"] != "e4m3":
        return {"y": y, "scales": None, "total": total}
    group, scales = s["group"] or s["width"], []
    for at in range(0, s["width"], group):
        part = y[:, at:at + group]
        scales.append((part.abs().amax(1) / TOP).clamp(min=LEAST))
        part /= scales[-1][:, None]                                 # codes before their rounding
    return {"y": y, "scales": torch.stack(scales, 1), "total": total}
