"""GPU tests of the paged cache's operators called together and in unusual ways:
captured on a stream of their own, batches whose queries are not one to a
sequence, batches padded past their last sequence."""
import numpy as np
import pytest
import torch

import deepseek_sparse_attention_gb300 as dsa
import paged_util as ref
from test_gpu_paged import DEV, SCALE, AttnCase, _lib, dev, host, i64, prefix  # noqa: F401 (_lib: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("q", [[2, 0, 1], [0, 3, 0], [0, 0, 3], [3, 0, 0], [0, 1, 2]])
def test_as_many_queries_as_sequences_but_not_one_each(q, dense, dtype):
    c = AttnCase(61, [200, 75, 3100], q=q, page=16, top_k=128, dense=dense, dtype=dtype)
    out, lse, code = c.call()
    assert code == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [2, 70, 160])
def test_a_batch_padded_past_its_last_query(n_q, dtype):
    """Queries that no sequence has are reported; the others are as ever."""
    if dtype == "f32" and n_q == 160:
        n_q = 40
    c = AttnCase(63, [700], q=[n_q], page=16, top_k=300, dtype=dtype)
    t, b = c.tensors(), c.batch()
    pad = 3
    for name in ("q", "idx", "n_sel", "out", "lse"):
        t[name] = torch.cat([t[name], t[name][:1].expand(pad, *t[name].shape[1:])]).contiguous()
    b.n_q = n_q + pad
    ws = dsa.alloc_workspace(c.shape, b, dsa.OP_PAGED_MLA)
    c.launch(t, b, ws)
    assert dsa.dsa_check_device_error(ws) == 2
    c.check(host(t["out"][:n_q]), host(t["lse"][:n_q]), [0, n_q // 2, n_q - 1])


@pytest.mark.parametrize("fmt", ["e4m3", "s8"])
def test_a_captured_step_of_plan_append_and_attention(fmt):
    """One decode step of five rows captured on a stream of its own and replayed
    from step to step, the lengths alone renewed: rows grow over pages, one ends
    and begins anew, pages pass from row to row."""
    rng = np.random.default_rng(65)
    n, page, ld, n_pages = 5, 16, 6, 22
    pages = dsa.make_pages(page, n_pages, ld, fmt)
    sh = dsa.make_shape(scale=SCALE)
    codes = torch.zeros((n_pages, page, 576), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n_pages, 2), dtype=torch.uint8, device=DEV)
    table = torch.full((n, ld), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    n_free = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    row_off, q_off = (torch.zeros(n + 1, dtype=torch.int64, device=DEV) for _ in range(2))
    slots = torch.zeros(n, dtype=torch.int64, device=DEV)
    key_off = i64(np.arange(n + 1) * ld * page)
    lens = [torch.zeros(n, dtype=torch.int64, device=DEV) for _ in range(3)]
    rows = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    q_abs = torch.zeros((n, 64, 576), dtype=torch.bfloat16, device=DEV)
    out, lse = torch.zeros((n, 64, 512), device=DEV), torch.zeros((n, 64), device=DEV)
    b = dsa.make_batch(row_off, key_off, q_off, n, 1, ld * page, n * ld * page, n * ld * page,
                       dsa.FLAG_DENSE)
    ws = [dsa.alloc_workspace(sh, b, op) for op in
          (dsa.OP_PAGE_PLAN, dsa.OP_CACHE_APPEND, dsa.OP_PAGED_MLA)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        dsa.dsa_page_plan(pages, *lens, free, n_free, table, row_off, q_off, slots, ws[0], stream=side)
        dsa.dsa_cache_append(sh, b, pages, rows, slots, codes, scales, ws[1], stream=side)
        dsa.dsa_paged_mla_attn(sh, b, pages, q_abs, codes, scales, table, None, None, out, lse, ws[2],
                               stream=side)
    held = np.zeros(n, dtype=np.int64)
    c_ref, s_ref = host(codes).copy(), host(scales).copy()
    for step in range(70):
        at = held.copy()                                # rows that stay
        if step in (20, 41, 60):
            at[step % n] = 0                            # ends; another begins in its place
        kv, q = at + 1, np.ones(n, dtype=np.int64)
        new = torch.tensor(rng.normal(size=(n, 576)) * np.exp(0.5 * rng.normal(size=(n, 1)))).bfloat16()
        qa = torch.tensor(rng.normal(size=(n, 64, 576))).bfloat16()
        for x, y in zip(lens, (held, kv, q)):
            x.copy_(i64(y))
        rows.copy_(new)
        q_abs.copy_(qa)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert [dsa.dsa_check_device_error(w) for w in ws] == [0, 0, 0]
        t, f = host(table), host(free)[:n_free.item()]
        used = [p for s in range(n) for p in t[s, :ref.pages_for(kv[s], page)]]
        assert sorted(used + list(f)) == list(range(n_pages))
        want = [int(t[s, at[s] // page]) * page + at[s] % page for s in range(n)]
        assert np.array_equal(host(slots), want) and np.array_equal(host(row_off), prefix(kv))
        c_ref, s_ref = ref.append(page, kv, q, new.double().numpy(), host(slots), c_ref, s_ref, fmt)
        assert np.array_equal(c_ref, host(codes)) and np.array_equal(s_ref, host(scales))
        if step % 10 == 9:
            pool, o, l = ref.widen(c_ref, s_ref, fmt), host(out), host(lse)
            for s in range(n):
                pos = np.arange(kv[s])
                pg = t[s][pos // page]
                unit = np.exp2(s_ref[pg, 0].astype(np.float64) - 127)
                w, wl, weight, reach, floor = ref.attention(qa[s].double().numpy(), pool[pg, pos % page], pos,
                                                            SCALE, unit)
                tol, tol_l = ref.attention_bounds("bf16", 576, int(kv[s]), weight, reach, wl, floor)
                assert np.all(np.abs(o[s] - w) <= tol) and np.all(np.abs(l[s] - wl) <= tol_l)
        held = kv
