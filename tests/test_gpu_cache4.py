"""4-bit caches on the GPU against the float64 oracle: writing and reading back
(exact), page scores, selected attention, and a serving run of all of them."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_basiskv_b200 as bkv
from oracle import basiskv_oracle as O
from oracle import span_oracle as SO
from span_harness import (FMT_WEIGHT, Paged, assert_rows, bf16, dims_of, random_rows,
                                reference, table_of)

pytestmark = pytest.mark.gpu


def status_clean():
    assert bkv.read_device_status() == 0


def _write_case(rng, B, n, Hkv, d, rv, rk, page, lens, cap_pages, offset=0):
    """Rows with every kind of block: normal, tiny, huge, zero, ties."""
    def rows(w):
        x = rng.standard_normal((B, n, Hkv, w)) * np.exp(2 * rng.standard_normal((B, n, Hkv, 1)))
        kind = rng.integers(0, 12, (B, n, Hkv, w // 16))
        blk = x.reshape(B, n, Hkv, w // 16, 16)
        blk[kind == 0] = 0.0
        blk[kind == 1] *= 1e-7           # below the smallest scale
        blk[kind == 2] *= 2e-5           # scales in steps of 2^-17
        blk[kind == 3] *= 3e4            # saturates above 61440
        m = kind == 4                    # multiples of 1/4 of a block maximum of 6: ties
        blk[m] = rng.integers(-24, 25, blk[m].shape) / 4.0
        return bf16(blk.reshape(B, n, Hkv, w))
    return rows(d), rows(rv), rows(rk)


def _dev(t, offset=0):
    """On the device, `offset` elements past the allocation's start."""
    buf = torch.empty(t.numel() + offset + 8, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("B,n,Hkv,d,rv,rk,page,lens,offset", [
    (1, 1, 1, 64, 32, 16, 16, [0], 0),
    (3, 1, 8, 128, 64, 32, 16, [0, 15, 16], 0),
    (2, 37, 2, 128, 96, 64, 32, [5, 31], 0),
    (2, 100, 3, 64, 128, 32, 16, [0, 7], 8),      # rows that are 16- but not 32-byte aligned
    (1, 700, 8, 128, 64, 32, 16, [3], 0),
    (5, 9, 16, 128, 128, 64, 32, [0, 1, 60, 2, 33], 0),  # more blocks a token than threads
])
def test_write_then_read_is_the_oracle(B, n, Hkv, d, rv, rk, page, lens, offset):
    rng = np.random.default_rng(n + d)
    mp = -(-(max(lens) + n) // page) + 1
    phys = B * mp + 3
    table = table_of(rng, B, mp, phys)
    dims = dims_of(B, 8 * Hkv, Hkv, d, rv, rk, page, mp, phys)
    parts = _write_case(rng, B, n, Hkv, d, rv, rk, page, lens, mp)
    ws = (d, rv, rk)
    caches = [torch.full((bkv.cache4_bytes(dims, w),), 0xA5, dtype=torch.uint8, device="cuda")
              for w in ws]
    assert all(c.numel() == phys * Hkv * page * w * 9 // 16 for c, w in zip(caches, ws))
    before = [c.clone() for c in caches]
    rows = [_dev(p, offset) for p in parts]
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(L, -7)
    bkv.basiskv_cache4_write(dims, *rows, n, L, out, torch.from_numpy(table).cuda(), *caches)
    status_clean()
    assert L.tolist() == lens and out.tolist() == [x + n for x in lens]
    want = [SO.round4(p.double().numpy()) for p in parts]
    # read back a window that starts before and ends behind the live tokens
    first = torch.tensor([x - 2 for x in lens], dtype=torch.int32, device="cuda")
    count = n + 5
    outs = [_dev(torch.full((B, count, Hkv, w), 77.0, dtype=torch.bfloat16), offset) for w in ws]
    bkv.basiskv_cache4_read(dims, first, count, out, torch.from_numpy(table).cuda(), *caches, *outs)
    status_clean()
    for o, wv in zip(outs, want):
        o = o.cpu().double().numpy()
        for b in range(B):
            np.testing.assert_array_equal(o[b, 2:2 + n], wv[b])
            assert np.all(o[b, 2 + n:] == 77.0)        # behind the last token: left alone
            if lens[b] < 2:
                assert np.all(o[b, :2 - lens[b]] == 77.0)  # before the first
    # the tiles' bytes, and nothing else, were written
    for c, c0, w, p in zip(caches, before, ws, parts):
        c, c0 = (t.cpu().numpy().reshape(phys, Hkv, -1) for t in (c, c0))
        mask = np.zeros_like(c, dtype=bool)
        for b in range(B):
            for j in range(n):
                t = lens[b] + j
                pg, r = table[b, t // page], t % page
                mask[pg, :, r * w // 2:(r + 1) * w // 2] = True
                s0 = page * w // 2 + r * w // 16
                mask[pg, :, s0:s0 + w // 16] = True
        np.testing.assert_array_equal(c[~mask], c0[~mask])


def test_write_in_place_overflow_and_optional_parts():
    rng = np.random.default_rng(3)
    B, n, Hkv, d, rv, rk, page, mp = 3, 5, 2, 64, 64, 32, 16, 2
    phys = B * mp
    table = table_of(rng, B, mp, phys)
    dims = dims_of(B, 8, Hkv, d, rv, rk, page, mp, phys)
    k, z, e = (_dev(p) for p in _write_case(rng, B, n, Hkv, d, rv, rk, page, None, mp))
    K, Z, E = (torch.zeros(bkv.cache4_bytes(dims, w), dtype=torch.uint8, device="cuda")
               for w in (d, rv, rk))
    tab = torch.from_numpy(table).cuda()
    L = torch.tensor([0, 28, 27], dtype=torch.int32, device="cuda")  # 28 + 5 passes 32
    K0 = K.clone()
    bkv.basiskv_cache4_write(dims, k, z, None, n, L, L, tab, K, Z, None)
    assert bkv.read_device_status() == bkv.DEV_OVERFLOW
    assert L.tolist() == [5, 28, 32]
    ko = torch.zeros(B, n, Hkv, d, dtype=torch.bfloat16, device="cuda")
    first = torch.tensor([0, 28, 27], dtype=torch.int32, device="cuda")
    bkv.basiskv_cache4_read(dims, first, n, L, tab, K, None, None, ko, None, None)
    status_clean()
    want = SO.round4(k.cpu().double().numpy())
    np.testing.assert_array_equal(ko[0].cpu().double().numpy(), want[0])
    np.testing.assert_array_equal(ko[2].cpu().double().numpy(), want[2])
    assert torch.all(ko[1] == 0)  # none of its rows was written
    pages1 = K.view(phys, -1)[torch.from_numpy(table[1]).long().cuda()]
    assert torch.all(pages1 == 0) and torch.equal(K0, torch.zeros_like(K0))
    # lengths not asked for
    L2 = torch.tensor([3, 3, 3], dtype=torch.int32, device="cuda")
    bkv.basiskv_cache4_write(dims, k, z, e, n, L2, None, tab, K, Z, E)
    status_clean()
    assert L2.tolist() == [3, 3, 3]
    # a table entry out of range: its rows are skipped and reported
    bad = tab.clone()
    bad[0, 0] = phys
    bkv.basiskv_cache4_write(dims, k, z, e, n, L2, None, bad, K, Z, E)
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    ko.fill_(9.0)
    bkv.basiskv_cache4_read(dims, L2, n, torch.full_like(L2, 8), bad, K, None, None, ko, None,
                            None)
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    assert torch.all(ko[0] == 9.0) and not torch.any(ko[1] == 9.0)


def _cache_problem(seed, B, G, Hkv, d, rv, rk, page, lens, spare=1, scale=1.0):
    rng = np.random.default_rng(seed)
    mp = max(1, -(-max(lens) // page)) + spare
    phys = B * mp + 2
    table = table_of(rng, B, mp, phys)
    dims = dims_of(B, G * Hkv, Hkv, d, rv, rk, page, mp, phys)
    K = Paged(random_rows(rng, lens, Hkv, d, scale), "4bit", page, table, phys)
    Z = Paged(random_rows(rng, lens, Hkv, rv), "4bit", page, table, phys)
    E = Paged(random_rows(rng, lens, Hkv, rk), "4bit", page, table, phys)
    for b, L in enumerate(lens):  # entries past the live pages are never looked up
        table[b, -(-L // page):] = -1
    q = bf16(rng.standard_normal((B, G * Hkv, d)) * scale)
    P_K = bf16(rng.standard_normal((Hkv, rv, d)) / np.sqrt(rv))
    U_K = bf16(np.linalg.qr(rng.standard_normal((Hkv, d, rk)))[0])
    return rng, dims, table, K, Z, E, q, P_K, U_K


def _workspace(dims, top_k, msl):
    return torch.full((bkv.workspace_size(dims, top_k, msl),), 0x7F, dtype=torch.uint8,
                      device="cuda")


@pytest.mark.parametrize("B,G,Hkv,d,rv,rk,page,lens,top_k", [
    (1, 4, 1, 64, 32, 16, 16, [1], 2),
    (2, 1, 2, 128, 64, 16, 32, [33, 0], 2),
    (3, 4, 2, 128, 64, 32, 16, [500, 17, 16], 8),
    (2, 8, 2, 128, 96, 64, 32, [1000, 95], 9),
    (2, 2, 3, 64, 128, 32, 16, [255, 256], 16),
    (4, 8, 1, 64, 96, 16, 16, [31, 0, 64, 700], 5),
])
def test_page_scores_and_selection(B, G, Hkv, d, rv, rk, page, lens, top_k):
    rng, dims, table, K, Z, E, q, P_K, U_K = _cache_problem(7, B, G, Hkv, d, rv, rk, page, lens)
    msl = max(lens) + 1
    mp = table.shape[1]
    scores = torch.full((B, Hkv, mp), 123.0, dtype=torch.float32, device="cuda")
    sel = torch.full((B, Hkv, top_k), -9, dtype=torch.int32, device="cuda")
    ws = _workspace(dims, top_k, msl)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bkv.basiskv_cache4_route(dims, q.cuda(), L, msl, torch.from_numpy(table).cuda(), P_K.cuda(),
                             U_K.cuda(), Z.tensor, E.tensor, top_k, scores, sel, ws)
    status_clean()
    scores, sel = scores.cpu().double().numpy(), sel.cpu().numpy()
    clean = 0
    for b in range(B):
        P = -(-lens[b] // page)
        assert np.all(scores[b, :, P:] == 123.0)  # behind the last page: left alone
        for g in range(Hkv):
            if P == 0:
                assert np.all(sel[b, g] == -1)
                continue
            kh = (Z.values[b][:, g] @ P_K[g].double().numpy()
                  + E.values[b][:, g] @ U_K[g].double().numpy().T)
            qg = q[b, g * G:(g + 1) * G].double().numpy()
            s = (qg @ kh.T).max(0)
            ref = np.array([s[p * page:(p + 1) * page].max() for p in range(P)])
            # fp32 folds and products of r_v + r_k terms, 22-bit queries: 2^-20 of
            # the products' magnitudes
            mag = (np.abs(qg) @ (np.abs(Z.values[b][:, g]) @ np.abs(P_K[g].double().numpy())
                                 + np.abs(E.values[b][:, g])
                                 @ np.abs(U_K[g].double().numpy()).T).T).max()
            assert np.abs(scores[b, g, :P] - ref).max() <= 2.0 ** -20 * mag
            rsel, tie = O.select_pages(ref.astype(np.float32), top_k, 1, 1)
            if not tie:
                clean += 1
                np.testing.assert_array_equal(sel[b, g], rsel)
    assert clean > 0


def test_route_reports_bad_pages_and_lengths():
    B, G, Hkv, d, rv, rk, page, lens = 2, 4, 2, 128, 64, 32, 16, [100, 90]
    rng, dims, table, K, Z, E, q, P_K, U_K = _cache_problem(8, B, G, Hkv, d, rv, rk, page, lens)
    ws = _workspace(dims, 2, 100)
    scores = torch.full((B, Hkv, table.shape[1]), 5.0, device="cuda")
    bad = table.copy()
    bad[1, 2] = dims.num_phys_pages
    run = lambda t, L: bkv.basiskv_cache4_route(
        dims, q.cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"), 100,
        torch.from_numpy(t).cuda(), P_K.cuda(), U_K.cuda(), Z.tensor, E.tensor, 2, scores, None,
        ws)
    run(table, lens)
    status_clean()
    good = scores.clone()
    scores.fill_(5.0)
    run(bad, lens)
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    assert torch.all(scores[1, :, 2] == -float("inf"))
    scores[1, :, 2] = good[1, :, 2]
    assert torch.equal(scores, good)
    for L in ([101, 90], [-1, 90]):
        scores.fill_(5.0)
        run(table, L)
        assert bkv.read_device_status() == bkv.DEV_BAD_LENGTH
        assert torch.all(scores[0] == 5.0) and torch.equal(scores[1], good[1])


@pytest.mark.parametrize("B,G,Hkv,d,rv,rk,page,lens,top_k,scale", [
    (1, 1, 2, 64, 32, 16, 16, [1], 2, 1.0),
    (2, 4, 2, 128, 64, 32, 16, [300, 7], 5, 1.0),
    (3, 8, 2, 128, 96, 64, 32, [200, 0, 33], 4, 1.0),
    (2, 2, 2, 64, 128, 32, 16, [255, 1000], 33, 1.0),
    (1, 4, 8, 128, 64, 32, 16, [4000], 64, 3.0),   # peaked: the reference moves
    (2, 8, 1, 64, 32, 16, 32, [64, 65], 2, 1.0),
])
def test_selected_attention(B, G, Hkv, d, rv, rk, page, lens, top_k, scale):
    rng, dims, table, K, Z, E, q, P_K, U_K = _cache_problem(9, B, G, Hkv, d, rv, rk, page, lens,
                                                            scale=scale)
    sel = np.full((B, Hkv, top_k), -1, dtype=np.int32)
    for b in range(B):
        P = -(-lens[b] // page)
        for g in range(Hkv):
            if P == 0:
                sel[b, g, 0] = 0  # a page past the length contributes nothing
                continue
            p = rng.permutation(P)[:top_k]
            pick = np.unique(np.append(p[:-1], P - 1)) if len(p) > 1 else np.array([P - 1])
            at = np.sort(rng.permutation(top_k)[:len(pick)])  # -1 anywhere between
            sel[b, g, at] = pick
    msl = max(lens) + 3
    out = torch.full((B, G * Hkv, rv), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = _workspace(dims, top_k, min(msl, table.shape[1] * page))
    args = (dims, q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            min(msl, table.shape[1] * page), torch.from_numpy(table).cuda(), K.tensor, Z.tensor,
            torch.from_numpy(sel).cuda(), top_k, out, ws)
    bkv.basiskv_cache4_attend(*args)
    status_clean()
    got = out.cpu().double().numpy()
    for b in range(B):
        for g in range(Hkv):
            t = np.concatenate([np.arange(p * page, min((p + 1) * page, lens[b]))
                                for p in sel[b, g] if p >= 0] or [np.arange(0)]).astype(int)
            see = np.zeros((G, max(lens[b], 1)), dtype=bool)
            see[:, t] = True
            Kb = K.values[b][:, g] if lens[b] else np.zeros((1, d))
            Zb = Z.values[b][:, g] if lens[b] else np.zeros((1, rv))
            if not lens[b]:
                see[:] = False
            a, A, X = reference(q[b, g * G:(g + 1) * G].double().numpy(), Kb, Zb, see)
            assert_rows(got[b, g * G:(g + 1) * G], a, A, X, FMT_WEIGHT["4bit"], f"b{b} g{g}")
    first = out.clone()
    out.zero_()
    bkv.basiskv_cache4_attend(*args)  # the same call gives the same bits
    assert torch.equal(out, first)


def test_a_page_selected_twice_counts_twice():
    G, Hkv, d, rv, page, L = 4, 2, 128, 64, 16, 100
    rng, dims, table, K, Z, E, q, *_ = _cache_problem(12, 1, G, Hkv, d, rv, 32, page, [L])
    sel = np.array([[[0, 3, 3, 6], [6, -1, 6, 6]]], dtype=np.int32)
    out = torch.zeros(1, G * Hkv, rv, dtype=torch.bfloat16, device="cuda")
    bkv.basiskv_cache4_attend(dims, q.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                              L, torch.from_numpy(table).cuda(), K.tensor, Z.tensor,
                              torch.from_numpy(sel).cuda(), 4, out, _workspace(dims, 4, L))
    status_clean()
    for g in range(Hkv):
        t = np.concatenate([np.arange(p * page, min((p + 1) * page, L)) for p in sel[0, g]
                            if p >= 0])
        a, A, X = reference(q[0, g * G:(g + 1) * G].double().numpy(), K.values[0][t][:, g],
                            Z.values[0][t][:, g], np.ones((G, len(t)), dtype=bool))
        assert_rows(out[0, g * G:(g + 1) * G].cpu().double().numpy(), a, A, X,
                    FMT_WEIGHT["4bit"], f"g{g}")


def test_selected_attention_reports_bad_pages():
    B, G, Hkv, d, rv, rk, page, lens = 1, 4, 2, 128, 64, 32, 16, [100]
    rng, dims, table, K, Z, E, q, *_ = _cache_problem(10, B, G, Hkv, d, rv, rk, page, lens)
    ws = _workspace(dims, 3, 100)
    out = torch.zeros(B, G * Hkv, rv, dtype=torch.bfloat16, device="cuda")

    def run(sel, tab):
        bkv.basiskv_cache4_attend(dims, q.cuda(), torch.tensor(lens, dtype=torch.int32,
                                                               device="cuda"), 100,
                                  torch.from_numpy(tab).cuda(), K.tensor, Z.tensor,
                                  torch.tensor(sel, dtype=torch.int32, device="cuda"), 3, out, ws)
        return bkv.read_device_status(), out.clone()

    st, ref = run([[[0, 3, -1], [1, 2, 6]]], table)
    assert st == 0
    bad = table.copy()
    bad[0, 5] = -4
    st, got = run([[[0, 3, 5], [1, 2, 6]]], bad)   # the page is left out
    assert st == bkv.DEV_BAD_PAGE and torch.equal(got, ref)
    st, got = run([[[0, 3, table.shape[1]], [1, 2, 6]]], table)  # a page behind the row
    assert st == bkv.DEV_BAD_PAGE and torch.equal(got, ref)


def test_serving_run_of_all_of_them():
    """A prompt written and attended, then decode steps that write a token, score
    and select pages, attend them and project: every stage against the oracle on
    the cached values, on a second stream, eager and as a replayed graph."""
    rng = np.random.default_rng(20)
    B, G, Hkv, d, rv, rk, page, n, steps, top_k = 2, 4, 2, 64, 32, 16, 16, 70, 3, 4
    Hq, mp = G * Hkv, 6
    phys = B * mp
    table = table_of(rng, B, mp, phys)
    dims = dims_of(B, Hq, Hkv, d, rv, rk, page, mp, phys)
    msl = mp * page
    st = torch.cuda.Stream()
    tab = torch.from_numpy(table).cuda()
    caches = [torch.zeros(bkv.cache4_bytes(dims, w), dtype=torch.uint8, device="cuda")
              for w in (d, rv, rk)]
    rows = [bf16(rng.standard_normal((B, n + steps, Hkv, w))) for w in (d, rv, rk)]
    P_K, U_K = bf16(rng.standard_normal((Hkv, rv, d)) / 6), bf16(
        np.linalg.qr(rng.standard_normal((Hkv, d, rk)))[0])
    W = bf16(rng.standard_normal((128, Hq * rv)) / 16)
    qs = bf16(rng.standard_normal((B, n + steps, Hq, d)))
    L = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = _workspace(dims, top_k, msl)
    wws = torch.zeros(bkv.window_workspace_size(dims, n, msl, 2, 40), dtype=torch.uint8,
                      device="cuda")
    a_prompt = torch.zeros(B, n, Hq, rv, dtype=torch.bfloat16, device="cuda")
    prompt = [r[:, :n].contiguous().cuda() for r in rows]
    tok = [torch.zeros(B, 1, Hkv, w, dtype=torch.bfloat16, device="cuda") for w in (d, rv, rk)]
    q1 = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    sel = torch.zeros(B, Hkv, top_k, dtype=torch.int32, device="cuda")
    a1 = torch.zeros(B, Hq, rv, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(B, 128, dtype=torch.bfloat16, device="cuda")
    Pk, Uk, Wd, qp = P_K.cuda(), U_K.cuda(), W.cuda(), qs[:, :n].contiguous().cuda()
    torch.cuda.synchronize()

    def step():
        bkv.basiskv_cache4_write(dims, *tok, 1, L, L, tab, *caches, stream=st)
        bkv.basiskv_cache4_route(dims, q1, L, msl, tab, Pk, Uk, caches[1], caches[2], top_k, None,
                                 sel, ws, stream=st)
        bkv.basiskv_cache4_attend(dims, q1, L, msl, tab, caches[0], caches[1], sel, top_k, a1, ws,
                                  stream=st)
        bkv.basiskv_outproj_sources(dims, a1, 1, Wd, y, ws, stream=st)

    with torch.cuda.stream(st):
        bkv.basiskv_cache4_write(dims, *prompt, n, L, L, tab, *caches, stream=st)
        bkv.basiskv_attend_window(dims, qp, n, L, msl, tab, caches[0], caches[1], 2, 40, a_prompt,
                                  wws, stream=st, cache4=True)
    st.synchronize()
    status_clean()
    assert L.tolist() == [n] * B
    vals = [SO.round4(r.double().numpy()) for r in rows]
    for b in range(B):
        for g in range(Hkv):
            see = np.repeat(SO.window_mask(n, n, 40, 2), G, 0)
            a, A, X = reference(qs[b, :n, g * G:(g + 1) * G].double().numpy().reshape(-1, d),
                                vals[0][b, :n, g], vals[1][b, :n, g], see)
            assert_rows(a_prompt[b, :, g * G:(g + 1) * G].cpu().double().numpy().reshape(-1, rv),
                        a, A, X, FMT_WEIGHT["4bit"], f"prompt b{b} g{g}")
    graph = None
    for i in range(steps):
        t = n + i
        with torch.cuda.stream(st):
            for x, r in zip(tok, rows):
                x.copy_(r[:, t:t + 1])
            q1.copy_(qs[:, t])
        st.synchronize()
        if i == 0:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    step()
                assert L.tolist() == [n + 1] * B  # capturing runs nothing
            with torch.cuda.stream(st):
                graph.replay()
        st.synchronize()
        status_clean()
        assert L.tolist() == [t + 1] * B
        T = t + 1
        for b in range(B):
            for g in range(Hkv):
                qg = q1[b, g * G:(g + 1) * G].cpu().double().numpy()
                kh = (vals[1][b, :T, g] @ P_K[g].double().numpy()
                      + vals[2][b, :T, g] @ U_K[g].double().numpy().T)
                s = (qg @ kh.T).max(0)
                sc = np.array([s[p:p + page].max() for p in range(0, T, page)])
                rsel, tie = O.select_pages(sc.astype(np.float32), top_k, 1, 1)
                gsel = sel[b, g].cpu().numpy()
                if not tie:
                    np.testing.assert_array_equal(gsel, rsel)
                see = np.zeros((G, T), dtype=bool)
                for p in gsel[gsel >= 0]:
                    see[:, p * page:(p + 1) * page] = True
                a, A, X = reference(qg, vals[0][b, :T, g], vals[1][b, :T, g], see)
                assert_rows(a1[b, g * G:(g + 1) * G].cpu().double().numpy(), a, A, X,
                            FMT_WEIGHT["4bit"], f"step {i} b{b} g{g}")
            ya = a1[b].cpu().double().numpy().reshape(-1)
            ref = W.double().numpy() @ ya
            mag = np.abs(W.double().numpy()) @ np.abs(ya)
            assert np.all(np.abs(y[b].cpu().double().numpy() - ref)
                          <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * mag)


@pytest.mark.parametrize("lens_out", ["none", "other", "in_place"])
@pytest.mark.parametrize("bad", [28, 32, -1])
def test_overflow_is_reported_whatever_becomes_of_the_lengths(lens_out, bad):
    """A sequence whose rows do not fit is skipped whole and reported, and its length
    stays, whether the lengths are advanced in place, in another buffer or not at all."""
    rng = np.random.default_rng(4)
    B, n, Hkv, d, rv, rk, page, mp = 3, 5, 2, 64, 32, 16, 16, 2
    phys = B * mp
    table = table_of(rng, B, mp, phys)
    dims = dims_of(B, 8, Hkv, d, rv, rk, page, mp, phys)
    k, z, e = (_dev(p) for p in _write_case(rng, B, n, Hkv, d, rv, rk, page, None, mp))
    caches = [torch.full((bkv.cache4_bytes(dims, w),), 0x5A, dtype=torch.uint8, device="cuda")
              for w in (d, rv, rk)]
    lens = [0, bad, 27]
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = {"none": None, "other": torch.full_like(L, -9), "in_place": L}[lens_out]
    bkv.basiskv_cache4_write(dims, k, z, e, n, L, out, torch.from_numpy(table).cuda(), *caches)
    assert bkv.read_device_status() == bkv.DEV_OVERFLOW
    if out is not None:
        assert out.tolist() == [5, bad, 32]
    if lens_out != "in_place":
        assert L.tolist() == lens
    for c in caches:
        c = c.view(phys, -1)
        assert torch.all(c[torch.from_numpy(table[1]).long().cuda()] == 0x5A)
        assert not torch.all(c[int(table[0, 0])] == 0x5A)


@pytest.mark.parametrize("long", [101, 130, 2 ** 31 - 1])
def test_selection_of_a_bad_length_is_empty(long):
    """A length outside [0, max_seq_len] gets no scores, and so no selection: never one
    of what lay in the workspace or in the caller's scores."""
    B, G, Hkv, d, rv, rk, page, lens = 3, 4, 2, 128, 64, 32, 16, [100, 90, 64]
    rng, dims, table, K, Z, E, q, P_K, U_K = _cache_problem(8, B, G, Hkv, d, rv, rk, page, lens,
                                                            spare=3)
    top_k, msl = 3, 100
    tab = torch.from_numpy(table).cuda()

    def run(L, fill, own_scores):
        ws = torch.full((bkv.workspace_size(dims, top_k, msl),), fill, dtype=torch.uint8,
                        device="cuda")
        scores = None
        if own_scores:
            scores = torch.randn(B, Hkv, table.shape[1], device="cuda") * 100
        sel = torch.full((B, Hkv, top_k), -9, dtype=torch.int32, device="cuda")
        bkv.basiskv_cache4_route(dims, q.cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"),
                                 msl, tab, P_K.cuda(), U_K.cuda(), Z.tensor, E.tensor, top_k,
                                 scores, sel, ws)
        return bkv.read_device_status(), sel.cpu()

    st, good = run(lens, 0, False)
    assert st == 0 and torch.all(good >= 0)
    for fill, own_scores in ((0, False), (0x7F, False), (0x3C, False), (0, True)):
        for L in ([long, 90, 64], [100, long, -1]):
            st, sel = run(L, fill, own_scores)
            assert st == bkv.DEV_BAD_LENGTH
            for b in range(B):
                if 0 <= L[b] <= msl:
                    assert torch.equal(sel[b], good[b])
                else:
                    assert torch.all(sel[b] == -1)


def test_selected_attention_of_a_bad_length_is_zero():
    """A sequence whose length is outside [0, max_seq_len] is taken as empty."""
    B, G, Hkv, d, rv, rk, page, lens = 3, 4, 2, 128, 64, 32, 16, [100, 90, 64]
    rng, dims, table, K, Z, E, q, *_ = _cache_problem(11, B, G, Hkv, d, rv, rk, page, lens)
    ws = _workspace(dims, 3, 100)
    out = torch.zeros(B, G * Hkv, rv, dtype=torch.bfloat16, device="cuda")
    sel = torch.tensor([[[0, 3, -1], [1, 2, 3]]] * B, dtype=torch.int32, device="cuda")

    def run(L):
        out.fill_(7.0)
        bkv.basiskv_cache4_attend(dims, q.cuda(), torch.tensor(L, dtype=torch.int32,
                                                               device="cuda"), 100,
                                  torch.from_numpy(table).cuda(), K.tensor, Z.tensor, sel, 3, out,
                                  ws)
        return bkv.read_device_status(), out.clone()

    st, good = run(lens)
    assert st == 0
    for L in ([101, 90, 64], [100, -1, 2 ** 31 - 1]):
        st, got = run(L)
        assert st == bkv.DEV_BAD_LENGTH
        for b in range(B):
            assert torch.equal(got[b], good[b]) if 0 <= L[b] <= 100 else torch.all(got[b] == 0)


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
def test_lengths_near_the_end_of_32_bits_overflow(length):
    """The length after a write is not taken in 32 bits."""
    B, n, Hkv, d, rv, page, mp = 2, 5, 2, 64, 32, 16, 2
    phys = B * mp
    dims = dims_of(B, 8, Hkv, d, rv, 16, page, mp, phys)
    tab = torch.arange(phys, dtype=torch.int32, device="cuda").view(B, mp)
    rows = [torch.ones(B, n, Hkv, w, dtype=torch.bfloat16, device="cuda") for w in (d, rv)]
    K, Z = (torch.zeros(bkv.cache4_bytes(dims, w), dtype=torch.uint8, device="cuda")
            for w in (d, rv))
    L = torch.tensor([length, 3], dtype=torch.int32, device="cuda")
    bkv.basiskv_cache4_write(dims, *rows, None, n, L, L, tab, K, Z, None)
    assert bkv.read_device_status() == bkv.DEV_OVERFLOW
    assert L.tolist() == [length, 8]
    assert torch.all(K.view(phys, -1)[:mp] == 0)
