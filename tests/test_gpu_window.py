"""Windowed attention on the GPU against the float64 oracle: single tokens,
drafts and prompt chunks, over bf16, E4M3 and 4-bit caches."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_basiskv_b200 as bkv
from oracle import span_oracle as SO
from span_harness import (FMT_WEIGHT, Paged, assert_rows, bf16, dims_of, random_rows,
                                reference, table_of)

pytestmark = pytest.mark.gpu


class Problem:
    def __init__(self, fmt, B, G, Hkv, d, rv, page, lens, n, window, sink, seed=0, scale=1.0,
                 lead=None, spare=1):
        rng = np.random.default_rng(seed + 1000 * n + len(lens))
        self.__dict__.update(fmt=fmt, B=B, G=G, Hkv=Hkv, d=d, rv=rv, page=page, lens=lens, n=n,
                             window=window, sink=sink)
        mp = max(1, -(-max(lens + [n]) // page)) + spare
        phys = B * mp + 1
        table = table_of(rng, B, mp, phys)
        kw = {}
        if lead:
            kw = dict(route_r_v=lead, route_r_k=16)
        self.dims = dims_of(B, G * Hkv, Hkv, d, rv, 32, page, mp, phys,
                            cache_fp8=1 if fmt == "e4m3" else 0, **kw)
        self.K = Paged(random_rows(rng, lens, Hkv, d, scale), fmt, page, table, phys)
        self.Z = Paged(random_rows(rng, lens, Hkv, rv), fmt, page, table, phys, lead=lead)
        # pages that no query sees may be anything: the table says they are gone
        for b, L in enumerate(lens):
            live = np.zeros(mp * page, dtype=bool)
            if L:
                live[:L] = SO.window_mask(L, n, window, sink).any(0)
            for p in range(mp):
                if not live[p * page:(p + 1) * page].any():
                    table[b, p] = 1 << 30 if p % 2 else -1
        self.table = torch.from_numpy(table).cuda()
        self.q = bf16(rng.standard_normal((B, n, G * Hkv, d)) * scale)
        self.qd = self.q.cuda()
        self.L = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.msl = min(max(max(lens), 1) + 2, mp * page)
        self.ws = torch.full((bkv.window_workspace_size(self.dims, n, self.msl, sink, window),),
                             0x7F, dtype=torch.uint8, device="cuda")
        self.out = torch.full((B, n, G * Hkv, rv), 9.0, dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None, out=None, ws=None):
        out = self.out if out is None else out
        bkv.basiskv_attend_window(self.dims, self.qd, self.n, self.L, self.msl, self.table,
                                  self.K.tensor, self.Z.tensor, self.sink, self.window, out,
                                  self.ws if ws is None else ws, stream=stream,
                                  cache4=self.fmt == "4bit")
        return out

    def check(self, out=None, kind=None):
        got = (self.out if out is None else out).cpu().double().numpy()
        kind = kind or self.fmt
        if kind == "bf16":
            kind = "bf16_token" if self.n * self.G <= 16 else "bf16_prompt"
        for b, L in enumerate(self.lens):
            if L == 0:
                assert np.all(got[b] == 0)
                continue
            see = np.repeat(SO.window_mask(L, self.n, self.window, self.sink), self.G, 0)
            for g in range(self.Hkv):
                hs = slice(g * self.G, (g + 1) * self.G)
                a, A, X = reference(self.q[b, :, hs].double().numpy().reshape(-1, self.d),
                                    self.K.values[b][:, g], self.Z.values[b][:, g], see)
                assert_rows(got[b, :, hs].reshape(-1, self.rv), a, A, X, FMT_WEIGHT[kind],
                            f"{self.fmt} n{self.n} b{b} g{g}")


def _go(*a, **kw):
    p = Problem(*a, **kw)
    p.run()
    assert bkv.read_device_status() == 0
    p.check()
    return p


FMTS = ["bf16", "e4m3", "4bit"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,d,rv,page", [(1, 64, 32, 16), (2, 128, 64, 32), (4, 128, 64, 16),
                                         (8, 128, 96, 32), (8, 64, 128, 16), (4, 64, 96, 16)])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_shapes(fmt, G, d, rv, page, n):
    _go(fmt, 2, G, 2, d, rv, page, [150, 37], n, 50, 3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 5, 33])
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (1, 1), (16, 0), (17, 16), (64, 130),
                                         (128, 5), (1000, 1000), (0, 7)])
def test_masks(fmt, n, window, sink):
    """Windows of one token and of all, sinks past the window, lengths of zero and
    one, and more queries than tokens (rows that see nothing are zero)."""
    _go(fmt, 6, 4, 1, 64, 32, 16, [0, 1, 4, 17, 129, 300], n, window, sink)


@pytest.mark.parametrize("fmt,page", [("bf16", 8), ("e4m3", 8), ("bf16", 32), ("4bit", 32)])
@pytest.mark.parametrize("n", [1, 3, 65])
def test_pages(fmt, page, n):
    _go(fmt, 3, 4, 2, 128, 64, page, [131, 8, 77], n, 30, 9)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("G,rv,page,lead", [(4, 64, 16, 16), (8, 96, 32, 32), (4, 96, 16, 16)])
def test_split_latent_tiles_of_a_narrow_router(fmt, n, G, rv, page, lead):
    _go(fmt, 2, G, 1, 128, rv, page, [100, 61], n, 40, 2, lead=lead)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("scale", [0.0, 3.0, 7.0])
def test_peaked_and_flat_scores(fmt, n, scale):
    """Scores of all zeros, and ones hundreds apart, that move the reference
    within a run, by much more than the weights' types hold."""
    _go(fmt, 2, 4, 2, 128, 64, 16, [400, 390], n, 0, 0, scale=scale)


@pytest.mark.parametrize("fmt", FMTS)
def test_growing_scores(fmt):
    """Every later token scores higher: the reference moves at every step."""
    for n in (1, 20):
        p = Problem(fmt, 1, 4, 1, 64, 32, 16, [700], n, 0, 0)
        ramp = np.linspace(-4, 4, 700)[:, None, None] * np.ones((1, 1, 64))
        table = p.table.cpu().numpy()
        p.K = Paged([ramp], fmt, 16, table, p.dims.num_phys_pages)
        p.q = bf16(np.full((1, n, 4, 64), 3.0))
        p.qd = p.q.cuda()
        p.run()
        assert bkv.read_device_status() == 0
        p.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,G,Hkv,n,lens", [
    (1, 4, 1, 128, [700]),           # two row tiles
    (1, 8, 2, 16, [900]),            # one row tile, runs of KV tiles
    (1, 4, 2, 300, [300]),           # a whole prompt, a last item of one row tile
    (3, 2, 1, 200, [1500, 40, 260]),  # ragged, one shorter than the chunk
    (2, 1, 1, 400, [400, 401]),
])
def test_prompts(fmt, B, G, Hkv, n, lens):
    _go(fmt, B, G, Hkv, 64, 64, 16, lens, n, 0 if n % 2 else 250, 4)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sink", [(0, 0), (1024, 5)])
@pytest.mark.parametrize("G,d,rv,page,n", [(4, 128, 64, 16, 5), (8, 64, 96, 32, 3),
                                           (8, 128, 128, 32, 4), (1, 64, 128, 16, 31),
                                           (4, 64, 64, 32, 7), (2, 128, 32, 16, 9)])
def test_streamed_drafts(fmt, window, sink, G, d, rv, page, n):
    """17 to 32 rows a group over 64 contexts of a thousand tokens and more."""
    p = Problem(fmt, 8, G, 8, d, rv, page, [1300, 3, 0, 17, 1100, 1029, 900, 1301], n, window,
                sink)
    p.run()
    assert bkv.read_device_status() == 0
    p.check(kind="bf16_token" if fmt == "bf16" else fmt)


def test_drafts_over_small_pages():
    """Pages of 8 tokens in the sizes that are streamed otherwise."""
    for fmt in ("bf16", "e4m3"):
        _go(fmt, 8, 4, 8, 128, 64, 8, [1100, 3, 0, 17, 1029, 1040, 900, 1101], 6, 0, 0)


def test_many_items():
    """More items than SMs: whole ones, and a last round that is cut into runs."""
    p = _go("bf16", 5, 8, 4, 64, 32, 16, [300, 290, 310, 280, 305], 260, 200, 4)
    assert p.B * p.Hkv * -(-260 // 32) > torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 24])
def test_long_context_in_one_sequence(fmt, n):
    _go(fmt, 1, 4, 1, 64, 32, 16, [5000], n, 0, 0)


@pytest.mark.parametrize("n", [1, 24])
def test_repeat_streams_and_graphs(n):
    """The same call gives the same bits, on another stream, as a replayed graph,
    and in two graphs that share a workspace."""
    p = _go("bf16", 3, 4, 2, 64, 64, 16, [500, 90, 333], n, 100, 4)
    first = p.out.clone()
    for _ in range(3):
        p.out.fill_(3.0)
        assert torch.equal(p.run(), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.zeros_like(p.out)
    p.run(stream=s, out=other)
    s.synchronize()
    assert torch.equal(other, first)
    o1, o2 = torch.zeros_like(p.out), torch.zeros_like(p.out)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s):
        p.run(stream=s, out=o1)
    with torch.cuda.graph(g2, stream=s):
        p.run(stream=s, out=o2)
    for g in (g1, g2, g1):
        o1.zero_(), o2.zero_()
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, first) and torch.equal(o2, first)
    # new lengths and queries under the same graph
    p.L.copy_(torch.tensor([300, 0, 1], dtype=torch.int32))
    p.qd.copy_(p.qd.flip(0))
    g1.replay()
    torch.cuda.synchronize()
    eager = p.run(out=torch.zeros_like(p.out))
    # (the pages of the old window may be gone from the table: only equality counts)
    torch.cuda.synchronize()
    bkv.read_device_status()
    assert torch.equal(o1, eager)


@pytest.mark.parametrize("n", [1, 24])
def test_two_calls_at_once(n):
    p = _go("4bit", 3, 4, 2, 64, 64, 16, [500, 90, 333], n, 0, 0)
    first = p.out.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2, w2 = torch.zeros_like(p.out), torch.zeros_like(p.out), p.ws.clone()
    torch.cuda.synchronize()
    for _ in range(10):
        p.run(stream=s1, out=o1)
        p.run(stream=s2, out=o2, ws=w2)
    torch.cuda.synchronize()
    assert torch.equal(o1, first) and torch.equal(o2, first)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 24])
def test_bad_lengths_and_pages_are_reported(fmt, n):
    p = Problem(fmt, 3, 4, 1, 64, 32, 16, [100, 60, 80], n, 0, 0)
    p.run()
    assert bkv.read_device_status() == 0
    good = p.out.clone()
    p.L.copy_(torch.tensor([p.msl + 1, 60, -5], dtype=torch.int32))
    p.run()
    assert bkv.read_device_status() == bkv.DEV_BAD_LENGTH
    assert torch.all(p.out[0] == 0) and torch.all(p.out[2] == 0)
    assert torch.equal(p.out[1], good[1])
    p.L.copy_(torch.tensor(p.lens, dtype=torch.int32))
    keep = p.table.clone()
    p.table[1, 1] = p.dims.num_phys_pages
    p.run()
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    assert torch.equal(p.out[0], good[0]) and torch.equal(p.out[2], good[2])
    assert torch.all(torch.isfinite(p.out[1].float()))
    p.table.copy_(keep)


def test_a_bad_page_is_left_out_of_a_tokens_softmax():
    p = Problem("bf16", 1, 4, 1, 64, 32, 16, [100], 1, 0, 0)
    p.table[0, 2] = -1
    p.run()
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    see = np.ones((4, 100), dtype=bool)
    see[:, 32:48] = False
    a, A, X = reference(p.q[0, 0].double().numpy(), p.K.values[0][:, 0], p.Z.values[0][:, 0], see)
    assert_rows(p.out[0, 0].cpu().double().numpy(), a, A, X, FMT_WEIGHT["bf16_token"])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 5, 24, 200])
@pytest.mark.parametrize("G,d,rv,page,window,sink", [(4, 64, 32, 16, 0, 0), (4, 128, 128, 32, 0, 0),
                                                     (8, 128, 64, 16, 90, 40)])
def test_bad_pages_are_left_out_of_the_softmax(fmt, n, G, d, rv, page, window, sink):
    """Tokens of pages whose table entry is out of range have no part in any row's
    softmax, by either kernel: the oracle does not see them.  Bad pages lie among the
    sinks, in the middle, in both halves of a 128-token tile, side by side, and at the
    end; a sequence whose every page is bad gives zeros."""
    lens = [1000, 390, 50]
    p = Problem(fmt, 3, G, 2, d, rv, page, lens, n, window, sink)
    bad = [[0, 5, 6, 17, 18, 19, (1000 - 1) // page], [2, (390 - 1) // page], range(-(-50 // page))]
    seen = [SO.window_mask(L, n, window, sink) for L in lens]
    hit = False
    for b, pages in enumerate(bad):
        for x in pages:
            live = seen[b][:, x * page:(x + 1) * page]
            hit |= bool(live.any())
            live[:] = False
            p.table[b, x] = p.dims.num_phys_pages if x % 2 else -3
    assert hit
    p.run()
    assert bkv.read_device_status() == bkv.DEV_BAD_PAGE
    got = p.out.cpu().double().numpy()
    kind = fmt if fmt != "bf16" else "bf16_token" if n * G <= 16 else "bf16_prompt"
    for b, L in enumerate(lens):
        see = np.repeat(seen[b], G, 0)
        for g in range(2):
            hs = slice(g * G, (g + 1) * G)
            a, A, X = reference(p.q[b, :, hs].double().numpy().reshape(-1, d),
                                p.K.values[b][:, g], p.Z.values[b][:, g], see)
            assert_rows(got[b, :, hs].reshape(-1, rv), a, A, X, FMT_WEIGHT[kind],
                        f"{fmt} n{n} b{b} g{g}")
    assert np.all(got[2] == 0)


@pytest.mark.parametrize("G,d,rv,page,n", [(4, 128, 64, 16, 40), (8, 64, 128, 32, 200),
                                           (4, 128, 128, 16, 300), (2, 64, 32, 8, 90)])
@pytest.mark.parametrize("scale", [1.0, 3.0])
def test_bf16_prompts_hold_their_weights_in_16_bits(G, d, rv, page, n, scale):
    """Prompts over bf16 caches are as accurate as single tokens: a weight is its upper
    8 bits (what they leave is below 2^-7 of it) and a bf16 rounding of the rest, off by
    at most 2^-16 of the weight."""
    p = Problem("bf16", 2, G, 2, d, rv, page, [700, 333], n, 0, 0, scale=scale)
    p.run()
    assert bkv.read_device_status() == 0
    p.check(kind="bf16_token")


@pytest.mark.parametrize("n", [1, 6, 100])
def test_large_latents(n):
    """Latents of 2^70, where a token in 200 scores 60 (log2) above the others: the
    sums stay finite, whichever token a reference was taken from."""
    lens = [700, 650, 600, 690]
    p = Problem("bf16", 4, 4, 8, 64, 32, 16, lens, n, 0, 0)
    table = p.table.cpu().numpy()
    rng = np.random.default_rng(5)
    spike = 60 / 1.4427 * 8 / 64  # of all 64 columns, under queries of ones
    p.K = Paged([spike * (rng.random((L, 8, 1)) < 1 / 200) * np.ones((1, 1, 64)) for L in lens],
                "bf16", 16, table, p.dims.num_phys_pages)
    p.Z = Paged([rng.standard_normal((L, 8, 32)) * 2.0 ** 70 for L in lens], "bf16", 16, table,
                p.dims.num_phys_pages)
    p.q = bf16(np.ones((4, n, 32, 64)))
    p.qd = p.q.cuda()
    p.run()
    assert bkv.read_device_status() == 0
    p.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,d,rv,page", [(4, 128, 128, 16), (8, 128, 128, 32), (4, 128, 32, 32),
                                         (8, 128, 32, 16), (2, 128, 96, 16), (1, 64, 96, 32)])
@pytest.mark.parametrize("n,window,sink,lens", [(80, 0, 0, [700, 33, 260]),
                                                (300, 130, 70, [650, 301])])
def test_prompts_of_every_width(fmt, G, d, rv, page, n, window, sink, lens):
    """The prompt kernel's instances differ in their stages and in where the queries
    lie (r_v 128 at d 128 has none of them in tensor memory)."""
    p = _go(fmt, len(lens), G, 2, d, rv, page, lens, n, window, sink)
    p.check(kind="bf16_token" if fmt == "bf16" else fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bound", [2500, 4300, 6500])
@pytest.mark.parametrize("G,d,rv,page,n", [(4, 128, 64, 16, 5), (8, 64, 96, 32, 3),
                                           (8, 128, 128, 32, 4), (1, 64, 128, 16, 31),
                                           (4, 64, 32, 32, 7), (2, 128, 96, 16, 13)])
def test_drafts_whose_bound_passes_the_contexts(fmt, bound, G, d, rv, page, n):
    """17 to 32 rows a group with bounds on the lengths on both sides of the sizes from
    which they are streamed (64 times 2048, 4096 and 6144 tokens): the same answers."""
    lens = [700, 3, 0, 17, 512, 429, 300, 699]
    p = Problem(fmt, 8, G, 8, d, rv, page, lens, n, 0, 0)
    wide = torch.full((8, -(-bound // page)), -1, dtype=torch.int32, device="cuda")
    wide[:, :p.table.shape[1]] = p.table
    p.table, p.dims.max_pages_per_seq, p.msl = wide, wide.shape[1], bound
    p.ws = torch.full((bkv.window_workspace_size(p.dims, n, bound, 0, 0),), 0x7F,
                      dtype=torch.uint8, device="cuda")
    p.run()
    assert bkv.read_device_status() == 0
    p.check(kind="bf16_token" if fmt == "bf16" else fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 6, 24, 200])
def test_the_same_call_gives_the_same_bits(fmt, n):
    p = _go(fmt, 4, 4, 4, 128, 64, 16, [1500, 90, 1333, 700], n, 600, 4)
    first = p.out.clone()
    for fill in (0x00, 0x3C, 0x7F):
        p.ws.fill_(fill)
        p.out.fill_(3.0)
        assert torch.equal(p.run(), first)
