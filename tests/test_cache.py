"""GPU tests of the paged cache: attn_cache_append and attn_fwd_cache against
the FP64 oracle at the sizes and masks where they can go wrong, and both as a
server runs them."""
from __future__ import annotations

import math

import pytest
import torch

import cache_oracle as ref
from scaled_dot_product_10_b200 import attn

pytestmark = pytest.mark.gpu
NAN8, NAN16 = 0x7F, 0x7FC0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


class Pool:
    """A CPU pool with its device copy; every slot that no sequence holds is NaN."""

    def __init__(self, lens, page, h_kv, kind, seed, heads_first=False, extra=2, spread=2.0,
                 filled=None):
        g = torch.Generator().manual_seed(seed)
        self.page, self.h_kv, self.kind = page, h_kv, kind
        pages_of = [-(-max(n, 0) // page) for n in lens]
        self.num = sum(pages_of) + extra
        self.max_pages = max(max(pages_of), 1)
        order = torch.randperm(self.num, generator=g).tolist()
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        e4m3 = kind == "e4m3"
        shape = (self.num, page, h_kv, 128)
        self.scale = [None, None]
        self.pages = []
        for t in range(2):
            x = torch.randn(shape, generator=g)
            if e4m3:
                # scales of any value, not only powers of two
                self.scale[t] = 2.0 ** (spread * torch.randn(self.num, h_kv, generator=g) - 6)
                x = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            else:
                x = x.to(torch.bfloat16)
            self.pages.append(x)
        bits = torch.uint8 if e4m3 else torch.int16
        free = torch.ones(self.num, page, dtype=torch.bool)
        for b, n in enumerate(lens if filled is None else filled):
            for j in range(pages_of[b]):
                pid = order.pop()
                self.table[b, j] = pid
                free[pid, :max(0, min(page, n - j * page))] = False
        for x in self.pages:
            x.view(bits)[free] = NAN8 if e4m3 else NAN16
        self.device(heads_first)

    def device(self, heads_first):
        def put(x):
            if x is None:
                return None
            if heads_first and x.dim() == 4:
                return x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
            return x.cuda()
        self.d_pages = [put(x) for x in self.pages]
        self.d_scale = [put(x) for x in self.scale]
        self.cache = attn.KVCache(*self.d_pages, *self.d_scale)
        self.d_table = self.table.cuda()


def run_attend(pool, lens, news, h_q, causal=True, window=-1, scale=None, pad=0, seed=5, size=1.0,
               max_q=None, uniform=False):
    g = torch.Generator().manual_seed(seed)
    rows = sum(news)
    q = (torch.randn(rows + pad, h_q, 128, generator=g) * size).to(torch.bfloat16)
    scale = 1 / math.sqrt(128) if scale is None else scale
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    o = torch.full((rows + pad, h_q, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((h_q, rows + pad), 7.0, device="cuda")
    attn.attn_fwd_cache(q.cuda(), pool.cache, pool.d_table,
                        torch.tensor(lens, dtype=torch.int32).cuda(),
                        cu_seqlens_q=None if uniform else cu.cuda(),
                        max_seqlen_q=max_q or max(news), causal=causal, window_left=window,
                        scale=scale, o=o, lse=lse)
    assert attn.attn_status() == attn.ATTN_OK
    if pad:
        assert bool((o[rows:] == 7).all()) and bool((lse[:, rows:] == 7).all())
    want = ref.attend(q[:rows], *pool.pages, *pool.scale, pool.table, lens, news, causal, window,
                      scale)
    ref.assert_attend(o, lse, want)
    return q, o, lse


# One token: lengths around a tile and a page, every width of the row tile.
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [257, 1, 40], [1000]])
def test_single_token(kind, lens):
    pool = Pool(lens, 16, 2, kind, seed=sum(lens))
    run_attend(pool, lens, [1] * len(lens), 8, uniform=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (4, 4), (6, 2), (16, 1), (24, 2), (40, 1), (64, 1),
                                      (100, 1), (130, 2)])
def test_head_layouts(kind, h_q, h_kv):
    lens = [200, 77]
    pool = Pool(lens, 32, h_kv, kind, seed=h_q)
    run_attend(pool, lens, [1, 1], h_q)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 48, 64, 128, 136, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_page_sizes(kind, page, heads_first):
    lens = [300, 5, page, page + 1]
    pool = Pool(lens, page, 2, kind, seed=page, heads_first=heads_first)
    run_attend(pool, lens, [1] * 4, 8)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[2, 2], [5, 1], [17, 3], [64, 33], [130, 200]])
@pytest.mark.parametrize("causal", [True, False])
def test_several_rows(kind, news, causal):
    lens = [n + extra for n, extra in zip(news, (150, 0))]
    pool = Pool(lens, 16, 2, kind, seed=sum(news))
    run_attend(pool, lens, news, 6, causal=causal)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 1, 100, 127, 128, 300, 5000, 2 ** 31 - 1])
def test_windows(kind, window):
    lens, news = [700, 130, 60], [1, 130, 7]
    pool = Pool(lens, 32, 2, kind, seed=window)
    run_attend(pool, lens, news, 8, window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_empty_and_padded_rows(kind):
    # a sequence without keys, one without rows, one with more rows than keys
    lens, news = [0, 50, 3, 0, 260], [2, 0, 6, 0, 3]
    pool = Pool(lens, 16, 2, kind, seed=3)
    _, o, lse = run_attend(pool, lens, news, 4, pad=5)
    assert bool((o[:2] == 0).all()) and bool(torch.isinf(lse[:, :2]).all())
    assert bool((o[2:5] == 0).all()) and bool(torch.isinf(lse[:, 2:5]).all())
    run_attend(pool, lens, news, 4, causal=False, pad=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences(kind):
    # more sequences than a CTA has threads, and many of no rows
    lens = [(37 * i) % 150 for i in range(500)]
    news = [0 if i % 5 == 0 else min(1 + i % 3, max(lens[i], 1)) for i in range(500)]
    pool = Pool(lens, 16, 1, kind, seed=11)
    run_attend(pool, lens, news, 2, pad=3)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_cache_is_split(kind):
    lens = [20011, 3]
    pool = Pool(lens, 64, 1, kind, seed=2)
    run_attend(pool, lens, [1, 1], 8)
    run_attend(pool, lens, [3, 2], 8, window=9000)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,h_q", [(1, 1), (1, 12), (7, 4), (40, 1), (33, 5)])
def test_shares_of_many_tiles_and_items(kind, n, h_q):
    """Every CTA has several key tiles, most of them of more than one item."""
    lens = [1400 + 97 * (i % 13) for i in range(90)]
    if n * h_q > 100:
        lens = lens[:30]
    news = [max(1, n - i % 3) for i in range(len(lens))]
    pool = Pool(lens, 48, 1, kind, seed=n)
    run_attend(pool, lens, news, h_q, pad=2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales_of_the_scores(kind, scale):
    lens = [300, 40]
    pool = Pool(lens, 16, 2, kind, seed=21, spread=0.5)
    run_attend(pool, lens, [2, 1], 4, scale=scale)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 1e4])
def test_query_sizes_e4m3(size):
    lens = [140]
    pool = Pool(lens, 16, 1, "e4m3", seed=8)
    run_attend(pool, lens, [1], 8, size=size, scale=0.1 / size)


def test_sink_and_tail_e4m3():
    """One key that takes nearly all the weight and a long even tail: the tail's
    weights, 2^-20 of the largest, keep their bits."""
    n, page = 16384, 64
    pool = Pool([n], page, 1, "e4m3", seed=1, spread=0.0)
    k = torch.zeros(pool.pages[0].shape)
    pool.pages[0] = k.to(torch.float8_e4m3fn)
    pool.pages[0][int(pool.table[0, 0]), 0] = 16.0
    pool.scale[0][:] = 1.0
    pool.device(False)
    q = torch.full((1, 8, 128), 0.0)
    q[..., 0] = 0.875  # the sink's score is 14: the tail's weights are e^-14
    cu = torch.tensor([0, 1], dtype=torch.int32)
    o, lse = attn.attn_fwd_cache(q.to(torch.bfloat16).cuda(), pool.cache, pool.d_table,
                                 torch.tensor([n], dtype=torch.int32).cuda(),
                                 cu_seqlens_q=cu.cuda(), max_seqlen_q=1, scale=1.0)
    want = ref.attend(q.to(torch.bfloat16), *pool.pages, *pool.scale, pool.table, [n], [1], True,
                      -1, 1.0)
    ref.assert_attend(o, lse, want)


def test_scales_of_pages_far_apart_e4m3():
    """V's scales from 0 and 2^-60 to 2^40, and a page of zeros that takes the weight."""
    lens = [512]
    pool = Pool(lens, 32, 1, "e4m3", seed=4)
    for j in range(16):
        pool.scale[1][int(pool.table[0, j]), 0] = (0.0, 2.0 ** -60, 1.0, 2.0 ** 40)[j % 4]
    pool.device(False)
    run_attend(pool, lens, [1], 4)
    pool.scale[1][:] = 0.0
    pool.device(False)
    _, o, _ = run_attend(pool, lens, [1], 4)
    assert bool((o == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_page_numbers_outside_the_pool(kind):
    """They read as zeros and no address follows them."""
    lens = [100]
    pool = Pool(lens, 16, 1, kind, seed=6)
    pool.table[0, 2], pool.table[0, 4] = pool.num, -1
    pool.device(False)
    run_attend(pool, lens, [1], 4)
    # a length past the table's room: the keys there do not exist
    run_attend(Pool([112], 16, 1, kind, seed=6), [5000], [1], 4, causal=False)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,h_q", [([1, 1], 8), ([5, 2], 8), ([1, 1], 128), ([130, 7], 8)])
@pytest.mark.parametrize("window", [0, 50, 200])
def test_slots_before_the_window_hold_anything(kind, news, h_q, window):
    """A server hands pages before the window to others: NaN there, in keys,
    values and the scales of whole pages, changes nothing."""
    lens = [900, 333]
    pool = Pool(lens, 16, 2, kind, seed=window + h_q)
    for b, (length, n) in enumerate(zip(lens, news)):
        first = length - n - window
        for j in range(-(-first // 16)):
            pid, last = int(pool.table[b, j]), min(first - 16 * j, 16)
            for x in pool.d_pages:
                bits = torch.uint8 if kind == "e4m3" else torch.int16
                x.view(bits)[pid, :last] = NAN8 if kind == "e4m3" else NAN16
            if kind == "e4m3" and last == 16:
                for x in pool.d_scale:
                    x[pid] = float("nan")
    run_attend(pool, lens, news, h_q, window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,h_q", [([300, 200], 8), ([300, 200], 128), ([9000, 1200], 8),
                                      ([9000, 1200], 128)])
def test_nan_in_a_seen_key_reaches_the_rows(kind, lens, h_q):
    """Short tables and shares that are joined, few rows and many."""
    pool = Pool(lens, 16, 2, kind, seed=h_q)
    clean = run_attend(pool, lens, [1, 1], h_q)[1:]
    bits, nan = (torch.uint8, NAN8) if kind == "e4m3" else (torch.int16, NAN16)
    at = (int(pool.table[0, 10]), 3, 1)
    seen = slice(h_q // 2, h_q)  # the query heads of key/value head 1

    def run():
        q = torch.randn(2, h_q, 128, generator=torch.Generator().manual_seed(5))
        cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
        return attn.attn_fwd_cache(q.to(torch.bfloat16).cuda(), pool.cache, pool.d_table,
                                   torch.tensor(lens, dtype=torch.int32).cuda(), cu_seqlens_q=cu,
                                   max_seqlen_q=1)
    for t, dims in ((0, slice(0, 128)), (1, slice(7, 8))):
        keep = pool.d_pages[t][at].clone()
        pool.d_pages[t].view(bits)[at][7] = nan
        o, lse = run()
        pool.d_pages[t][at] = keep
        assert attn.attn_status() == attn.ATTN_OK
        assert bool(o[0, seen, dims].isnan().all())
        assert bool(lse[seen, 0].isnan().all()) == (t == 0)
        o[0, seen, dims] = clean[0][0, seen, dims]
        if t == 0:
            lse[seen, 0] = clean[1][seen, 0]
        assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


def test_strided_queries_stream_and_graph():
    lens = [400, 90, 33]
    pool = Pool(lens, 16, 2, "e4m3", seed=9)
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    wide = torch.randn(3, 20, 128, device="cuda").to(torch.bfloat16)
    q = wide[:, 4:12]
    want = ref.attend(q.cpu(), *pool.pages, *pool.scale, pool.table, lens, [1, 1, 1], True, -1,
                      128 ** -0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = attn.attn_fwd_cache(q, pool.cache, pool.d_table, seqlens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref.assert_attend(o, lse, want)
    ws = torch.empty(attn.cache_workspace_bytes(8, 2, 1), dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # nothing in it has to be set
    o.zero_(), lse.zero_()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs share a workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.attn_fwd_cache(q, pool.cache, pool.d_table, seqlens, o=o, lse=lse, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    ref.assert_attend(o, lse, want)
    first = o.clone(), lse.clone()
    graphs[0].replay()
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)  # no order of sums by chance
    # the graph follows its tensors: other lengths
    seqlens.copy_(torch.tensor([17, 90, 0], dtype=torch.int32))
    graphs[1].replay()
    ref.assert_attend(o, lse, ref.attend(q.cpu(), *pool.pages, *pool.scale, pool.table, [17, 90, 0],
                                         [1, 1, 1], True, -1, 128 ** -0.5))
    assert attn.attn_status() == attn.ATTN_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_streams_at_once(kind):
    """Calls side by side, each with a workspace of its own."""
    lens = [3000, 700]
    pool = Pool(lens, 64, 1, kind, seed=14)
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    news = [1, 40]
    streams = [torch.cuda.Stream() for _ in news]
    cases = []
    for n in news:
        q = torch.randn(2 * n, 4, 128, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
        want = ref.attend(q, *pool.pages, *pool.scale, pool.table, lens, [n, n], True, -1, 128 ** -0.5)
        cases.append((q.cuda(), want))
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [attn.attn_fwd_cache(q, pool.cache, pool.d_table, seqlens, stream=s)
                for (q, _), s in zip(cases, streams)]
        torch.cuda.synchronize()
        for (o, lse), (_, want) in zip(outs, cases):
            ref.assert_attend(o, lse, want)
    assert attn.attn_status() == attn.ATTN_OK


def test_launches_and_bounds():
    """One launch for short tables; rows past max_seqlen_q are left alone."""
    pool = Pool([500, 512], 16, 2, "e4m3", seed=15)
    run_attend(pool, [500, 512], [1, 1], 8)
    assert attn.last_launch_count() == 1
    pool = Pool([500, 513], 16, 2, "e4m3", seed=15)
    run_attend(pool, [500, 513], [1, 1], 8)
    assert attn.last_launch_count() == 2
    q = torch.randn(8, 4, 128).to(torch.bfloat16).cuda()
    sl = torch.tensor([500, 513], dtype=torch.int32).cuda()
    o = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 8), 7.0, device="cuda")
    attn.attn_fwd_cache(q, pool.cache, pool.d_table, sl, max_seqlen_q=3, o=o, lse=lse)
    whole, _ = attn.attn_fwd_cache(q, pool.cache, pool.d_table, sl)
    assert attn.attn_status() == attn.ATTN_OK
    for i in range(8):
        if i % 4 == 3:
            assert bool((o[i] == 7).all()) and bool((lse[:, i] == 7).all())
        else:
            assert float((o[i].float() - whole[i].float()).abs().max()) < 2.0 ** -5


# ------------------------------------------------------------------ append
def inv_freq_of(rotary):
    if rotary == 0:
        return None
    return (10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / rotary)).float()


def run_append(pool, lens, news, h_q, rotary=128, interleaved=False, uniform=False, pad=0, seed=5,
               size=1.0, first_shift=0):
    g = torch.Generator().manual_seed(seed)
    rows, h_kv = sum(news), pool.h_kv
    qkv = torch.randn(rows + pad, h_q + 2 * h_kv, 128, generator=g) * size
    qkv = qkv.to(torch.bfloat16)
    q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
    inv = inv_freq_of(rotary)
    d = qkv.cuda()
    dq, dk, dv = d[:, :h_q], d[:, h_q:h_q + h_kv], d[:, h_q + h_kv:]
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    before = [x.cpu().clone() for x in pool.d_pages]
    want = ref.append(k[:rows], v[:rows], *before,
                      *[None if s is None else s.cpu() for s in pool.d_scale], pool.table, lens,
                      news, inv, interleaved)
    q_out = torch.full((rows + pad, h_q, 128), 7.0, dtype=torch.bfloat16, device="cuda") \
        if h_q else None
    got = attn.attn_cache_append(pool.cache, dk, dv, pool.d_table,
                                 torch.tensor(lens, dtype=torch.int32).cuda(),
                                 cu_seqlens=None if uniform else cu.cuda(), max_seqlen=max(news),
                                 q=dq if h_q else None, q_out=q_out,
                                 inv_freq=None if inv is None else inv.cuda(),
                                 interleaved=interleaved)
    torch.cuda.synchronize()
    assert got is q_out
    e4m3 = pool.kind == "e4m3"
    for t in range(2):
        ref.assert_pages(pool.d_pages[t], want[t], e4m3, want[4], before[t])
        if e4m3:
            assert torch.equal(pool.d_scale[t].cpu().double(), want[2 + t])
    if h_q:
        row = 0
        for length, n in zip(lens, news):
            y = ref.rotate(q[row:row + n].double(), length - n, inv, interleaved)
            off = (q_out[row:row + n].cpu().double() - y).abs()
            assert bool((off <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * size * 6).all())
            row += n
        if pad:
            assert bool((q_out[rows:] == 7).all())
    return qkv


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rotary", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotations(kind, rotary, interleaved):
    lens, news = [40, 9, 3], [7, 9, 1]
    pool = Pool(lens, 16, 2, kind, seed=rotary, filled=[a - b for a, b in zip(lens, news)])
    run_append(pool, lens, news, 4, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [8, 24, 64, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append_pages(kind, page, heads_first):
    # from a page's middle, over its end, whole pages, one row, no rows, padding
    lens, news = [page + 3, 300, page, 1, 20], [5, 290, page, 1, 0]
    pool = Pool(lens, page, 3, kind, seed=page, heads_first=heads_first,
                filled=[a - b for a, b in zip(lens, news)])
    run_append(pool, lens, news, 6, pad=4)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_single_tokens(kind):
    lens = [1 + 13 * i % 70 for i in range(300)]
    pool = Pool(lens, 16, 1, kind, seed=1, filled=[n - 1 for n in lens])
    run_append(pool, lens, [1] * 300, 2, uniform=True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_scale_growth(interleaved):
    """Token after token of growing size into the same pages: the scale grows,
    the older tokens are coded again; smaller ones leave it."""
    page, h_kv = 16, 2
    pool = Pool([page], page, h_kv, "e4m3", seed=5, filled=[0])
    for t in range(page):
        size = [1.0, 3.0, 0.1, 40.0, 0.5, 1e4, 2.0, 1e-3][t % 8]
        run_append(pool, [t + 1], [1], 0, seed=t, size=size, interleaved=interleaved)


@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-20, 1e20, 1e36])
def test_append_extreme_sizes(size):
    lens, news = [12, 30], [12, 2]
    pool = Pool(lens, 8, 1, "e4m3", seed=2, filled=[0, 28])
    for s in pool.d_scale:
        s.zero_()
    for x in pool.d_pages:
        x.view(torch.uint8).zero_()
    run_append(pool, lens, news, 0, rotary=0, size=size)


def test_append_scale_borders():
    """Bounds at, just under and just over 448 times a power of two."""
    page = 8
    for i, top in enumerate([448.0, 450.0, 446.0, 1.75, 1.7578125, 3.5, 0.875]):
        pool = Pool([page], page, 1, "e4m3", seed=3, filled=[0])
        x = torch.zeros(page, 1, 128)
        x[2, 0, 5] = -top
        x = x.to(torch.bfloat16).cuda()
        attn.attn_cache_append(pool.cache, x, x, pool.d_table,
                               torch.tensor([page], dtype=torch.int32).cuda())
        want = ref.pow2_scale(float(x.float().abs().max()))
        for s in pool.d_scale:
            assert float(s[int(pool.table[0, 0]), 0]) == want


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_far_positions(kind):
    """Positions past 2^24, where FP32 angles lose their phase: the pages of all
    but the last tokens are outside the pool."""
    page, n = 64, 5
    length = (1 << 24) + 77
    pool = Pool([page * 2], page, 1, kind, seed=4, filled=[(length - n) % page])
    table = torch.full((1, length // page + 1), -1, dtype=torch.int32)
    table[0, (length - n) // page:] = pool.table[0, 0]
    pool.table, pool.d_table = table, table.cuda()
    assert (length - n) // page == (length - 1) // page
    run_append(pool, [length], [n], 2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_refuses_bad_places(kind):
    """Negative positions, pages outside the pool and past the table are left."""
    pool = Pool([40], 8, 1, kind, seed=7, filled=[20])
    pool.table[0, 3] = pool.num + 5
    pool.d_table = pool.table.cuda()
    run_append(pool, [40], [20], 2)
    pool = Pool([40], 8, 1, kind, seed=8, filled=[0])
    run_append(pool, [3], [10], 2)     # seven rows before the start
    pool = Pool([40], 8, 1, kind, seed=9, filled=[30])
    run_append(pool, [60], [30], 2)    # twenty past the table


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_captured_and_on_a_stream(kind):
    """A captured step appends wherever its tensors point when it is replayed."""
    lens, page = [20, 5], 8
    pool = Pool([40, 40], page, 2, kind, seed=12, filled=[19, 4])
    g = torch.Generator().manual_seed(3)
    inv = inv_freq_of(64)
    k, v = (torch.randn(2, 2, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    dk, dv, dinv = k.cuda(), v.cuda(), inv.cuda()
    seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attn_cache_append(pool.cache, dk, dv, pool.d_table, seqlens, inv_freq=dinv)
    side = torch.cuda.Stream()
    for step in range(12):
        before = [x.cpu().clone() for x in pool.d_pages]
        want = ref.append(k, v, *before, *[None if s is None else s.cpu() for s in pool.d_scale],
                          pool.table, lens, [1, 1], inv, False)
        if step % 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            attn.attn_cache_append(pool.cache, dk, dv, pool.d_table, seqlens, inv_freq=dinv,
                                   stream=side)
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for t in range(2):
            ref.assert_pages(pool.d_pages[t], want[t], kind == "e4m3", want[4], before[t])
            if kind == "e4m3":
                assert torch.equal(pool.d_scale[t].cpu().double(), want[2 + t])
        lens = [n + 1 for n in lens]
        k = k * (1.5 if step % 3 else 0.2)
        dk.copy_(k)
        seqlens.copy_(torch.tensor(lens, dtype=torch.int32))


def test_append_rows_past_the_bound():
    """max_seqlen cuts a sequence's rows; the others keep their positions."""
    for kind in ("bf16", "e4m3"):
        pool = Pool([30], 8, 1, kind, seed=13, filled=[20])
        x = torch.randn(10, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        before = [p.cpu().clone() for p in pool.d_pages]
        d = x.cuda()
        attn.attn_cache_append(pool.cache, d[:, :1], d[:, 1:], pool.d_table,
                               torch.tensor([30], dtype=torch.int32).cuda(), max_seqlen=6,
                               inv_freq=inv_freq_of(128).cuda())
        # the first six rows, at positions 20 .. 25
        want = ref.append(x[:6, :1], x[:6, 1:], *before,
                          *[None if s is None else s.clone() for s in pool.scale], pool.table,
                          [26], [6], inv_freq_of(128), False)
        for t in range(2):
            ref.assert_pages(pool.d_pages[t], want[t], kind == "e4m3", want[4], before[t])


def test_offsets_past_32_bits():
    """A pool of over 2^32 elements: pages at its far end."""
    page, h_kv = 64, 1
    num = (1 << 32) // (page * 128) + 8
    k = torch.empty(num, page, h_kv, 128, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    ks = torch.zeros(num, h_kv, device="cuda")
    vs = torch.zeros_like(ks)
    cache = attn.KVCache(k, v, ks, vs)
    ids = [num - 1, 3, num - 5]
    table = torch.tensor([ids], dtype=torch.int32)
    n = 150
    x = torch.randn(n, 2, 128).to(torch.bfloat16)
    seqlens = torch.tensor([n], dtype=torch.int32).cuda()
    d = x.cuda()
    attn.attn_cache_append(cache, d[:, :1], d[:, 1:], table.cuda(), seqlens)
    sk, sv = k[ids].cpu(), v[ids].cpu()
    small = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    blank = torch.zeros(3, page, h_kv, 128, dtype=torch.float8_e4m3fn)
    want = ref.append(x[:, :1], x[:, 1:], blank, blank, torch.zeros(3, 1), torch.zeros(3, 1),
                      small, [n], [n], None, False)
    keep = want[4] == 2
    for got, w in ((sk, want[0]), (sv, want[1])):
        off = (got[keep].double() - w[keep]).abs()
        assert bool((off <= 2.0 ** -4 * w[keep].abs() + 2.0 ** -10).all())
    q = torch.randn(1, 4, 128).to(torch.bfloat16)
    o, lse = attn.attn_fwd_cache(q.cuda(), cache, table.cuda(), seqlens)
    ref.assert_attend(o, lse, ref.attend(q, sk, sv, ks[ids].cpu(), vs[ids].cpu(), small, [n], [1],
                                         True, -1, 128 ** -0.5))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_server_run(kind):
    """Prompts of different lengths, then tokens one by one, each step appended
    and attended over; against attention over all keys as they were given,
    within what the cache's type rounds."""
    h_q, h_kv, page, steps = 8, 2, 16, 20
    prompts = [37, 1, 64]
    total = [n + steps for n in prompts]
    pool = Pool(total, page, h_kv, kind, seed=31, filled=[0, 0, 0])
    inv = inv_freq_of(128)
    g = torch.Generator().manual_seed(77)
    keys = [torch.zeros(0, h_kv, 128, dtype=torch.float64) for _ in prompts]
    vals = [torch.zeros(0, h_kv, 128, dtype=torch.float64) for _ in prompts]
    for step in range(steps + 1):
        news = prompts if step == 0 else [1, 1, 1]
        lens = [n + step for n in prompts]
        qkv = torch.randn(sum(news), h_q + 2 * h_kv, 128, generator=g).to(torch.bfloat16)
        d = qkv.cuda()
        cu = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
        sl = torch.tensor(lens, dtype=torch.int32).cuda()
        q = attn.attn_cache_append(pool.cache, d[:, h_q:h_q + h_kv], d[:, h_q + h_kv:],
                                   pool.d_table, sl, cu_seqlens=cu, max_seqlen=max(news),
                                   q=d[:, :h_q], inv_freq=inv.cuda())
        o, lse = attn.attn_fwd_cache(q, pool.cache, pool.d_table, sl, cu_seqlens_q=cu,
                                     max_seqlen_q=max(news))
        held = [x.cpu() for x in pool.d_pages], [None if s is None else s.cpu()
                                                 for s in pool.d_scale]
        ref.assert_attend(o, lse, ref.attend(q.cpu(), *held[0], *held[1], pool.table, lens, news,
                                             True, -1, 128 ** -0.5))
        row = 0
        for b, n in enumerate(news):
            part = qkv[row:row + n].double()
            keys[b] = torch.cat((keys[b], ref.rotate(part[:, h_q:h_q + h_kv], lens[b] - n, inv,
                                                     False)))
            vals[b] = torch.cat((vals[b], part[:, h_q + h_kv:]))
            row += n
    # The cache holds what was appended: one rounding for each growth of a
    # scale and one more (a power of two shifts exponents: only subnormals,
    # 2^-10 of the scale, are rounded again).
    for b in range(len(prompts)):
        for t, want in ((0, keys[b]), (1, vals[b])):
            for h in range(h_kv):
                got = ref.page_rows(held[0][t], held[1][t], pool.table[b], h, total[b])
                if kind == "bf16":
                    bound = 2.0 ** -8 * want[:, h].abs() + 2.0 ** -18
                else:
                    unit = torch.stack([held[1][t][int(pool.table[b, j // page]), h].double()
                                        for j in range(total[b])])[:, None]
                    bound = 2.0 ** -4 * want[:, h].abs() + 2.0 ** -9 * unit
                assert bool(((got - want[:, h]).abs() <= bound).all())
    assert attn.attn_status() == attn.ATTN_OK
