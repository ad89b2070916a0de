"""Pages of a paged cache: copying, forking, reserving, freeing, compacting.

On the CPU: the host oracle (oracle/pages.py) keeps the counts equal to what
the tables hold and every sequence's tokens unchanged over random sequences of
calls, and the entry points refuse what they should. On the GPU: every call
equals the oracle's bit for bit, tables, counts, pages and error bits, and a
serving run over the 4-bit cache (prompt, samples, growth, retirement) attends
as it would without sharing.
"""
import ctypes

import numpy as np
import pytest

import synth
import w8a8_quantized_decode_gb300 as a8w8
from gpu_util import to_dev, to_host
from oracle import kv_i4, pages

gpu = pytest.mark.gpu
FAKE = 0x10000
BITS = dict(BLOCK=a8w8.DEVERR_BLOCK, CTX=a8w8.DEVERR_CTX, ROW=a8w8.DEVERR_ROW,
            PAGES=a8w8.DEVERR_PAGES, ALIAS=a8w8.DEVERR_ALIAS)


@pytest.fixture(scope="module")
def lib():
    a8w8.build()
    return a8w8.lib()


class State:
    """Tables and a pool on the host (and, with on_gpu, the same on the device)."""

    def __init__(self, seed, B, M, N, page, words=(8, 2, 3)):
        rng = np.random.default_rng(seed)
        self.page, self.rng = page, rng
        self.pool = [rng.integers(-2 ** 31, 2 ** 31, (N, page, w)).astype(np.int32) for w in words]
        self.bt = np.full((B, M), -1, np.int32)
        self.ctx = np.zeros(B, np.int32)
        self.ref = np.zeros(N, np.int32)

    def on_gpu(self):
        self.g = [to_dev(a) for a in (self.bt, self.ctx, self.ref)]
        self.gp = [to_dev(c) for c in self.pool]
        self.handle = a8w8.PagePool(self.gp, len(self.ref), self.page)
        return self

    def check(self, errors=()):
        want = 0
        for e in errors:
            want |= BITS[e]
        assert a8w8.read_device_errors() == want
        for got, host in zip(self.g + self.gp, [self.bt, self.ctx, self.ref] + self.pool):
            assert np.array_equal(to_host(got), host)

    def sequences(self):
        """Every row's tokens, by value."""
        out = []
        for b, n in enumerate(self.ctx):
            t = np.arange(n)
            p = self.bt[b][t // self.page]
            out.append([c[p, t % self.page] for c in self.pool])
        return out

    def counts_match(self):
        held = np.bincount(self.bt[self.bt >= 0], minlength=len(self.ref))
        return np.array_equal(held, self.ref)


def _fill(s, rows, lens):
    """Rows with pages and contexts, in place, from the front of the free pages."""
    pages.reserve(s.page, s.bt, s.ref, rows, lens)
    s.ctx[rows] = lens


def _same(a, b):
    return all(np.array_equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


# ---------------------------------------------------------------------------
# oracle (CPU)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(4))
def test_oracle_keeps_counts_and_sequences(seed):
    s = State(seed, 12, 6, 40, 4)
    rng = np.random.default_rng(seed)
    _fill(s, [0, 1, 2], [9, 16, 1])
    for _ in range(40):
        live, empty = np.flatnonzero(s.ctx), np.flatnonzero((s.ctx == 0) & (s.bt[:, 0] < 0))
        what = rng.integers(4)
        before = s.sequences()
        if what == 0 and len(live) and len(empty):
            p, c = rng.choice(live, 2), rng.permutation(empty)[:2]
            err = pages.fork(s.pool, s.page, s.bt, s.ctx, s.ref, p, c)
            assert err <= {"PAGES"}
            after = s.sequences()
            assert _same([before[b] for b in live], [after[b] for b in live])
            for i, b in enumerate(c):
                if s.ctx[b]:
                    assert _same([before[p[i]]], [after[b]])
        elif what == 1:
            pages.reserve(s.page, s.bt, s.ref, [0, 5], rng.integers(0, 24, 2))
        elif what == 2 and len(live) > 2:
            pages.free(s.bt, s.ctx, s.ref, rng.choice(live, 2))
        else:
            err, n = pages.compact(s.pool, s.bt, s.ref)
            assert not err and (s.ref[:n] > 0).all() and not s.ref[n:].any()
            assert _same(before, s.sequences())
        assert s.counts_match()


def test_oracle_copy_by_hand():
    pool = [np.arange(6).reshape(6, 1)]
    assert pages.copy_pages(pool, [0, 1, -1, 5, 2], [3, 4, 0, 5, -1]) == set()
    assert pool[0][:, 0].tolist() == [0, 1, 2, 0, 1, 5]
    # the first of two pairs into a page; no pair into a page that is read; no page out of range
    assert pages.copy_pages(pool, [5, 2, 0, 9], [1, 1, 2, 0]) == {"ALIAS", "BLOCK"}
    assert pool[0][:, 0].tolist() == [0, 5, 2, 0, 1, 5]


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------

def test_page_operation_validation(lib):
    INV, SHAPE, WS = a8w8.ERR_INVALID_ARG, a8w8.ERR_UNSUPPORTED_SHAPE, a8w8.ERR_WORKSPACE

    def pool(n=2, ptr=FAKE, size=1024):
        return (ctypes.c_void_p * n)(*[ptr] * n), (ctypes.c_size_t * n)(*[size] * n), n

    def copy(c=None, N=8, src=FAKE, n=4):
        return lib.paged_copy_pages(*(c or pool()), N, src, FAKE, n, None)

    def fork(c=None, N=8, page=16, bt=FAKE, B=4, M=4, n=2, ws=FAKE, wsb=1 << 30):
        return lib.paged_fork(*(c or pool()), N, page, bt, FAKE, FAKE, B, M, FAKE, FAKE, n, ws, wsb,
                              None)

    def reserve(N=8, page=16, bt=FAKE, B=4, M=4, n=2, ws=FAKE, wsb=1 << 30):
        return lib.paged_reserve(bt, FAKE, B, M, N, page, FAKE, FAKE, n, ws, wsb, None)

    def free(N=8, bt=FAKE, B=4, M=4, n=2):
        return lib.paged_free(bt, FAKE, FAKE, B, M, N, FAKE, n, None)

    def compact(c=None, N=8, bt=FAKE, B=4, M=4, live=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.paged_compact(*(c or pool()), N, bt, FAKE, B, M, live, ws, wsb, None)

    for f in (copy, fork, compact):
        assert f(c=pool(n=257)) == SHAPE
        assert f(c=pool(size=1022)) == SHAPE          # not 4-byte words
        assert f(c=pool(size=0)) == SHAPE
        assert f(c=pool(size=1 << 31)) == SHAPE
        assert f(c=pool(ptr=None)) == INV
        assert f(c=pool(ptr=FAKE + 4)) == INV
        assert f(c=(None, None, 2)) == INV
        assert f(c=pool()[:2] + (0,)) == INV
        assert f(N=1 << 21) == SHAPE
        assert f(N=0) == INV
    assert fork(c=pool(size=16 * 4 + 4)) == SHAPE     # not 4-byte words per token
    for f in (fork, reserve, free, compact):
        assert f(B=0) == INV and f(M=0) == INV and f(bt=None) == INV and f(bt=FAKE + 8) == INV
        assert f(N=1 << 21) == SHAPE
        assert f(M=(1 << 24) + 1) == SHAPE
    for f in (fork, reserve):
        assert f(page=0) == INV
        assert f(M=1 << 22, page=16) == SHAPE
    for f in (copy, fork, reserve, free):
        assert f(n=-1) == INV
        assert f(n=0) == a8w8.OK
    assert copy(src=None) == INV
    assert compact(live=FAKE + 2) == INV
    for f, n in ((fork, 2), (reserve, 2), (compact, 0)):
        need = lib.a8w8_pages_workspace_bytes(8, 4, n)
        assert need > 0 and f(ws=None) == WS and f(wsb=need - 1) == WS and f(ws=FAKE + 8) == WS
    assert lib.a8w8_pages_workspace_bytes(0, 4, 1) == 0
    assert lib.a8w8_pages_workspace_bytes(8, 4, -1) == 0


def test_pool_refuses_host_tensors():
    import torch
    with pytest.raises(a8w8.A8W8Error):
        a8w8.PagePool([torch.zeros(4, 4)], 4, 1)
    with pytest.raises(a8w8.A8W8Error):
        a8w8.PagePool([], 4, 1)


# ---------------------------------------------------------------------------
# each call against the oracle (GPU)
# ---------------------------------------------------------------------------

def _i32(v):
    return to_dev(np.asarray(v, np.int32))


@gpu
@pytest.mark.parametrize("words", [(4,), (8, 2, 3), (1, 5000)])
@pytest.mark.parametrize("n", [1, 7, 200])
def test_copy(words, n):
    s = State(n, 2, 2, 500, 3, words).on_gpu()
    p = s.rng.permutation(500).astype(np.int32)
    src, dst = p[:n].copy(), p[n:2 * n].copy()
    if n > 1:
        src[1] = -1
        dst[3] = src[3]
        src[5] = src[4]                    # one page copied twice
    a8w8.read_device_errors()
    a8w8.paged_copy_pages(s.handle, _i32(src), _i32(dst))
    assert pages.copy_pages(s.pool, src, dst) == set()
    s.check()


@gpu
def test_copy_conflicts_and_ranges():
    s = State(3, 2, 2, 30, 4).on_gpu()
    src = [0, 1, 2, 30, 5, 6, 7, 8, 9, 9, 2 ** 31 - 1, 12]
    dst = [10, 10, 0, 11, 31, 13, 14, 7, 9, 15, 16, -2 ** 31]
    a8w8.read_device_errors()
    a8w8.paged_copy_pages(s.handle, _i32(src), _i32(dst))
    err = pages.copy_pages(s.pool, src, dst)
    assert err == {"ALIAS", "BLOCK"}
    s.check(err)
    # random lists, mostly in conflict, over several checking batches
    src, dst = (s.rng.integers(-1, 30, 400).astype(np.int32) for _ in range(2))
    a8w8.paged_copy_pages(s.handle, _i32(src), _i32(dst))
    s.check(pages.copy_pages(s.pool, src, dst))
    a8w8.paged_copy_pages(s.handle, _i32([]), _i32([]))
    s.check()


@gpu
@pytest.mark.parametrize("page,words", [(16, (4, 1)), (5, (3, 8)), (1, (4,)), (64, (512, 4))])
def test_fork(page, words):
    B, M, N = 40, 9, 300
    s = State(page, B, M, N, page, words)
    lens = [1, page, page + 1, M * page, 3 * page, 4 * page - 1, 2]
    _fill(s, np.arange(7) * 2, lens)
    s.on_gpu()
    parents = np.array([0, 2, 4, 4, 6, 8, 10, 10, 10, 12, -1, 20, 4], np.int32)
    children = np.array([1, 3, 5, 7, 9, 11, 13, 15, 17, 19, 21, 23, -3], np.int32)
    a8w8.read_device_errors()
    a8w8.paged_fork(s.handle, *s.g, _i32(parents), _i32(children))
    assert pages.fork(s.pool, page, s.bt, s.ctx, s.ref, parents, children) == set()
    assert s.counts_match()
    s.check()


@gpu
def test_fork_refusals_and_full_pool():
    page, B, M = 4, 16, 4
    s = State(1, B, M, 12, page)
    _fill(s, [0, 1, 2, 3], [6, 8, 3, 16])          # 9 pages of 12
    s.bt[4, 0] = 11                                # in use though empty
    s.ref[11] = 1
    s.ctx[5], s.bt[5, :2] = 7, [99, 0]             # a bad block id
    s.ctx[6] = 17                                  # context out of range
    s.on_gpu()
    parents = [0, 0, 1, 0, 16, 0, 0, 5, 6, 2, 0, 3, 2]
    children = [7, 7, 3, 4, 8, 16, 1, 9, 10, 11, 12, 13, 14]
    a8w8.read_device_errors()
    a8w8.paged_fork(s.handle, *s.g, _i32(parents), _i32(children))
    err = pages.fork(s.pool, page, s.bt, s.ctx, s.ref, parents, children)
    assert err == {"ALIAS", "ROW", "BLOCK", "CTX", "PAGES"}
    s.check(err)
    assert s.ctx[13] == 16 and s.ctx[12] == 0      # a fork that needs no page is carried out


@gpu
@pytest.mark.parametrize("seed", range(3))
def test_fork_many(seed):
    """More forks than the plan has warps or threads, and a nearly full pool."""
    page, B, M, N = 8, 3000, 5, 4099
    s = State(seed, B, M, N, page, (2,))
    parents = np.arange(500)
    _fill(s, parents, s.rng.integers(0, M * page + 1, 500))
    s.on_gpu()
    p = s.rng.integers(0, 500, 2400).astype(np.int32)
    c = (500 + s.rng.permutation(2500)[:2400]).astype(np.int32)
    a8w8.read_device_errors()
    a8w8.paged_fork(s.handle, *s.g, _i32(p), _i32(c))
    err = pages.fork(s.pool, page, s.bt, s.ctx, s.ref, p, c)
    assert s.counts_match()
    s.check(err)


@gpu
def test_reserve():
    page, B, M, N = 16, 50, 70, 900
    s = State(2, B, M, N, page, (1,))
    _fill(s, [3, 4], [40, 16])
    s.bt[5, [0, 2, 40]] = [880, 881, 882]          # holes inside a row are filled
    s.ref[[880, 881, 882]] = 1
    s.on_gpu()
    rows = [3, 9, 4, -1, 5, 10, 11, 9, 50, 12, 13]
    tokens = [41, 0, 16 * 70, 5, 16 * 45, 1, -1, 30, 4, 16 * 70 + 1, 100]
    a8w8.read_device_errors()
    a8w8.paged_reserve(s.handle, s.g[0], s.g[2], _i32(rows), _i32(tokens))
    err = pages.reserve(page, s.bt, s.ref, rows, tokens)
    assert err == {"ALIAS", "ROW", "CTX"}
    s.check(err)
    # until the pool is full: the first row that does not fit, and those behind it
    rows = np.arange(14, 50)
    tokens = s.rng.integers(1, M * page, len(rows))
    a8w8.paged_reserve(s.handle, s.g[0], s.g[2], _i32(rows), _i32(tokens))
    err = pages.reserve(page, s.bt, s.ref, rows, tokens)
    assert err == {"PAGES"}
    s.check(err)
    assert s.counts_match()


@gpu
def test_reserve_many_rows():
    page, B, M, N = 4, 2500, 3, 6001
    s = State(7, B, M, N, page, (1,)).on_gpu()
    rows = s.rng.permutation(B)
    tokens = s.rng.integers(0, M * page + 1, B)
    a8w8.read_device_errors()
    a8w8.paged_reserve(s.handle, s.g[0], s.g[2], _i32(rows), _i32(tokens))
    s.check(pages.reserve(page, s.bt, s.ref, rows, tokens))


@gpu
@pytest.mark.parametrize("n", [1, 40, 1500])
def test_reserve_far_more_than_the_pool(n):
    page, B, M, N = 1, 2000, 5000, 37
    s = State(n, B, M, N, page, (1,)).on_gpu()
    rows = s.rng.permutation(B)[:n]
    tokens = np.full(n, M)
    tokens[n // 2:] = 30
    a8w8.read_device_errors()
    a8w8.paged_reserve(s.handle, s.g[0], s.g[2], _i32(rows), _i32(tokens))
    err = pages.reserve(page, s.bt, s.ref, rows, tokens)
    assert err == ({"PAGES"} if n > 1 else set()) and (n > 1 or s.ref.sum() == 30)
    s.check(err)


@gpu
def test_free():
    page, B, M = 4, 20, 40
    s = State(5, B, M, 400, page)
    _fill(s, np.arange(10), s.rng.integers(1, M * page + 1, 10))
    pages.fork(s.pool, page, s.bt, s.ctx, s.ref, [0, 0, 1], [10, 11, 12])
    s.on_gpu()
    rows = [0, 3, 3, -1, 12, 19, 10, 3]
    a8w8.read_device_errors()
    a8w8.paged_free(s.handle, *s.g, _i32(rows))
    assert pages.free(s.bt, s.ctx, s.ref, rows) == set()
    assert s.counts_match()
    s.check()
    # pages that are free already, ids and rows out of range
    s.ref[s.bt[5, 0]] = 0
    s.bt[6, 1] = 400
    s.g[2].copy_(to_dev(s.ref))
    s.g[0].copy_(to_dev(s.bt))
    rows = [5, 6, 20]
    a8w8.paged_free(s.handle, *s.g, _i32(rows))
    err = pages.free(s.bt, s.ctx, s.ref, rows)
    assert err == {"BLOCK", "ROW"}
    s.check(err)


@gpu
@pytest.mark.parametrize("N,words", [(1, (4,)), (37, (4, 1)), (4101, (3,)), (9000, (64, 8))])
def test_compact(N, words):
    page, B, M = 2, 64, 70
    s = State(N, B, M, N, page, words)
    order = s.rng.permutation(N)
    used = order[:N // 2 + 1]
    at = s.rng.permutation(B * M)[:min(len(used), B * M)]
    s.bt.reshape(-1)[at] = used[:len(at)]
    s.ref[:] = np.bincount(s.bt[s.bt >= 0], minlength=N)
    s.on_gpu()
    a8w8.read_device_errors()
    live = a8w8.paged_compact(s.handle, s.g[0], s.g[2])
    err, n = pages.compact(s.pool, s.bt, s.ref)
    assert not err and int(live) == n
    s.check()
    a8w8.paged_compact(s.handle, s.g[0], s.g[2])       # nothing left to move
    s.check()


@gpu
def test_compact_bad_entries_and_full_pool():
    s = State(8, 4, 6, 20, 2)
    s.bt[0, :3], s.bt[1, :2] = [19, 3, 25], [15, 18]   # page 18 is free, 25 does not exist
    s.ref[[19, 3, 15]] = [2, 1, 1]
    s.bt[2, 0] = 19
    s.on_gpu()
    a8w8.read_device_errors()
    a8w8.paged_compact(s.handle, s.g[0], s.g[2])
    err, _ = pages.compact(s.pool, s.bt, s.ref)
    assert err == {"BLOCK"}
    s.check(err)
    s.ref[:] = 1
    s.g[2].copy_(to_dev(s.ref))
    s.bt[:] = -1
    s.g[0].copy_(to_dev(s.bt))
    assert int(a8w8.paged_compact(s.handle, s.g[0], s.g[2])) == 20
    s.check()


@gpu
@pytest.mark.parametrize("seed", range(3))
def test_random_calls(seed):
    """Random calls in a row, captured state compared after each."""
    s = State(seed, 40, 8, 150, 4, (5, 4)).on_gpu()
    rng = np.random.default_rng(seed + 50)
    a8w8.read_device_errors()
    for _ in range(60):
        what, n = rng.integers(5), int(rng.integers(1, 12))
        a, b = rng.integers(-1, 41, n), rng.integers(-1, 41, n)
        if what == 0:
            a8w8.paged_fork(s.handle, *s.g, _i32(a), _i32(b))
            err = pages.fork(s.pool, 4, s.bt, s.ctx, s.ref, a, b)
        elif what in (1, 2):
            tok = rng.integers(0, 34, n)
            a8w8.paged_reserve(s.handle, s.g[0], s.g[2], _i32(a), _i32(tok))
            err = pages.reserve(4, s.bt, s.ref, a, tok)
            for r in a[(a >= 0) & (a < 40)]:           # the rows take tokens into their pages
                front = (np.cumprod(s.bt[r] >= 0)).sum() * 4
                if s.ctx[r] < front:
                    s.ctx[r] = rng.integers(s.ctx[r], front + 1)
            s.g[1].copy_(to_dev(s.ctx))
        elif what == 3:
            a = a[:3]
            a8w8.paged_free(s.handle, *s.g, _i32(a))
            err = pages.free(s.bt, s.ctx, s.ref, a)
        else:
            live = a8w8.paged_compact(s.handle, s.g[0], s.g[2])
            err, n = pages.compact(s.pool, s.bt, s.ref)
            assert int(live) == n
        s.check(err)
        assert s.counts_match()


@gpu
def test_captured_on_another_stream_with_shared_workspace():
    """fork, reserve and compact captured into two graphs that share a workspace of arbitrary
    contents, replayed in turn."""
    import torch
    page = 8
    s = State(4, 16, 6, 64, page)
    _fill(s, [0, 1], [20, 33])
    s.on_gpu()
    ws = torch.full((a8w8.pages_workspace_bytes(64, 16, 8),), 0xA5, dtype=torch.uint8, device="cuda")
    p, c, tok = [_i32(v) for v in ([0, 1, 0], [4, 5, 6], [30, 48, 21])]
    side = torch.cuda.Stream()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    a8w8.read_device_errors()
    with torch.cuda.graph(g1, stream=side):
        a8w8.paged_fork(s.handle, *s.g, p, c, ws=ws)
        a8w8.paged_reserve(s.handle, s.g[0], s.g[2], c, tok, ws=ws)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = _i32([0, 4])
    with torch.cuda.graph(g2, stream=side):
        a8w8.paged_free(s.handle, *s.g, rows)
        a8w8.paged_compact(s.handle, s.g[0], s.g[2], num_live=live, ws=ws)
    s.check()                                          # capturing ran nothing
    for k in range(2):
        g1.replay()
        g2.replay()
        err = pages.fork(s.pool, page, s.bt, s.ctx, s.ref, [0, 1, 0], [4, 5, 6])
        err |= pages.reserve(page, s.bt, s.ref, [4, 5, 6], [30, 48, 21])
        err |= pages.free(s.bt, s.ctx, s.ref, [0, 4])
        e, n = pages.compact(s.pool, s.bt, s.ref)
        s.check(err | e)
        assert int(live) == n


@gpu
def test_copy_and_compact_all_layers():
    """The 160 caches of a 40-layer 4-bit pool: 96 page copies, then a compaction."""
    import torch
    L, N, page, Hkv, D = 40, 256, 128, 8, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (2 * L, N, page, Hkv, D // 2), dtype=torch.uint8, device="cuda",
                          generator=g)
    meta = torch.randint(-2 ** 15, 2 ** 15, (2 * L, N, page, Hkv, 2), dtype=torch.int16,
                         device="cuda", generator=g)
    pool = a8w8.PagePool([c[i] for i in range(2 * L) for c in (codes, meta)], N, page)
    p = torch.randperm(N, device="cuda", generator=g).to(torch.int32)
    src, dst = p[:96].contiguous(), p[96:192].contiguous()
    want = codes.clone(), meta.clone()
    a8w8.read_device_errors()
    a8w8.paged_copy_pages(pool, src, dst)
    for c, w in zip((codes, meta), want):
        w[:, dst.long()] = w[:, src.long()]
        assert torch.equal(c, w)
    ref = torch.zeros(N, dtype=torch.int32, device="cuda")
    bt = p[:100].reshape(10, 10).clone()
    ref[p[:100].long()] = 1
    live = a8w8.paged_compact(pool, bt, ref)
    assert int(live) == 100 and int(ref[:100].sum()) == 100 and int(bt.max()) == 99
    for c, w in zip((codes, meta), want):
        assert torch.equal(c[:, bt.reshape(-1).long()], w[:, p[:100].long()])
    assert a8w8.read_device_errors() == 0


@gpu
def test_pages_past_4_gib():
    import torch
    page_bytes, N = 1 << 20, 4200
    pool = torch.zeros((N, page_bytes // 4), dtype=torch.int32, device="cuda")
    pool[4150] = torch.arange(page_bytes // 4, dtype=torch.int32, device="cuda")
    h = a8w8.PagePool([pool], N, 16)
    a8w8.read_device_errors()
    a8w8.paged_copy_pages(h, _i32([4150]), _i32([4199]))
    assert torch.equal(pool[4199], pool[4150]) and not pool[103].any() and not pool[4198].any()
    bt, ref = _i32([[4199, 4150]]), torch.zeros(N, dtype=torch.int32, device="cuda")
    ref[[4199, 4150]] = 1
    assert int(a8w8.paged_compact(h, bt, ref)) == 2
    assert to_host(bt).tolist() == [[1, 0]]
    assert torch.equal(pool[0], pool[4150]) and torch.equal(pool[1], pool[4150])
    assert a8w8.read_device_errors() == 0


# ---------------------------------------------------------------------------
# a serving run over the 4-bit cache (GPU)
# ---------------------------------------------------------------------------

@gpu
def test_serving_run_over_the_4_bit_cache():
    """A prompt written once and forked into samples, each grown by tokens of its own, retired
    and compacted: every row attends exactly as over its own unshared tokens."""
    import torch
    page, Hq, Hkv, D, N, B, M = 16, 10, 2, 128, 40, 6, 8
    shape = lambda w, t: torch.zeros((N * page, Hkv, w), dtype=t, device="cuda")  # noqa: E731
    cache = [shape(D // 2, torch.uint8), shape(D // 2, torch.uint8),
             shape(2, torch.bfloat16), shape(2, torch.bfloat16)]
    pool = a8w8.PagePool(cache, N, page)
    bt = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    ctx, ref = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, N))
    rng = np.random.default_rng(1)
    toks = {}                                          # row -> (k, v) of its tokens

    def append(row, n, seed):
        k, v = (synth.bf16_normal(seed + i, (n, Hkv, D)) for i in (0, 1))
        old = toks.get(row)
        n0 = 0 if old is None else len(old[0])
        toks[row] = (k, v) if old is None else tuple(np.concatenate(z) for z in zip(old, (k, v)))
        a8w8.paged_reserve(pool, bt, ref, _i32([row]), _i32([n0 + n]))
        t = n0 + np.arange(n)
        slots = to_host(bt)[row][t // page] * page + t % page
        a8w8.paged_kv_write_i4(to_dev(k), to_dev(v), _i32(slots), *cache, page)
        ctx[row] = n0 + n

    def attend():
        q = synth.bf16_normal(77, (B, Hq, D))
        return q, to_host(a8w8.paged_decode_attention_i4kv(to_dev(q), *cache, bt, ctx, page))

    def check():
        q, got = attend()
        for r in range(B):
            if r not in toks:
                assert not got[r].any()
                continue
            k, v = toks[r]
            n = len(k)
            own = [np.zeros((-(-n // page) * page, Hkv, w), t) for w, t in
                   ((D // 2, np.uint8), (D // 2, np.uint8), (2, np.uint16), (2, np.uint16))]
            kv_i4.kv_write(k, v, np.arange(n), *own)
            table = np.arange(-(-n // page))[None]
            want, bound = kv_i4.attention(q[r:r + 1], *own, table, [n], page)
            g = kv_i4.bf16_to_f64(got[r:r + 1])
            assert (np.abs(g - want) <= bound + (np.abs(want) + bound) * 2.0 ** -8).all()
        return got

    a8w8.read_device_errors()
    append(0, 41, 10)
    append(1, 32, 20)
    a8w8.paged_fork(pool, bt, ctx, ref, _i32([0, 0, 1]), _i32([2, 3, 4]))
    toks.update({2: toks[0], 3: toks[0], 4: toks[1]})
    check()
    for i, r in enumerate((0, 2, 3, 4, 1)):
        append(r, [1, 9, 30, 2, 17][i], 100 + 10 * i)
    check()
    a8w8.paged_free(pool, bt, ctx, ref, _i32([0, 1]))
    del toks[0], toks[1]
    before = check()
    live = int(a8w8.paged_compact(pool, bt, ref))
    held = to_host(bt)[to_host(bt) >= 0]
    assert live == len(np.unique(held)) and held.max() == live - 1
    assert np.array_equal(before, check())             # moved pages, the same bits
    assert np.array_equal(np.bincount(held, minlength=N), to_host(ref))
    assert a8w8.read_device_errors() == 0


@gpu
def test_calls_on_another_stream_with_work_pending_on_the_current_one():
    """Workspaces and counts of calls on another stream are not taken from what the current stream
    gave back with a kernel still queued that writes it."""
    import torch
    page = 8
    s = State(14, 16, 6, 64, page)
    _fill(s, [0, 1], [20, 33])
    s.on_gpu()
    a = torch.randn((8192, 8192), device="cuda", dtype=torch.bfloat16)
    p, c, tok = [_i32(v) for v in ([0, 1, 0], [4, 5, 6], [30, 48, 21])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a8w8.read_device_errors()
    left = [torch.empty(a8w8.pages_workspace_bytes(64, 16, n), dtype=torch.uint8, device="cuda")
            for n in (3, 3, 0)] + [torch.empty(1, dtype=torch.int32, device="cuda")]
    for _ in range(20):                                    # some 10 ms on the current stream
        a @ a
    for x in left:
        x.fill_(1)
    del left, x
    a8w8.paged_fork(s.handle, *s.g, p, c, stream=side)
    a8w8.paged_reserve(s.handle, s.g[0], s.g[2], c, tok, stream=side)
    live = a8w8.paged_compact(s.handle, s.g[0], s.g[2], stream=side)
    torch.cuda.synchronize()
    err = pages.fork(s.pool, page, s.bt, s.ctx, s.ref, [0, 1, 0], [4, 5, 6])
    err |= pages.reserve(page, s.bt, s.ref, [4, 5, 6], [30, 48, 21])
    e, n = pages.compact(s.pool, s.bt, s.ref)
    assert int(live) == n
    s.check(err | e)


@gpu
def test_lists_written_by_the_kernel_just_before():
    """Page lists drawn by the sampler (one logit far above the others) into a buffer that is used
    again and again, and copied from at once."""
    import torch
    N, n, rounds, page = 200, 24, 30, 4
    s = State(21, 2, 2, N, page, (16,)).on_gpu()
    src = s.rng.integers(0, 100, (rounds, n)).astype(np.int32)
    logits = torch.zeros((rounds, n, N), dtype=torch.float32, device="cuda")
    logits.scatter_(2, to_dev(src.astype(np.int64))[:, :, None], 100.0)
    dst = _i32(100 + s.rng.permutation(100)[:n])
    out = torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(a8w8.lib().a8w8_sample_workspace_bytes(n, N), dtype=torch.uint8, device="cuda")
    got = torch.zeros((rounds, n, page, 16), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    a8w8.read_device_errors()
    for i in range(rounds):
        a8w8.a8w8_sample(logits[i], 1.0, 1.0, 3, i, out=out, ws=ws)
        a8w8.paged_copy_pages(s.handle, out, dst)
        got[i] = s.gp[0][dst.long()]
    assert a8w8.read_device_errors() == 0
    assert np.array_equal(to_host(got), s.pool[0][src])


class _FakeCache:
    """What PagePool asks of a CUDA tensor."""

    def __init__(self, page_bytes, blocks, ptr=FAKE):
        self.bytes, self.ptr, self.device = page_bytes * blocks, ptr, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return self.bytes

    def element_size(self):
        return 1

    def data_ptr(self):
        return self.ptr


def test_pool_refuses_what_its_operations_would(lib):
    """Too many caches, pages that are not words, empty or misaligned caches and too many pages are
    refused when the pool is made, not when an operation first meets them."""
    c = lambda **k: _FakeCache(**{**dict(page_bytes=1024, blocks=8), **k})  # noqa: E731
    assert len(a8w8.PagePool([c()] * 256, 8, 16).caches) == 256
    a8w8.PagePool([c(page_bytes=20)], 8, 16)          # no whole words a token: refused by fork alone
    for caches, blocks in (([c()] * 257, 8), ([c(), c(page_bytes=1022)], 8), ([c(page_bytes=0)], 8),
                           ([c(ptr=FAKE + 4)], 8), ([c(ptr=0)], 8),
                           ([c(page_bytes=1 << 31)], 8),
                           ([c(page_bytes=4, blocks=1 << 21)], 1 << 21)):
        with pytest.raises(a8w8.A8W8Error, match="PagePool: "):
            a8w8.PagePool(caches, blocks, 16)


def test_lists_too_long_are_refused(lib):
    """Entries are counted in int with strides past the end, and copy units in 64 bits."""
    n = (1 << 30) + 1
    pool = ((ctypes.c_void_p * 1)(FAKE), (ctypes.c_size_t * 1)(1024), 1)
    tables, ws = (FAKE, FAKE, FAKE), (FAKE, 1 << 50, None)
    SHAPE = a8w8.ERR_UNSUPPORTED_SHAPE
    assert lib.paged_copy_pages(*pool, 8, FAKE, FAKE, n, None) == SHAPE
    assert lib.paged_fork(*pool, 8, 16, *tables, 4, 4, FAKE, FAKE, n, *ws) == SHAPE
    assert lib.paged_reserve(FAKE, FAKE, 4, 4, 8, 16, FAKE, FAKE, n, *ws) == SHAPE
    assert lib.paged_free(*tables, 4, 4, 8, FAKE, n, None) == SHAPE


@gpu
def test_copy_long_list():
    """20,000 pairs of small pages, some in conflict, over many CTAs' shares."""
    s = State(22, 2, 2, 50000, 1, (4, 1)).on_gpu()
    p = s.rng.permutation(50000).astype(np.int32)
    src, dst = p[:20000].copy(), p[20000:40000].copy()
    dst[[17000, 9000, 19999]] = dst[[5, 3, 0]]             # destinations of earlier pairs
    dst[4000] = src[15000]                                 # a page that is read
    dst[7], src[8] = -1, 50000
    a8w8.read_device_errors()
    a8w8.paged_copy_pages(s.handle, _i32(src), _i32(dst))
    ok = np.ones(20000, bool)
    ok[[17000, 9000, 19999, 4000, 7, 8]] = False
    for c in s.pool:
        c[dst[ok]] = c[src[ok]]
    s.check({"ALIAS", "BLOCK"})


@gpu
def test_fork_all_layers():
    """64 forks of 16 rows through the 160 caches of a 40-layer 4-bit pool, then their pages for 160
    more tokens: tables and counts as the oracle's, every child's tokens its parent's."""
    import torch
    L, N, page, Hkv, D, B, M = 40, 448, 128, 8, 128, 96, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, (2 * L, N, page, Hkv, D // 2), dtype=torch.uint8, device="cuda",
                          generator=g)
    meta = torch.randint(-2 ** 15, 2 ** 15, (2 * L, N, page, Hkv, 2), dtype=torch.int16,
                         device="cuda", generator=g)
    pool = a8w8.PagePool([c[i] for i in range(2 * L) for c in (codes, meta)], N, page)
    s = State(31, B, M, N, page, (1,))
    _fill(s, np.arange(16), 100 + np.arange(16) * 173)
    s.on_gpu()
    p, c = np.arange(64, dtype=np.int32) % 16, 20 + np.arange(64, dtype=np.int32)
    tokens = s.ctx[p] + 160
    a8w8.read_device_errors()
    a8w8.paged_fork(pool, *s.g, _i32(p), _i32(c))
    a8w8.paged_reserve(pool, s.g[0], s.g[2], _i32(c), _i32(tokens))
    assert pages.fork(s.pool, page, s.bt, s.ctx, s.ref, p, c) == set()
    assert pages.reserve(page, s.bt, s.ref, c, tokens) == set()
    for got, host in zip(s.g, (s.bt, s.ctx, s.ref)):
        assert np.array_equal(to_host(got), host)
    assert a8w8.read_device_errors() == 0 and s.counts_match()
    for i in range(0, 64, 7):
        n = int(s.ctx[c[i]])
        if n % page == 0:
            continue                                       # no page in part: all shared
        own, of = s.bt[c[i]][n // page], s.bt[p[i]][n // page]
        assert own != of
        for x in (codes, meta):
            assert torch.equal(x[:, int(own), :n % page], x[:, int(of), :n % page])
