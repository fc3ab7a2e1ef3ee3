"""Entries and pages on the move, on the GPU, against lists (tree_ref.py): all of
it exact."""
import numpy as np
import pytest

import tree_ref
from test_gpu_kv import bits_of, i32, make_cache, sv, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def np_of(t):
    return t.cpu().numpy()


def contents(cache):
    return [bits_of(x) if x.element_size() != 1 or "float8" in str(x.dtype) else np_of(x)
            for x in (cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp) if x is not None]


# ------------------------------------------------------------------ compact
def random_path(rng, N):
    """Node 0 and some others in order."""
    n = int(rng.integers(0, N))
    return [0] + sorted(rng.choice(np.arange(1, N), n, replace=False).tolist())


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("D,S,H,B,N,prefix", [(64, 16, 1, 4, 20, 0), (80, 32, 3, 3, 7, 10), (96, 64, 2, 5, 64, 0),
                                              (128, 128, 8, 2, 33, 130), (128, 16, 4, 40, 26, 0), (64, 16, 2, 1, 512, 0)])
def test_compact(sv, fmt, D, S, H, B, N, prefix):  # noqa: F811
    rng = np.random.default_rng(D + N)
    own = rng.integers(0, 100, B)
    mp = -(-(100 + N) // S)
    n, table, _ = tables(rng, B, mp, 0)
    cache = make_cache(sv, rng, fmt, n, H, S, D)[0]
    want = contents(cache)
    path, acc = np.full((B, N), -1), np.zeros(B, int)
    for b in range(B):
        way = random_path(rng, N) if b != 1 else list(range(N))  # one whose entries all stay
        path[b, :len(way)], acc[b] = way, len(way) - 1
        for j, i in enumerate(way):
            to, origin = own[b] + j, own[b] + i
            for x in want:
                x[table[b, to // S], :, to % S] = x[table[b, origin // S], :, origin % S]
    st = sv.spec_kv_compact(cache, i32(table), i32(own + prefix), i32(path), i32(acc), prefix_len=prefix, with_status=True)
    assert (np_of(st) == 0).all()
    for x, y in zip(contents(cache), want):
        assert np.array_equal(x, y)


def test_compact_errors(sv):  # noqa: F811
    """Rows in error move nothing; a page that is not there keeps its entries from moving, no others."""
    rng = np.random.default_rng(7)
    B, N, S = 8, 12, 16
    n, table, _ = tables(rng, B, 3, 0)
    cache = make_cache(sv, rng, "e4m3", n, 2, S, 64)[0]
    path = np.tile(np.array([0, 2, 5, 6, 9] + [-1] * 7), (B, 1))
    acc, own = np.full(B, 4), np.full(B, 10)
    path[0, 2] = 2                      # not increasing
    path[1, 4] = 12                     # past the step
    acc[2] = 12                         # past the path
    acc[3] = -1
    own[4] = 3 * S - 8                  # passes the table
    own[5] = -3
    table[6, 1] = n + 3                 # positions 16 .. 31
    path[7, 0] = 1
    want = contents(cache)
    for j, i in ((1, 2), (2, 5)):       # 12 -> 11, 15 -> 12; 16 and 19 lie on the page
        for x in want:
            x[table[6, 0], :, 10 + j] = x[table[6, 0], :, 10 + i]
    st = sv.spec_kv_compact(cache, i32(table), i32(own), i32(path), i32(acc), with_status=True)
    bad = tree_ref.BAD_TREE
    assert list(np_of(st)) == [bad, bad, bad, bad, tree_ref.BAD_LENGTH, tree_ref.BAD_LENGTH, tree_ref.BAD_PAGE, bad]
    for x, y in zip(contents(cache), want):
        assert np.array_equal(x, y)


# --------------------------------------------------------------------- copy
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("D,S,H", [(64, 16, 1), (80, 32, 3), (96, 64, 2), (128, 128, 8)])
def test_copy(sv, fmt, D, S, H):  # noqa: F811
    rng = np.random.default_rng(D)
    cache = make_cache(sv, rng, fmt, 40, H, S, D)[0]
    want = contents(cache)
    ids = rng.permutation(40)
    rows = [(ids[i], ids[20 + i], int(rng.integers(0, S + 1))) for i in range(14)]
    rows += [(ids[0], ids[34], S), (ids[0], ids[35], 1), (-1, ids[36], 3), (ids[1], 40, 3), (ids[2], ids[37], 0),
             (ids[2], ids[38], S + 9), (ids[3], ids[39], -4)]
    for s, d, n in rows:
        if 0 <= s < 40 and 0 <= d < 40 and n > 0:
            for x in want:
                x[d, :, :n] = x[s, :, :n]
    sv.spec_kv_copy(cache, i32(np.array(rows)))
    for x, y in zip(contents(cache), want):
        assert np.array_equal(x, y)
    sv.spec_kv_copy(cache, i32(np.zeros((0, 3))))


def test_copy_and_compact_past_32_bits_and_in_strided_pages(sv):  # noqa: F811
    """Keys and values as two halves of one allocation, the last pages beyond 2^32 bytes."""
    import torch
    H, S, D = 8, 128, 128
    n = (1 << 32) // (2 * H * S * D) + 40
    both = torch.empty((n, 2, H, S, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    exps = [torch.zeros((n, H, S), dtype=torch.int8, device="cuda") for _ in range(2)]
    big, small = sv.KVCache(both[:, 0], both[:, 1], *exps), sv.KVCache.empty(6, H, S, D)
    rng = np.random.default_rng(4)
    x, y = (torch.from_numpy(rng.standard_normal((2, 300, H, D)).astype(np.float32)).cuda() for _ in range(2))
    ids = np.arange(6).reshape(2, 3)
    res = []
    for c, t in ((big, ids + n - 6), (small, ids)):
        sv.spec_kv_append(c, x, y, i32(t), i32([0, 0]))
        sv.spec_kv_compact(c, i32(t), i32([100, 250]), i32([[0, 3, 40, -1] + [-1] * 60, [0, 2, 3, 9] + [-1] * 60]), i32([2, 3]))
        sv.spec_kv_copy(c, i32([[t[0, 0], t[1, 1], 77]]))
        res.append(sv.spec_kv_read(c, i32(t), i32([300, 300]), 300))
    for a, b in zip(*res):
        assert torch.equal(a, b)


# ------------------------------------------------------------------- tables
def pool_of(rng, B, wide, n_pages, S, lens, shared=0.0):
    """A pool with rows of these lengths, `shared` of the other pages held elsewhere."""
    held = [0 if x < 0 else -(-x // S) for x in lens]
    ids = rng.permutation(n_pages)
    table, at = rng.integers(-3, n_pages, (B, wide)), 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    refs = np.zeros(n_pages, int)
    refs[ids[:at]] = 1
    others = ids[at:at + int(shared * (n_pages - at))]
    refs[others] = rng.integers(1, 4, len(others))
    return refs, table, held


def same(pool, refs, table, held):
    """Counts, what is held, and the entries in use: what stands behind them is free."""
    assert np.array_equal(np_of(refs), pool.refs)
    assert np.array_equal(np_of(held), pool.held)
    t = np_of(table)
    for b, h in enumerate(pool.held):
        if 0 <= h <= t.shape[1]:
            assert list(t[b, :h]) == pool.table[b][:h], b


@pytest.mark.parametrize("B,S,n_pages,top,n", [(1, 16, 40, 300, 5), (7, 32, 100, 500, 0), (64, 16, 5000, 900, 9),
                                               (513, 128, 3001, 500, 400), (4, 64, 20000, 60000, 3), (4096, 16, 9000, 30, 3)])
@pytest.mark.parametrize("off", [0, 1])
def test_resize(sv, B, S, n_pages, top, n, off):  # noqa: F811
    """Rows grow, shrink and are given back, again and again; where the pool runs
    out the first rows are served.  off: counts that are not 16-byte aligned, a strided table."""
    import torch
    rng = np.random.default_rng(B + n_pages)
    wide = -(-(top + n) // S)
    lens = rng.integers(-1, top // 4, B)
    refs, table, held = pool_of(rng, B, wide, n_pages, S, lens, 0.3)
    pool = tree_ref.Pool(refs, table, held, S)
    store = torch.zeros(n_pages + off, dtype=torch.int32, device="cuda")[off:]
    store.copy_(i32(refs))
    tab = torch.zeros((B, wide + 3 * off), dtype=torch.int32, device="cuda")[:, off:off + wide]
    tab.copy_(i32(table))
    h = i32(held)
    for step in range(6):
        lens = np.where(rng.random(B) < 0.2, -1, rng.integers(0, top, B) if step % 2 else np.minimum(lens + 7, top))
        st = sv.spec_kv_resize(store, tab, h, i32(lens), n, S, with_status=True)
        want = pool.resize(lens.tolist(), n)
        assert list(np_of(st)) == want
        same(pool, store, tab, h)


def test_resize_many_pages(sv):  # noqa: F811
    """More pages than are looked at in one round (8 x 1024 x 32), free ones in the first, last and middle ones."""
    rng = np.random.default_rng(9)
    n_pages, S, wide = 700001, 16, 4000
    refs = np.ones(n_pages, int)
    refs[[5, 77, 262143, 262144, 300000, 524287, 524288, 700000]] = 0
    refs[rng.choice(n_pages, 3000, replace=False)] = 0
    free = int((refs <= 0).sum())
    table, held = np.full((3, wide), -1), [0, 0, 0]
    pool = tree_ref.Pool(refs, table, held, S)
    r, t, h = i32(refs), i32(table), i32(held)
    for lens in ([16 * 100, 16 * 1000, 0], [16 * 90, 16 * 1000, 16 * (free - 1090)], [16 * 91, 16 * 1000, 0],
                 [16 * 91, 16 * 1000, 16 * (free - 1090)], [-1, -1, -1]):
        st = sv.spec_kv_resize(r, t, h, i32(lens), 0, S, with_status=True)
        assert list(np_of(st)) == pool.resize(lens, 0)
        same(pool, r, t, h)
    assert int((np_of(r) <= 0).sum()) == free


@pytest.mark.parametrize("n_pages,busy,B,off", [(600001, 0.95, 50, 0), (262144, 0.0, 64, 0), (262145, 0.6, 9, 3), (40000, 0.5, 300, 0)])
def test_resize_by_many_ctas(sv, n_pages, busy, B, off):  # noqa: F811
    """Thousands of pages for a call, from a pool that is mostly taken, empty, or taken in long runs."""
    import torch
    rng = np.random.default_rng(n_pages)
    refs = (rng.random(n_pages) < busy).astype(int)
    if B == 300:  # runs
        refs = np.repeat(rng.random(n_pages // 500) < busy, 500).astype(int)
    free = int((refs == 0).sum())
    wide = 2 * free // B + 1
    table, held = np.full((B, wide), -1), [0] * B
    pool = tree_ref.Pool(refs, table, held, 16)
    r = torch.zeros(n_pages + off, dtype=torch.int32, device="cuda")[off:]
    r.copy_(i32(refs))
    t, h = i32(table), i32(held)
    for top in (free // B // 2, 2 * free // B, free // B, 0):  # what there is, too many, fewer again, nothing
        lens = rng.integers(0, 16 * top + 1, B) if top else np.full(B, -1)
        st = sv.spec_kv_resize(r, t, h, i32(lens), 0, 16, with_status=True)
        assert list(np_of(st)) == pool.resize(lens.tolist(), 0)
        same(pool, r, t, h)
    assert int((np_of(r) <= 0).sum()) == free


def test_resize_errors(sv):  # noqa: F811
    rng = np.random.default_rng(10)
    S, wide = 16, 6
    lens = [40, 40, 40, 40, 40, 40, 40]
    refs, table, held = pool_of(rng, 7, wide, 60, S, lens)
    held[1], held[2] = -1, wide + 1
    table[3, 1], table[3, 2] = 60, -5
    pool = tree_ref.Pool(refs, table, held, S, prefix=20)
    r, t, h = i32(refs), i32(table), i32(held)
    lens = [-2, 60, 60, 21, 20 + 16 * wide + 1, 10, 20 + 16 * wide]
    st = sv.spec_kv_resize(r, t, h, i32(lens), 0, S, prefix_len=20, with_status=True)
    want = pool.resize(lens, 0)
    L = tree_ref.BAD_LENGTH
    assert want == [L, L, L, tree_ref.BAD_PAGE, L, L, 0] and list(np_of(st)) == want
    same(pool, r, t, h)


@pytest.mark.parametrize("B,S,n_pages,n,prefix", [(5, 16, 60, 3, 0), (64, 32, 700, 40, 50), (300, 128, 900, 250, 0),
                                                  (4096, 16, 9000, 4000, 0)])
def test_fork(sv, B, S, n_pages, n, prefix):  # noqa: F811
    """Random forks, some of them refused: rows named twice, rows in use, rows that
    are not there, no pages left."""
    rng = np.random.default_rng(B + n)
    for trial in range(4):
        lens = np.where(rng.random(B) < 0.7, -1, rng.integers(0, 150 if B < 1000 else 30, B))
        refs, table, held = pool_of(rng, B, 12, n_pages, S, lens, 0.2 + 0.25 * trial)
        kv = [int(x) if x < 0 else int(x) + prefix for x in lens]
        src, dst = rng.integers(-1 if trial else 0, B, n), rng.permutation(B)[:n]
        if trial:
            dst[rng.random(n) < 0.1] = dst[0]
            dst[-1] = B
            held[int(src[0])] = 13
        if trial == 3:
            table[rng.integers(0, B, 5), 0] = n_pages
        pool = tree_ref.Pool(refs, table, held, S, prefix)
        r, t, h, k = i32(refs), i32(table), i32(held), i32(kv)
        copies, st = sv.spec_kv_fork(r, t, h, k, i32(src), i32(dst), S, prefix_len=prefix, with_status=True)
        wc, ws = pool.fork(kv, src.tolist(), dst.tolist())
        assert list(np_of(st)) == ws
        assert np_of(copies).tolist() == wc
        assert list(np_of(k)) == kv
        same(pool, r, t, h)


def test_fork_then_give_back(sv):  # noqa: F811
    """Counts return to what they were; shared pages are free only when the last row gives them back."""
    S = 16
    refs, table, held, kv = (i32(x) for x in (np.zeros(20), np.full((3, 5), -1), np.zeros(3), [40, -1, -1]))
    sv.spec_kv_resize(refs, table, held, kv, 0, S)
    copies = sv.spec_kv_fork(refs, table, held, kv, i32([0, 0]), i32([1, 2]), S)
    assert np_of(copies).tolist() == [[2, 3, 8], [2, 4, 8]] and list(np_of(kv)) == [40, 40, 40]
    assert list(np_of(refs)[:6]) == [3, 3, 1, 1, 1, 0]
    sv.spec_kv_resize(refs, table, held, i32([-1, 40, 40]), 0, S)
    assert list(np_of(refs)[:6]) == [2, 2, 0, 1, 1, 0]
    sv.spec_kv_resize(refs, table, held, i32([-1, 40, -1]), 30, S)
    assert list(np_of(refs)[:6]) == [1, 1, 1, 1, 1, 0] and list(np_of(table)[1]) == [0, 1, 3, 2, 4]
    sv.spec_kv_resize(refs, table, held, i32([-1, -1, -1]), 30, S)
    assert (np_of(refs) == 0).all() and (np_of(held) == 0).all()


def test_empty_calls(sv):  # noqa: F811
    e = lambda *s: i32(np.zeros(s))  # noqa: E731
    assert sv.spec_kv_resize(e(5), e(0, 3), e(0), e(0), 4, 16, with_status=True).shape == (0,)
    assert sv.spec_kv_fork(e(5), e(2, 3), e(2), e(2), e(0), e(0), 16).shape == (0, 3)
    held, refs = e(2), e(0)
    st = sv.spec_kv_resize(refs, e(2, 0), held, i32([0, -1]), 0, 16, with_status=True)  # no pages, no columns
    assert list(np_of(st)) == [0, 0]
    st = sv.spec_kv_resize(refs, e(2, 4), held, i32([0, 3]), 0, 16, with_status=True)
    assert list(np_of(st)) == [0, tree_ref.NO_PAGES] and list(np_of(held)) == [0, 0]


def test_tables_in_a_graph(sv):  # noqa: F811
    """Resize, fork, copy and resize again, captured once and replayed over new lengths."""
    import torch
    rng = np.random.default_rng(12)
    B, S, n_pages = 32, 16, 600
    cache = make_cache(sv, rng, "e4m3", n_pages, 2, S, 64)[0]
    lens = rng.integers(0, 60, B)
    lens[16:] = -1
    refs, table, held = pool_of(rng, B, 12, n_pages, S, lens, 0.2)
    r, t, h, kv = i32(refs), i32(table), i32(held), i32(lens)
    src, dst, extra = i32(np.arange(16)), i32(np.arange(16, 32)), i32(lens)
    pool = tree_ref.Pool(refs, table, held, S)

    def step():
        sv.spec_kv_resize(r, t, h, extra, 9, S)
        copies = sv.spec_kv_fork(r, t, h, kv, src, dst, S)
        sv.spec_kv_copy(cache, copies)
        sv.spec_kv_resize(r, t, h, extra, 0, S)
        return copies
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    keep = [x.clone() for x in (r, t, h, kv)]
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        copies = step()
    for x, y in zip((r, t, h, kv), keep):
        x.copy_(y)
    want = contents(cache)
    for k in range(3):
        now = np.where(np.arange(B) < 16, lens + 5 * k, -1)
        kv.copy_(i32(now))
        extra.copy_(kv)
        g.replay()
        torch.cuda.synchronize()
        state = now.tolist()
        pool.resize(state, 9)
        wc, _ = pool.fork(state, list(range(16)), list(range(16, 32)))
        pool.resize(now.tolist(), 0)
        assert np_of(copies).tolist() == wc and list(np_of(kv)) == state
        same(pool, r, t, h)
        for s, d, n in wc:
            if s >= 0:
                for x in want:
                    x[d, :, :n] = x[s, :, :n]
        for x, y in zip(contents(cache), want):
            assert np.array_equal(x, y)


def test_calls_on_a_given_stream(sv):  # noqa: F811
    """Each call behind a long wait and a write of its inputs on the same stream;
    what it returns is used on the caller's stream behind a wait for it."""
    import torch
    rng = np.random.default_rng(13)
    B, N, S, n_pages = 5, 33, 16, 60
    parents = tree_ref.random_parents(rng, B, N - 1)
    draft, target = rng.integers(0, 3, (B, N - 1)), rng.integers(0, 3, (B, N))
    own = rng.integers(0, 20, B)
    cache = make_cache(sv, rng, "e4m3", n_pages, 2, S, 64)[0]
    lens = i32(np.zeros(B))
    dev = {k: torch.full_like(i32(v), -7) for k, v in dict(parents=parents, draft=draft, target=target, own=own).items()}
    real = dict(parents=i32(parents), draft=i32(draft), target=i32(target), own=i32(own))
    refs, table, held = i32(np.zeros(n_pages)), i32(np.full((B + 1, 8), -1)), i32(np.zeros(B + 1))
    kv = torch.full((B + 1,), -1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        for k in dev:
            dev[k].copy_(real[k])
        kv[:B].copy_(real["own"])
    mask, depth = sv.spec_tree_mask(dev["parents"], stream=side)
    acc, nxt, path, tok = sv.spec_tree_accept(dev["target"], dev["draft"], dev["parents"], stream=side)
    sv.spec_kv_resize(refs, table, held, kv, N, S, stream=side)
    sv.spec_kv_compact(cache, table[:B], dev["own"], path, acc, stream=side)
    sv.spec_kv_resize(refs, table, held, kv, 0, S, stream=side)
    copies = sv.spec_kv_fork(refs, table, held, kv, i32([0]), i32([B]), S, stream=side)
    sv.spec_kv_copy(cache, copies, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    bits, want = tree_ref.sees(parents, np.full(B, N - 1))
    assert np.array_equal(np_of(mask), tree_ref.words(bits)) and np.array_equal(np_of(depth), want)
    for b in range(B):
        a, t, way = tree_ref.accept(target[b], draft[b], parents[b], N - 1)
        assert (int(acc[b]), int(nxt[b])) == (a, t) and list(np_of(path)[b, :a + 1]) == way
    pool = tree_ref.Pool(np.zeros(n_pages, int), np.full((B + 1, 8), -1), [0] * (B + 1), S)
    state = own.tolist() + [-1]
    pool.resize(state, N)
    pool.resize(state, 0)
    wc, _ = pool.fork(state, [0], [B])
    assert np_of(copies).tolist() == wc and list(np_of(kv)) == state
    same(pool, refs, table, held)
    assert (np_of(lens) == 0).all()


def test_calls_from_threads(sv):  # noqa: F811
    """Calls of several threads, whose checks, outputs and launches come between one another's."""
    import threading
    rng = np.random.default_rng(14)
    runs = [tree_ref.random_parents(rng, 4, 20 + k) for k in range(4)]
    wrong = []

    def work(k):
        p, want = i32(runs[k]), tree_ref.words(tree_ref.sees(runs[k], np.full(4, 20 + k))[0])
        refs, table, held = i32(np.zeros(50)), i32(np.full((3, 8), -1)), i32(np.zeros(3))
        for step in range(200):
            mask, depth, st = sv.spec_tree_mask(p, with_status=True)
            sv.spec_kv_resize(refs, table, held, i32([16 * (step % 5), 20, -1]), 0, 16)
            if not np.array_equal(np_of(mask), want) or list(np_of(held)) != [step % 5, 2, 0]:
                wrong.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_calls_leave_no_references(sv):  # noqa: F811
    """What the calls take and give is freed with its last name, also behind errors."""
    import gc
    import sys

    import torch
    p, q, z = i32(np.zeros((2, 3))), i32(np.zeros((2, 4))), torch.zeros((2, 4, 30), device="cuda")
    seq, n = i32(np.zeros((2, 5))), i32([3, 4])
    calls = [lambda: sv.spec_tree_mask(p, with_status=True), lambda: sv.spec_tree_accept(q, p, p),
             lambda: sv.spec_adjust(z, seq, n, p, out=z)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    gc.collect()
    before, held = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in (p, q, z, seq, n)]
    for _ in range(100):
        for call in calls:
            call()
        for bad in (lambda: sv.spec_tree_mask(p, gamma_per_row=n[:1]), lambda: sv.spec_adjust(z, seq, n),
                    lambda: sv.spec_tree_accept(q, p, q)):
            with pytest.raises(ValueError):
                bad()
    gc.collect()
    assert [sys.getrefcount(t) for t in (p, q, z, seq, n)] == held
    assert torch.cuda.memory_allocated() == before


def test_compact_of_tables_without_columns(sv):  # noqa: F811
    """Sequences that hold the shared prefix alone and accepted nothing: nothing moves."""
    cache = make_cache(sv, np.random.default_rng(15), "bf16", 4, 2, 16, 64)[0]
    want = contents(cache)
    args = i32(np.zeros((2, 0))), i32([40, 40]), i32([[0, 1, -1], [0, 1, 2]])
    st = sv.spec_kv_compact(cache, *args, i32([0, 0]), prefix_len=40, with_status=True)
    assert list(np_of(st)) == [0, 0]
    st = sv.spec_kv_compact(cache, *args, i32([0, 1]), prefix_len=40, with_status=True)
    assert list(np_of(st)) == [0, tree_ref.BAD_LENGTH]
    for x, y in zip(contents(cache), want):
        assert np.array_equal(x, y)
