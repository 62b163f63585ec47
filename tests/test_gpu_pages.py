"""Page operations on the GPU against the page oracle: tables, counts, lengths and every byte of the cache, for the
8-bit and the packed cache; refusals, device errors, captured graphs."""
import random

import numpy as np
import pytest
import torch

from oracle import pages
from packed_decode_attention_b200 import bgtq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def cache(kind, dev, batch, cap, pool, layers=2, hkv=2, seed=0):
    """A paged cache whose every byte is random."""
    if kind == "packed":
        kv = bgtq.PackedKVCache(bgtq.Config(n_layers=layers, n_kv_heads=hkv, n_q_heads=hkv, max_batch=batch,
                                            capacity_tokens=cap, k_avg_bits=3, v_avg_bits=2, page_pool_tiles=pool), dev)
    else:
        kv = bgtq.ByteKVCache(bgtq.ByteConfig(n_layers=layers, n_kv_heads=hkv, n_q_heads=hkv, max_batch=batch,
                                              capacity_tokens=cap, code=kind, page_pool_tiles=pool), dev)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kv.cache.copy_(torch.randint(0, 256, kv.cache.shape, generator=g, device=dev, dtype=torch.uint8))
    return kv


def slots(kv):
    """The cache's arrays as bytes [L, Hkv, pages, bytes of a slot]."""
    c = kv.cfg
    if isinstance(kv, bgtq.ByteKVCache):
        a = (kv.k_codes(), kv.k_scales(), kv.v_codes(), kv.v_scales())
    else:
        a = (kv.k_tiles(), kv.k_norms(), kv.v_tiles(), kv.v_norms())
    return [x.view(torch.uint8).reshape(c.n_layers, c.n_kv_heads, c.page_pool_tiles, -1).cpu().numpy().copy() for x in a]


def moved(arrays, pairs):
    for a in arrays:
        before = a.copy()
        for src, dst in pairs:
            a[:, :, dst] = before[:, :, src]
    return arrays


def same_bytes(kv, want):
    return all(np.array_equal(a, b) for a, b in zip(slots(kv), want))


def state(rng, batch, width, pool, other=3, most=None):
    """A random table [batch][width] with shared whole pages, counts with other owners, and lengths."""
    ids = list(range(pool))
    rng.shuffle(ids)
    table, lens, refs = [], [], [0] * pool
    for b in range(batch):
        n = 0 if rng.random() < 0.1 else rng.randint(1, min(64 * width, most or 64 * width))
        row = []
        for t in range(pages.held(n)):
            if table and rng.random() < 0.2 and len(table[0]) > t and table[0][t] >= 0 and 64 * (t + 1) <= min(n, lens[0]):
                row.append(table[0][t])
            else:
                row.append(ids.pop())
            refs[row[-1]] += 1
        table.append(row + [-1] * (width - len(row)))
        lens.append(n)
    for _ in range(other):
        refs[rng.randrange(pool)] += 1
    return table, refs, lens


KINDS = ["e4m3", "int8", "packed"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [0, 1, 2, 7, 30])
def test_copy(dev, kind, n):
    kv = cache(kind, dev, 1, 64, 61, layers=3)
    ids = random.Random(n).sample(range(61), 2 * n)
    src, dst = ids[:n], ids[n:]
    if n > 2:
        src[1] = src[0]                       # one page to two places
        src[2] = dst[2]                       # onto itself: nothing
    want = moved(slots(kv), list(zip(src, dst)))
    kv.copy_pages(i32(src, dev), i32(dst, dev))
    assert same_bytes(kv, want) and kv.device_error() == 0


def test_copy_skips_bad_pages(dev):
    kv = cache("int8", dev, 1, 64, 9)
    want = moved(slots(kv), [(2, 5)])
    kv.copy_pages(i32([-1, 2, 3, 9, 4], dev), i32([0, 5, 9, 1, -2147483648], dev))
    assert same_bytes(kv, want) and kv.device_error() == bgtq.DEVERR_PAGE


def run_fork(kv, dev, parent, table, refs, lens, in_place):
    tb, rf, ln = i32(table, dev), i32(refs, dev), i32(lens, dev)
    marked = i32(np.full(np.shape(table), -7), dev)
    refs_out = rf if in_place else torch.empty_like(rf)
    lens_out = ln if in_place else torch.empty_like(ln)
    kv.fork_sequences(i32(parent, dev), tb, rf, ln, marked, refs_out, lens_out)
    return marked.cpu().tolist(), refs_out.cpu().tolist(), lens_out.cpu().tolist()


def check_fork(kv, dev, parent, table, refs, lens, in_place=False, flags=0):
    rows, r, n, pairs, short = pages.fork(parent, table, refs, lens)
    want = moved(slots(kv), pairs)
    got, gr, gn = run_fork(kv, dev, parent, table, refs, lens, in_place)
    assert gn == n and gr == r
    for b in range(len(parent)):
        t = pages.held(lens[parent[b]]) if parent[b] >= 0 else 0
        assert got[b] == rows[b][:t] + [-7] * (len(got[b]) - t), b    # entries behind a row: as they were
    assert same_bytes(kv, want) and kv.device_error() == (flags or (bgtq.DEVERR_POOL if short else 0))
    return rows, r, n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(6))
def test_fork_matches_oracle(dev, kind, seed):
    rng = random.Random(seed)
    batch, width = rng.randint(1, 20), rng.randint(1, 9)
    pool = batch * width + batch + rng.randint(0, 40)
    kv = cache(kind, dev, batch + 1, 64 * width, pool, layers=rng.randint(1, 3), seed=seed)
    table, refs, lens = state(rng, batch, width, pool)
    parent = [rng.randint(-1, batch - 1) for _ in range(batch)]
    check_fork(kv, dev, parent, table, refs, lens, in_place=seed % 2 == 1)


def test_fork_of_more_rows_than_one_cta_plans(dev):
    rng = random.Random(11)
    batch, width, pool = 257, 3, 900
    table, refs, lens = state(rng, batch, width, pool)
    parent = [rng.choice([b, 0, rng.randint(-1, batch - 1)]) for b in range(batch)]
    check_fork(cache("int8", dev, batch, 64 * width, pool, layers=1), dev, parent, table, refs, lens)


@pytest.mark.parametrize("case", ["stay", "all_of_one", "free_all", "rotate"])
def test_fork_patterns(dev, case):
    batch, width, pool = 9, 5, 70
    table, refs, lens = state(random.Random(5), batch, width, pool)
    lens[3] = max(lens[3], 1)
    parent = {"stay": list(range(batch)), "all_of_one": [3] * batch, "free_all": [-1] * batch,
              "rotate": [(b + 1) % batch for b in range(batch)]}[case]
    check_fork(cache("e4m3", dev, batch, 64 * width, pool), dev, parent, table, refs, lens)


def test_fork_of_many_rows_and_a_large_pool(dev):
    """More rows than a CTA has threads, a pool of several chunks, tables wider than a warp's share."""
    rng = random.Random(8)
    batch, width, pool = 700, 150, 21000
    kv = cache("int8", dev, batch, 64 * width, pool, layers=1, hkv=1)
    table, refs, lens = state(rng, batch, width, pool, other=500, most=64 * 25)
    lens[0] = 64 * width - 7
    ids = [p for p in range(pool) if refs[p] == 0]
    for t in range(width):
        if table[0][t] >= 0:
            refs[table[0][t]] -= 1
        table[0][t] = ids[t]
        refs[ids[t]] += 1
    parent = [rng.choice([b, rng.randint(-1, batch - 1)]) for b in range(batch)]
    check_fork(kv, dev, parent, table, refs, lens)


def test_fork_with_too_few_pages(dev):
    table = [[b, 10 + b] for b in range(5)]
    refs = [1] * 5 + [0] * 2 + [1] * 3 + [1] * 5
    kv = cache("packed", dev, 5, 128, 15)
    check_fork(kv, dev, [0, 0, 0, 0, 4], table, refs, [100] * 5)      # rows 1, 2, 3's pages come free
    table = [[0, 1], [2, 3], [4, 5]]
    kv = cache("e4m3", dev, 3, 128, 7)
    rows, r, n = check_fork(kv, dev, [0, 0, 0], table, [1] * 6 + [2], [100, 128, 128])
    kv = cache("e4m3", dev, 4, 128, 5)
    rows, r, n = check_fork(kv, dev, [0, 0, 0, 0], [[0, 1], [2, -1], [-1, -1], [-1, -1]], [1, 1, 1, 3, 1], [70, 64, 0, 0])
    assert n == [70, 70, 64, 64]


def test_fork_bad_inputs(dev):
    kv = cache("int8", dev, 4, 256, 12)
    before = slots(kv)
    table = [[0, 1, -1, -1], [2, 99, -1, -1], [3, 4, -5, -1], [5, -1, -1, -1]]
    got, r, n = run_fork(kv, dev, [0, 4, -2, 3], table, [1] * 6 + [0] * 6, [100, 0, 0, 64], False)
    assert kv.device_error() == bgtq.DEVERR_ARG and n == [100, 0, 0, 64] and r == [1] * 6 + [0] * 6
    got, r, n = run_fork(kv, dev, [0, 1, 2, 3], table, [1] * 6 + [0] * 6, [100, 128, 300, 64], False)
    assert kv.device_error() == bgtq.DEVERR_PAGE | bgtq.DEVERR_SEQ_LEN and n == [100, 128, 0, 64]
    assert got[1][:2] == [2, 99]
    got, r, n = run_fork(kv, dev, [2, 2, 2, 2], table, [1] * 6 + [0] * 6, [0, 0, 130, 0], False)
    assert kv.device_error() == bgtq.DEVERR_PAGE      # a partly filled page outside the pool is nobody's
    assert same_bytes(kv, before)


def check_resize(kv, dev, table, refs, lens, new, out="other"):
    rows, r, n, pairs, short = pages.resize(table, refs, lens, new)
    want = moved(slots(kv), pairs)
    tb, rf, ln, nw = i32(table, dev), i32(refs, dev), i32(lens, dev), i32(new, dev)
    got = {"other": torch.empty_like(ln), "lens": ln, "new": nw}[out]
    kv.resize_sequences(tb, rf, ln, nw, got)
    assert got.cpu().tolist() == n and rf.cpu().tolist() == r and tb.cpu().tolist() == rows
    assert same_bytes(kv, want) and kv.device_error() == (bgtq.DEVERR_POOL if short else 0)
    return rows, r, n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(6))
def test_resize_matches_oracle(dev, kind, seed):
    rng = random.Random(100 + seed)
    batch, width = rng.randint(1, 20), rng.randint(2, 9)
    pool = batch * width + batch + 8
    kv = cache(kind, dev, batch, 64 * width, pool, layers=rng.randint(1, 3), seed=seed)
    table, refs, lens = state(rng, batch, width, pool)
    # forks first, so that pages are shared, then lengths cut into shared pages, then growth out of them
    parent = [rng.randint(-1, batch - 1) for _ in range(batch)]
    rows, refs, lens, _, _ = pages.fork(parent, table, refs, lens)
    new = [rng.choice([0, n, max(0, n - 1), rng.randint(0, n)]) for n in lens]
    table, refs, lens = check_resize(kv, dev, rows, refs, lens, new, ["other", "lens", "new"][seed % 3])
    new = [rng.choice([n, min(64 * width, n + 1), rng.randint(n, 64 * width), 64 * width]) for n in lens]
    check_resize(kv, dev, table, refs, lens, new, ["new", "other", "lens"][seed % 3])


def test_resize_and_compact_of_a_large_pool(dev):
    """A pool past what one CTA's shared memory plans."""
    rng = random.Random(9)
    batch, width, pool = 300, 70, 17000
    kv = cache("int8", dev, batch, 64 * width, pool, layers=1, hkv=1)
    table, refs, lens = state(rng, batch, width, pool, other=300)
    parent = [rng.choice([b, rng.randint(-1, batch - 1)]) for b in range(batch)]
    table, refs, lens = check_fork(kv, dev, parent, table, refs, lens)
    table = [r[:pages.held(n)] + [-1] * (width - pages.held(n)) for r, n in zip(table, lens)]
    new = [rng.choice([0, n, n // 2, min(64 * width, n + 70)]) for n in lens]
    table, refs, lens = check_resize(kv, dev, table, refs, lens, new)
    rows, r, to, n, pairs = pages.compact(table, refs, lens)
    want = moved(slots(kv), pairs)
    tb, rf = i32(table, dev), i32(refs, dev)
    mp, live = torch.empty_like(rf), i32([0], dev)
    kv.compact_pages(tb, rf, i32(lens, dev), tb, rf, mp, live)
    assert live.item() == n and mp.tolist() == to and rf.tolist() == r and tb.tolist() == rows
    assert same_bytes(kv, want) and kv.device_error() == 0
    # and where the pool runs out
    new = [64 * width] * batch
    check_resize(kv, dev, rows, r, lens, new)


def test_resize_with_too_few_pages(dev):
    # rows 0 and 1 share a partly filled page; pages for the copy run out, then for the growth
    table, refs = [[0, 1, -1, -1], [0, 1, -1, -1], [2, -1, -1, -1]], [2, 2, 1, 0, 0]
    kv = cache("int8", dev, 3, 256, 5)
    rows, r, n = check_resize(kv, dev, table, refs, [100, 100, 64], [256, 256, 256])
    assert n == [256, 100, 64]
    kv = cache("int8", dev, 3, 256, 5)
    rows, r, n = check_resize(kv, dev, table, refs, [100, 100, 64], [101, 256, 256])
    assert n == [101, 192, 64]
    kv = cache("packed", dev, 2, 1 << 20, 40)        # wants far beyond the pool
    rows, r, n = check_resize(kv, dev, [[-1] * 16384] * 2, [0] * 40, [0, 0], [1 << 20, 1 << 20])
    assert n == [2560, 0]


def test_resize_bad_inputs(dev):
    kv = cache("e4m3", dev, 4, 256, 9)
    before = slots(kv)
    tb, rf = i32([[0, 1, -1, -1], [2, -1, -1, -1], [3, 77, -1, -1], [4, -1, -1, -1]], dev), i32([1] * 5 + [0] * 4, dev)
    got = i32([9] * 4, dev)
    kv.resize_sequences(tb, rf, i32([100, 64, 70, 10], dev), i32([257, -1, 72, 10], dev), got)
    assert kv.device_error() == bgtq.DEVERR_SEQ_LEN | bgtq.DEVERR_PAGE and got.tolist() == [100, 64, 72, 10]
    assert rf.tolist() == [1] * 5 + [0] * 4 and tb.tolist()[2] == [3, 77, -1, -1]
    kv.resize_sequences(tb, rf, i32([0, 0, 0, 300], dev), i32([0, 0, 0, 10], dev), got)
    assert kv.device_error() == bgtq.DEVERR_SEQ_LEN and got.tolist() == [0, 0, 0, 10]
    assert tb.tolist()[3][0] == 5 and same_bytes(kv, before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_matches_oracle(dev, kind, seed, in_place):
    rng = random.Random(200 + seed)
    batch, width = rng.randint(1, 20), rng.randint(1, 9)
    pool = batch * width + 1 + (0 if seed == 0 else rng.randint(0, 3000))
    kv = cache(kind, dev, batch, 64 * width, pool, layers=rng.randint(1, 2), hkv=1, seed=seed)
    table, refs, lens = state(rng, batch, width, pool, other=0 if seed == 1 else 20)
    if seed == 2:
        table, refs, lens = [[-1] * width] * batch, [0] * pool, [0] * batch          # nothing lives
    if seed == 3:
        refs = [max(1, r) for r in refs]                                              # everything does
    rows, r, to, n, pairs = pages.compact(table, refs, lens)
    want = moved(slots(kv), pairs)
    tb, rf = i32(table, dev), i32(refs, dev)
    to_table, to_refs = (tb, rf) if in_place else (tb.clone(), torch.full_like(rf, -9))
    to_map, live = torch.empty_like(rf), i32([-1], dev)
    kv.compact_pages(tb, rf, i32(lens, dev), to_table, to_refs, to_map, live)
    assert live.item() == n and to_map.tolist() == to and to_refs.tolist() == r and to_table.tolist() == rows
    assert same_bytes(kv, want) and kv.device_error() == 0


def test_compact_bad_inputs(dev):
    kv = cache("int8", dev, 3, 128, 6)
    tb = i32([[5, 9], [0, -1], [4, 1]], dev)
    rf, mp, live = i32([0, 0, 0, 0, 1, 1], dev), i32([7] * 6, dev), i32([0], dev)
    want = moved(slots(kv), [(4, 0), (5, 1)])
    kv.compact_pages(tb, rf, i32([70, 1, 129], dev), tb, rf, mp, live)
    # page 9 does not exist, page 0 is free, length 129 does not fit
    assert kv.device_error() == bgtq.DEVERR_PAGE | bgtq.DEVERR_SEQ_LEN
    assert tb.tolist() == [[1, -1], [-1, -1], [4, 1]] and rf.tolist() == [1, 1, 0, 0, 0, 0] and live.item() == 2
    assert mp.tolist() == [-1, -1, -1, -1, 0, 1] and same_bytes(kv, want)


def test_refusals(dev):
    def status(fn, *a):
        with pytest.raises(bgtq.BgtqError) as e:
            fn(*a)
        return e.value.status

    flat = bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, 2, 128), dev)
    z = torch.zeros(4096, dtype=torch.int32, device=dev)
    a, b, c, d, e, f, g, s = (z[512 * i:512 * i + 512] for i in range(8))
    assert status(bgtq.bgtq_page_scratch_bytes, flat.state) == -1
    assert status(bgtq.bgtq_copy_pages, flat.state, a, b, 1) == -1
    for kv in (cache("int8", dev, 2, 128, 8), cache("packed", dev, 2, 128, 8)):
        st = kv.state
        fork = lambda *x, n=2: bgtq.bgtq_fork_sequences(st, *x[:4], n, *x[4:])  # noqa: E731
        fork(a, b, c, d, e, f, g, s)
        for i in range(8):
            args = [a, b, c, d, e, f, g, s]
            args[i] = None
            assert status(fork, *args) == -2
            args[i] = [a, b, c, d, e, f, g, s][i].data_ptr() + 2
            assert status(fork, *args) == -8
        assert status(lambda: fork(a, b, c, d, e, f, g, s, n=0)) == -1
        assert status(lambda: fork(a, b, c, d, e, f, g, s, n=3)) == -1
        assert status(fork, a, b, c, d, b, f, g, s) == -1          # table_out is table
        assert status(fork, a, b, c, d, b[2:], f, g, s) == -1      # or overlaps it
        assert status(fork, a, b, c, d, e, c[1:], g, s) == -1      # refs_out overlaps refs
        assert status(fork, a, b, c, d, e, f, a, s) == -1          # lens_out is parent
        assert status(fork, a, b, c, d, e, f, e, s) == -1          # two outputs overlap
        assert status(fork, a, b, c, d, e, f, g, b) == -1          # the scratch is an input
        fork(a, b, c, d, e, c, d, s)                               # in place
        resize = lambda *x: bgtq.bgtq_resize_sequences(st, *x[:4], 2, *x[4:])  # noqa: E731
        resize(a, b, c, d, e, s)
        resize(a, b, c, d, c, s)
        resize(a, b, c, d, d, s)
        assert status(resize, a, a, c, d, e, s) == -1 and status(resize, a, b, a, d, e, s) == -1
        assert status(resize, a, b, c, d, c[1:], s) == -1 and status(resize, a, b, c, d, e, None) == -2
        compact = lambda *x: bgtq.bgtq_compact_pages(st, *x[:3], 2, *x[3:])  # noqa: E731
        compact(a, b, c, a, b, f, g, s)
        assert status(compact, a, b, c, a, b, b, g, s) == -1 and status(compact, a, b, c, d, e, f, f, s) == -1
        assert status(compact, a, b, c, d, e, f, None, s) == -2
        assert status(bgtq.bgtq_copy_pages, st, a, b, -1) == -1 and status(bgtq.bgtq_copy_pages, st, None, b, 1) == -2
        assert status(bgtq.bgtq_copy_pages, st, a.data_ptr() + 1, b, 1) == -8
        kv.device_error()


def test_captured_and_on_streams(dev):
    rng = random.Random(3)
    batch, width, pool = 6, 4, 60
    kv = cache("e4m3", dev, batch, 64 * width, pool)
    table, refs, lens = state(rng, batch, width, pool)
    parent = [1, 1, 0, -1, 2, 5]
    tb, rf, ln, pr = i32(table, dev), i32(refs, dev), i32(lens, dev), i32(parent, dev)
    to, ro, lo = torch.full_like(tb, -1), torch.empty_like(rf), torch.empty_like(ln)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kv.fork_sequences(pr, tb, rf, ln, to, ro, lo)
        tb.copy_(to)
        rf.copy_(ro)
        ln.copy_(lo)
    for _ in range(3):
        rows, refs, n, pairs, short = pages.fork(parent, table, refs, lens)
        want = moved(slots(kv), pairs)
        graph.replay()
        torch.cuda.synchronize()
        assert ln.tolist() == n and rf.tolist() == refs and same_bytes(kv, want)
        table, lens = rows, n
        for b in range(batch):
            assert tb.tolist()[b][:pages.held(n[b])] == rows[b][:pages.held(n[b])]
    assert kv.device_error() == 0
