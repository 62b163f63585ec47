"""Page copies of many items a warp (its lookups run ahead in groups of 32), byte for byte."""
import random

import pytest
import torch

from packed_decode_attention_b200 import bgtq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def make(kind, dev, pool, batch=1, cap=64):
    """A paged cache of 37 x 4 (layer, head) pairs whose every byte is random, and the warps that a copy runs on it."""
    common = dict(n_layers=37, n_kv_heads=4, n_q_heads=4, max_batch=batch, capacity_tokens=cap, page_pool_tiles=pool)
    if kind == "packed":
        kv, slot = bgtq.PackedKVCache(bgtq.Config(k_avg_bits=3, v_avg_bits=2, **common), dev), 1024 * 5 + 512 + 128
    else:
        kv, slot = bgtq.ByteKVCache(bgtq.ByteConfig(code=kind, **common), dev), 16384
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    kv.cache.random_(0, 256, generator=g)
    return kv, min(8, 100 * 1024 // (3 * slot)) * torch.cuda.get_device_properties(dev).multi_processor_count


def arrays(kv):
    a = (kv.k_codes(), kv.k_scales(), kv.v_codes(), kv.v_scales()) if isinstance(kv, bgtq.ByteKVCache) else (
        kv.k_tiles(), kv.k_norms(), kv.v_tiles(), kv.v_norms())
    return [x.view(torch.uint8).reshape(37 * 4, kv.cfg.page_pool_tiles, -1) for x in a]


def copied(kv, pairs):
    """What the cache holds after the copies."""
    want = kv.cache.clone()
    base, start = kv.cache.data_ptr(), kv.cache
    src, dst = (torch.tensor([p[i] for p in pairs], device=start.device) for i in (0, 1))
    for x in arrays(kv):
        at = x.data_ptr() - base
        w = want[at:at + x.numel()].view(x.shape)
        w[:, dst] = x[:, src]
    return want


@pytest.mark.parametrize("kind", ["e4m3", "packed"])
def test_copies_of_many_items_a_warp(dev, kind):
    kv, warps = make(kind, dev, 800)
    rng = random.Random(2)
    for items in (15, 16, 17, 30, 31, 32, 33, 34, 47, 48, 49, 63, 64, 65, 79, 97):
        n = -(-items * warps // 148)                   # pairs of 148 items each
        for skip in (0.0, 0.3):
            ids = rng.sample(range(800), 2 * n) if 2 * n <= 800 else [rng.randrange(300) for _ in range(n)] + rng.sample(
                range(300, 800), n)
            src, dst = ids[:n], ids[n:]
            bad = 0
            for i in range(n):
                if rng.random() < skip:                # a pair to itself, or with a page that does not exist
                    if rng.random() < 0.5:
                        src[i] = dst[i]
                    else:
                        src[i], bad = rng.choice([-1, 800, 2 ** 31 - 1]), 1
            want = copied(kv, [(s, d) for s, d in zip(src, dst) if 0 <= s < 800 and s != d])
            kv.copy_pages(i32(src, dev), i32(dst, dev))
            assert torch.equal(kv.cache, want), (items, skip)
            assert kv.device_error() == (bgtq.DEVERR_PAGE if bad else 0)


@pytest.mark.parametrize("kind", ["int8", "packed"])
def test_compaction_of_many_pages(dev, kind):
    """Some 60 items a warp behind a plan: the pairs come from the device."""
    pool = 1000
    kv, warps = make(kind, dev, pool, batch=2)
    rng = random.Random(4)
    n_live = 61 * warps // 148
    n_live = min(n_live, pool // 2)
    live = sorted(rng.sample(range(pool // 2, pool), n_live))
    refs = [0] * pool
    for p in live:
        refs[p] = 1
    want = copied(kv, list(zip(live, range(n_live))))
    rf, mp, count = i32(refs, dev), i32([0] * pool, dev), i32([0], dev)
    tb, ln = i32([[live[0]], [live[-1]]], dev), i32([64, 10], dev)
    kv.compact_pages(tb, rf, ln, tb, rf, mp, count)
    assert count.item() == n_live and tb.tolist() == [[0], [n_live - 1]]
    assert torch.equal(kv.cache, want) and kv.device_error() == 0
