"""The serving operators together, as a decode loop uses them: rows turned by rotary positions over three axes, pages
taken for them, rows appended, attention, beams forked, drafted tokens rejected, pages compacted.

The paged cache is held against a contiguous one whose rows are gathered by hand: the same rows appended in the same
order give the same codes, so the outputs are equal bit for bit, wherever the pages lie and whoever shares them."""
import random

import pytest
import torch

from packed_decode_attention_b200 import bgtq
from packed_decode_attention_b200 import workloads as wl

pytestmark = pytest.mark.gpu

BATCH, CAP, LAYERS, HKV, GROUP = 5, 640, 2, 2, 4
AXES = [j * 3 // 64 for j in range(64)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(kind, dev, pool):
    if kind == "packed":
        w = wl.scaled(wl.WORKLOADS["tiny"], n_layers=LAYERS, n_kv_heads=HKV, n_q_heads=HKV * GROUP, n_calib=64)
        cfg = dict(n_layers=LAYERS, n_kv_heads=HKV, n_q_heads=HKV * GROUP, max_batch=BATCH, capacity_tokens=CAP)
        kv = bgtq.PackedKVCache(bgtq.Config(**cfg, page_pool_tiles=pool), dev)
        kv.allocate(*(x.to(dev) for x in wl.calibration(w)))
        return kv
    return bgtq.ByteKVCache(bgtq.ByteConfig(n_layers=LAYERS, n_kv_heads=HKV, n_q_heads=HKV * GROUP, max_batch=BATCH,
                                            capacity_tokens=CAP, code=kind, rows="bf16", max_q_tokens=4,
                                            page_pool_tiles=pool), dev)


def arrays(kv):
    if isinstance(kv, bgtq.ByteKVCache):
        return kv.k_codes().view(torch.uint8), kv.k_scales(), kv.v_codes().view(torch.uint8), kv.v_scales()
    return kv.k_tiles(), kv.k_norms(), kv.v_tiles(), kv.v_norms()


def append(kv, k, v, start, count):
    (kv.encode_append if isinstance(kv, bgtq.PackedKVCache) else kv.append)(0, k, v, start, count, layer_count=LAYERS)


def attend(kv, q, lens):
    if isinstance(kv, bgtq.PackedKVCache):
        out = torch.empty_like(q[:, :, -1])
        kv.decode_attn(0, q[:, :, -1].contiguous(), lens, out, layer_count=LAYERS)
        return out
    out = torch.empty_like(q)
    kv.decode_attn(0, q, lens, out, layer_count=LAYERS, softcap=30.0, window=300, prefix=(lens > 0).int() * 4)
    return out


@pytest.mark.parametrize("kind", ["e4m3", "int8", "packed"])
@pytest.mark.parametrize("seed", [0, 1])
def test_decode_loop_over_shared_pages(dev, kind, seed):
    rng = random.Random(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    pool = BATCH * (CAP // 64) + 3
    paged, flat = make(kind, dev, pool), make(kind, dev, 0)
    dt = torch.float16 if kind == "packed" else torch.bfloat16
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.full((BATCH, CAP // 64), -1, dtype=torch.int32, device=dev)
    table2, refs, lens = table.clone(), i32([0] * pool), i32([0] * BATCH)
    refs[7] = 1                                               # a page somebody else keeps
    page_map, live = torch.empty_like(refs), i32([0])
    paged.set_block_table(table)

    def step(n, counts):
        """Rows for the next positions of every sequence, appended to both caches; attention of the last n tokens."""
        heads = HKV * (GROUP + 1)
        rows = (torch.randn((LAYERS, BATCH * n, heads, 128), generator=g, device=dev)).to(dt)
        v = torch.randn((LAYERS, BATCH, n, HKV, 128), generator=g, device=dev).to(dt)
        at = (lens[:, None] + torch.arange(n, device=dev, dtype=torch.int32)).reshape(-1)
        pos = torch.stack([at, at // 7, at % 7]).int()
        q, k = rows[:, :, :HKV * GROUP], rows[:, :, HKV * GROUP:]
        for l in range(LAYERS):
            bgtq.rope_axes(q[l], k[l], pos, AXES, 1e6, q[l], k[l])
        k = k.reshape(LAYERS, BATCH, n, HKV, 128).contiguous()
        count = i32(counts)
        new = lens + count
        paged.resize_sequences(table, refs, lens, new, new)
        assert torch.equal(new, lens + count)
        for kv in (paged, flat):
            append(kv, k, v, lens, count)
        lens.copy_(new)
        q = q.reshape(LAYERS, BATCH, n, HKV * GROUP, 128)[:, :, -min(n, 4):].contiguous()
        a, b = attend(paged, q, lens), attend(flat, q, lens)
        assert torch.equal(a, b) and torch.isfinite(a.float()).all() and a.float().abs().max() > 0

    step(200, [200, 130, 64, 1, 0])
    for _ in range(8):
        parent = [rng.choice([b, rng.randint(0, BATCH - 1)]) for b in range(BATCH)]
        if rng.random() < 0.5:
            parent[rng.randint(0, BATCH - 1)] = -1
        paged.fork_sequences(i32(parent), table, refs, lens, table2, refs, lens)
        table.copy_(table2)
        for a in arrays(flat):
            a.copy_(a[:, [max(p, 0) for p in parent]].clone())
        step(1, [1] * BATCH)
        step(4, [4] * BATCH)                                  # drafted; some are rejected
        paged.resize_sequences(table, refs, lens, lens - i32([rng.randint(0, 4) for _ in range(BATCH)]), lens)
        if rng.random() < 0.5:
            paged.compact_pages(table, refs, lens, table, refs, page_map, live)
            used = {p for row, m in zip(table.tolist(), lens.tolist()) for p in row[:-(-m // 64)]}
            assert live.item() <= len(used) + 1 and max(used) < live.item() and int((refs > 0).sum()) == live.item()
        step(70, [rng.randint(0, 40) for _ in range(BATCH)])
    # rows leave: what is left is the other owner's page
    paged.resize_sequences(table, refs, lens, torch.zeros_like(lens), lens)
    assert int((refs > 0).sum()) == 1 and refs[refs > 0].item() == 1 and not lens.any()
    for kv in (paged, flat):
        assert kv.device_error() == 0
