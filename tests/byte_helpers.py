"""Shared by the 8-bit cache's GPU tests: caches filled at random, their values in float64, the expected attention
and the error the arithmetic allows."""
import numpy as np
import torch

from oracle import byte_cache as bc
from packed_decode_attention_b200 import bgtq

HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}   # relative, of a rounding to the type
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}      # half the smallest subnormal


def values(codes, scales):
    """float64 values of codes [..., 64, 128] with scales [...]."""
    return codes.double().cpu().numpy() * scales.double().cpu().numpy()[..., None, None]


def random_fill(kv, g, spread=1.0):
    """Random codes in every place of the cache, keys with channels of unequal size and blocks of unequal scale."""
    for codes, scales, s in ((kv.k_codes(), kv.k_scales(), spread), (kv.v_codes(), kv.v_scales(), 0.0)):
        x = torch.randn(codes.shape, generator=g, device=codes.device)
        x *= torch.exp(s * torch.randn(128, generator=g, device=codes.device))
        x *= torch.exp2(torch.randint(-1, 2, codes.shape[:-2], generator=g, device=codes.device).float())[..., None, None]
        a = x.abs().amax(dim=(-1, -2))
        q = 448.0 if kv.cfg.code == "e4m3" else 127.0
        e = torch.ceil(torch.log2(a / q))
        y = x * torch.exp2(-e)[..., None, None]
        codes.copy_(y.to(codes.dtype) if kv.cfg.code == "e4m3" else y.round().clamp(-127, 127).to(torch.int8))
        scales.copy_(torch.exp2(e))


def rows_of(kv, arr, layer, b, h, length, table=None):
    """Values [length, 128] of one sequence and head; arr: float64 values of the whole cache."""
    n = -(-length // 64)
    blocks = arr[layer, h][table[b, :n]] if table is not None else arr[layer, b, h, :n]
    return blocks.reshape(-1, 128)[:length]


def expect(q, k, v, length, n_q, i, rows, score):
    """(expected [128], allowed error [128]) of one query row.

    The kernel's scores: 128 exact products summed in fp32 (each sum off by at
    most 2^-23 of the running magnitude, hence 2^-16 S), three scalings, the
    cap (1e-6 relative) and the exponent's fp32 argument (2^-22 of the
    largest score or bias in log2 units).  A score off by d moves its weight by 2 d
    relative, and the sum's by as much; the weights are rounded to fp16
    (2^-11) but the sum is of the rounded ones, so twice that at most; the
    sums over positions add 2^-20.  Weights are held as 2^14 of the running
    maximum's, so one far below it is off by half of fp16's least subnormal
    instead, 2^-25 / 2^14 of the largest weight, and the sum they are divided
    by is at least the largest: 2^-39 |v_t| a position.  Then the output's
    own rounding."""
    see = bc.visible(length, n_q, i, score.get("window", 0), score.get("prefix", 0), score.get("doc_start", 0))
    slope, pos = score.get("slope", 0.0), length - n_q + i
    scale = score.get("scale") or 128 ** -0.5
    want, mass, s = bc.attention_row(q, k, v, see, pos, scale, score.get("softcap", 0.0), slope)
    if not see.any():
        return want, np.zeros(128)
    at = np.nonzero(see)[0]
    bias = abs(slope) * (at.max() - at.min())
    cap = score.get("softcap", 0.0)
    top = min(s, cap) if cap else s
    d = s * 2.0 ** -16 + top * 2e-6 + (top + bias) * 2.0 ** -22
    allowed = mass * (2 * HALF_STEP["fp16"] + 4 * d + 2.0 ** -20) + 2.0 ** -39 * np.abs(v[see]).sum(axis=0)
    return want, allowed + HALF_STEP[rows] * (np.abs(want) + allowed) + TINY[rows]


def check_attention(kv, q, lens, out, layer=0, layer_count=1, table=None, softcap=0.0, slopes=None, window=0,
                    prefix=None, doc_start=None, scale=None):
    """Every query row of `out` against the oracle."""
    cfg = kv.cfg
    karr, varr = values(kv.k_codes(), kv.k_scales()), values(kv.v_codes(), kv.v_scales())
    qn, on = q.double().cpu().numpy(), out.double().cpu().numpy()
    tb = None if table is None else table.cpu().numpy()
    for l in range(layer_count):
        for b, n in enumerate(lens):
            for h in range(cfg.n_kv_heads):
                k = rows_of(kv, karr, layer + l, b, h, n, tb)
                v = rows_of(kv, varr, layer + l, b, h, n, tb)
                for i in range(q.shape[2]):
                    for hq in range(h * cfg.group_size, (h + 1) * cfg.group_size):
                        score = {"softcap": softcap, "window": window, "scale": scale,
                                 "prefix": prefix[b] if prefix is not None else 0,
                                 "doc_start": doc_start[b][i] if doc_start is not None else 0,
                                 "slope": slopes[hq] if slopes is not None else 0.0}
                        want, allowed = expect(qn[l, b, i, hq], k, v, n, q.shape[2], i, cfg.rows, score)
                        off = np.abs(on[l, b, i, hq] - want)
                        assert np.all(off <= allowed), (l, b, h, i, hq, off.max(), allowed[off.argmax()])


def make(dev, lens, hkv=1, group=4, code="e4m3", rows="fp16", n_q=1, layers=1, paged=False, cap=None, seed=0, spread=1.0):
    """(cache filled at random, q, out, device lens, block table or None)."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    cap = cap or max(64, max(lens))
    need = [-(-n // 64) for n in lens]
    pool = sum(need) + 2 if paged else 0
    cfg = bgtq.ByteConfig(n_layers=layers, n_kv_heads=hkv, n_q_heads=hkv * group, max_batch=len(lens),
                          capacity_tokens=cap, code=code, rows=rows, max_q_tokens=n_q, page_pool_tiles=pool)
    kv = bgtq.ByteKVCache(cfg, dev)
    random_fill(kv, g, spread)
    table = None
    if paged:
        ids = torch.randperm(pool, generator=g, device=dev).int()
        table = torch.full((len(lens), -(-cap // 64)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        kv.set_block_table(table)
    q = torch.randn((layers, len(lens), n_q, hkv * group, 128), generator=g, device=dev).to(kv.row_dtype)
    out = torch.full_like(q, float("nan"))
    return kv, q, out, torch.tensor(lens, dtype=torch.int32, device=dev), table
