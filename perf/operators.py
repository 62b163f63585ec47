"""The operators of the 8-bit cache, measured: append and attention over a cache of 8-bit codes with a scale for each
block of 64 positions and KV head, the page operations of a paged cache, and rotary positions over several axes.

``own`` false: plain forms in elementary torch operations.  ``own`` true: the calls a user makes of
packed_decode_attention_b200.  Shapes: D = 128; a cache's arrays are [L][B][H][T][64][128] (contiguous) or
[L][H][P][64][128] (paged, with a block table int32 [B][T]); scales are fp32, one for each 64 x 128 block.
"""
import math
import random

import numpy as np
import torch

own = False

D, TILE = 128, 64
E_MIN = -100
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
ROWS = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases -------------------------------------------------------------

def _attn(name, lens, hkv, hq, code, rows, n_q=1, paged=False, softcap=0.0, slopes=False, window=0, prefix="", docs=""):
    return {"name": name, "op": "attn", "lens": lens, "hkv": hkv, "hq": hq, "code": code, "rows": rows, "n_q": n_q,
            "paged": paged, "softcap": softcap, "slopes": slopes, "window": window, "prefix": prefix, "docs": docs}


def listed():
    ragged = random.Random(16)
    batch = ",".join(str(ragged.randint(16384, 32768)) for _ in range(16))
    return [
        # one KV head, four query heads, 4096 tokens: the smallest decode call, where latency counts
        _attn("attn_tiny_4k", "4096", 1, 4, "e4m3", "fp16"),
        # one layer of an 8-KV-head model at 32K, scores capped by a tanh
        _attn("attn_32k_int8_softcap", "32768", 8, 32, "int8", "fp16", softcap=50.0),
        # one layer of a 2-KV-head model at 128K: one sequence split over the whole GPU
        _attn("attn_128k_bf16", "131072", 2, 16, "e4m3", "bf16"),
        # ragged serving batch, 16 sequences of 16K to 32K, seven query heads to a KV head, paged
        _attn("attn_batch_ragged_paged", batch, 4, 28, "int8", "bf16", paged=True),
        # four drafted tokens verified at once, distance bias, packed documents and a prefix all queries see; one
        # sequence is empty, one is a single token
        _attn("attn_verify_bias_docs", "16381,9001,0,1,16384,5000", 8, 32, "e4m3", "fp16", n_q=4, slopes=True,
              prefix="65,0,0,0,200,10", docs="9000,0,0,0,12345,4000"),
        # a decode step's rows: one row for each of 16 sequences, inside blocks that hold rows already
        {"name": "append_step", "op": "append", "starts": ",".join(str(1000 + 37 * i) for i in range(16)),
         "counts": ",".join(["1"] * 16), "n": 1, "hkv": 4, "code": "int8", "rows": "bf16", "cap": 2048},
        # a 32K prefill of 8 KV heads
        {"name": "append_prefill_32k", "op": "append", "starts": "0", "counts": "32768", "n": 32768, "hkv": 8,
         "code": "e4m3", "rows": "fp16", "cap": 32768},
        # two pages of a one-layer cache copied: latency
        {"name": "pages_copy_2", "op": "copy", "layers": 1, "hkv": 2, "pool": 64, "pairs": 2, "code": "e4m3"},
        # beam search over 28 layers: 16 rows take over five parents' rows, four are freed
        {"name": "pages_fork_beams", "op": "fork", "layers": 28, "hkv": 4, "pool": 512, "cap": 2048,
         "lens": "1500,1700,640,0,1999,2000,1500,77,900,1,64,63,128,129,2047,300",
         "parents": "0,0,0,4,4,4,5,7,7,9,-1,-1,-1,12,-1,14", "held": 3, "code": "int8"},
        # a pool of 2048 pages, two fifths of them live after sequences left, moved together
        {"name": "pages_compact", "op": "compact", "layers": 8, "hkv": 4, "pool": 2048, "cap": 16384,
         "lens": ",".join(str(v) for v in (5000, 16384, 1, 0, 9000, 777, 12800, 7000)), "held": 5, "code": "e4m3"},
        # one decode step's q and k rows of 16 sequences turned by (time, height, width)
        {"name": "rope_step", "op": "rope", "tokens": 16, "hq": 28, "hkv": 4, "rows": "bf16", "axes": 3,
         "pairing": 0, "base": 1e6, "far": 131072},
        # a 32K-token prefill of text and images
        {"name": "rope_prefill_32k", "op": "rope", "tokens": 32768, "hq": 32, "hkv": 8, "rows": "fp16", "axes": 3,
         "pairing": 0, "base": 5e5, "far": 32768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "copy", "fork", "compact", "rope"])
    code, rows = rng.choice(["e4m3", "int8"]), rng.choice(["fp16", "bf16"])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "attn":
        g, n_q, batch = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 1, 1, 2, 3, 5, 8]), _log(rng, 1, 24)
        g = min(g, max(1, 64 // n_q))
        most = min(131072, 1_200_000 // (hkv * batch))
        lens = [0 if rng.random() < 0.05 else _log(rng, 1, most) for _ in range(batch)]
        c = _attn("", ",".join(map(str, lens)), hkv, hkv * g, code, rows, n_q, rng.random() < 0.5)
        if rng.random() < 0.4:
            c["softcap"] = rng.choice([15.0, 30.0, 50.0])
        if rng.random() < 0.4:
            c["slopes"] = True
        if rng.random() < 0.4:
            c["window"] = _log(rng, 1, 8192)
        if rng.random() < 0.4:
            c["prefix"] = ",".join(str(rng.randint(0, 300)) for _ in lens)
        if rng.random() < 0.3:
            c["docs"] = ",".join(str(rng.randint(0, v)) for v in lens)
    elif op == "append":
        batch = _log(rng, 1, 24)
        n = _log(rng, 1, 32768 // batch)
        counts = [n if rng.random() < 0.6 else rng.randint(0, n) for _ in range(batch)]
        starts = [rng.choice([0, rng.randint(0, 1500)]) for _ in range(batch)]
        c = {"op": "append", "starts": ",".join(map(str, starts)), "counts": ",".join(map(str, counts)), "n": n,
             "hkv": hkv, "code": code, "rows": rows, "cap": n + 1500}
    elif op == "copy":
        pool = _log(rng, 16, 1024)
        c = {"op": "copy", "layers": rng.randint(1, 8), "hkv": hkv, "pool": pool, "pairs": rng.randint(1, pool // 2),
             "code": code}
    elif op == "rope":
        g = rng.choice([1, 2, 4, 7, 8])
        c = {"op": "rope", "tokens": _log(rng, 1, 262144 // (hkv * max(g, 4))), "hq": hkv * g, "hkv": hkv,
             "rows": rows, "axes": rng.randint(1, 4), "pairing": rng.randint(0, 1), "base": rng.choice([1e4, 5e5, 1e6]),
             "far": _log(rng, 100, 1 << 20)}
    else:
        batch = _log(rng, 1, 48)
        cap = 64 * rng.randint(2, 64)
        lens = [0 if rng.random() < 0.1 else _log(rng, 1, cap) for _ in range(batch)]
        held = rng.randint(0, 6)
        pool = sum(-(-v // TILE) for v in lens) + held + batch + rng.randint(0, 200)
        layers = rng.randint(1, max(1, min(8, 32768 // (pool * hkv))))
        c = {"op": op, "layers": layers, "hkv": hkv, "pool": pool, "cap": cap, "lens": ",".join(map(str, lens)),
             "held": held, "code": code}
        if op == "fork":
            c["parents"] = ",".join(str(rng.randint(-1, batch - 1)) for _ in lens)
    c.pop("name", None)
    return c


def _ints(text, n=None):
    got = [int(v) for v in text.split(",")] if text else [0] * (n or 0)
    return got


# ---- the inputs ------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _blocks(shape, code, g, spread):
    """Random codes [*shape, 64, 128] and scales [*shape] as quantised rows have them: channels of unequal size (a
    key's rotary pairs differ by an order of magnitude), each block scaled to its largest element."""
    codes = torch.empty(shape + (TILE, D), dtype=CODE[code], device="cuda")
    scales = torch.empty(shape, dtype=torch.float32, device="cuda")
    sigma = torch.exp(spread * torch.randn(D, generator=g, device="cuda"))
    flat, s = codes.view(-1, TILE, D), scales.view(-1)
    for i in range(0, flat.shape[0], 4096):
        x = torch.randn(flat[i:i + 4096].shape, generator=g, device="cuda") * sigma
        e = _exponent(x.abs().amax(dim=(1, 2)), code)
        flat[i:i + 4096] = _round(torch.ldexp(x, -e[:, None, None]), code)
        s[i:i + 4096] = torch.ldexp(torch.ones_like(s[i:i + 4096]), e)
    return codes, scales


def _exponent(a, code):
    """The least e >= E_MIN with a <= QMAX 2^e."""
    m, k = torch.frexp(a)
    top, bits = (0.875, 9) if code == "e4m3" else (127 / 128, 7)
    return torch.where(a > 0, k - bits + (m > top).int(), torch.full_like(k, E_MIN)).clamp(min=E_MIN)


def _round(y, code):
    return y.to(torch.float8_e4m3fn) if code == "e4m3" else torch.round(y).to(torch.int8)


def _table(lens, cap, pool, g):
    """Distinct random pages for every sequence's positions, -1 behind them, and the pages left over."""
    ids = torch.randperm(pool, generator=g, device="cuda").tolist()
    tiles = [-(-v // TILE) for v in lens]
    rows = np.full((len(lens), -(-cap // TILE)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(tiles):
        rows[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(rows).cuda(), ids[at:]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _handle(c, batch, cap, layers=1, pool=0, n_q=1, hq=None):
    """A program's cache: created once, kept."""
    from packed_decode_attention_b200 import bgtq
    cfg = bgtq.ByteConfig(n_layers=layers, n_kv_heads=c["hkv"], n_q_heads=hq or c["hkv"], max_batch=batch,
                          capacity_tokens=cap, code=c["code"], rows=c.get("rows", "fp16"), max_q_tokens=n_q,
                          page_pool_tiles=pool)
    return bgtq.ByteKVCache(cfg, "cuda")


def _load(kv, s):
    """The handle takes over the state's cache arrays; they are its own from then on."""
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        view = getattr(kv, name)()
        view.copy_(s[name])
        s[name] = view
    s["kv"] = kv


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] == "attn":
        lens = _ints(c["lens"])
        batch, cap = len(lens), max(TILE, max(lens))
        tiles = -(-cap // TILE)
        pool = sum(-(-v // TILE) for v in lens) + 3 if c["paged"] else 0
        shape = (1, c["hkv"], pool) if c["paged"] else (1, batch, c["hkv"], tiles)
        s["k_codes"], s["k_scales"] = _blocks(shape, c["code"], g, 1.0)
        s["v_codes"], s["v_scales"] = _blocks(shape, c["code"], g, 0.0)
        s["q"] = (torch.randn((1, batch, c["n_q"], c["hq"], D), generator=g, device="cuda")).to(ROWS[c["rows"]])
        s["lens"] = _i32(lens)
        s["table"] = _table(lens, cap, pool, g)[0] if c["paged"] else None
        s["slopes"] = (torch.pow(2.0, -8.0 * torch.arange(1, c["hq"] + 1, device="cuda") / c["hq"]).float()
                       if c["slopes"] else None)
        s["prefix"] = _i32(_ints(c["prefix"])) if c["prefix"] else None
        # the queries of one sequence lie in one document: the last one
        s["docs"] = _i32(_ints(c["docs"]))[:, None].expand(batch, c["n_q"]).contiguous() if c["docs"] else None
        s["out"] = torch.empty_like(s["q"])
        if own:
            kv = _handle(c, batch, cap, pool=pool, n_q=c["n_q"], hq=c["hq"])
            _load(kv, s)
            if c["paged"]:
                kv.set_block_table(s["table"])
    elif c["op"] == "append":
        starts, counts = _ints(c["starts"]), _ints(c["counts"])
        batch, tiles = len(starts), -(-c["cap"] // TILE)
        shape = (1, batch, c["hkv"], tiles)
        s["k_codes"], s["k_scales"] = _blocks(shape, c["code"], g, 1.0)
        s["v_codes"], s["v_scales"] = _blocks(shape, c["code"], g, 0.0)
        # rows a little larger or smaller than those the blocks hold, so that some blocks' scales grow
        size = torch.exp2(torch.randint(-2, 3, (1, batch, c["n"], c["hkv"], 1), generator=g, device="cuda").float())
        rows = lambda: (torch.randn((1, batch, c["n"], c["hkv"], D), generator=g, device="cuda") * size).to(ROWS[c["rows"]])  # noqa: E731
        s["k"], s["v"] = rows(), rows()
        s["starts"], s["counts"] = _i32(starts), _i32(counts)
        if own:
            _load(_handle(c, batch, c["cap"]), s)
    elif c["op"] in ("copy", "fork", "compact"):
        shape = (c["layers"], c["hkv"], c["pool"])
        s["k_codes"], s["k_scales"] = _blocks(shape, c["code"], g, 1.0)
        s["v_codes"], s["v_scales"] = _blocks(shape, c["code"], g, 0.0)
        if c["op"] == "copy":
            ids = torch.randperm(c["pool"], generator=g, device="cuda").int()
            s["src"], s["dst"] = ids[:c["pairs"]].contiguous(), ids[c["pairs"]:2 * c["pairs"]].contiguous()
            batch, cap = 1, TILE * c["pool"]
        else:
            lens = _ints(c["lens"])
            batch, cap = len(lens), c["cap"]
            s["table"], rest = _table(lens, cap, c["pool"], g)
            s["lens"] = _i32(lens)
            refs = torch.zeros(c["pool"], dtype=torch.int32, device="cuda")
            used = s["table"][s["table"] >= 0].long()
            refs[used] = 1
            # pages that no row holds, but somebody else does (a prompt kept for later requests)
            refs[torch.tensor(rest[:c["held"]], dtype=torch.long, device="cuda")] = 1
            if c["op"] == "fork" and used.numel():
                refs[used[torch.randint(0, used.numel(), (c["held"],), generator=g, device="cuda")]] += 1
            s["refs"] = refs
            s["table_out"], s["refs_out"], s["lens_out"] = s["table"].clone().fill_(-1), refs.clone(), s["lens"].clone()
            if c["op"] == "fork":
                s["parents"] = _i32(_ints(c["parents"]))
            else:
                s["map"], s["live"] = refs.clone(), _i32([0])
        if own:
            _load(_handle(c, batch, cap, layers=c["layers"], pool=c["pool"]), s)
    else:
        shape = (c["tokens"],)
        dt = ROWS[c["rows"]]
        s["q"] = torch.randn(shape + (c["hq"], D), generator=g, device="cuda").to(dt)
        s["k"] = torch.randn(shape + (c["hkv"], D), generator=g, device="cuda").to(dt)
        s["pos"] = torch.randint(0, c["far"], (c["axes"], c["tokens"]), generator=g, device="cuda", dtype=torch.int32)
        # 64 rotary blocks dealt to the axes in sections, the first the shortest
        s["axis"] = [min(c["axes"] - 1, (j * c["axes"] + 20) // 64) if c["axes"] > 1 else 0 for j in range(64)]
        s["axis_dev"] = torch.tensor(s["axis"], device="cuda")
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    return {"attn": _run_attn, "append": _run_append, "copy": _run_copy, "fork": _run_fork,
            "compact": _run_compact, "rope": _run_rope}[s["c"]["op"]](s)


def _take(codes, scales, at):
    """Values of the blocks at[...] of each leading row: fp32."""
    raw = codes.view(torch.uint8)[:, at].view(codes.dtype).float()
    return raw * scales[:, at][..., None, None]


def _visible(c, lens, prefix, docs, n_keys):
    """[B, n_q, n_keys] truth values and the queries' positions [B, n_q]."""
    p = lens[:, None].long() - c["n_q"] + torch.arange(c["n_q"], device=lens.device)
    t = torch.arange(n_keys, device=lens.device)
    lo = torch.zeros_like(p) if docs is None else docs.long()
    if c["window"]:
        lo = torch.maximum(lo, p - c["window"] + 1)
    vis = (t >= lo[..., None]) & (t <= p[..., None])
    if prefix is not None:
        vis |= t < torch.minimum(prefix, lens)[:, None, None]
    return vis, p


def _run_attn(s):
    c = s["c"]
    if own:
        s["kv"].decode_attn(0, s["q"], s["lens"], s["out"], softcap=c["softcap"], slopes=s["slopes"],
                            window=c["window"], prefix=s["prefix"], doc_start=s["docs"])
        return s["out"]
    batch, n_q, hkv, grp = s["lens"].shape[0], c["n_q"], c["hkv"], c["hq"] // c["hkv"]
    if s["table"] is not None:
        at = s["table"].clamp(min=0).long()
        k = _take(s["k_codes"][0], s["k_scales"][0], at).transpose(0, 1)
        v = _take(s["v_codes"][0], s["v_scales"][0], at).transpose(0, 1)
    else:
        k = s["k_codes"][0].float() * s["k_scales"][0][..., None, None]
        v = s["v_codes"][0].float() * s["v_scales"][0][..., None, None]
    k, v = k.reshape(batch, hkv, -1, D), v.reshape(batch, hkv, -1, D)
    q = s["q"][0].float().view(batch, n_q, hkv, grp, D).permute(0, 2, 1, 3, 4).reshape(batch, hkv, n_q * grp, D)
    x = (q @ k.transpose(2, 3)).view(batch, hkv, n_q, grp, -1) / math.sqrt(D)
    del k
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    vis, p = _visible(c, s["lens"], s["prefix"], s["docs"], x.shape[-1])
    vis = vis[:, None, :, None, :]
    if s["slopes"] is not None:
        far = (p[..., None] - torch.arange(x.shape[-1], device=x.device))[:, None, :, None, :]
        x = x.double() - s["slopes"].double().view(1, hkv, 1, grp, 1) * far
    x = torch.where(vis, x, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    w = torch.where(vis, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0).float()
    total = w.sum(dim=-1, keepdim=True)
    o = (w.view(batch, hkv, n_q * grp, -1) @ v).view(batch, hkv, n_q, grp, D)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"][0] = o.permute(0, 2, 1, 3, 4).reshape(batch, n_q, c["hq"], D).to(s["out"].dtype)
    return s["out"]


def _cache(s):
    return {n: s[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def _run_append(s):
    c = s["c"]
    if own:
        s["kv"].append(0, s["k"], s["v"], s["starts"], s["counts"])
        return _cache(s)
    batch, tiles = s["starts"].shape[0], s["k_scales"].shape[-1]
    p = torch.arange(tiles * TILE, device="cuda")
    r = p - s["starts"].long()[:, None]                                 # the row that position p takes
    new = ((r >= 0) & (r < s["counts"][:, None])).view(batch, 1, tiles, TILE, 1)
    r = r.clamp(0, c["n"] - 1)
    anew = new[:, :, :, 0, 0]                                           # the block's first position is written
    hit = new.any(dim=3)[..., 0]
    for rows, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        x = torch.gather(rows[0].float(), 1, r[:, :, None, None].expand(-1, -1, c["hkv"], D))
        x = x.view(batch, tiles, TILE, c["hkv"], D).permute(0, 3, 1, 2, 4)
        e = _exponent(torch.where(new, x.abs(), 0.0).amax(dim=(3, 4)), c["code"])
        old = torch.frexp(scales[0])[1] - 1
        e = torch.where(hit, torch.where(anew, e, torch.maximum(e, old)), old)
        kept = _round(torch.ldexp(codes[0].float(), torch.where(anew, 0, old - e)[..., None, None]), c["code"])
        made = _round(torch.ldexp(x, -e[..., None, None]), c["code"])
        put = torch.where(new, made.view(torch.uint8), kept.view(torch.uint8))
        codes[0] = put.view(codes.dtype)
        scales[0] = torch.ldexp(torch.ones_like(scales[0]), e)
    return _cache(s)


def _move(s, src, dst):
    for name in ("k_codes", "v_codes"):
        raw = s[name].view(torch.uint8)
        raw[:, :, dst] = raw[:, :, src]
    for name in ("k_scales", "v_scales"):
        s[name][:, :, dst] = s[name][:, :, src]


def _run_copy(s):
    if own:
        s["kv"].copy_pages(s["src"], s["dst"])
    else:
        _move(s, s["src"].long(), s["dst"].long())
    return _cache(s)


def _run_fork(s):
    c = s["c"]
    if own:
        s["kv"].fork_sequences(s["parents"], s["table"], s["refs"], s["lens"], s["table_out"], s["refs_out"],
                               s["lens_out"])
        return {"table": s["table_out"], "refs": s["refs_out"], "lens": s["lens_out"], **_cache(s)}
    par, pool = s["parents"].long(), c["pool"]
    width = torch.arange(s["table"].shape[1], device="cuda")
    lens = torch.where(par >= 0, s["lens"][par.clamp(min=0)], 0)
    rows = s["table"][par.clamp(min=0)]
    held, had = width < -(-lens // TILE)[:, None], width < -(-s["lens"] // TILE)[:, None]
    refs = s["refs"].clone()
    refs += torch.bincount(rows[held].long(), minlength=pool).int() - torch.bincount(s["table"][had].long(), minlength=pool).int()
    part = lens % TILE != 0
    last = (lens // TILE).long().clamp(max=width.numel() - 1)
    page = torch.where(part, rows.gather(1, last[:, None])[:, 0].long(), pool)   # `pool`: none
    b = torch.arange(par.numel(), device="cuda")
    first = torch.full((pool + 1,), par.numel(), device="cuda").scatter_reduce(0, page, b, "amin")
    users = torch.bincount(page, minlength=pool + 1)
    more = torch.cat([refs, refs.new_zeros(1)])[page] > users[page]
    takers = torch.nonzero(part & ((first[page] != b) | more))[:, 0]
    fresh = torch.nonzero(refs == 0)[:takers.numel(), 0]
    src = page[takers]
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    refs[fresh] = 1
    rows[takers, last[takers]] = fresh.int()
    _move(s, src, fresh)
    s["table_out"][held] = rows[held]
    s["refs_out"].copy_(refs)
    s["lens_out"].copy_(lens)
    return {"table": s["table_out"], "refs": s["refs_out"], "lens": s["lens_out"], **_cache(s)}


def _run_compact(s):
    if own:
        s["kv"].compact_pages(s["table"], s["refs"], s["lens"], s["table_out"], s["refs_out"], s["map"], s["live"])
        return {"table": s["table_out"], "refs": s["refs_out"], "map": s["map"], "live": s["live"], **_cache(s)}
    ids, live = torch.arange(s["c"]["pool"], device="cuda"), s["refs"] > 0
    n = live.sum()
    src, dst = torch.nonzero(live & (ids >= n))[:, 0], torch.nonzero(~live & (ids < n))[:, 0]
    to = torch.where(live, ids, -1)
    to[src] = dst
    held = torch.arange(s["table"].shape[1], device="cuda") < -(-s["lens"] // TILE)[:, None]
    s["table_out"][held] = to[s["table"][held].long()].int()
    refs = s["refs"].clone()
    refs[dst] = refs[src]
    refs[src] = 0
    _move(s, src, dst)
    s["refs_out"].copy_(refs)
    s["map"].copy_(to)
    s["live"].copy_(n.view(1))
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["map"], "live": s["live"], **_cache(s)}


def _run_rope(s):
    c = s["c"]
    if own:
        from packed_decode_attention_b200 import bgtq
        bgtq.rope_axes(s["q"], s["k"], s["pos"], s["axis"], c["base"], s["q_out"], s["k_out"], pairing=c["pairing"])
        return s["q_out"], s["k_out"]
    j = torch.arange(64, device="cuda", dtype=torch.float64)
    angle = s["pos"].t()[:, s["axis_dev"]].double() * torch.pow(c["base"], -2.0 * j / D)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        if c["pairing"]:
            a, b = y[..., 0::2], y[..., 1::2]
            z = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        else:
            a, b = y[..., :64], y[..., 64:]
            z = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        out.copy_(z)
    return s["q_out"], s["k_out"]


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c = case
    if c["op"] == "attn":
        lens = _ints(c["lens"])
        prefix, docs = _ints(c["prefix"], len(lens)), _ints(c["docs"], len(lens))
        seen = pairs = 0
        for n, pre, doc in zip(lens, prefix, docs):
            pre, first = min(pre, n), n
            for i in range(c["n_q"]):
                p = n - c["n_q"] + i
                lo = max(doc, p - c["window"] + 1 if c["window"] else 0, 0)
                if lo <= p:
                    first = min(first, lo)
                pairs += max(0, p + 1 - max(lo, pre)) + pre
            seen += n - max(first, pre) + pre if first < n else pre
        rows = len(lens) * c["n_q"] * c["hq"]
        return {"bytes": seen * c["hkv"] * (2 * D + 8 / TILE) + rows * D * 4, "flops": 4.0 * D * pairs * c["hq"]}
    if c["op"] == "append":
        blocks = elems = 0
        for a, n in zip(_ints(c["starts"]), _ints(c["counts"])):
            blocks += (a + n - 1) // TILE - a // TILE + 1 if n else 0
            elems += n * c["hkv"] * D
        return {"bytes": 2 * (elems * 3 + blocks * c["hkv"] * 4), "flops": 4.0 * elems}
    if c["op"] == "rope":
        rows = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": rows * D * 4 + 4 * c["axes"] * c["tokens"], "flops": 3.0 * rows * D}
    moved, held = c.get("pairs", 0), 0
    if c["op"] != "copy":
        lens = _ints(c["lens"])
        held = sum(-(-v // TILE) for v in lens)
        if c["op"] == "fork":
            par = _ints(c["parents"])
            moved = sum(1 for b, p in enumerate(par) if p >= 0 and lens[p] % TILE and p in par[:b])
        else:
            live = held + c["held"]
            moved = live * (c["pool"] - live) // c["pool"]              # expected: the pages lie anywhere
    page = (2 * TILE * D + 8) * c["layers"] * c["hkv"]
    return {"bytes": 2 * moved * page + 8 * held + 8 * (c["pool"] if c["op"] != "copy" else moved), "flops": 0.0}


# ---- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] in ("copy", "fork", "compact"):
        return None                                     # copies and whole numbers: nothing is computed in floating point
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "rope": _exact_rope}[c["op"]](s, c)


def _exact_attn(s, c):
    lens, grp = _ints(c["lens"]), c["hq"] // c["hkv"]
    prefix, docs = _ints(c["prefix"], len(lens)), _ints(c["docs"], len(lens))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(c["hkv"] if n else 0):
            tiles = -(-n // TILE)
            at = (0, h, s["table"][b, :tiles].long()) if s["table"] is not None else (0, b, h, slice(0, tiles))

            def values(codes, scales):
                whole = codes.view(torch.uint8)[at].view(codes.dtype).double() * scales[at].double()[:, None, None]
                return whole.reshape(-1, D)[:n]

            k, v = values(s["k_codes"], s["k_scales"]), values(s["v_codes"], s["v_scales"])
            t = torch.arange(n, device="cuda")
            for i in range(c["n_q"]):
                p = n - c["n_q"] + i
                lo = max(docs[b], p - c["window"] + 1 if c["window"] else 0)
                see = ((t >= lo) & (t <= p)) | (t < prefix[b])
                if not bool(see.any()):
                    continue
                x = s["q"][0, b, i, h * grp:(h + 1) * grp].double() @ k[see].T / D ** 0.5
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                if s["slopes"] is not None:
                    x = x + s["slopes"][h * grp:(h + 1) * grp, None].double() * (t[see] - p).double()
                out[0, b, i, h * grp:(h + 1) * grp] = torch.softmax(x, dim=-1) @ v[see]
    return out


def _exact_append(s, c):
    """Block by block, with the codes' grid written out: e4m3 has steps of 2^(floor(log2 |y|) - 3), at least 2^-9."""
    q = QMAX[c["code"]]

    def grid(y):
        if c["code"] == "int8":
            return np.rint(y)
        size = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
        step = np.exp2(size - 3)
        return np.rint(y / step) * step

    got = {}
    for rows, kind in ((s["k"], "k"), (s["v"], "v")):
        x = rows[0].double().cpu().numpy()
        codes = s[kind + "_codes"][0].to(torch.float32).cpu().numpy().astype(np.float64)
        scales = s[kind + "_scales"][0].double().cpu().numpy()
        for b, (a, n) in enumerate(zip(_ints(c["starts"]), _ints(c["counts"]))):
            for t in range(a // TILE, (a + n - 1) // TILE + 1 if n else 0):
                lo, hi = max(a, t * TILE), min(a + n, (t + 1) * TILE)
                for h in range(c["hkv"]):
                    new = x[b, lo - a:hi - a, h]
                    big = np.abs(new).max()
                    scale = max(2.0 ** E_MIN, 2.0 ** math.ceil(math.log2(big / q))) if big else 2.0 ** E_MIN
                    if lo > t * TILE:
                        scale = max(scale, scales[b, h, t])
                        codes[b, h, t] = grid(codes[b, h, t] * (scales[b, h, t] / scale))
                    scales[b, h, t] = scale
                    codes[b, h, t, lo - t * TILE:hi - t * TILE] = grid(new / scale)
        codes = torch.from_numpy(codes[None])
        got[kind + "_codes"] = codes.to(torch.int8) if c["code"] == "int8" else codes
        got[kind + "_scales"] = torch.from_numpy(scales[None])
    return got


def _exact_rope(s, c):
    base = np.float64(c["base"]) ** (-np.arange(64) / 64.0)
    angle = s["pos"].cpu().numpy().astype(np.float64)[np.array(s["axis"])].T * base
    turn = torch.polar(torch.ones(angle.shape, dtype=torch.float64), torch.from_numpy(angle)).cuda()[:, None]

    def turned(x):
        pairs = x.double().unflatten(-1, (64, 2)) if c["pairing"] else x.double().unflatten(-1, (2, 64)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        return (z if c["pairing"] else z.transpose(-1, -2)).flatten(-2)

    return turned(s["q"]), turned(s["k"])
