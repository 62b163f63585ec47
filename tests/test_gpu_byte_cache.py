"""The 8-bit cache on the GPU: append bit for bit and attention row by row
against the float64 oracle, over codes, row types, head layouts, lengths,
masks and paging; refusals; captured graphs; streams."""
import numpy as np
import pytest
import torch

from oracle import byte_cache as bc
from packed_decode_attention_b200 import bgtq

from byte_helpers import check_attention, make, values

pytestmark = pytest.mark.gpu

CODES, ROWS = ["e4m3", "int8"], ["fp16", "bf16"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# ---- append ----------------------------------------------------------------

def unscaled(codes):
    return codes.double().cpu().numpy()


def check_append(kv, calls, dev, table=None):
    """Appends in turn, the whole cache compared with the oracle's after each."""
    cfg = kv.cfg
    arrs = {}
    for kind, c, s in (("k", kv.k_codes(), kv.k_scales()), ("v", kv.v_codes(), kv.v_scales())):
        sc = s.double().cpu().numpy()
        arrs[kind] = (unscaled(c), np.where(sc > 0, np.log2(np.where(sc > 0, sc, 1)), bc.E_MIN), sc)
    for layer, k, v, start, count in calls:
        kv.append(layer, k, v, i32(start, dev), i32(count, dev), layer_count=k.shape[0])
        for kind, x in (("k", k), ("v", v)):
            vals, exps, raw = arrs[kind]
            xn = x.double().cpu().numpy()
            for l in range(k.shape[0]):
                for b in range(k.shape[1]):
                    for h in range(cfg.n_kv_heads):
                        if table is None:
                            bv, be = vals[layer + l, b, h], exps[layer + l, b, h]
                            bc.append(bv, be, xn[l, b, :count[b], h], start[b], cfg.capacity_tokens, cfg.code)
                        else:
                            bv, be = vals[layer + l, h][table[b]], exps[layer + l, h][table[b]]
                            bc.append(bv, be, xn[l, b, :count[b], h], start[b], cfg.capacity_tokens, cfg.code)
                            vals[layer + l, h][table[b]], exps[layer + l, h][table[b]] = bv, be
            got = kv.k_codes() if kind == "k" else kv.v_codes()
            assert np.array_equal(unscaled(got), vals), kind
            sc = (kv.k_scales() if kind == "k" else kv.v_scales()).double().cpu().numpy()
            written = sc > 0
            assert np.array_equal(sc[written], 2.0 ** exps[written]) and np.all(raw[~written] == 0)
    assert kv.device_error() == 0


def rows(g, dev, shape, dt, lo=-3, hi=4):
    size = torch.exp2(torch.randint(lo, hi, shape[:-2] + (shape[-2], 1), generator=g, device=dev).float())
    return (torch.randn(shape, generator=g, device=dev) * size).to(dt)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rt", ROWS)
def test_append_matches_oracle(dev, code, rt):
    """Prefill pieces that start and end inside blocks, then single rows whose size makes scales grow."""
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    cfg = bgtq.ByteConfig(n_layers=2, n_kv_heads=2, n_q_heads=2, max_batch=3, capacity_tokens=300, code=code, rows=rt)
    kv = bgtq.ByteKVCache(cfg, dev)
    mk = lambda n, L=1: (rows(g, dev, (L, 3, n, 2, 128), kv.row_dtype), rows(g, dev, (L, 3, n, 2, 128), kv.row_dtype))  # noqa: E731
    calls = []
    pos = [0, 0, 0]
    for n, counts in ((65, [65, 1, 0]), (130, [130, 63, 64]), (1, [1, 1, 1]), (2, [2, 2, 1]), (1, [1, 0, 1]),
                      (70, [3, 70, 64])):
        k, v = mk(n, 2)
        calls.append((0, k, v, list(pos), counts))
        pos = [p + c for p, c in zip(pos, counts)]
    k, v = mk(5)
    calls.append((1, k, v, [2, 64, 100], [5, 5, 5]))        # rows in the middle written again
    check_append(kv, calls, dev)


@pytest.mark.parametrize("code", CODES)
def test_append_paged_and_capacity(dev, code):
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    cfg = bgtq.ByteConfig(n_layers=1, n_kv_heads=3, n_q_heads=3, max_batch=2, capacity_tokens=150, code=code,
                          page_pool_tiles=9)
    kv = bgtq.ByteKVCache(cfg, dev)
    table = np.array([[7, 0, 4], [8, 2, 1]], dtype=np.int32)
    kv.set_block_table(torch.from_numpy(table).to(dev))
    mk = lambda n: (rows(g, dev, (1, 2, n, 3, 128), torch.float16), rows(g, dev, (1, 2, n, 3, 128), torch.float16))  # noqa: E731
    check_append(kv, [(0, *mk(100), [0, 0], [100, 90]), (0, *mk(40), [100, 90], [40, 40])], dev, table)
    # past the capacity: the rows that fit are written
    k, v = mk(40)
    kv.append(0, k, v, i32([140, 130], dev), i32([40, 10], dev))
    assert kv.device_error() == bgtq.DEVERR_CAPACITY
    got = values(kv.k_codes(), kv.k_scales())[0, 0, 4].reshape(-1, 128)
    # half a step: e4m3 2^-4 of the value (2^-10 of the scale among its subnormals), int8 half the scale
    x, unit = k[0, 0, :10, 0].double().cpu().numpy(), kv.k_scales()[0, 0, 4].item()
    step = np.maximum(np.abs(x) * 2.0 ** -4, unit * 2.0 ** -10) if code == "e4m3" else unit / 2
    assert np.all(np.abs(got[12:22] - x) <= step)
    assert np.array_equal(got[22:], np.zeros((42, 128)))    # behind the capacity: as it was


def test_append_of_no_rows_touches_nothing(dev):
    """No rows, or none within the capacity, in the middle of a block that nothing was written to."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(1, 2, 2, 3, 100), dev)
    before = kv.cache.clone()
    k = torch.ones((1, 3, 4, 2, 128), dtype=torch.float16, device=dev)
    kv.append(0, k, k, i32([70, 120, 2 ** 31 - 2], dev), i32([0, 3, 4], dev))
    assert torch.equal(kv.cache, before) and kv.device_error() == bgtq.DEVERR_CAPACITY


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rt", ROWS)
def test_append_special_values(dev, code, rt):
    """Infinities, NaN, zeros, the type's largest and smallest values."""
    cfg = bgtq.ByteConfig(n_layers=1, n_kv_heads=1, n_q_heads=1, max_batch=1, capacity_tokens=256, code=code, rows=rt)
    kv = bgtq.ByteKVCache(cfg, dev)
    dt = kv.row_dtype
    k = torch.zeros((1, 1, 256, 1, 128), dtype=dt, device=dev)
    f = torch.finfo(dt)
    k[0, 0, 64, 0, :4] = torch.tensor([f.max, f.tiny, f.min, 1.0], dtype=dt)
    k[0, 0, 128, 0, :4] = torch.tensor([float("inf"), float("nan"), float("-inf"), 3.0], dtype=dt)
    k[0, 0, 192, 0, :2] = torch.tensor([f.smallest_normal, f.tiny / 4 if rt == "fp16" else f.tiny], dtype=dt)
    kv.append(0, k, k, i32([0], dev), i32([256], dev))
    assert kv.device_error() == bgtq.DEVERR_NONFINITE
    vals, exps = np.zeros((4, 64, 128)), np.zeros(4)
    bc.append(vals, exps, k[0, 0, :, 0].double().cpu().numpy(), 0, 256, code)
    assert np.array_equal(unscaled(kv.k_codes())[0, 0, 0], vals)
    assert np.array_equal(kv.v_scales()[0, 0, 0].double().cpu().numpy(), 2.0 ** exps)
    assert exps[0] == bc.E_MIN


def test_append_argument_errors(dev):
    cfg = bgtq.ByteConfig(n_layers=1, n_kv_heads=1, n_q_heads=1, max_batch=3, capacity_tokens=128, page_pool_tiles=4)
    kv = bgtq.ByteKVCache(cfg, dev)
    k = torch.ones((1, 3, 2, 1, 128), dtype=torch.float16, device=dev)
    with pytest.raises(bgtq.BgtqError) as e:
        kv.append(0, k, k, i32([0, 0, 0], dev), i32([1, 1, 1], dev))
    assert e.value.status == -5                              # no block table yet
    kv.set_block_table(i32([[0, 1], [2, 3], [9, -1]], dev))
    kv.append(0, k, k, i32([-1, 0, 0], dev), i32([1, 3, 0], dev))
    assert kv.device_error() == bgtq.DEVERR_ARG
    assert not kv.cache.any()
    kv.append(0, k, k, i32([0, 0, 0], dev), i32([1, 0, 1], dev))
    assert kv.device_error() == bgtq.DEVERR_PAGE
    assert kv.k_codes()[0, 0, 0].float().any() and not kv.k_codes()[0, 0, 1:].float().any()


# ---- attention ---------------------------------------------------------------

LENS = [[1], [64], [65, 0, 3], [4096], [700, 1, 2500, 63]]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rt", ROWS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_attention_lengths(dev, code, rt, lens):
    kv, q, out, sl, _ = make(dev, lens, hkv=2, group=4, code=code, rows=rt)
    kv.decode_attn(0, q, sl, out)
    check_attention(kv, q, lens, out)
    assert kv.device_error() == 0


@pytest.mark.parametrize("group,n_q", [(1, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (1, 8), (4, 4), (7, 3), (16, 16)])
@pytest.mark.parametrize("code", CODES)
def test_attention_head_layouts(dev, group, n_q, code):
    lens = [260, 5, 129]
    kv, q, out, sl, table = make(dev, lens, hkv=2, group=group, n_q=n_q, code=code, paged=True, rows="bf16")
    kv.decode_attn(0, q, sl, out)
    check_attention(kv, q, lens, out, table=table)
    assert kv.device_error() == 0


MASKS = [
    dict(softcap=5.0), dict(softcap=0.01), dict(softcap=1e4), dict(window=1), dict(window=64), dict(window=100),
    dict(window=5, prefix=[4, 70, 0, 900]), dict(prefix=[400, 1, 0, 64]),
    dict(doc=True), dict(doc=True, prefix=[1, 1, 0, 130]), dict(slopes=True), dict(slopes=True, window=70),
    dict(slopes=True, softcap=2.0, window=10, prefix=[3, 64, 1, 129], doc=True), dict(scale=0.3),
    dict(empty=True), dict(empty=True, slopes=True, prefix=[0, 2, 0, 0]),
]


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: ",".join(m))
@pytest.mark.parametrize("n_q,group", [(1, 4), (3, 4)])
def test_attention_masks(dev, mask, n_q, group):
    lens = [330, 2, 0, 1000]
    kv, q, out, sl, _ = make(dev, lens, hkv=1, group=group, n_q=n_q, code="int8", cap=1024)
    opt = {k: mask[k] for k in ("softcap", "window", "scale") if k in mask}
    dev_opt = dict(opt)
    if "prefix" in mask:
        opt["prefix"], dev_opt["prefix"] = mask["prefix"], i32(mask["prefix"], dev)
    if mask.get("slopes"):
        s = torch.tensor([0.5, 0.0, 2.0 ** -8, 3.0][:group], device=dev)
        opt["slopes"], dev_opt["slopes"] = s.double().tolist(), s
    if mask.get("doc") or mask.get("empty"):
        d = [[n if mask.get("empty") else max(0, n - 70 - 65 * i) for i in range(n_q)] for n in lens]
        opt["doc_start"], dev_opt["doc_start"] = d, i32(d, dev)
    kv.decode_attn(0, q, sl, out, **dev_opt)
    check_attention(kv, q, lens, out, **opt)
    assert kv.device_error() == 0


def test_far_prefix_keeps_its_distances(dev):
    """Only a far prefix is visible: the bias differences among its positions must survive the large distances."""
    n = 1 << 17
    kv, q, out, sl, _ = make(dev, [n], hkv=1, group=4, code="int8")
    s = torch.tensor([0.5, 0.25, 1.0, 0.125], device=dev)
    doc = i32([[n]], dev)
    kv.decode_attn(0, q, sl, out, slopes=s, prefix=i32([100], dev), doc_start=doc)
    check_attention(kv, q, [n], out, slopes=s.tolist(), prefix=[100], doc_start=[[n]])


@pytest.mark.parametrize("code", CODES)
def test_long_and_many(dev, code):
    """Units over many CTAs beside units that share one; several layers in one call."""
    lens = [30000, 0, 17, 5000, 64, 1, 129, 9999]
    kv, q, out, sl, table = make(dev, lens, hkv=2, group=5, code=code, layers=3, paged=True)
    kv.decode_attn(1, q[1:], sl, out[1:], layer_count=2)
    check_attention(kv, q[1:], lens, out[1:], layer=1, layer_count=2, table=table)
    one = torch.full_like(out[2:], float("nan"))
    kv.decode_attn(2, q[2:], sl, one)
    check_attention(kv, q[2:], lens, one, layer=2, table=table)
    assert torch.isnan(out[0]).all()


def test_batch_larger_than_a_cta(dev):
    """More sequences than a CTA has threads."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 90, size=600)]
    kv, q, out, sl, _ = make(dev, lens, hkv=1, group=1)
    kv.decode_attn(0, q, sl, out)
    check_attention(kv, q, lens, out)


def test_garbage_behind_the_sequence(dev):
    """NaN codes behind seq_lens, and whole blocks nothing refers to, do not reach the result."""
    lens = [70, 128, 1]
    for rt in ROWS:
        kv, q, out, sl, _ = make(dev, lens, hkv=1, group=2, code="e4m3", rows=rt, cap=256)
        want = torch.empty_like(q)
        kv.decode_attn(0, q, sl, want)
        for b, n in enumerate(lens):
            for c in (kv.k_codes(), kv.v_codes()):
                c.view(torch.uint8)[0, b].view(1, -1, 128)[:, n:] = 0x7F
            for s in (kv.k_scales(), kv.v_scales()):
                s[0, b, :, -(-n // 64):] = float("nan")
        kv.decode_attn(0, q, sl, out)
        assert torch.equal(out, want)


def test_query_extremes(dev):
    """Queries near the type's largest and smallest values, a zero row, and a NaN row that stays alone."""
    for rt in ROWS:
        kv, q, out, sl, _ = make(dev, [100], hkv=1, group=5, code="int8", rows=rt)
        f = torch.finfo(q.dtype)
        q[0, 0, 0, 0] *= f.max / 2 ** 8
        q[0, 0, 0, 1] *= f.tiny * 64
        q[0, 0, 0, 2] = 0
        q[0, 0, 0, 3, 7] = float("nan")
        kv.decode_attn(0, q, sl, out)
        assert torch.isnan(out[0, 0, 0, 3]).all()
        keep = [0, 1, 2, 4]
        assert torch.isfinite(out[0, 0, 0, keep]).all()
        v = values(kv.v_codes(), kv.v_scales())[0, 0, 0].reshape(-1, 128)[:100]
        k = values(kv.k_codes(), kv.k_scales())[0, 0, 0].reshape(-1, 128)[:100]
        best = (k @ q[0, 0, 0, 0].double().cpu().numpy()).argmax()     # a softmax this steep picks one position
        assert np.abs(out[0, 0, 0, 0].double().cpu().numpy() - v[best]).max() <= 2.0 ** -8 * np.abs(v[best]).max()
        assert np.abs(out[0, 0, 0, 2].double().cpu().numpy() - v.mean(0)).max() <= 2.0 ** -7 * np.abs(v).mean()


def test_lengths_out_of_range_and_bad_pages(dev):
    lens = [100, 100]
    kv, q, out, sl, table = make(dev, lens, hkv=1, group=2, paged=True, cap=128)
    good = torch.empty_like(out)
    kv.decode_attn(0, q, sl, good)
    kv.decode_attn(0, q, i32([100, 129], dev), out)
    assert kv.device_error() == bgtq.DEVERR_SEQ_LEN
    assert torch.equal(out[0, 0], good[0, 0]) and not out[0, 1].any()
    kv.decode_attn(0, q, i32([-5, 100], dev), out)
    assert kv.device_error() == bgtq.DEVERR_SEQ_LEN and not out[0, 0].any()
    table[1, 1] = 77
    kv.decode_attn(0, q, sl, out)
    assert kv.device_error() == bgtq.DEVERR_PAGE and torch.equal(out[0, 0], good[0, 0])


def test_repeats_bit_for_bit_on_streams_and_in_graphs(dev):
    lens = [3000, 10, 700]
    kv, q, out, sl, _ = make(dev, lens, hkv=2, group=4, code="e4m3", cap=4096)
    first = torch.empty_like(out)
    kv.decode_attn(0, q, sl, first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kv.decode_attn(0, q, sl, out)
    s.synchronize()
    assert torch.equal(out, first)
    k = torch.randn((1, 3, 1, 2, 128), device=dev).half()
    start, one = sl.clone(), i32([1, 1, 1], dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.append(0, k, k, start, one)
        start += 1
        kv.decode_attn(0, q, start, out)
    for step in range(3):
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        check_attention(kv, q, [n + step + 1 for n in lens], out)
    assert kv.device_error() == 0


def test_timeout_is_reported(dev):
    """A block whose copies are never issued: the waits end, the flag is set, the state stays usable."""
    kv, q, out, sl, _ = make(dev, [640], hkv=1, group=4)
    want = torch.empty_like(out)
    kv.decode_attn(0, q, sl, want)
    kv.test_drop_tile_copies(3)
    kv.decode_attn(0, q, sl, out)
    assert kv.device_error() == bgtq.DEVERR_TIMEOUT
    kv.test_drop_tile_copies(-1)
    kv.decode_attn(0, q, sl, out)
    assert kv.device_error() == 0 and torch.equal(out, want)


def test_states_refuse_each_others_calls(dev):
    byte = bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, 1, 64), dev)
    packed = bgtq.PackedKVCache(bgtq.Config(1, 1, 1, 1, 64), dev)
    z = torch.zeros(1 << 12, dtype=torch.float16, device=dev)
    n = i32([0], dev)

    def status(fn, *a):
        with pytest.raises(bgtq.BgtqError) as e:
            fn(*a)
        return e.value.status

    st = byte.state
    assert status(bgtq.bgtq_allocate, st, z, 1, z, 1) == -1
    assert status(bgtq.bgtq_set_allocation, st, np.full((1, 1, 64), 3)) == -1
    assert status(bgtq.bgtq_encode_append, st, 0, 1, z, z, n, n, 1, 1) == -5
    assert status(bgtq.bgtq_decode_attn, st, 0, 1, z, n, 1, z) == -5
    assert status(bgtq.bgtq_decode_split, st, 0, 1, z, n, 1) == -5
    assert status(bgtq.bgtq_rotate_query, st, 0, 1, z, 1, z) == -5
    assert status(bgtq.bgtq_logit_mae, st, 0, 1, 0, 0, 1, z, z, z) == -5
    assert status(bgtq.bgtq_get_allocation, st, 1, 1) == -5
    assert status(bgtq.bgtq_get_layout, st, 0, 0) == -5
    assert status(bgtq.bgtq_set_split_tokens, st, 64) == -1
    assert status(bgtq.bgtq_set_decode_path, st, 0) == -1
    assert status(bgtq.bgtq_get_decode_path, st) == -1
    assert status(bgtq.bgtq_byte_append, packed.state, 0, 1, z, z, n, n, 1, 1) == -1
    assert status(bgtq.bgtq_byte_decode_attn, packed.state, 0, 1, z, n, 1, 1, z) == -1
