"""The 8-bit cache's attention at random over what its documentation allows together: sequences from none to hundreds,
head groups, query tokens, layers a call, paging, row and code types, masks and biases, blocks of very unequal scale."""
import random

import pytest
import torch

from byte_helpers import check_attention, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(dev, seed):
    rng = random.Random(seed)
    batch = [1, 1, 2, 5, 31, 32, 33, 200, 400][seed % 9]
    group, n_q = rng.choice([1, 2, 3, 4, 7, 8, 9, 16]), rng.choice([1, 1, 2, 3, 4, 7, 16])
    hkv, layers = rng.choice([1, 1, 2, 3]), rng.choice([1, 1, 2])
    rows = batch * group * n_q * hkv * layers
    most = max(40, min(9000, 6_000_000 // rows))
    lens = [rng.choice([0, 1, 31, 32, 33, 64, 65, n_q, rng.randint(0, most)]) if rng.random() < 0.4 else
            rng.randint(1, most) for _ in range(batch)]
    code, rt, paged = rng.choice(["e4m3", "int8"]), rng.choice(["fp16", "bf16"]), rng.random() < 0.5
    kv, q, out, sl, table = make(dev, lens, hkv=hkv, group=group, code=code, rows=rt, n_q=n_q, layers=layers,
                                 paged=paged, seed=seed)
    if rng.random() < 0.3:
        # scales of neighbouring blocks up to 2^12 apart
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        v = kv.v_scales()
        v.mul_(torch.exp2(torch.randint(-6, 7, v.shape, generator=g, device=dev).float()))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    kw, score = {}, {}
    if rng.random() < 0.4:
        kw["softcap"] = score["softcap"] = rng.choice([2.0, 30.0])
    if rng.random() < 0.4:
        s = [2.0 ** -rng.randint(1, 9) for _ in range(hkv * group)]
        kw["slopes"], score["slopes"] = torch.tensor(s, device=dev), s
    if rng.random() < 0.4:
        kw["window"] = score["window"] = rng.choice([1, 5, 40, 700])
    if rng.random() < 0.4:
        p = [rng.choice([0, 3, 70, 10 ** 6]) for _ in lens]
        kw["prefix"], score["prefix"] = i32(p), p
    if rng.random() < 0.4:
        d = [[rng.randint(-2, n + 2) for _ in range(n_q)] for n in lens]
        kw["doc_start"], score["doc_start"] = i32(d), d
    if rng.random() < 0.3:
        kw["scale"] = score["scale"] = 0.05
    kv.decode_attn(0, q, sl, out, layer_count=layers, **kw)
    check_attention(kv, q, lens, out, layer_count=layers, table=table, **score)
    again = torch.full_like(out, float("nan"))
    kv.decode_attn(0, q, sl, again, layer_count=layers, **kw)
    assert torch.equal(out, again) and kv.device_error() == 0


@pytest.mark.parametrize("hkv,group,n_q", [(1, 4, 1), (3, 8, 1), (2, 16, 1), (148, 1, 1), (75, 2, 1), (5, 3, 5)])
def test_one_sequence_shared_by_the_whole_gpu(dev, hkv, group, n_q):
    """A unit's steps in equal shares, units fewer and more than the SMs, lengths around the shares' borders."""
    for n in (1, 33, 385, 4735, 4737, 9999 if hkv < 50 else 500):
        kv, q, out, sl, _ = make(dev, [n], hkv=hkv, group=group, n_q=n_q, code="int8", seed=n)
        kv.decode_attn(0, q, sl, out)
        check_attention(kv, q, [n], out)
