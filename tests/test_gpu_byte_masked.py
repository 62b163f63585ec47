"""What no query of a call sees does not reach its result: NaN codes and scales in masked places of the 8-bit cache."""
import pytest
import torch

from oracle import byte_cache as bc

from byte_helpers import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


CASES = [dict(doc=5), dict(doc=33), dict(doc=100), dict(window=1), dict(window=40), dict(window=130),
         dict(window=20, prefix=7), dict(doc=150, prefix=70), dict(doc=10 ** 6), dict(doc=10 ** 6, prefix=3),
         dict(doc=60, window=75, prefix=1)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("group,n_q", [(4, 1), (4, 3), (16, 1), (8, 5)])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_unseen_positions_may_hold_anything(dev, code, group, n_q, case):
    """Left-padded and gapped sequences: NaN codes (e4m3) at every position that no query sees, NaN scales of the
    blocks that hold none that one sees."""
    lens = [200, 37, 512, 64]
    kv, q, out, sl, _ = make(dev, lens, hkv=1, group=group, n_q=n_q, code=code, rows="bf16", cap=512)
    opt, prefix, doc = {}, [0] * 4, [[0] * n_q] * 4
    if "window" in case:
        opt["window"] = case["window"]
    if "prefix" in case:
        prefix = [case["prefix"], 2, 300, 0]
        opt["prefix"] = i32(prefix, dev)
    if "doc" in case:
        # the queries' documents start at different places
        doc = [[case["doc"] + 3 * i for i in range(n_q)], [20 + i for i in range(n_q)], [case["doc"]] * n_q, [63] * n_q]
        opt["doc_start"] = i32(doc, dev)
    want = torch.empty_like(q)
    kv.decode_attn(0, q, sl, want, **opt)
    assert torch.isfinite(want).all()
    for b, n in enumerate(lens):
        seen = torch.zeros(512, dtype=torch.bool)
        for i in range(n_q):
            seen[:n] |= torch.from_numpy(bc.visible(n, n_q, i, case.get("window", 0), prefix[b], doc[b][i]))
        for codes, scales in ((kv.k_codes(), kv.k_scales()), (kv.v_codes(), kv.v_scales())):
            if code == "e4m3":
                raw = codes.view(torch.uint8)[0, b, 0].view(512, 128)
                raw[(~seen).to(dev)] = 0xFF
            else:
                codes[0, b, 0].view(512, 128)[(~seen).to(dev)] = -128
            scales[0, b, 0, (~seen.view(-1, 64).any(1)).to(dev)] = float("nan")
    kv.decode_attn(0, q, sl, out, **opt)
    assert torch.equal(out, want) and kv.device_error() == 0


def test_the_widest_window(dev):
    """A window past the capacity, at lengths shorter than the call's queries: as none."""
    lens = [3, 0, 200]
    kv, q, out, sl, _ = make(dev, lens, hkv=1, group=2, n_q=16)
    want = torch.empty_like(q)
    kv.decode_attn(0, q, sl, want)
    for window in (200, 2 ** 31 - 1):
        kv.decode_attn(0, q, sl, out.fill_(1), window=window)
        assert torch.equal(out, want)
