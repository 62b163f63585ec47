"""Attention over the 8-bit cache at the ends of its ranges: scores, scales and biases of any size, values up to the type's
largest, biases that grow with the distance."""
import numpy as np
import pytest
import torch

from oracle import byte_cache as bc
from packed_decode_attention_b200 import bgtq

from byte_helpers import HALF_STEP, TINY, check_attention, make, values

pytestmark = pytest.mark.gpu

CODES = ["e4m3", "int8"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def close(got, want, mass, rows):
    """Weights of 0 or of one size: only fp32 sums (2^-19 of sum p |v|) and the output's rounding are off."""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    allowed = 2.0 ** -19 * mass
    return np.all(np.abs(got - want) <= allowed + HALF_STEP[rows] * (np.abs(want) + allowed) + TINY[rows])


@pytest.mark.parametrize("code", CODES)
def test_scores_of_every_size(dev, code):
    """One position, and two of one score, with scores from 2^4 to 2^45 and their negatives in log2 units: the
    weights are finite, so the result is the value, or the mean of both."""
    kv, q, out, sl, _ = make(dev, [1, 2], hkv=1, group=4, code=code, rows="bf16")
    kv.k_codes().copy_(torch.ones((), device=dev).to(kv.k_codes().dtype))
    v = values(kv.v_codes(), kv.v_scales())[0, :, 0, 0]
    q[:] = torch.tensor([1.0, -1.0, 1.375, -1.75], device=dev, dtype=q.dtype)[:, None]
    for e in range(42):
        kv.k_scales().fill_(2.0 ** e)
        kv.decode_attn(0, q, sl, out)
        for r in range(4):
            assert close(out[0, 0, 0, r], v[0, 0], np.abs(v[0, 0]), "bf16"), (e, r)
            assert close(out[0, 1, 0, r], v[1, :2].mean(0), np.abs(v[1, :2]).mean(0), "bf16"), (e, r)


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_scores_past_fp32(dev, softcap):
    """Scores that fp32 does not hold: the largest one wins, and zero codes under a huge scale score 0."""
    kv, q, out, sl, _ = make(dev, [5, 1], hkv=1, group=4, code="int8", rows="bf16")
    k = kv.k_codes()
    k.zero_()
    k[0, 0, 0, 0, 2, 0], k[0, 0, 0, 0, 4, 0], k[0, 0, 0, 0, 3, 1], k[0, 1, 0, 0, 0, :2] = 1, -1, -1, -1
    kv.k_scales().fill_(2.0 ** 100)
    q.zero_()
    q[..., 0, 0], q[..., 1, 0], q[..., 2, 1] = 2.0 ** 120, -2.0 ** 120, 2.0 ** 120
    kv.decode_attn(0, q, sl, out, softcap=softcap)
    v = values(kv.v_codes(), kv.v_scales())[0, :, 0, 0]
    sign = np.array([[0, 0, 1, 0, -1], [0, 0, -1, 0, 1], [0, 0, 0, -1, 0], [0, 0, 0, 0, 0]])
    for r in range(4):
        x = sign[r] * (softcap or 1e30)
        w = np.exp(x - x.max())
        w /= w.sum()
        # capped scores: tanh's 1e-6 of 5, twice in a weight and its sum; weights in fp16 (2^-11, twice)
        extra = (4e-5 + 2.0 ** -10) * (w @ np.abs(v[0, :5])) if softcap else 0.0
        got = out[0, 0, 0, r].double().cpu().numpy()
        want = w @ v[0, :5]
        allowed = extra + (2.0 ** -10 + 2.0 ** -19) * (w @ np.abs(v[0, :5]))   # the mean of 4 or 5: equal weights
        assert np.all(np.abs(got - want) <= allowed + HALF_STEP["bf16"] * (np.abs(want) + allowed)), r
        assert close(out[0, 1, 0, r], v[1, 0], np.abs(v[1, 0]), "bf16"), r


def test_scale_bounds(dev):
    kv, q, out, sl, _ = make(dev, [70], hkv=1, group=4, rows="bf16")
    kv.decode_attn(0, q, sl, out, scale=16384.0)
    assert torch.isfinite(out).all()
    for bad in (16385.0, 1e30, float("inf"), float("nan"), -1.0):
        with pytest.raises(bgtq.BgtqError) as e:
            kv.decode_attn(0, q, sl, out, scale=bad)
        assert e.value.status == -1


@pytest.mark.parametrize("rt", ["fp16", "bf16"])
def test_slopes_of_the_largest_size(dev, rt):
    """A bias so steep that one position is left: the nearest, or the farthest where the slope is negative."""
    kv, q, out, sl, _ = make(dev, [700], hkv=1, group=4, code="int8", rows=rt)
    big = torch.finfo(torch.float32).max
    kv.decode_attn(0, q, sl, out, slopes=torch.tensor([big, 1e30, -big, -1e30], device=dev), prefix=i32([5], dev),
                   window=100)
    v = values(kv.v_codes(), kv.v_scales())[0, 0, 0].reshape(-1, 128)
    for r, at in enumerate((699, 699, 0, 0)):
        assert close(out[0, 0, 0, r], v[at], np.abs(v[at]), rt), r


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("lens,hkv", [([1], 1), ([5, 700], 1), ([4000], 1), ([4000, 1, 3000, 70], 4)])
def test_values_up_to_the_largest(dev, code, lens, hkv):
    """Values near bf16's largest: sums over the positions must not overflow where the weighted mean does not."""
    kv, q, out, sl, _ = make(dev, lens, hkv=hkv, group=4, code=code, rows="bf16")
    kv.v_scales().fill_(2.0 ** (118 if code == "e4m3" else 120))
    kv.decode_attn(0, q, sl, out)
    assert torch.isfinite(out).all()
    check_attention(kv, q, lens, out)
    kv.v_scales().fill_(2.0 ** -100)
    kv.decode_attn(0, q, sl, out)
    check_attention(kv, q, lens, out)


@pytest.mark.parametrize("opt", [{}, {"window": 70000}, {"prefix": 100}, {"prefix": 9, "window": 1000}], ids=str)
@pytest.mark.parametrize("n_q", [1, 3])
def test_negative_slopes_keep_the_far_positions(dev, opt, n_q):
    """With a negative slope the farthest positions weigh most: the bias must be exact there, however far they are.

    The error allowed is byte_helpers.expect's, with the bias of each position counted from the heaviest one
    (2^-22 of it) and weighed by the position's own weight."""
    n = 1 << 17
    kv, q, out, sl, _ = make(dev, [n], hkv=1, group=4, code="int8", n_q=n_q, rows="fp16")
    slopes = [-1.0, -0.3, -2.0 ** -12, 0.25]
    dopt = dict(opt)
    if "prefix" in opt:
        dopt["prefix"] = i32([opt["prefix"]], dev)
    kv.decode_attn(0, q, sl, out, slopes=torch.tensor(slopes, device=dev), **dopt)
    k = values(kv.k_codes(), kv.k_scales())[0, 0, 0].reshape(-1, 128)
    v = values(kv.v_codes(), kv.v_scales())[0, 0, 0].reshape(-1, 128)
    for i in range(n_q):
        see = bc.visible(n, n_q, i, opt.get("window", 0), opt.get("prefix", 0))
        t = np.arange(n)[see]
        for r, slope in enumerate(torch.tensor(slopes).double().tolist()):
            qr = q[0, 0, i, r].double().cpu().numpy()
            x = k[see] @ qr / np.sqrt(128)
            s = (np.abs(k[see]) @ np.abs(qr)).max() / np.sqrt(128)
            bias = slope * (t - (t.min() if slope < 0 else t.max()))      # <= 0
            w = np.exp(x + bias - (x + bias).max())
            w /= w.sum()
            want = w @ v[see]
            d = s * 2.0 ** -16 + s * 2e-6 + (s + np.abs(bias)) * 2.0 ** -22
            allowed = (w * (2 * HALF_STEP["fp16"] + 2 * d + 2 * (w @ d) + 2.0 ** -20)) @ np.abs(v[see])
            allowed = allowed + 2.0 ** -39 * np.abs(v[see]).sum(axis=0)
            got = out[0, 0, i, r].double().cpu().numpy()
            allowed = allowed + HALF_STEP["fp16"] * (np.abs(want) + allowed) + TINY["fp16"]
            assert np.all(np.abs(got - want) <= allowed), (i, r, np.abs(got - want).max(), allowed.min())
