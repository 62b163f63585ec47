"""Attention over the 8-bit cache at the ends of its ranges: scores of any size."""
import numpy as np
import pytest
import torch

from byte_helpers import HALF_STEP, TINY, make, values

pytestmark = pytest.mark.gpu

CODES = ["e4m3", "int8"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


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
