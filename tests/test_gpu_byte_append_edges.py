"""Appends of nothing to the 8-bit cache, and into blocks whose scale was never written."""
import numpy as np
import pytest
import torch

from oracle import byte_cache as bc
from packed_decode_attention_b200 import bgtq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def test_no_rows_past_the_capacity_are_no_error(dev):
    """Idle rows: count 0, wherever the sequence stands."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(1, 2, 2, 4, 100), dev)
    before = kv.cache.clone()
    k = torch.ones((1, 4, 4, 2, 128), dtype=torch.float16, device=dev)
    kv.append(0, k, k, i32([100, 101, 5000, 2 ** 31 - 1], dev), i32([0, 0, 0, 0], dev))
    assert torch.equal(kv.cache, before) and kv.device_error() == 0
    kv.append(0, k, k, i32([99, 101, 100, 0], dev), i32([2, 0, 0, 0], dev))
    assert kv.device_error() == bgtq.DEVERR_CAPACITY


def test_a_call_of_no_rows(dev):
    """n = 0: torch's empty tensors have no address."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(2, 2, 2, 3, 100), dev)
    before = kv.cache.clone()
    k = torch.empty((2, 3, 0, 2, 128), dtype=torch.float16, device=dev)
    kv.append(0, k, k, i32([0, 5, 99], dev), i32([0, 0, 0], dev), layer_count=2)
    kv._ctx = None                                            # and by the Python checks
    kv.append(0, k, k, i32([0, 5, 99], dev), i32([0, 0, 0], dev), layer_count=2)
    assert torch.equal(kv.cache, before) and kv.device_error() == 0
    with pytest.raises(bgtq.BgtqError) as e:
        kv.append(1, k, k, i32([0, 5, 99], dev), i32([0, 0, 0], dev), layer_count=2)
    assert e.value.status == -1
    with pytest.raises(bgtq.BgtqError) as e:
        bgtq.bgtq_byte_append(kv.state, 0, 1, None, None, i32([0], dev), i32([0], dev), 1, 1)
    assert e.value.status == -2


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_a_scale_that_is_no_power_of_two_is_none(dev, code):
    """A block that starts in its middle, in a buffer that held something else before."""
    cfg = bgtq.ByteConfig(n_layers=1, n_kv_heads=1, n_q_heads=1, max_batch=1, capacity_tokens=64, code=code)
    kv = bgtq.ByteKVCache(cfg, dev)
    k = torch.randn((1, 1, 20, 1, 128), device=dev).half()
    vals, exps = np.zeros((1, 64, 128)), np.full(1, bc.E_MIN)
    bc.append(vals, exps, k[0, 0, :, 0].double().cpu().numpy(), 7, 64, code)
    inf = float("inf")
    for was in (0.0, 3e20, 1.5 * 2.0 ** 60, 2.0 ** 60 + 2.0 ** 37, -2.0 ** 60, 2.0 ** -101, 2.0 ** -140, inf, -inf, float("nan")):
        kv.cache.zero_()
        for s in (kv.k_scales(), kv.v_scales()):
            s.fill_(was)
        kv.append(0, k, k, i32([7], dev), i32([20], dev))
        assert kv.v_scales().item() == kv.k_scales().item() == 2.0 ** exps[0], was
        assert np.array_equal(kv.k_codes().double().cpu().numpy()[0, 0, 0, 0, 7:27], vals[0, 7:27]), was
    assert kv.device_error() == 0
