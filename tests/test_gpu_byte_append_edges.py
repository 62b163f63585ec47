"""Appends of nothing to the 8-bit cache."""
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
