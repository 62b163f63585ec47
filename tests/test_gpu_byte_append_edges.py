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
