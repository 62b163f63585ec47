"""Forks of rows whose lengths are out of range; lengths that are input and output at once."""
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


@pytest.mark.parametrize("batch,pool", [(4, 12), (300, 900), (4, 9000)])
def test_fork_flags_lengths_nobody_forks_from(dev, batch, pool):
    """Every row's length is checked, also those of rows that end with the call."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, batch, 128, page_pool_tiles=pool), dev)
    table = [[2 * b, 2 * b + 1] for b in range(batch)]
    lens, parent = [128] * batch, list(range(batch))
    for bad in (129, -1):
        lens[1], parent[1] = bad, -1
        tb, refs, ln = i32(table, dev), i32([1] * (2 * batch) + [0] * (pool - 2 * batch), dev), i32(lens, dev)
        out, r, n = torch.full_like(tb, -7), torch.empty_like(refs), torch.empty_like(ln)
        kv.fork_sequences(i32(parent, dev), tb, refs, ln, out, r, n)
        assert kv.device_error() == bgtq.DEVERR_SEQ_LEN
        assert n.tolist() == [0 if b == 1 else 128 for b in range(batch)]
        assert torch.equal(r, refs) and out[1].tolist() == [-7, -7] and torch.equal(out[2:], tb[2:])
        parent[1] = 1                                   # forked from by itself: the same
        kv.fork_sequences(i32(parent, dev), tb, refs, ln, out, r, n)
        assert kv.device_error() == bgtq.DEVERR_SEQ_LEN and n[1].item() == 0


@pytest.mark.parametrize("pool", [6, 9000])
def test_resize_to_the_lengths_it_has(dev, pool):
    """One array as the lengths, the new lengths and the lengths granted: nothing changes."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, 3, 128, page_pool_tiles=pool), dev)
    table, refs, lens = i32([[0, 1], [2, -1], [0, -1]], dev), i32([2, 1, 1] + [0] * (pool - 3), dev), i32([100, 7, 64], dev)
    before = [t.clone() for t in (table, refs, lens)]
    kv.resize_sequences(table, refs, lens, lens, lens)
    assert all(torch.equal(a, b) for a, b in zip((table, refs, lens), before)) and kv.device_error() == 0
    with pytest.raises(bgtq.BgtqError) as e:
        kv.resize_sequences(table, refs, table[:, 0].contiguous(), lens, refs[:3])
    assert e.value.status == -1
