"""The binding around the compiled calls: what needs them."""
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


@pytest.mark.parametrize("pages", [0, 8])
def test_packed_cache_without_the_compiled_calls(dev, monkeypatch, pages):
    """Only the serving operators need _marshal.so; the packed cache is made and used without it."""
    def missing():
        raise RuntimeError("_marshal.so is missing")
    monkeypatch.setattr(bgtq, "marshal", missing)
    kv = bgtq.PackedKVCache(bgtq.Config(1, 1, 2, 1, 200, page_pool_tiles=pages), dev)
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    x = lambda *s: torch.randn(s, generator=g, device=dev).half()  # noqa: E731
    kv.allocate(x(1, 32, 2, 128), x(1, 32, 1, 128))
    if pages:
        kv.set_block_table(i32([[3, 1, 0, 7]], dev))
    k, v = x(1, 1, 130, 1, 128), x(1, 1, 130, 1, 128)
    kv.encode_append(0, k, v, i32([0], dev), i32([130], dev))
    out = torch.zeros((1, 1, 2, 128), dtype=torch.float16, device=dev)
    kv.decode_attn(0, x(1, 1, 2, 128), i32([130], dev), out)
    assert out.any() and torch.isfinite(out).all() and kv.device_error() == 0
    if pages:
        with pytest.raises(RuntimeError, match="_marshal"):
            kv.copy_pages(i32([0], dev), i32([2], dev))
    with pytest.raises(RuntimeError, match="_marshal"):
        bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, 1, 64), dev)
