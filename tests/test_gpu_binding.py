"""The binding around the compiled calls: what needs them, and what other threads do meanwhile."""
import threading
import time

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


def operators(dev):
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(1, 1, 1, 1, 128, page_pool_tiles=4), dev)
    kv.set_block_table(i32([[0, 1]], dev))
    k, q = torch.ones((1, 1, 1, 1, 128), device=dev).half(), torch.ones((1, 1, 1, 1, 128), device=dev).half()
    n, one, out = i32([3], dev), i32([1], dev), torch.empty_like(q)
    table, refs, table_out, refs_out, lens_out = i32([[0, 1]], dev), i32([1, 1, 0, 0], dev), i32([[0, 0]], dev), i32([0] * 4, dev), i32([0], dev)
    page_map, live, zero = i32([0] * 4, dev), i32([0], dev), i32([0], dev)
    src, dst = i32([0], dev), i32([2], dev)
    rows, pos = torch.ones((1, 1, 128), device=dev).half(), i32([[3]], dev)
    rows_out = torch.empty_like(rows)
    return kv, {
        "append": lambda: kv.append(0, k, k, n, one),
        "decode_attn": lambda: kv.decode_attn(0, q, n, out),
        "copy_pages": lambda: kv.copy_pages(src, dst),
        "fork_sequences": lambda: kv.fork_sequences(zero, table, refs, n, table_out, refs_out, lens_out),
        "resize_sequences": lambda: kv.resize_sequences(table, refs, n, n, lens_out),
        "compact_pages": lambda: kv.compact_pages(table, refs, n, table_out, refs_out, page_map, live),
        "rope_axes": lambda: bgtq.rope_axes(rows, None, pos, [0] * 64, 1e4, rows_out),
    }


@pytest.mark.parametrize("name", ["append", "decode_attn", "copy_pages", "fork_sequences", "resize_sequences",
                                  "compact_pages", "rope_axes"])
def test_other_threads_run_while_a_launch_waits(dev, name):
    """Behind a second of other work the launch queue fills and a call waits for a place in it: meanwhile another
    Python thread goes on."""
    kv, todo = operators(dev)
    todo[name]()
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    torch.cuda._sleep(2_000_000_000)                    # cycles: about a second
    t0 = time.perf_counter()
    try:
        for _ in range(3000):
            todo[name]()
    finally:
        stop.set()
        other.join()
    waited = time.perf_counter() - t0
    torch.cuda.synchronize()
    assert waited > 0.5, "the queue never filled"
    assert max(gaps) < 0.25, max(gaps)
    assert kv.device_error() == 0
