"""CPU checks of the 8-bit cache: sizes, refused configs, and tensors refused before a pointer reaches the library."""
import pytest
import torch

from packed_decode_attention_b200 import bgtq
from packed_decode_attention_b200 import build as pkg_build

ERR_INVALID_ARG, ERR_NULL = -1, -2


def status(fn, *args, **kw):
    with pytest.raises(bgtq.BgtqError) as e:
        fn(*args, **kw)
    return e.value.status


@pytest.fixture()
def kv(monkeypatch):
    pkg_build.build()
    monkeypatch.setattr(bgtq, "_stream", lambda s: 0)
    obj = object.__new__(bgtq.ByteKVCache)
    obj.cfg = bgtq.ByteConfig(n_layers=3, n_kv_heads=2, n_q_heads=8, max_batch=4, capacity_tokens=300, max_q_tokens=2)
    obj.device = torch.device("cpu")
    obj.state = None
    return obj


def test_required_bytes_and_refused_configs():
    pkg_build.build()
    base = dict(n_layers=28, n_kv_heads=4, n_q_heads=28, max_batch=16, capacity_tokens=32768)
    cache, ws = bgtq.bgtq_byte_required_bytes(bgtq.ByteConfig(**base))
    blocks = 28 * 4 * 16 * 512
    assert blocks * (2 * 8192 + 8) <= cache < blocks * (2 * 8192 + 8) + 4 * 256
    paged, ws_p = bgtq.bgtq_byte_required_bytes(bgtq.ByteConfig(**base, page_pool_tiles=100))
    assert 28 * 4 * 100 * (2 * 8192 + 8) <= paged < 28 * 4 * 100 * (2 * 8192 + 8) + 4 * 256 and ws_p == ws
    for change in (dict(head_dim=64), dict(n_q_heads=30), dict(n_q_heads=68), dict(max_batch=0), dict(n_layers=0),
                   dict(n_layers=65536), dict(capacity_tokens=0), dict(capacity_tokens=(1 << 30) + 1),
                   dict(max_q_tokens=0), dict(max_q_tokens=17), dict(page_pool_tiles=-1), dict(code="e5m2"),
                   dict(rows="fp32"), dict(max_batch=1 << 20, capacity_tokens=1 << 30)):
        assert status(bgtq.bgtq_byte_required_bytes, bgtq.ByteConfig(**{**base, **change})) == ERR_INVALID_ARG, change


def test_tensors_are_checked(kv):
    h = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k, q, out, sl = h(1, 4, 5, 2, 128), h(1, 4, 2, 8, 128), h(1, 4, 2, 8, 128), i(4)
    assert status(kv.append, 0, k, k, sl, sl) == ERR_NULL
    assert status(kv.decode_attn, 0, q, sl, out, slopes=h(8, dt=torch.float32), prefix=sl, doc_start=i(4, 2)) == ERR_NULL
    for bad in (dict(k=h(1, 4, 5, 3, 128)), dict(k=k.bfloat16()), dict(v=h(1, 4, 4, 2, 128)), dict(start=i(3)),
                dict(count=sl.long()), dict(k=h(2, 4, 5, 2, 128)),
                dict(k=h(1, 4, 5, 128, 2).transpose(3, 4), v=h(1, 4, 5, 2, 128))):
        a = dict(k=k, v=k, start=sl, count=sl)
        a.update(bad)
        assert status(kv.append, 0, a["k"], a["v"], a["start"], a["count"]) == ERR_INVALID_ARG, bad
    for bad in (dict(q=h(1, 4, 8, 128)), dict(q=q.bfloat16()), dict(out=h(1, 4, 1, 8, 128)), dict(seq_lens=i(5)),
                dict(slopes=h(8)), dict(slopes=h(7, dt=torch.float32)), dict(prefix=i(3)), dict(doc_start=i(4)),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        a = dict(q=q, seq_lens=sl, out=out)
        a.update(bad)
        assert status(kv.decode_attn, 0, **a) == ERR_INVALID_ARG, bad
