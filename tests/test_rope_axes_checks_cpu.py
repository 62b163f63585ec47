"""Refusals of bgtq_rope_axes and of the page operations' tensors, before anything is launched (no GPU)."""
import pytest
import torch

from packed_decode_attention_b200 import bgtq
from packed_decode_attention_b200 import build as pkg_build


def status(fn, *a, **kw):
    with pytest.raises(bgtq.BgtqError) as e:
        fn(*a, **kw)
    return e.value.status


@pytest.fixture(autouse=True)
def built(monkeypatch):
    pkg_build.build()
    monkeypatch.setattr(bgtq, "_stream", lambda s: 0)


BASE = dict(n_q_heads=2, n_kv_heads=1, pairing=0, dtype=0, axis=[0] * 64, base=1e4, d_q=1 << 20, q_stride=256,
            d_k=1 << 30, k_stride=128, d_pos=1 << 12, n_axes=1, tokens=10, d_q_out=1 << 24, q_out_stride=256,
            d_k_out=1 << 28, k_out_stride=128)


@pytest.mark.parametrize("change,want", [
    (dict(d_q=None), -2), (dict(d_q_out=None), -2), (dict(d_k=None), -2), (dict(d_k_out=None), -2), (dict(d_pos=None), -2),
    (dict(n_q_heads=-1), -1), (dict(n_q_heads=0, n_kv_heads=0), -1), (dict(n_q_heads=65537, q_stride=1 << 28), -1),
    (dict(pairing=2), -1), (dict(dtype=2), -1), (dict(head_dim=64), -1),
    (dict(base=1.0), -1), (dict(base=float("nan")), -1), (dict(base=float("inf")), -1),
    (dict(n_axes=0), -1), (dict(n_axes=65), -1), (dict(axis=[0] * 63 + [1]), -1), (dict(axis=[0] * 63), -1),
    (dict(axis=[256] + [0] * 63), -1), (dict(axis=[-1] + [0] * 63), -1), (dict(axis=[0.5] + [0] * 63), -1),
    (dict(tokens=-1), -1), (dict(tokens=(1 << 30) + 1), -1),
    (dict(q_stride=255), -1), (dict(q_stride=260), -1), (dict(k_stride=120), -1), (dict(q_out_stride=-256), -1),
    (dict(k_out_stride=(1 << 30) + 8), -1),
    (dict(d_q=(1 << 20) + 8), -8), (dict(d_k_out=(1 << 28) + 2), -8), (dict(d_pos=(1 << 12) + 2), -8),
    (dict(d_q_out=(1 << 20) + 16), -1),                           # overlaps q, not q itself
    (dict(d_q_out=1 << 20, q_out_stride=512), -1),                # q, with another stride
    (dict(d_k_out=(1 << 20) + 256 * 4), -1),                      # overlaps q
    (dict(d_k_out=(1 << 24) + 256 * 2), -1),                      # overlaps q_out
    (dict(d_q_out=(1 << 12) - 256), -1),                          # overlaps pos
    # slices of one buffer whose rows run into one another
    (dict(d_k=(1 << 20) + 2 * 128, k_stride=384, q_stride=384, d_q_out=1 << 20, q_out_stride=384), -1),
])
def test_rope_refusals(change, want):
    assert status(bgtq.bgtq_rope_axes, **{**BASE, **change}) == want


def test_rope_of_no_tokens_launches_nothing():
    bgtq.bgtq_rope_axes(**{**BASE, "tokens": 0})
    # slices of one buffer, in place: accepted up to the launch
    s = dict(d_k=(1 << 20) + 512, k_stride=384, q_stride=384, d_q_out=1 << 20, q_out_stride=384, d_k_out=(1 << 20) + 512,
             k_out_stride=384)
    bgtq.bgtq_rope_axes(**{**BASE, **s, "tokens": 0})


def test_rope_tensors():
    h = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    q, k, pos = h(5, 4, 128), h(5, 2, 128), torch.zeros((3, 5), dtype=torch.int32)
    ax = [0] * 64
    for bad in (dict(q=None, k=None), dict(q=h(5, 4, 64)), dict(q=h(5, 4, 128, dt=torch.float32)), dict(q=h(5, 512)),
                dict(k=k.bfloat16()), dict(k=h(4, 2, 128)), dict(pos=pos.long()), dict(pos=pos[:, :4].contiguous()),
                dict(pos=pos.t()), dict(q_out=h(5, 3, 128)), dict(q_out=q.bfloat16()), dict(k=None, k_out=h(5, 2, 128)),
                dict(q=h(4, 5, 128).transpose(0, 1)), dict(q=h(5, 4, 256)[..., ::2]), dict(axis=[0] * 65)):
        a = dict(q=q, k=k, pos=pos, axis=ax, base=1e4)
        a.update(bad)
        assert status(bgtq.rope_axes, **a) == -1, bad


def test_page_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kv = object.__new__(bgtq.ByteKVCache)
    kv.cfg = bgtq.ByteConfig(n_layers=1, n_kv_heads=1, n_q_heads=1, max_batch=4, capacity_tokens=200, page_pool_tiles=9)
    kv.device, kv.state = torch.device("cpu"), None
    p, t, r, n, t2, r2, n2 = i(4), i(4, 4), i(9), i(4), i(4, 4), i(9), i(4)
    assert status(kv.fork_sequences, p, t, r, n, t2, r2, n2) == -2
    assert status(kv.resize_sequences, t, r, n, n2, n) == -2
    assert status(kv.compact_pages, t, r, n, t, r, r2, i(1)) == -2
    assert status(kv.copy_pages, i(2), i(2)) == -2
    assert kv.copy_pages(i(0), i(0)) is None
    for args in ((p, i(4, 3), r, n, t2, r2, n2), (p, t, i(8), n, t2, r2, n2), (p, t, r, i(3), t2, r2, n2),
                 (p.long(), t, r, n, t2, r2, n2), (p, t, r, n, i(3, 4), r2, n2), (p, t, r, n, t2, r2, i(5)),
                 (p, i(4, 8)[:, ::2], r, n, t2, r2, n2)):
        assert status(kv.fork_sequences, *args) == -1
    assert status(kv.resize_sequences, t, r, n, i(3), n) == -1 and status(kv.copy_pages, i(2), i(3)) == -1
    assert status(kv.compact_pages, t, r, n, t, r, r2, i(2)) == -1
    assert status(kv.compact_pages, t, r, n, t, r, i(4), i(1)) == -1


def test_a_state_is_made_on_the_current_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert bgtq._device("cuda") == torch.device("cuda", 0) == bgtq._device("cuda:0")
    assert bgtq._device("cpu") == torch.device("cpu")
    assert status(bgtq._device, "cuda:1") == -1


def test_numbers_that_do_not_fit():
    assert status(bgtq.bgtq_rope_axes, **{**BASE, "n_q_heads": 1 << 40}) == -1
    assert status(bgtq.bgtq_rope_axes, **{**BASE, "base": "x"}) == -1
    for bad in (dict(window=1.5), dict(window=1 << 40), dict(softcap="x")):
        assert status(bgtq.bgtq_byte_decode_attn, None, 0, 1, 16, 16, 1, 1, 16, **bad) == -1
