"""The compiled checks in front of the serving operators: they make the calls, and refuse what the Python checks refuse,
with the same errors."""
import pytest
import torch

from packed_decode_attention_b200 import bgtq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device="cuda")


def calls(dev, rt):
    """Each method with good arguments by name."""
    kv = bgtq.ByteKVCache(bgtq.ByteConfig(n_layers=2, n_kv_heads=2, n_q_heads=4, max_batch=3, capacity_tokens=200,
                                          rows=rt, max_q_tokens=2, page_pool_tiles=20), "cuda")
    packed = bgtq.PackedKVCache(bgtq.Config(n_layers=1, n_kv_heads=1, n_q_heads=1, max_batch=3, capacity_tokens=200,
                                            page_pool_tiles=20), "cuda")
    kv.set_block_table(torch.arange(12, dtype=torch.int32, device=dev).view(3, 4))
    h = lambda *s: torch.randn(s, device=dev).to(kv.row_dtype)  # noqa: E731
    k, q = h(2, 3, 5, 2, 128), h(2, 3, 2, 4, 128)
    qr, kr = h(7, 4, 128), h(7, 2, 128)
    attn = dict(layer=0, q=q, seq_lens=i32(3) + 5, out=h(2, 3, 2, 4, 128), layer_count=2, scale=0.1, softcap=20.0,
                slopes=torch.ones(4, device=dev), window=3, prefix=i32(3) + 1, doc_start=i32(3, 2))
    fork = dict(parent=i32(3), table=i32(3, 4), refs=i32(20), lens=i32(3), table_out=i32(3, 4), refs_out=i32(20),
                lens_out=i32(3))
    resize = dict(table=i32(3, 4), refs=i32(20), lens=i32(3), new_lens=i32(3) + 70, lens_out=i32(3))
    compact = dict(table=i32(3, 4), refs=i32(20), lens=i32(3), table_out=i32(3, 4), refs_out=i32(20), page_map=i32(20),
                   n_live=i32(1))
    return kv, [(kv.append, dict(layer=0, k=k, v=k, start=i32(3), count=i32(3) + 5, layer_count=2)),
                (kv.decode_attn, attn), (kv.decode_attn, {n: attn[n] for n in ("layer", "q", "seq_lens", "out", "layer_count")}),
                (kv.copy_pages, dict(src=i32(2) + 1, dst=torch.arange(5, 7, dtype=torch.int32, device=dev))),
                (kv.copy_pages, dict(src=i32(0), dst=i32(0))),
                (kv.fork_sequences, fork), (kv.resize_sequences, resize), (kv.compact_pages, compact),
                (packed.fork_sequences, fork), (packed.resize_sequences, {**resize, "refs": i32(20), "table": i32(3, 4)}),
                (bgtq.rope_axes, dict(q=qr, k=kr, pos=i32(3, 7), axis=[0] * 64, base=1e4, q_out=torch.empty_like(qr),
                                      k_out=torch.empty_like(kr), pairing=1)),
                (bgtq.rope_axes, dict(q=None, k=kr, pos=i32(1, 7), axis=(0,) * 64, base=10000, k_out=torch.empty_like(kr)))]


def outputs(kv, kw):
    return [kv.cache] + [t for t in kw.values() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("rt", ["fp16", "bf16"])
def test_compiled_calls_do_what_the_python_ones_do(dev, rt, monkeypatch):
    def run(compiled):
        torch.manual_seed(0)
        kv, todo = calls(dev, rt)
        kv.cache.zero_()
        got = []
        with monkeypatch.context() as m:
            if compiled:
                def no(*a, **k):
                    raise AssertionError("not compiled")
                for n in ("bgtq_byte_append", "bgtq_byte_decode_attn", "bgtq_copy_pages", "bgtq_fork_sequences",
                          "bgtq_resize_sequences", "bgtq_compact_pages", "bgtq_rope_axes"):
                    m.setattr(bgtq, n, no)
            else:
                class Python:
                    def __getattr__(self, name):
                        return lambda *a: None
                m.setattr(bgtq, "marshal", Python)
                kv._ctx = None
                todo[-1][0], todo[-4][0].__self__.__setattr__("_ctx", None), todo[-3][0].__self__.__setattr__("_ctx", None)
            for fn, kw in todo:
                fn(**kw)
                torch.cuda.synchronize()
                got.append([t.clone() for t in outputs(kv, kw)])
        assert kv.device_error() == 0
        return got

    for a, b in zip(run(True), run(False)):
        assert len(a) == len(b)
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_refusals_are_the_python_ones(dev):
    _, todo = calls(dev, "fp16")
    for fn, kw in todo:
        for name, t in kw.items():
            if not isinstance(t, torch.Tensor):
                continue
            bad = [None, 5, t.cpu(), t.double(), t[None], torch.zeros((3,) + tuple(t.shape), dtype=t.dtype, device=dev)]
            if t.dim() > 1 and t.shape[0] > 1 and fn is not bgtq.rope_axes:
                bad.append(torch.zeros(tuple(t.shape[::-1]), dtype=t.dtype, device=dev).permute(*range(t.dim())[::-1]))
            for x in bad:
                if x is None and (name in ("slopes", "prefix", "doc_start") or (fn is bgtq.rope_axes and name.endswith("_out"))):
                    continue
                if isinstance(x, torch.Tensor) and x.is_contiguous() and x.shape == t.shape and x.dtype == t.dtype and x.is_cuda:
                    continue
                with pytest.raises(bgtq.BgtqError) as e:
                    fn(**{**kw, name: x})
                assert e.value.status in (-1, -2), (fn, name, x)
    kv = todo[0][0].__self__
    with pytest.raises(bgtq.BgtqError) as e:
        kv.append(2, *(todo[0][1][n] for n in ("k", "v", "start", "count")), layer_count=2)
    assert e.value.status == -1
    kv.close()
    with pytest.raises(bgtq.BgtqError) as e:
        kv.append(**todo[0][1])
    assert e.value.status == -2
