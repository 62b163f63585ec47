"""Rotary positions over several axes on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import rope
from packed_decode_attention_b200 import bgtq

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def sections(n_axes):
    return [j * n_axes // 64 for j in range(64)]


def check(x, got, pos, axis, base, pairing):
    """Sines: the angle's fraction in fp32 (2^-25 turns: 2^-22 in the sine), its sine's own rounding (2^-23), two
    products and a difference (2^-23 in all): 2^-21 of |a| + |b|.  The angle in fp64: five roundings of the turns
    here, one of the angle in the oracle, 2^-50 of the angle.  Then the output's rounding."""
    n, heads = x.shape[0], x.shape[1]
    xd, gd, pn = x.double().cpu().numpy(), got.double().cpu().numpy(), pos.cpu().numpy()
    reach = np.abs(pn).max(axis=0) if n else 0
    for h in range(heads):
        want = rope.apply_rope_axes(xd[:, h], pn, axis, base, pairing)
        pair = np.empty_like(want)
        for a, b in rope.block_dims(128, pairing):
            pair[:, a] = pair[:, b] = np.abs(xd[:, h, a]) + np.abs(xd[:, h, b])
        allowed = pair * (2.0 ** -21 + reach[:, None] * 2.0 ** -50)
        allowed = allowed + HALF_STEP[x.dtype] * (np.abs(want) + allowed) + TINY[x.dtype]
        assert np.all(np.abs(gd[:, h] - want) <= allowed), h


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("tokens,hq,hkv,axes,far", [(1, 1, 1, 1, 10), (3, 28, 4, 3, 131072), (17, 7, 1, 2, 2 ** 31 - 1),
                                                    (130, 5, 3, 4, 1 << 20), (2500, 9, 2, 3, 5000), (33, 16, 16, 64, 999)])
def test_matches_oracle(dev, dt, pairing, tokens, hq, hkv, axes, far):
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    q = torch.randn((tokens, hq, 128), generator=g, device=dev).to(dt)
    k = (torch.randn((tokens, hkv, 128), generator=g, device=dev) * 30).to(dt)
    pos = torch.randint(-far, far, (axes, tokens), generator=g, device=dev, dtype=torch.int32)
    axis, base = sections(axes), 1e4 if pairing else 1e6
    qo, ko = bgtq.rope_axes(q, k, pos, axis, base, pairing=pairing)
    check(q, qo, pos, axis, base, pairing)
    check(k, ko, pos, axis, base, pairing)
    # in place, and each alone: the same bits
    q2, k2 = q.clone(), k.clone()
    bgtq.rope_axes(q2, k2, pos, axis, base, q2, k2, pairing=pairing)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(bgtq.rope_axes(q, None, pos, axis, base, pairing=pairing)[0], qo)
    assert torch.equal(bgtq.rope_axes(None, k, pos, axis, base, pairing=pairing)[1], ko)


def test_slices_of_a_projection(dev):
    tokens, hq, hkv = 50, 6, 2
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    qkv = torch.randn((tokens, (hq + 2 * hkv) * 128 + 8), generator=g, device=dev).half()
    q = qkv[:, :hq * 128].view(tokens, hq, 128)
    k = qkv[:, hq * 128:(hq + hkv) * 128].view(tokens, hkv, 128)
    rest = qkv[:, (hq + hkv) * 128:].clone()
    pos = torch.randint(0, 9999, (3, tokens), generator=g, device=dev, dtype=torch.int32)
    want = bgtq.rope_axes(q.contiguous(), k.contiguous(), pos, sections(3), 5e5)
    out = bgtq.rope_axes(q, k, pos, sections(3), 5e5)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    bgtq.rope_axes(q, k, pos, sections(3), 5e5, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, (hq + hkv) * 128:], rest)               # what lies between the rows stays
    # one token of it
    one = bgtq.rope_axes(q[:1], k[:1], pos[:, :1].contiguous(), sections(3), 5e5)
    two = bgtq.rope_axes(q[:2], k[:2], pos[:, :2].contiguous(), sections(3), 5e5)
    assert torch.equal(one[0][0], two[0][0]) and torch.equal(one[1][0], two[1][0])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_zero_positions_and_extremes(dev, dt):
    top = torch.finfo(dt).max
    x = torch.tensor([0.0, top, -top, torch.finfo(dt).tiny, float("inf"), float("nan"), 1.0, -0.0], dtype=dt, device=dev)
    q = x.repeat(16)[None, None].contiguous()
    pos = torch.zeros((2, 1), dtype=torch.int32, device=dev)
    got = bgtq.rope_axes(q, None, pos, sections(2), 1e4)[0]
    keep = torch.isfinite(q) & torch.isfinite(q.roll(64, -1))
    assert torch.equal(got[keep], q[keep])                            # position 0 turns nothing
    # a pair whose turn leaves the type's range becomes infinite, and touches no other pair
    one = torch.ones((1, 1), dtype=torch.int32, device=dev)
    q = torch.ones((1, 1, 128), dtype=dt, device=dev)
    plain = bgtq.rope_axes(q, None, one, [0] * 64, 1e4)[0]
    q[0, 0, 3], q[0, 0, 67] = float("nan"), 1.0
    got = bgtq.rope_axes(q, None, one, [0] * 64, 1e4)[0]
    assert torch.isnan(got[0, 0, [3, 67]]).all()
    rest = [d for d in range(128) if d % 64 != 3]
    assert torch.equal(got[0, 0, rest], plain[0, 0, rest])


def test_no_tokens_and_captured(dev):
    q = torch.empty((0, 4, 128), dtype=torch.float16, device=dev)
    pos = torch.empty((3, 0), dtype=torch.int32, device=dev)
    assert bgtq.rope_axes(q, None, pos, sections(3), 1e4)[0].shape == q.shape
    q, pos = torch.randn((9, 4, 128), device=dev).half(), torch.ones((1, 9), dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        bgtq.rope_axes(q, None, pos, [0] * 64, 1e4, q_out=out)
        pos += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(q, out, pos - 1, [0] * 64, 1e4, 0)
