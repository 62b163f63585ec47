"""Pins of the 8-bit cache's float64 oracle by hand-worked values, torch's own
e4m3 conversion and closed forms."""
import numpy as np
import pytest
import torch

from oracle import byte_cache as bc


def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mine = bc.e4m3_values()
    assert np.array_equal(np.isnan(codes), np.isnan(mine))
    assert np.array_equal(codes[~np.isnan(codes)], mine[~np.isnan(mine)])
    y = np.concatenate([np.linspace(-448, 448, 20001), np.geomspace(2.0 ** -12, 448, 5000),
                        (mine[:126] + mine[1:127]) / 2])        # ties among them
    got = torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy()
    y = torch.from_numpy(y).float().double().numpy()
    assert np.array_equal(bc.to_grid(y, "e4m3"), got)


def test_special_values():
    y = np.array([np.nan, np.inf, -np.inf, 1e30, 0.5, 1.5, -2.5])
    assert bc.to_grid(y, "int8").tolist() == [0, 127, -127, 127, 0, 2, -2]
    assert bc.to_grid(y[:4], "e4m3").tolist() == [0, 448, -448, 448]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_exponent_is_the_least(code):
    for a in (0.0, 1e-40, 1.0, 127.0, 127.5, 128.0, 448.0, 449.0, 3.3e38):
        e = bc.exponent(a, code)
        assert a <= bc.QMAX[code] * 2.0 ** e
        assert e == bc.E_MIN or a > bc.QMAX[code] * 2.0 ** (e - 1)


def test_a_growing_block_by_hand():
    vals, exps = np.zeros((1, 64, 128)), np.full(1, 7)
    row = np.zeros(128)
    row[:4] = [127.0, 3.0, 1.0, -1.0]
    bc.append(vals, exps, [row], 0, 64, "int8")              # starts the block anew: 2^0
    assert exps[0] == 0 and vals[0, 0, :4].tolist() == [127, 3, 1, -1]
    bc.append(vals, exps, [row * 0.25], 1, 64, "int8")       # smaller rows keep the scale
    assert exps[0] == 0 and vals[0, 1, :4].tolist() == [32, 1, 0, 0]
    bc.append(vals, exps, [row * 2], 2, 64, "int8")          # 254: 2^1, old codes halved, ties to even
    assert exps[0] == 1 and vals[0, 0, :4].tolist() == [64, 2, 0, 0] and vals[0, 2, :4].tolist() == [127, 3, 1, -1]


def test_visible_by_hand():
    see = lambda **k: np.nonzero(bc.visible(8, **k))[0].tolist()  # noqa: E731
    assert see(n_q=1, i=0) == list(range(8))
    assert see(n_q=3, i=0) == [0, 1, 2, 3, 4, 5]
    assert see(n_q=1, i=0, window=3) == [5, 6, 7]
    assert see(n_q=1, i=0, window=3, prefix=2) == [0, 1, 5, 6, 7]
    assert see(n_q=2, i=0, doc_start=6) == [6]
    assert see(n_q=2, i=0, doc_start=7) == []
    assert see(n_q=2, i=0, doc_start=7, prefix=100) == list(range(8))
    assert np.nonzero(bc.visible(1, 3, 0))[0].tolist() == [] and np.nonzero(bc.visible(1, 3, 2))[0].tolist() == [0]


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v, q = rng.normal(size=(9, 128)), rng.normal(size=(9, 128)), rng.normal(size=128)
    every = np.ones(9, dtype=bool)
    o, _, _ = bc.attention_row(np.zeros(128), k, v, every, 8)
    assert np.allclose(o, v.mean(0))
    one = np.zeros(9, dtype=bool)
    one[4] = True
    assert np.allclose(bc.attention_row(q, k, v, one, 8, softcap=5.0, slope=0.3)[0], v[4])
    # a steep bias leaves the nearest position; a tiny cap leaves equal weights
    assert np.allclose(bc.attention_row(q, k, v, every, 8, slope=1e3)[0], v[8])
    assert np.allclose(bc.attention_row(q, k, v, every, 8, softcap=1e-9)[0], v.mean(0))
    assert np.array_equal(bc.attention_row(q, k, v, ~every, 8)[0], np.zeros(128))
