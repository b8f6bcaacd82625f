"""Pins of the paged cache's oracle: formats, nearest codes, growth, masks and
eviction against closed forms and brute force (no GPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.paged_oracle as po


def _cache(pages, H, D, fmt, pos=True, weight=True):
    return {"k": np.full((pages, H, 64, D), 0x7F, np.uint8), "v": np.full((pages, H, 64, D), 0x7F, np.uint8),
            "k_scale": np.full((pages, H), np.nan, np.float32), "v_scale": np.full((pages, H), np.nan, np.float32),
            "pos": np.full((pages, H, 64), -7, np.int32) if pos else None,
            "weight": np.full((pages, H, 64), 9.0, np.float32) if weight else None, "fmt": fmt}


def test_e4m3_table_and_rounding_match_torch():
    raw = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(raw).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(po.code_values(raw, "e4m3"), t, equal_nan=True)
    g = np.random.default_rng(0)
    x = np.concatenate([g.normal(size=4000) * 2.0 ** g.integers(-12, 9, 4000), po._E4M3_POS[:-1] / 2 + po._E4M3_POS[1:] / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(po.encode(x, "e4m3"), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_the_nearest_of_the_real_quotient(fmt):
    g = np.random.default_rng(1)
    vals = po.code_values(np.arange(256, dtype=np.uint8), fmt)
    vals = [v for v in vals if np.isfinite(v) and (fmt == "e4m3" or v != -128)]
    for _ in range(40):
        x = (g.normal(size=16) * 10.0 ** g.integers(-6, 6)).astype(np.float32)
        s = po.fresh_scale(np.abs(x).max(), fmt)
        codes = po.code_values(po.quotient_codes(x, s, fmt), fmt)
        for xi, ci in zip(x, codes):
            q = Fraction(float(xi)) / Fraction(float(s))
            best = min(abs(Fraction(v) - q) for v in vals)
            assert abs(Fraction(float(ci)) - q) == best


def test_scales_at_their_borders():
    assert po.fresh_scale(np.float32(127), "int8") == 1.0
    assert po.fresh_scale(np.float32(1e-45), "int8") == np.float32(2.0 ** -126)
    assert po.fresh_scale(np.float32(448), "e4m3") == 1.0
    assert po.fresh_scale(np.nextafter(np.float32(448), np.float32(1e9)), "e4m3") == 2.0
    assert po.grown(1.0, np.float32(127.5), "int8") == (2.0, 1)
    assert po.grown(1.0, np.nextafter(np.float32(127.5), np.float32(0)), "int8") == (1.0, 0)
    assert po.grown(1.0, np.float32(448), "e4m3") == (1.0, 0)
    assert po.grown(0.5, np.float32(1000), "e4m3") == (4.0, 3)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_page_filled_token_by_token_is_within_one_step(fmt):
    g = np.random.default_rng(2)
    x = (g.normal(size=(1, 1, 64, 64)) * np.exp(np.linspace(-3, 3, 64))[None, None, :, None]).astype(np.float32)
    c = _cache(1, 1, 64, fmt)
    for t in range(64):
        po.append(c, [[0]], [t], [1], x[:, :, t:t + 1], x[:, :, t:t + 1])
    k, _ = po.read(c, [[0]], 0, 0, 0, 64)
    if fmt == "int8":
        bound = c["k_scale"][0, 0] * np.ones_like(k)
    else:  # half a step of the value's own binade, and the subnormal steps of the growing scales
        bound = np.abs(x[0, 0]) * 2.0 ** -4 + c["k_scale"][0, 0] * 2.0 ** -9
    assert (np.abs(k - x[0, 0]) <= bound * (1 + 1e-6)).all()
    assert np.array_equal(c["pos"][0, 0], np.arange(64)) and (c["weight"] == 0).all()


def test_attention_closed_forms_and_masks():
    c = _cache(2, 1, 64, "int8", pos=False)
    g = np.random.default_rng(3)
    x = g.normal(size=(1, 1, 70, 64)).astype(np.float32)
    po.append(c, [[0, 1]], [0], [70], x, x)
    v = po.read(c, [[0, 1]], 0, 0, 0, 70)[1].astype(np.float64)
    q = np.zeros((3, 64))
    z, _ = po.scores(c, [[0, 1]], 0, 0, 0, 70, q, 0.125, q_len=3, causal=True)
    out, lse, w = po.attention(z, v)
    for i in range(3):  # zero queries: the mean of what is seen
        assert np.allclose(out[i], v[:68 + i].mean(0)) and np.isclose(lse[i], np.log(68 + i))
    assert np.allclose(w.sum(1), 1)
    z, _ = po.scores(c, [[0, 1]], 0, 0, 0, 70, q, 0.125, q_len=3, causal=True, first=[69, 70, 0])
    out, lse, _ = po.attention(z, v)
    assert lse[0] == -np.inf and (out[0] == 0).all() and lse[1] == -np.inf and np.isclose(lse[2], np.log(70))
    z, _ = po.scores(c, [[0, 1]], 0, 0, 0, 5, np.zeros((5, 64)), 0.125, q_len=5, causal=True, prefix=3)
    assert (np.isfinite(z).sum(1) == [3, 3, 3, 4, 5]).all()
    z, _ = po.scores(c, [[0, 1]], 0, 0, 0, 2, q[:1], 0.125, q_len=1, slope=0.5, q_pos=10)
    assert np.allclose(z, [[-5.0, -4.5]])
    q = g.normal(size=(1, 64)) * 100
    z, _ = po.scores(c, [[0, 1]], 0, 0, 0, 70, q, 1.0, q_len=1, cap=5.0)
    assert np.abs(z).max() <= 5.0


def test_eviction_order():
    w = np.array([5, 1, np.nan, 3, 3, 3, -0.0, 0.0, 2, 7], np.float32)
    assert po.keep_slots(w, 10, 10, 0, 0) == list(range(10))
    assert po.keep_slots(w, 10, 5, 1, 1) == [0, 3, 4, 5, 9]
    assert po.keep_slots(w, 10, 4, 1, 1) == [0, 3, 4, 9]
    assert po.keep_slots(w, 10, 9, 0, 0) == [0, 1, 3, 4, 5, 6, 7, 8, 9]
    assert po.keep_slots(w, 10, 2, 1, 1) == [0, 9]
    assert po.keep_slots(w, 10, 4, 0, 2) == [0, 3, 8, 9]


@pytest.mark.parametrize("mistake", ["floor", "levels", "no_ties", "causal", "recent"])
def test_planted_mistakes_are_seen(mistake, monkeypatch):
    """Each mistake in the oracle makes one of the pins above fail."""
    if mistake == "floor":
        monkeypatch.setattr(po, "encode", lambda x, fmt: np.clip(np.floor(x), -127, 127).astype(np.int8).view(np.uint8))
        with pytest.raises(AssertionError):
            test_codes_are_the_nearest_of_the_real_quotient("int8")
    elif mistake == "levels":
        monkeypatch.setattr(po, "fresh_scale", lambda a, fmt: np.float32(a) / np.float32(128))
        with pytest.raises(AssertionError):
            test_scales_at_their_borders()
    elif mistake == "no_ties":
        monkeypatch.setattr(po, "keep_slots", lambda w, n, keep, s, r: sorted(
            sorted(range(n), key=lambda j: (-np.nan_to_num(w[j]), -j))[:keep]))
        with pytest.raises(AssertionError):
            test_eviction_order()
    elif mistake == "causal":
        real = po.scores
        monkeypatch.setattr(po, "scores", lambda *a, **kw: real(*a, **{**kw, "causal": False}))
        with pytest.raises(AssertionError):
            test_attention_closed_forms_and_masks()
    else:
        real_keep = po.keep_slots
        monkeypatch.setattr(po, "keep_slots", lambda w, n, keep, s, r: real_keep(w, n, keep, s, 0))
        with pytest.raises(AssertionError):
            test_eviction_order()


def test_a_large_cap_is_close_to_none():
    c = _cache(1, 1, 64, "int8", pos=False)
    x = np.random.default_rng(4).normal(size=(1, 1, 60, 64)).astype(np.float32)
    po.append(c, [[0]], [0], [60], x, x)
    q = np.random.default_rng(5).normal(size=(2, 64))
    z0, e0 = po.scores(c, [[0]], 0, 0, 0, 60, q, 0.125, q_len=2)
    z1, e1 = po.scores(c, [[0]], 0, 0, 0, 60, q, 0.125, q_len=2, cap=1e6)
    assert np.abs(z1 - z0).max() <= 1e-9 and (e1 - e0 <= np.abs(z0) * 2.0 ** -18).all()
