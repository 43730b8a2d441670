"""Pins of the layer operators' oracle."""

import math

import numpy as np
import pytest

from oracle import layer as oy
from oracle import lmhead as ol


def test_attention_matches_plain_loops():
    rng = np.random.default_rng(1)
    P, L, Q, Hq, Hkv, D = 5, 3, 4, 4, 2, 6
    q = rng.standard_normal((Q, Hq, D))
    pk, pv = rng.standard_normal((2, P, Hkv, D))
    k, v = rng.standard_normal((2, L + Q - 1, Hkv, D))
    out, lse, weight, spread = oy.prefix_attention(q, pk, pv, k, v, L, 0.3)
    for i in range(Q):
        for h in range(Hq):
            keys = [(pk[j, h // 2], pv[j, h // 2]) for j in range(P)]
            keys += [(k[j, h // 2], v[j, h // 2]) for j in range(L + i)]
            e = [math.exp(0.3 * math.fsum(q[i, h] * kk)) for kk, _ in keys]
            assert math.isclose(lse[i, h], math.log(math.fsum(e)), rel_tol=1e-12)
            for d in range(D):
                ref = math.fsum(p * vv[d] for p, (_, vv) in zip(e, keys)) / math.fsum(e)
                assert math.isclose(out[i, h, d], ref, rel_tol=1e-10, abs_tol=1e-12)
            assert (np.abs(out[i, h]) <= weight[i, h] + 1e-15).all() and spread[i, h] > 0


def test_attention_single_equal_and_no_key():
    D = 4
    q = np.arange(2 * D, dtype=float).reshape(2, 1, D)
    none = np.zeros((0, 1, D))
    v = np.array([[[1.0, 2, 3, 4]], [[5.0, 6, 7, 8]]])
    # position 0 sees nothing, position 1 one key: its value, whatever the score
    out, lse, _, _ = oy.prefix_attention(q, none, none, np.ones((1, 1, D)), v[:1], 0, 0.5)
    assert (out[0] == 0).all() and lse[0, 0] == -math.inf
    np.testing.assert_allclose(out[1, 0], v[0, 0])
    # two equal keys: the mean of their values
    out, _, _, _ = oy.prefix_attention(q[:1], np.ones((2, 1, D)), v, none, none, 0, 0.5)
    np.testing.assert_allclose(out[0, 0], v[:, 0].mean(0))


def test_sequence_flags():
    ok = dict(k=2, K=3, length=5, max_pages=4, page_size=2, table_row=[0, 1, 2, 3],
              prefix_pages=[7], num_pages=8)
    assert oy.sequence_flags(**ok) == 0
    assert oy.sequence_flags(**{**ok, "k": 4}) == oy.FLAG_BAD_K
    assert oy.sequence_flags(**{**ok, "k": -1}) == oy.FLAG_BAD_K
    assert oy.sequence_flags(**{**ok, "length": 7}) == oy.FLAG_BAD_N
    assert oy.sequence_flags(**{**ok, "length": -1}) == oy.FLAG_BAD_N
    assert oy.sequence_flags(**{**ok, "table_row": [0, 1, 2, -1]}) == oy.FLAG_BAD_PAGE
    assert oy.sequence_flags(**{**ok, "table_row": [0, 1, 2, -1], "length": 4}) == 0
    assert oy.sequence_flags(**{**ok, "prefix_pages": [8]}) == oy.FLAG_BAD_PAGE


def test_norm_matches_the_final_norm():
    rng = np.random.default_rng(2)
    x, r, w = rng.standard_normal((3, 40)), rng.standard_normal((3, 40)), rng.standard_normal(40)
    s, y = oy.rmsnorm_residual(x, r, w, 1e-5)
    np.testing.assert_array_equal(s, x + r)
    np.testing.assert_allclose(y, ol.rmsnorm(x + r, w, 1e-5))
    c = oy.row_scale(y)
    np.testing.assert_allclose(np.abs(y / c[:, None]).max(1), 448.0)
    assert oy.row_scale(np.zeros((1, 4)))[0] == 2.0 ** -126


def test_e4m3_values_are_torchs():
    torch = pytest.importorskip("torch")
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    want = np.unique(np.abs(every[np.isfinite(every)]))
    np.testing.assert_array_equal(oy.e4m3_values(), want)


def test_linear_matches_triple_loop_and_activations():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    x, W = rng.standard_normal((3, 7)), rng.standard_normal((5, 7))
    sx, sw, bias, res = (rng.standard_normal(n) for n in (3, 5, 5, 15))
    res = res.reshape(3, 5)
    F = torch.nn.functional
    acts = [lambda z: z, F.relu, F.silu, F.gelu, lambda z: F.gelu(z, approximate="tanh")]
    for act in range(5):
        out, absp = oy.linear(x, W, sx, sw, bias, act, res)
        for m in range(3):
            for n in range(5):
                z = sx[m] * sw[n] * math.fsum(x[m] * W[n]) + bias[n]
                ref = float(acts[act](torch.tensor(z, dtype=torch.float64))) + res[m, n]
                assert math.isclose(out[m, n], ref, rel_tol=1e-12, abs_tol=1e-13)
                assert math.isclose(absp[m, n], abs(sx[m] * sw[n]) * math.fsum(np.abs(x[m] * W[n])))
