"""Pins of the oracle's definitions of what ends a decode step against closed forms, the
quantizer oracle and torch's own functions in f64."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import answer


def test_values_of_blocks():
    """Q1_0 and q8_0 values are those that the products' oracle multiplies."""
    rows, K, n = 5, 384, 2
    w, a = wl.q1_weights_aos(rows, K, 1), wl.q8_acts_aos(K, 2, n)
    t, off = answer.product(answer.q1_values(w), answer.q8_values(a, n), None, 0)
    y = np.asarray(oracle.q1_q8_gemv_aos(w, a, rows, K, n)).reshape(n, rows)
    assert (np.abs(y - t) <= off).all() and (off < 1e-2 * np.abs(t).max()).all()
    d = np.zeros((1, 1, 18), np.uint8)
    d[0, 0, :2] = np.array([0.5], np.float16).view(np.uint8)
    d[0, 0, 2] = 0b101
    assert list(answer.q1_values(d)[0, :4]) == [0.5, -0.5, 0.5, -0.5]


@pytest.mark.parametrize("code", range(6))
def test_activations(code):
    torch = pytest.importorskip("torch")
    F = torch.nn.functional
    t = np.linspace(-30, 30, 4001)
    x = torch.from_numpy(t)
    want = [x, F.relu(x), F.relu(x) ** 2, F.gelu(x), F.gelu(x, approximate="tanh"), F.silu(x)][code].numpy()
    assert np.allclose(answer.act(t, code), want, rtol=1e-12, atol=1e-12)
    slope = np.abs(np.diff(want) / np.diff(t))
    assert (slope <= answer.act_slope(t[1:], t[1] - t[0], code) + 1e-9).all()


@pytest.mark.parametrize("scale,cap", [(1.0, 0.0), (0.5, 0.0), (2.0, 15.0)])
def test_logprobs(scale, cap):
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(3).standard_normal(200).astype(np.float32) * 8
    x[7] = -np.inf
    z = torch.from_numpy(x.astype(np.float64))
    z = scale * (cap * torch.tanh(z / cap) if cap else z)
    z[7] = -float("inf")
    want = torch.log_softmax(z, 0).numpy()
    tokens = np.array([0, 7, 199, -1, 200])
    lp, entropy, ids, tops = answer.logprobs(x, tokens, 9, scale, cap)
    assert np.allclose(lp, [want[0], -np.inf, want[199], 0, 0])
    assert np.isclose(entropy, -np.nansum(np.exp(want) * np.where(np.isfinite(want), want, 0)))
    assert list(ids) == list(np.argsort(-x, kind="stable")[:9]) and np.allclose(tops, want[ids])


def test_logprobs_of_rows_with_little_left():
    inf = np.inf
    lp, entropy, ids, tops = answer.logprobs(np.array([-inf, -inf]), np.array([1, -1]), 3)
    assert list(lp) == [-inf, 0] and entropy == 0 and list(ids) == [-1] * 3 and list(tops) == [-inf] * 3
    lp, entropy, ids, tops = answer.logprobs(np.array([-inf, 2.0, 2.0]), np.array([1]), 3)
    assert np.isclose(lp[0], -np.log(2)) and np.isclose(entropy, np.log(2)) and list(ids) == [1, 2, -1]
    for bad in (np.nan, inf):
        lp, entropy, ids, tops = answer.logprobs(np.array([bad, 1.0]), np.array([1, -1]), 1)
        assert np.isnan(lp[0]) and lp[1] == 0 and np.isnan(entropy) and ids[0] == -1 and np.isnan(tops[0])


def test_tokens_outside_the_vocabulary_are_padding():
    """Of rows that hold a NaN or an infinity too."""
    for x in ([1.0, 2.0], [np.nan, 2.0], [np.inf, 2.0], [-np.inf, -np.inf]):
        lp = answer.logprobs(np.array(x), np.array([-1, 2, 7]), 1)[0]
        assert list(lp) == [0, 0, 0]
