"""Pins of the oracle's norm, rotary and 8-bit cache definitions against closed
forms, the quantizer oracle and plain loops."""
import numpy as np
import pytest

import oracle
from oracle import layer


def test_norm_of_unit_weights_quantizes_the_normalised_row():
    """With weight 1 the codes are those of the row itself (a common factor
    leaves them), and the scales those of the row over its root mean square."""
    rng = np.random.default_rng(1)
    h = rng.standard_normal((3, 96)).astype(np.float32)
    codes, scale = layer.rmsnorm_codes(h, np.ones(96), 0.0, 32)
    for r in range(3):
        want, s = oracle.quantize_absmax_int8(h[r].reshape(3, 32))
        assert np.array_equal(codes[r].reshape(3, 32), want)
        rms = np.sqrt(np.mean(h[r].astype(np.float64) ** 2))
        assert np.allclose(scale[r], s / rms, rtol=1e-6)


def test_norm_zero_group_and_whole_row_scale():
    h = np.zeros((1, 64), np.float32)
    h[0, 40] = -3.0
    codes, scale = layer.rmsnorm_codes(h, np.full(64, 2.0), 1e-5, 32)
    assert not codes[0, :32].any() and scale[0, 0] == 0
    assert codes[0, 40] == -127 and scale[0, 1] > 0
    codes, scale = layer.rmsnorm_codes(h, np.full(64, 2.0), 0.0, 64)
    assert scale.shape == (1, 1)
    assert np.isclose(codes[0, 40] * scale[0, 0], -3 * 2 / np.sqrt(9 / 64), rtol=1e-6)


def test_rows_quantize_like_the_block_format():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 64)).astype(np.float32)
    x[2, :32] = 0
    codes, d = layer.q8_rows(x)
    raw = oracle.quantize_q8_0(x).reshape(5, 2, 34)
    assert np.array_equal(codes.view(np.uint8).reshape(5, 2, 32), raw[:, :, 2:])
    assert np.array_equal(d.view(np.uint8).reshape(5, 2, 2), raw[:, :, :2])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 16)).astype(np.float32)
    table = layer.rope_table(9, 8, 100.0).astype(np.float32)
    pos = [0, 8, 3, 3]
    y = layer.rotate(x, table, pos, interleaved)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.array_equal(y[0], x[0])   # position 0 turns nothing
    for n in range(4):
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
            z = (x[n, :, a] + 1j * x[n, :, b]) * np.exp(1j * pos[n] * 100.0 ** (-2 * i / 8))
            assert np.allclose(y[n, :, a] + 1j * y[n, :, b], z, atol=1e-6)


def test_scaled_frequencies():
    f = layer.rope_freqs(64, 10000.0)[0]
    assert f[0] == 1 and np.isclose(f[-1], 10000.0 ** (-62 / 64))
    assert np.allclose(layer.rope_freqs(64, 10000.0, {"kind": "linear", "factor": 4.0})[0], f / 4)
    ntk = layer.rope_freqs(64, 10000.0, {"kind": "ntk", "factor": 4.0})[0]
    assert ntk[0] == 1 and np.isclose(ntk[-1], f[-1] / 4)   # the slowest pair is interpolated fully
    y, factor = layer.rope_freqs(64, 10000.0, {"kind": "yarn", "factor": 4.0, "original_len": 4096, "low": 1, "high": 32})
    assert np.allclose(y[:5], f[:5]) and np.allclose(y[-3:], f[-3:] / 4) and np.isclose(factor, 0.1 * np.log(4) + 1)
    g = layer.rope_freqs(64, 500000.0, {"kind": "llama3", "factor": 8.0, "original_len": 8192, "low": 1, "high": 4})[0]
    f = layer.rope_freqs(64, 500000.0)[0]
    assert np.allclose(g[:3], f[:3]) and np.allclose(g[-3:], f[-3:] / 8)
    assert np.all(g <= f) and np.all(g >= f / 8)


def test_attention_rows_match_the_single_token_oracle():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    sees = np.ones((2, 9), bool)
    sees[0, 5:] = False
    out, vmax, smax = layer.attention_rows(q, k, v, sees, 0.5)
    assert np.allclose(out[0], oracle.attention_decode(q[0], k[:, :5], v[:, :5], 0.5), atol=1e-13)
    assert np.allclose(out[1], oracle.attention_decode(q[1], k, v, 0.5), atol=1e-13)
    assert vmax == np.abs(v).max() and smax > 0
    far, _, _ = layer.attention_rows(q, k, v, sees, 0.5, cap=1e6)
    assert np.allclose(far, out, atol=1e-9)   # a cap far above the scores changes nothing
    none, _, _ = layer.attention_rows(q, k, v, np.zeros((2, 9), bool), 0.5)
    assert not none.any()
    flat, _, _ = layer.attention_rows(q * 1e9, k, v, sees, 0.5, cap=1e-9)
    assert np.allclose(flat[1, 0], v[0].mean(0), atol=1e-7)   # a cap of nothing: the mean


def off_by_a_tie(values, a, b):
    """The codes a and b of rows `values` [n, 32] (of up to 24 bits each) differ by one, upwards from the half that both lie
    beside, in exact arithmetic; how many."""
    at = np.argwhere(a != b)
    for r, i in at:
        v, top = int(values[r, i] * 2.0 ** 40), int(np.abs(values[r]).max() * 2.0 ** 40)
        assert v * 2.0 ** -40 == values[r, i] and top * 2.0 ** -40 == np.abs(values[r]).max()
        lower = min(int(a[r, i]), int(b[r, i]))
        assert abs(int(a[r, i]) - int(b[r, i])) == 1 and 2 * 127 * v == (2 * lower + 1) * top
    return len(at)


def test_the_two_factors_differ_at_exact_halves_only():
    """The cache's factor 127 * (1 / absmax) and the quantizers' 127 / absmax give one block other codes only where a value is
    an exact half of a step; the scales are the same."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((20000, 32)).astype(np.float32)
    x = np.where(np.abs(x) < 2.0 ** -10, np.float32(0.5), x)   # whole multiples of 2^-40, for exact arithmetic
    coarse = (x.view(np.uint32) & 0xffff0000).view(np.float32)   # bf16 values
    for values, ties in ((coarse, True), (x, False)):
        codes, scale = layer.q8_rows(values)
        want, s = oracle.quantize_absmax_int8(values)
        assert np.array_equal(scale[:, 0], s.astype(np.float16))
        assert (off_by_a_tie(values.astype(np.float64), codes, want) > 0) == ties
