"""Pins of the 8-bit path's float64 definitions (oracle/dsmoe_q8.py) to things other than
themselves: torch's e4m3 and e8m0 types, brute force over the format, central differences."""
import numpy as np
import pytest
import torch

from oracle import dsmoe_q8 as Q


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(Q.e4m3_values(), nan=1e9))
    s = torch.arange(1, 256, dtype=torch.uint8)  # byte 0 is a subnormal power that no block gets
    np.testing.assert_array_equal(np.nan_to_num(s.view(torch.float8_e8m0fnu).double().numpy(), nan=1e9),
                                  np.nan_to_num(Q.decode_scale(s.numpy()), nan=1e9))


def test_e4m3_rounding_is_nearest_even():
    """Every midpoint of two neighbours, the values beside it, and random ones, against torch's
    conversion and against the nearest value by brute force."""
    v = Q.e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 1e9), np.nextafter(mid, 0),
                        np.random.default_rng(0).uniform(-448, 448, 2000)])
    x = np.concatenate([x, -x])
    x32 = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x32).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(Q.decode_e4m3(Q.encode_e4m3(x32)), want)
    best = np.abs(x[:, None] - np.concatenate([v, -v])[None, :]).min(axis=1)
    np.testing.assert_array_equal(np.abs(Q.decode_e4m3(Q.encode_e4m3(x)) - x), best)


def test_scale_is_the_smallest_power():
    rng = np.random.default_rng(1)
    a = np.abs(rng.standard_normal(500)) * 10.0 ** rng.uniform(-30, 30, 500)
    a = np.concatenate([a, 448.0 * 2.0 ** np.arange(-20, 20), np.nextafter(448.0 * 2.0 ** np.arange(-20, 20), 1e30)])
    s = Q.decode_scale(Q.scale_byte(a))
    assert (a <= 448 * s).all() and (a > 448 * s / 2).all()
    assert list(Q.scale_byte([0.0, 1e-45, 448 * 2.0 ** -126, np.inf, np.nan])) == [1, 1, 1, 255, 255]


@pytest.mark.parametrize("C", [16, 128, 144, 512, 528, 704])
def test_rows_round_trip(C):
    """Each value within half a step of e4m3: 2^-4 of itself, or half the smallest step of its block."""
    rng = np.random.default_rng(C)
    x = Q.round_bf16(rng.standard_normal((9, C)) * 10.0 ** rng.uniform(-5, 5, (9, 1)))
    x[3] = 0
    q, s = Q.quantize_rows(x)
    assert s.shape == (9, Q.scale_cols(C)) and (s[:, -(-C // 128):] == 127).all()
    step = np.repeat(Q.decode_scale(s)[:, :-(-C // 128)], 128, axis=1)[:, :C]
    assert (np.abs(Q.dequantize_rows(q, s) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()
    assert (Q.dequantize_rows(q, s)[3] == 0).all()


def test_a_block_with_an_infinity_or_nan_is_nan():
    x = np.ones((3, 256))
    x[0, 5], x[1, 200] = np.inf, np.nan
    q, s = Q.quantize_rows(x)
    d = Q.dequantize_rows(q, s)
    assert np.isnan(d[0, :128]).all() and (d[0, 128:] == 1).all() and np.isnan(d[1, 128:]).all() and (d[2] == 1).all()


def test_weights_blocks_are_square():
    W = np.random.default_rng(0).standard_normal((2, 200, 144))
    q, s = Q.quantize_weights(W)
    q1, s1 = Q.quantize_rows(W[1, 128:200, 128:144].reshape(1, -1)[:, :1] * 0 + np.abs(W[1, 128:200, 128:144]).max())
    assert s.shape == (2, 2, 4) and s[1, 1, 1] == s1[0, 0]
    assert np.abs(Q.dequantize_weights(q, s) - W).max() <= 2.0 ** -4 * np.abs(W).max()


def test_round_bf16_is_torchs():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(3000) * 10.0 ** rng.uniform(-38, 38, 3000)).astype(np.float32)
    np.testing.assert_array_equal(Q.round_bf16(x), torch.from_numpy(x).bfloat16().double().numpy())


@pytest.mark.parametrize("T,d", [(1, 64), (3, 192)])
def test_norm_gradient_is_that_of_differences(T, d):
    rng = np.random.default_rng(3)
    r, w, g = rng.standard_normal((T, d)), 1 + 0.3 * rng.standard_normal(d), rng.standard_normal((T, d))
    dres = rng.standard_normal((T, d))
    f = lambda r, w: float((Q.norm(r, w, 1e-5)[0] * g).sum() + (dres * r).sum())  # noqa: E731
    dx, dw = Q.norm_backward(g, dres, r, w, 1e-5)
    h = 1e-6
    for t in range(T):
        for i in range(0, d, 17):
            e = np.zeros((T, d))
            e[t, i] = h
            assert abs((f(r + e, w) - f(r - e, w)) / (2 * h) - dx[t, i]) < 1e-6
    for i in range(0, d, 13):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(r, w + e) - f(r, w - e)) / (2 * h) - dw[i]) < 1e-6


def test_norm_against_autograd():
    torch.manual_seed(0)
    r = torch.randn(4, 128, dtype=torch.float64, requires_grad=True)
    w = torch.randn(128, dtype=torch.float64, requires_grad=True)
    g = torch.randn(4, 128, dtype=torch.float64)
    u = torch.nn.functional.rms_norm(r, (128,), w, eps=1e-6)
    np.testing.assert_allclose(Q.norm(r.detach().numpy(), w.detach().numpy(), 1e-6)[0], u.detach().numpy(), rtol=1e-12)
    u.backward(g)
    dx, dw = Q.norm_backward(g.numpy(), None, r.detach().numpy(), w.detach().numpy(), 1e-6)
    np.testing.assert_allclose(dx, r.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_grouped_leaves_rows_of_no_group():
    a, W = np.eye(5), np.arange(2 * 3 * 5, dtype=float).reshape(2, 3, 5)
    y = Q.grouped(a, W, [1, 2, 4])
    np.testing.assert_array_equal(y[1], W[0, :, 1])
    np.testing.assert_array_equal(y[2:4], W[1, :, 2:4].T)
    assert np.isnan(y[0]).all() and np.isnan(y[4]).all()
