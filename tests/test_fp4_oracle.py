"""Pins of the microscaled 4-bit oracle by independent checks (CPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle import fp4_oracle as F

FMTS = [F.MX, F.NV]


def test_tables():
    assert np.array_equal(F.e4m3_table(), torch.arange(127, dtype=torch.uint8)
                          .view(torch.float8_e4m3fn).double().numpy())
    # E2M1: sign-exponent-mantissa with bias 1
    want = [(m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)]
    assert np.array_equal(F.E2M1, want)


def test_nearest_against_brute_force():
    for table in (F.E2M1, F.e4m3_table()):
        mids = (table[1:] + table[:-1]) / 2
        v = np.concatenate([table, mids, mids * (1 + 1e-12), mids * (1 - 1e-12),
                            np.random.default_rng(0).uniform(0, table[-1] * 1.2, 500)])
        for x, i in zip(v, F.nearest(v, table)):
            d = np.abs(table - x)
            best = [j for j in range(len(table)) if d[j] == d.min()]
            assert i == (best[0] if len(best) == 1 else next(j for j in best if j % 2 == 0))


def test_e4m3_rounding_agrees_with_torch():
    x = torch.from_numpy(np.random.default_rng(1).uniform(0, 448, 20000)).float()
    assert np.array_equal(F.e4m3_table()[F.nearest(x.double().numpy(), F.e4m3_table())],
                          x.to(torch.float8_e4m3fn).double().numpy())


def test_gscale():
    for e in range(-100, 100, 7):
        assert F.gscale(2688.0 * 2.0 ** e) == 2.0 ** e
        assert F.gscale(np.nextafter(2688.0 * 2.0 ** e, np.inf)) == 2.0 ** (e + 1)
    assert F.gscale(0.0) == 1.0 and F.gscale(2.0 ** -140) == 2.0 ** -126


@pytest.mark.parametrize("fmt", FMTS)
def test_grid_values_round_trip(fmt):
    """Values on the grid of a scale are stored exactly when a 6 fixes the block's scale."""
    rng = np.random.default_rng(2)
    b = F.BLOCK[fmt]
    codes = rng.integers(0, 16, (8, 6 * b))
    codes[:, ::b] = 7
    v = np.where(codes >= 8, -F.E2M1[codes & 7], F.E2M1[codes & 7])
    x = v * 2.0 ** rng.integers(-3, 4, (8, 6)).repeat(b, 1)
    assert np.array_equal(F.dequant(F.quantize(x, fmt)), x)


@pytest.mark.parametrize("fmt", FMTS)
def test_error_bound_and_best_code(fmt):
    """Each stored value is a nearest representable one of its block's scale, and off by at
    most a sixth of the block's largest magnitude, but for the saturation that a rounded-down
    scale allows."""
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (5, 4 * 32))
    q = F.quantize(x, fmt)
    v = F.dequant(q)
    b = F.BLOCK[fmt]
    step = np.abs(F.dequant({**q, "codes": np.full_like(q["codes"], 2)}))  # value of code "1.0"
    grid = np.concatenate([F.E2M1, -F.E2M1])[:, None, None] * step
    assert np.allclose(np.abs(v - x), np.abs(grid - x).min(0))
    amax = np.abs(x).reshape(5, -1, b).max(2).repeat(b, 1)
    assert np.all(np.abs(v - x) <= amax / 4 + 1e-12)


@pytest.mark.parametrize("fmt", FMTS)
def test_weight_and_transpose_hold_the_same_values(fmt):
    W = np.random.default_rng(4).normal(0, 0.02, (64, 96))
    w, wt = F.quantize_weight(W, fmt)
    assert np.array_equal(F.dequant(w), F.dequant(wt).T)
    assert np.linalg.norm(F.dequant(w) - W) < 0.2 * np.linalg.norm(W)


def test_non_finite_values_stay_in_their_block():
    x = np.ones((3, 64))
    x[1, 20], x[2, 40] = np.nan, -np.inf
    for fmt in FMTS:
        v = F.dequant(F.quantize(x, fmt))
        b = F.BLOCK[fmt]
        assert np.isnan(v[1, 20 // b * b:(20 // b + 1) * b]).all() and np.isnan(v).sum() == 2 * b


def test_scale_positions_are_a_bijection():
    for R, B in itertools.product([1, 31, 128, 300], [2, 4, 9]):
        i = F.scale_index(R, B)
        assert len(np.unique(i)) == R * B and i.max() < F.store_scales(np.zeros((R, B), np.uint8)).size
    assert F.scale_index(300, 9)[129, 5] == (1 * 3 + 1) * 512 + 1 * 16 + 0 + 1


def test_forward_by_triple_loop_and_backward_by_adjoint():
    """On inputs that the 4-bit grid holds exactly the layer is bilinear: the forward is the
    plain sum, and <dX, V> is the derivative of <Y, dY> along V."""
    rng = np.random.default_rng(5)
    M, N, K, r, scale = 3, 32, 64, 8, 0.5
    for fmt in FMTS:
        w, _ = F.quantize_weight(rng.normal(0, 1, (N, K)), fmt)
        X = F.dequant(F.quantize(rng.normal(0, 1, (M, K)), fmt))
        X = F.dequant(F.quantize(X, fmt)) if fmt == F.MX else X
        dY = F.dequant(F.quantize(rng.normal(0, 1, (M, N)), fmt))
        A, B = rng.normal(0, 1, (K, r)), rng.normal(0, 1, (r, N))
        Y, T = F.linear_forward(X, w, A, B, scale)
        Xq, W = F.dequant(F.quantize(X, fmt)), F.dequant(w)
        want = [[sum(Xq[m, k] * W[n, k] for k in range(K)) +
                 scale * sum(T[m, j] * B[j, n] for j in range(r)) for n in range(N)] for m in range(M)]
        assert np.allclose(Y, want)
        dX, dA, dB = F.linear_backward(dY, X, w, A, B, scale)
        dYq = F.dequant(F.quantize(dY, fmt))
        f = lambda X_, A_, B_: np.sum((X_ @ W.T) * dYq) + scale * np.sum((X_ @ A_ @ B_) * dY)
        for g, i in ((dX, 0), (dA, 1), (dB, 2)):
            V = rng.normal(0, 1, g.shape)
            at = [X, A, B]
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + V, at[i] - V
            assert np.allclose((f(*hi) - f(*lo)) / 2, np.sum(g * V))
