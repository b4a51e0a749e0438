"""4-bit products of rows whose elements lie far apart: an element that meets a
weight of zero, or one of a group with a small scale, is in no term, or in a small
one, and must not cost its neighbours their bits.

Bound: the header's, 1e-5 of the sum of |terms|, and 2^-126 for sums below f32's
normal range; the gated pair as in test_q4_gpu.py."""
import numpy as np
import pytest
import torch

import synth
from conftest import dev
from test_q4_gpu import F16, F32, Matrix, plain_values, product

pytestmark = pytest.mark.gpu


def matrix(q8d, seed, p, n, group, zeros, small=(), scale=1.0):
    """Codes 0 .. 15 under one scale, 8 (the value zero) in the columns `zeros`;
    the groups that start at the columns `small` under a scale of 2^-20."""
    w = synth.stream(seed, "spread.w").integers(-8, 8, (p, n)).astype(np.float32)
    w[:, ::32] = -8
    for c in zeros:
        w[:, c] = 0
    w *= np.float32(scale)
    for c in small:
        w[:, c:c + group] *= np.float32(2.0 ** -20 / scale)
    W = Matrix(q8d, 1, p, n, group)
    q8d.q8d_q4_pack(dev(w), F32, n, W.bytes, p, n, group)
    W.values = plain_values(w, group).astype(np.float64)
    return W


def check(y, W, v):
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)
    ref, tol = v @ W.values.T, 1e-5 * (np.abs(v) @ np.abs(W.values).T) + 2.0 ** -126
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


def rows(m, n, far, top, at, kind=np.float32):
    x = synth.normal_f32(m, "spread.x", (m, n)).astype(np.float64) * top * far
    x[:, at] = top
    return x.astype(kind)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 4, 7, 11, 16])
@pytest.mark.parametrize("top,far", [(1.0, 2.0 ** -20), (1.0, 2.0 ** -24), (1.0, 1e-8), (1.0, 1e-9), (3.0, 2.0 ** -34),
                                     (1e10, 2.0 ** -40), (1e18, 1e-30), (1e35, 1e-60), (1e-20, 1e-12), (3e38, 1e-70)])
def test_outliers_on_zero_weights(q8d, group, m, top, far):
    n, at = 384, [5, 133, 250]
    W = matrix(q8d, 1, 70, n, group, at)
    x = rows(m, n, far, top, at)
    check(product(q8d, W, dev(x), F32, n, m), W, x.astype(np.float64))


@pytest.mark.parametrize("top,far", [(60000.0, 2.0 ** -20), (60000.0, 2.0 ** -30), (60000.0, 2.0 ** -38), (1.0, 2.0 ** -22)])
@pytest.mark.parametrize("m", [1, 8, 16])
@pytest.mark.parametrize("group", [32, 128])
def test_outliers_of_f16_rows(q8d, group, m, top, far):
    n, at = 384, [5, 133, 250]
    W = matrix(q8d, 2, 70, n, group, at)
    x = rows(m, n, far, top, at, np.float16)
    check(product(q8d, W, dev(x), F16, n, m), W, x.astype(np.float64))


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("far", [2.0 ** -26, 2.0 ** -30, 2.0 ** -34])
def test_outliers_in_groups_of_small_scales(q8d, group, far):
    """Terms of one size: elements of 1 under scales of 2^-20, of `far` under others."""
    n, m = 256, 5
    W = matrix(q8d, 3, 40, n, group, [], [64, 192], 2.0 ** -20 / far)
    x = synth.normal_f32(m, "spread.x", (m, n))
    big = np.isin(np.arange(n) // group * group, [64, 192])
    x[:, ~big] *= np.float32(far)
    check(product(q8d, W, dev(x), F32, n, m), W, x.astype(np.float64))


@pytest.mark.parametrize("m,p,n,group", [(1, 3584, 18944, 32), (16, 100, 18944, 128), (16, 18944, 3584, 32), (3, 300_001, 96, 64),
                                         (16, 80000, 160, 32), (2, 77, 32768, 64)])
@pytest.mark.parametrize("far", [1e-9, 1e-20])
def test_outliers_of_large_calls(q8d, m, p, n, group, far):
    """Some tiles of some rows, wherever a row's columns and the rows are cut."""
    at = list(range(7, n, 997))
    W = matrix(q8d, 4, p, n, group, at)
    x = rows(m, n, far, 1.0, at)
    x[m // 2] = synth.normal_f32(5, "spread.plain", n)
    x[0, n // 2:] = synth.normal_f32(6, "spread.half", n - n // 2)
    check(product(q8d, W, dev(x), F32, n, m), W, x.astype(np.float64))


@pytest.mark.parametrize("m,p,n,group", [(1, 100, 384, 32), (6, 3000, 1024, 64), (16, 500, 4736, 128)])
@pytest.mark.parametrize("far", [1e-9, 1e-20])
def test_gated_outliers(q8d, m, p, n, group, far):
    at = list(range(7, n, 131))
    G, U = matrix(q8d, 7, p, n, group, at), matrix(q8d, 8, p, n, group, at)
    x = rows(m, n, far, 1.0 / far / n, at)
    h = torch.full((m, p), 7.0, device="cuda")
    q8d.q8d_q4_gated(dev(x), F32, n, G.bytes, U.bytes, group, h, p, m, n, p)
    torch.cuda.synchronize()
    v = x.astype(np.float64)
    g, gt = v @ G.values.T, 1e-5 * (np.abs(v) @ np.abs(G.values).T)
    u, ut = v @ U.values.T, 1e-5 * (np.abs(v) @ np.abs(U.values).T)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    tol = 1.1 * gt * (np.abs(u) + ut) + np.abs(silu) * ut + 2.0 ** -20 * np.abs(silu * u) + 1e-37
    assert np.all(np.abs(h.cpu().numpy().astype(np.float64) - silu * u) <= tol)
