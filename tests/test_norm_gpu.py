"""q8d_rmsnorm_rows against the formula in 64 bits, and its 8-bit rows byte by
byte against the formula in f32 steps.

Tolerance of an f32 output: the sum, the factor and two products are rounded,
each by 2^-24 of its value at most, and the factor follows the rounded sums by
2^-24 more: 5 * 2^-24 of |y| (and half a step of the output's own type)."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
F32, F16, Q8_0 = kp.F32, kp.F16, kp.Q8_0
NP = {F32: np.float32, F16: np.float16}
TT = {F32: torch.float32, F16: torch.float16}


def rows_of(a, kind, ld, offset):
    """Device rows `ld` apart, `offset` elements into a buffer filled with sevens."""
    buf = np.full(offset + a.shape[0] * ld, 7, NP[kind])
    for i, row in enumerate(a):
        buf[offset + i * ld:offset + i * ld + a.shape[1]] = row
    return dev(buf)[offset:]


def steps(x, r, w, eps):
    """(h, y) in the operator's f32 steps."""
    h = x.astype(np.float32)
    if r is not None:
        h = (h + r.astype(np.float32)).astype(np.float32)
    with np.errstate(all="ignore"):
        m = np.square(h.astype(np.float64)).mean(1, keepdims=True)
        inv = (1 / np.sqrt(m + np.float64(np.float32(eps)))).astype(np.float32)
        return h, ((h * inv).astype(np.float32) * w).astype(np.float32)


def inputs(seed, rows, n, kind, spread=True):
    x = synth.normal_f32(seed, "norm.x", (rows, n)).astype(np.float64)
    if spread:
        x *= 10.0 ** (np.arange(rows) % 6 - 3)[:, None]
    return x.astype(NP[kind])


CASES = [  # rows, n, ldx, ldr, lds, ldy, offset
    (1, 1, 1, 1, 1, 1, 0),
    (1, 3584, 3584, 3584, 3584, 3584, 0),
    (3, 32, 32, 32, 32, 32, 0),
    (7, 64, 64, 68, 72, 64, 0),
    (5, 33, 40, 33, 33, 37, 1),          # off every boundary
    (2, 8192, 8192, 8192, 8192, 8192, 0),
    (1, 16384, 16384, 16384, 16384, 16384, 0),
    (2, 16383, 16383, 16383, 16383, 16383, 0),
    (9, 8193, 8193, 8200, 8193, 8194, 3),
    (700, 896, 896, 896, 896, 896, 0),
    (301, 100, 104, 100, 100, 104, 0),
    (2500, 128, 128, 128, 128, 128, 0),
    (1900, 1184, 1184, 1184, 1184, 1184, 0),
    (400, 5000, 5000, 5000, 5000, 5000, 0),
]


@pytest.mark.parametrize("src", [F32, F16])
@pytest.mark.parametrize("dst", [F32, F16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,n,ldx,ldr,lds,ldy,offset", CASES)
def test_norm(q8d, src, dst, residual, rows, n, ldx, ldr, lds, ldy, offset):
    x = inputs(1, rows, n, src)
    r = inputs(2, rows, n, src) if residual else None
    w = (1 + 0.1 * synth.normal_f32(3, "norm.w", n)).astype(np.float32)
    dx, dw = rows_of(x, src, ldx, offset), dev(w)
    dr = rows_of(r, src, ldr, offset) if residual else None
    fill = np.full((rows, n), 5, np.float32)
    ds = rows_of(fill, src, lds, offset) if residual else None
    dy = rows_of(fill, dst, ldy, offset)
    q8d.q8d_rmsnorm_rows(dx, dr, ds, src, ldx, ldr, lds, dw, 1e-6, dy, dst, ldy, rows, n)
    torch.cuda.synchronize()
    h = x.astype(np.float64) + (r.astype(np.float64) if residual else 0)
    y = h / np.sqrt(np.square(h).mean(1, keepdims=True) + np.float64(np.float32(1e-6))) * w
    got = dy.cpu().numpy()
    for i in range(rows):
        g = got[i * ldy:i * ldy + n].astype(np.float64)
        tol = 5 * 2.0 ** -24 * np.abs(y[i]) + (2.0 ** -11 * np.abs(y[i]) + 2.0 ** -25 if dst == F16 else 0)
        # (a sum next to zero is off by half a step of its terms, not of itself: 2^-24 |x + r| covers f32 inputs only
        # where they do not cancel; the sum of two f16 is exact in f32 here)
        if src == F32 and residual:
            tol += 2.0 ** -24 * np.abs(y[i])
        assert np.all(np.abs(g - y[i]) <= tol), i
        assert np.all(got[i * ldy + n:(i + 1) * ldy] == 7)
    if residual:
        s = ds.cpu().numpy()
        want = (x.astype(np.float32) + r.astype(np.float32)).astype(NP[src])
        for i in range(rows):
            assert np.array_equal(s[i * lds:i * lds + n], want[i])
            assert np.all(s[i * lds + n:(i + 1) * lds] == 7)


@pytest.mark.parametrize("src", [F32, F16])
@pytest.mark.parametrize("rows,n,ldx,ldy,offset", [
    (1, 32, 32, 32, 0), (3, 96, 96, 128, 0), (5, 3584, 3584, 3584, 0), (1, 16384, 16384, 16384, 0),
    (600, 1024, 1024, 1024, 0), (33, 160, 161, 160, 1), (2000, 4864, 4864, 4864, 0), (4000, 64, 64, 64, 0)])
def test_norm_8_bit_rows(q8d, src, rows, n, ldx, ldy, offset):
    x, r = inputs(4, rows, n, src), inputs(5, rows, n, src)
    w = (1 + 0.1 * synth.normal_f32(6, "norm.w8", n)).astype(np.float32)
    if n >= 96:
        w[32:64] = 0  # a block of zeros
    nb = ldy // 32 * 34
    dy = torch.full((rows, nb), 77, dtype=torch.uint8, device="cuda")
    dr = rows_of(r, src, ldx, offset)
    q8d.q8d_rmsnorm_rows(rows_of(x, src, ldx, offset), dr, dr, src, ldx, ldx, ldx, dev(w), 1e-6, dy, Q8_0, ldy, rows, n)
    torch.cuda.synchronize()
    h, y = steps(x, r, w, 1e-6)
    want = kp.q8_blocks(y.reshape(rows, -1, 32)).reshape(rows, -1)
    got = dy.cpu().numpy()
    assert np.array_equal(got[:, :n // 32 * 34], want)
    assert np.all(got[:, n // 32 * 34:] == 77)
    s = dr.cpu().numpy()
    for i in range(rows):  # (the residual's rows became the sums)
        assert np.array_equal(s[i * ldx:i * ldx + n], h[i].astype(NP[src]))


@pytest.mark.parametrize("n", [7, 32, 128, 3584, 9000])
def test_norm_of_extreme_rows(q8d, n):
    """Rows whose squares pass f32's range, of zeros, infinities and NaN, next
    to ordinary ones: what 64-bit arithmetic gives."""
    rows = [np.full(n, 1e30), np.full(n, 1e-30), np.zeros(n), np.full(n, 3e38), np.linspace(-1, 1, n) * 1e-20,
            np.arange(n) * 1.0, np.full(n, 1e-44)]
    rows += [np.where(np.arange(n) == n // 2, v, 1.0) for v in (np.inf, -np.inf, np.nan, 1e25, 1e-38)]
    x = np.stack(rows + [np.arange(n) - 3.0] * 3).astype(np.float32)
    w = np.linspace(0.5, 2, n).astype(np.float32)
    for eps in (1e-6, 0.0):
        y = torch.empty(len(x), n, device="cuda")
        q8d.q8d_rmsnorm_rows(dev(x), None, None, F32, n, n, n, dev(w), eps, y, F32, n, len(x), n)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            _, want = steps(x, None, w, eps)
        got = y.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.isinf(got), np.isinf(want))
        fine = np.isfinite(want)
        # (one unit of the factor, where two roundings of it differ, and the products')
        assert np.all(np.abs(got[fine].astype(np.float64) - want[fine]) <= 4 * 2.0 ** -24 * np.abs(want[fine]) + 2.0 ** -149)


def test_norm_rows_do_not_depend_on_their_neighbours(q8d):
    """A row's bits are the same alone, in a batch, in place and in a graph."""
    n, rows = 640, 900
    x, r = inputs(7, rows, n, F32), inputs(8, rows, n, F32)
    x[::7] *= np.float32(1e25)  # (rows of the wide path between the others)
    w = dev(np.ones(n, np.float32))
    y, one = torch.empty(rows, n, device="cuda"), torch.empty(1, n, device="cuda")
    dx, dr = dev(x), dev(r)
    q8d.q8d_rmsnorm_rows(dx, dr, None, F32, n, n, n, w, 1e-6, y, F32, n, rows, n)
    for i in (0, 1, 6, 7, 8, 699, 899):
        q8d.q8d_rmsnorm_rows(dx[i:], dr[i:], None, F32, n, n, n, w, 1e-6, one, F32, n, 1, n)
        torch.cuda.synchronize()
        assert torch.equal(one[0], y[i])
    again, g, st = torch.empty_like(y), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        q8d.q8d_rmsnorm_rows(dx, dr, dx, F32, n, n, n, w, 1e-6, again, F32, n, rows, n, st)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, y)
    assert torch.equal(dx, dev((x + r).astype(np.float32)))
