"""4-bit matrices: the quantizer against the plain one, the products against
64-bit sums of the matrices' own values, at the header's 1e-5 of the sum of
|terms|; the gated pair at that bound carried through silu and the product
(|silu'| <= 1.1, and 2^-20 for exp, division and product)."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
F32, F16, Q8_0 = kp.F32, kp.F16, kp.Q8_0
NP = {F32: np.float32, F16: np.float16}


def plain_values(w, group):
    """f32 values [p][n] of a matrix quantized in groups, and its f16 scales."""
    p, n = w.shape
    pad = -n % group
    g = np.pad(w, ((0, 0), (0, pad))).reshape(p, -1, group)
    m = np.take_along_axis(g, np.abs(g).argmax(-1)[..., None], -1)
    d = (m / np.float32(-8)).astype(np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(1) / d
    inv = np.where(np.isfinite(inv), inv, np.float32(0)).astype(np.float32)
    q = np.clip(np.floor(((g * inv).astype(np.float32) + np.float32(8.5)).astype(np.float32)), 0, 15)
    return ((q.astype(np.float32) - 8) * d.astype(np.float16).astype(np.float32)).reshape(p, -1)[:, :n]


def q8_rows(x):
    return kp.q8_blocks(x.reshape(len(x), -1, 32)).reshape(len(x), -1)


def q8_values(b):
    b = b.reshape(len(b), -1, 34)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    return (d * b[..., 2:].view(np.int8)).reshape(len(b), -1)


class Matrix:
    def __init__(self, q8d, seed, p, n, group, scale=1.0):
        self.p, self.n, self.group = p, n, group
        w = (synth.normal_f32(seed, "q4.w", (p, n)) * np.float32(scale / np.sqrt(n))).astype(np.float32)
        self.values = plain_values(w, group).astype(np.float64)
        self.bytes = torch.full((q8d.q8d_q4_matrix_bytes(p, n, group),), 255, dtype=torch.uint8, device="cuda")
        q8d.q8d_q4_pack(dev(w), F32, n, self.bytes, p, n, group)


SHAPES = [(1, 32), (16, 128), (17, 96), (33, 416), (250, 128), (40, 2080), (129, 160)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("p,n", SHAPES)
@pytest.mark.parametrize("src,ld,offset", [(F32, 0, 0), (F32, 3, 1), (F16, 0, 0), (F16, 5, 3), (Q8_0, 0, 0), (Q8_0, 64, 0)])
def test_pack_and_unpack(q8d, group, p, n, src, ld, offset):
    ld += n
    w = synth.normal_f32(11, "q4.pack", (p, n))
    w *= (10.0 ** (np.arange(p) % 7 - 3)).astype(np.float32)[:, None]
    if n >= 96:
        w[:, 32:64] = 0
        w[:, 64:96] = np.tile(np.array([8, -8, 2.5, -2.5, 0.5, -0.5, 127, -127], np.float32), 4)
    if src == Q8_0:
        b = q8_rows(w)
        w = q8_values(b).astype(np.float32)
        buf = np.full((p, ld // 32 * 34), 99, np.uint8)
        buf[:, :b.shape[1]] = b
        d = dev(buf)
    else:
        w = w.astype(NP[src])
        buf = np.full(offset + p * ld, 99, NP[src])
        buf[offset:].reshape(p, ld)[:, :n] = w
        d, w = dev(buf)[offset:], w.astype(np.float32)
    nb = q8d.q8d_q4_matrix_bytes(p, n, group)
    out = torch.full((nb + 16,), 255, dtype=torch.uint8, device="cuda")
    q8d.q8d_q4_pack(d, src, ld, out, p, n, group)
    want = plain_values(w, group)
    for dst, t in ((F32, torch.float32), (F16, torch.float16)):
        back = torch.full((offset + p * ld,), 7, dtype=t, device="cuda")
        q8d.q8d_q4_unpack(out, back[offset:], dst, ld, p, n, group)
        torch.cuda.synchronize()
        got = back[offset:].view(p, ld).cpu().numpy()
        with np.errstate(over="ignore"):
            assert np.array_equal(got[:, :n], want.astype(NP[dst]))
        assert np.all(got[:, n:] == 7)
    assert torch.all(out[nb:] == 255)


def activations(seed, m, n, kind, ld=None):
    """(device rows, f64 values, elements between rows)"""
    x = synth.normal_f32(seed, "q4.x", (m, n))
    x = (x * (10.0 ** (np.arange(m) % 5 - 2))[:, None]).astype(np.float32)
    if n >= 256:
        x[:, 5] *= 100
        x[:, 128:160] *= np.float32(1e-4)
    ld = ld or n
    if kind == Q8_0:
        b = q8_rows(x)
        buf = np.full((m, ld // 32 * 34), 99, np.uint8)
        buf[:, :b.shape[1]] = b
        return dev(buf), q8_values(b), ld
    x = x.astype(NP[kind])
    buf = np.full((m, ld), 99, NP[kind])
    buf[:, :n] = x
    return dev(buf), x.astype(np.float64), ld


def product(q8d, W, x, kind, ld, m, bias=None, res=None, ldy=None, in_place=False, stream=None):
    ldy = ldy or W.p
    y = torch.full((m, ldy), 7.0, device="cuda")
    if in_place:
        y[:, :W.p] = res
        res = y
    q8d.q8d_q4_matmul(x, kind, ld, W.bytes, W.group, bias, res, ldy if in_place else (0 if res is None else res.stride(0)), y,
                      ldy, m, W.n, W.p, stream)
    return y


def check(y, W, v, bias=None, res=None):
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)
    ref, tol = v @ W.values.T, np.abs(v) @ np.abs(W.values).T
    for more in (bias, res):
        if more is not None:
            ref, tol = ref + more, tol + np.abs(more)
    assert np.all(np.abs(got[:, :W.p] - ref) <= 1e-5 * tol)
    assert np.all(got[:, W.p:] == 7)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", [F32, F16, Q8_0])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("p,n", [(16, 32), (17, 96), (250, 1184), (2450, 128)])
def test_product(q8d, group, kind, m, p, n):
    W = Matrix(q8d, 20, p, n, group)
    x, v, ld = activations(21, m, n, kind)
    check(product(q8d, W, x, kind, ld, m), W, v)


@pytest.mark.parametrize("kind", [F32, F16, Q8_0])
@pytest.mark.parametrize("m,p,n,group", [
    (1, 16, 32768, 128), (16, 16, 32768, 64), (8, 64, 18944, 32), (16, 100, 18944, 128), (1, 3584, 3584, 32),
    (3, 4608, 3584, 64), (1, 40001, 896, 64), (7, 40001, 896, 128), (16, 80000, 160, 32)])
def test_product_sizes(q8d, kind, m, p, n, group):
    W = Matrix(q8d, 22, p, n, group)
    x, v, ld = activations(23, m, n, kind, n + 32)
    check(product(q8d, W, x, kind, ld, m, ldy=p + 3), W, v)


@pytest.mark.parametrize("kind", [F32, F16, Q8_0])
@pytest.mark.parametrize("m", [1, 6, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_bias_and_residual(q8d, kind, m, in_place):
    W = Matrix(q8d, 24, 333, 416, 32)
    x, v, ld = activations(25, m, 416, kind)
    bias, res = synth.normal_f32(26, "q4.b", 333), synth.normal_f32(27, "q4.r", (m, 333))
    db, dr = dev(bias), dev(res)
    check(product(q8d, W, x, kind, ld, m, db, dr, 340, in_place), W, v, bias.astype(np.float64), res.astype(np.float64))
    if not in_place:
        check(product(q8d, W, x, kind, ld, m, db), W, v, bias.astype(np.float64))
        check(product(q8d, W, x, kind, ld, m, None, dr), W, v, None, res.astype(np.float64))


@pytest.mark.parametrize("kind", [F32, F16, Q8_0])
@pytest.mark.parametrize("m,p,n,group", [(1, 16, 32, 32), (5, 77, 160, 64), (16, 4736, 1024, 128), (1, 18944, 896, 32),
                                         (9, 30, 18944, 64), (2, 12000, 96, 128)])
def test_gated(q8d, kind, m, p, n, group):
    G, U = Matrix(q8d, 28, p, n, group, 3.0), Matrix(q8d, 29, p, n, group)
    x, v, ld = activations(30, m, n, kind)
    h = torch.full((m, p + 1), 7.0, device="cuda")
    q8d.q8d_q4_gated(x, kind, ld, G.bytes, U.bytes, group, h, p + 1, m, n, p)
    torch.cuda.synchronize()
    got = h.cpu().numpy().astype(np.float64)
    g, gt = v @ G.values.T, 1e-5 * (np.abs(v) @ np.abs(G.values).T)
    u, ut = v @ U.values.T, 1e-5 * (np.abs(v) @ np.abs(U.values).T)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    tol = 1.1 * gt * (np.abs(u) + ut) + np.abs(silu) * ut + 2.0 ** -20 * np.abs(silu * u) + 1e-37
    assert np.all(np.abs(got[:, :p] - silu * u) <= tol)
    assert np.all(got[:, p:] == 7)


def test_exact_sums(q8d):
    """Whole numbers below 2^24 come out exactly: every column is met once."""
    p, n = 48, 1184
    rng = synth.stream(31, "q4.int")
    w = rng.integers(-8, 8, (p, n)).astype(np.float32)
    w[:, ::32] = -8  # (the largest magnitude: the scale is 1)
    W = Matrix(q8d, 1, p, n, 32)
    q8d.q8d_q4_pack(dev(w), F32, n, W.bytes, p, n, 32)
    x = rng.integers(-64, 64, (4, n)).astype(np.float32)
    y = product(q8d, W, dev(x), F32, n, 4)
    torch.cuda.synchronize()
    assert np.array_equal(y.cpu().numpy(), x @ w.T)
    eye = np.zeros((16, n), np.float32)
    for first in range(0, n, 16):
        eye[:] = 0
        eye[np.arange(16), first + np.arange(16)] = 1
        y = product(q8d, W, dev(eye), F32, n, 16)
        torch.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy(), w[:, first:first + 16].T)


def test_rows_with_nan_and_infinity_stay_alone(q8d):
    W = Matrix(q8d, 32, 100, 256, 64)
    for kind in (F32, F16):
        x, v, ld = activations(33, 4, 256, kind)
        x[1, 200] = float("nan")
        x[2, 3] = float("inf")
        y = product(q8d, W, x, kind, ld, 4)
        torch.cuda.synchronize()
        assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[2]).any()
        keep = [0, 3]
        check(y[keep], W, v[keep])


def test_range_of_activations(q8d):
    """Rows far from 1: a power of two for every 128 columns keeps their bits."""
    W = Matrix(q8d, 34, 100, 384, 32)
    x = synth.normal_f32(35, "q4.range", (8, 384))
    x = (x * np.float32(10.0) ** np.array([-37, -30, -12, -4, 4, 12, 30, 34])[:, None]).astype(np.float32)
    x[3, 128:256] *= np.float32(1e20)
    check(product(q8d, W, dev(x), F32, 384, 8), W, x.astype(np.float64))
    zero = torch.zeros(2, 384, device="cuda")
    assert torch.all(product(q8d, W, zero, F32, 384, 2) == 0)


def test_same_bits_every_time(q8d):
    """Repeated, on two streams at once, in a graph, and straight behind the
    kernels that write its operands."""
    W = Matrix(q8d, 36, 5000, 3584, 32)
    G = Matrix(q8d, 37, 5000, 3584, 32)
    x, v, ld = activations(38, 3, 3584, F32)
    first = product(q8d, W, x, F32, ld, 3)
    check(first, W, v)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [torch.empty(3, 5000, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        q8d.q8d_q4_matmul(x, F32, ld, W.bytes, 32, None, None, 0, y, 5000, 3, 3584, 5000, streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for y in outs)
    g, y, h = torch.cuda.CUDAGraph(), torch.empty(3, 5000, device="cuda"), torch.empty(3, 5000, device="cuda")
    q8d.q8d_q4_gated(x, F32, ld, W.bytes, G.bytes, 32, h, 5000, 3, 3584, 5000)
    torch.cuda.synchronize()
    want, back = h.clone(), torch.empty(5000, 3584, device="cuda")
    with torch.cuda.graph(g, stream=streams[0]):
        q8d.q8d_q4_matmul(x, F32, ld, W.bytes, 32, None, None, 0, y, 5000, 3, 3584, 5000, streams[0])
        # (the matrix read back and packed again between two products: the same bytes)
        q8d.q8d_q4_unpack(W.bytes, back, F32, 3584, 5000, 3584, 32, streams[0])
        q8d.q8d_q4_pack(back, F32, 3584, W.bytes, 5000, 3584, 32, streams[0])
        q8d.q8d_q4_gated(x, F32, ld, W.bytes, G.bytes, 32, h, 5000, 3, 3584, 5000, streams[0])
    for _ in range(3):
        y.zero_()
        h.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first) and torch.equal(h, want)


@pytest.mark.parametrize("m,p,n", [(1, 70, 224), (7, 200, 672), (14, 90, 2016)])
def test_first_call_of_a_size_in_a_capture(q8d, m, p, n):
    """Nothing of a size has to be known before a graph is captured."""
    W = Matrix(q8d, 39, p, n, 64)
    x, v, ld = activations(40, m, n, F32)
    y, st, g = torch.full((m, p), 7.0, device="cuda"), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        q8d.q8d_q4_matmul(x, F32, ld, W.bytes, 64, None, None, 0, y, p, m, n, p, st)
    torch.cuda.synchronize()
    assert torch.all(y == 7)
    g.replay()
    check(y, W, v)


@pytest.mark.parametrize("m", [9, 13, 16])
def test_sixteen_rows_of_a_large_matrix(q8d, m):
    """Rows that go in one launch or in two, with everything that has a row's place."""
    p, n = 18944, 3584
    W, U = Matrix(q8d, 41, p, n, 32), Matrix(q8d, 42, p, n, 32)
    x, v, ld = activations(43, m, n, F32, n + 4)
    bias, res = synth.normal_f32(44, "q4.b16", p), synth.normal_f32(45, "q4.r16", (m, p))
    check(product(q8d, W, x, F32, ld, m, dev(bias), dev(res), p + 5, True), W, v, bias.astype(np.float64),
          res.astype(np.float64))
    h = torch.full((m, p + 1), 7.0, device="cuda")
    q8d.q8d_q4_gated(x, F32, ld, W.bytes, U.bytes, 32, h, p + 1, m, n, p)
    torch.cuda.synchronize()
    g, u = v @ W.values.T, v @ U.values.T
    gt, ut = (1e-5 * (np.abs(v) @ np.abs(w.values).T) for w in (W, U))
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    tol = 1.1 * gt * (np.abs(u) + ut) + np.abs(silu) * ut + 2.0 ** -20 * np.abs(silu * u) + 1e-37
    got = h.cpu().numpy()
    assert np.all(np.abs(got[:, :p] - silu * u) <= tol) and np.all(got[:, p:] == 7)


@pytest.mark.parametrize("m,p,n,group,kind", [(1, 900_001, 64, 32, F32), (5, 700_000, 32, 64, F32), (16, 3584, 18944, 128, F32),
                                              (16, 30000, 2048, 64, Q8_0), (12, 400_000, 96, 128, F16)])
def test_many_strips(q8d, m, p, n, group, kind):
    """More strips than a CTA sums up at once."""
    W = Matrix(q8d, 46, p, n, group)
    x, v, ld = activations(47, m, n, kind)
    check(product(q8d, W, x, kind, ld, m), W, v)
    if p * n < 4e7:
        U = Matrix(q8d, 48, p, n, group)
        h, y = torch.empty(m, p, device="cuda"), product(q8d, U, x, kind, ld, m)
        q8d.q8d_q4_gated(x, kind, ld, W.bytes, U.bytes, group, h, p, m, n, p)
        g = product(q8d, W, x, kind, ld, m)
        torch.cuda.synchronize()
        g, y = g.double(), y.double()
        # (of the products as the other entry makes them, which cuts them up elsewhere: the bounds of both)
        tol = dev(np.abs(v) @ np.abs(W.values).T) * y.abs() + g.abs() * dev(np.abs(v) @ np.abs(U.values).T)
        assert torch.all((h.double() - g * torch.sigmoid(g) * y).abs() <= 2.5e-5 * tol + 2.0 ** -20 * (g * y).abs())
