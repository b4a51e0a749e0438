"""q8d_moe_ffn against a plain numpy form in f64.

Tolerance of Y: 1e-5 of the sum of |terms| A = sum_k w_k |Wd| (|h| + dh):
the products' contract is 1e-5 of their own sums of |terms|, and h's error
passes through Wd.  dh bounds h's: with Ag, Au the gate's and up's sums of
|terms|, |silu'| <= 1.1 and the relative error of a product at most 2e-7
(two f16 parts of x, 2^-22, and f32 sums), dh = 2e-7 (1.1 Ag |u| +
|silu(g)| Au), which the check adds to 1e-5 A.  Below f32's normal range a rounding is up
to 2^-150 whatever the value (a token of 1e-20 gives h of 1e-40): the
roundings of h reach Y through k * ffn entries of Wd of at most 1, and with
k * ffn <= 2^18 they and Y's own stay under 2^-131, so 2^-126 is added.  The weights are f32
roundings of f64 values: 2^-24 each, checked at 2^-22.  The choice has to be
equal."""
import numpy as np
import pytest
import torch

import synth
from conftest import dev

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def dequant(w, p, n):
    b = w.reshape(p, n // 32, 34)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    return (d * b[..., 2:].view(np.int8)).reshape(p, n)


def layer(seed, E, hidden, ffn):
    """router and the experts' matrices, one behind the other."""
    r = synth.normal_f32(seed, "moe.router", (E, hidden)) * np.float32(2 / np.sqrt(hidden))
    s = 1 / (73 * np.sqrt(hidden))
    sd = 1 / (73 * np.sqrt(ffn))
    return (r, synth.q8_matrix(seed, "moe.g", E * ffn, hidden, 0.5 * s, 1.5 * s),
            synth.q8_matrix(seed, "moe.u", E * ffn, hidden, 0.5 * s, 1.5 * s),
            synth.q8_matrix(seed, "moe.d", E * hidden, ffn, 0.5 * sd, 1.5 * sd))


def plain(L, x, E, hidden, ffn, k, norm, res):
    """(experts, weights, Y, the tolerance of Y) in f64."""
    r, wg, wu, wd = L
    m = x.shape[0]
    x = x.astype(np.float64)
    logits = x @ r.astype(np.float64).T
    rank = np.where(np.isnan(logits), -np.inf, logits)
    at = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    p = np.exp(logits - rank.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, at, 1)
    if norm:
        w = w / w.sum(1, keepdims=True)
    y = np.zeros((m, hidden)) if res is None else res.astype(np.float64)
    tol = 1e-6 * np.abs(y) + 2.0 ** -126
    for e in np.unique(at):
        t, j = np.nonzero(at == e)
        rows = wg.shape[1]
        G = dequant(wg.reshape(E, ffn, rows)[e], ffn, hidden)
        U = dequant(wu.reshape(E, ffn, rows)[e], ffn, hidden)
        D = dequant(wd.reshape(E, hidden, -1)[e], hidden, ffn)
        g, u = x[t] @ G.T, x[t] @ U.T
        ag, au = np.abs(x[t]) @ np.abs(G).T, np.abs(x[t]) @ np.abs(U).T
        with np.errstate(over="ignore"):
            s = g / (1 + np.exp(-g))
        h = s * u
        dh = 2e-7 * (1.1 * ag * np.abs(u) + np.abs(s) * au)
        wt = w[t, j][:, None]
        np.add.at(y, t, wt * (h @ D.T))
        np.add.at(tol, t, np.abs(wt) * ((1e-5 * np.abs(h) + dh) @ np.abs(D).T))
    return at.astype(np.int32), w, y, tol


def run(q8d, L, x, E, hidden, ffn, k, norm, res=None, ldx=None, ldy=None, outs=True, in_place=False, stream=None):
    m = x.shape[0]
    ldx, ldy = ldx or hidden, ldy or hidden
    X = torch.zeros(m, ldx, device="cuda")
    X[:, :hidden] = dev(x)
    Y = torch.full((m, ldy), -7.0, device="cuda")
    R = None
    if res is not None:
        R = Y if in_place else dev(res)
        if in_place:
            Y[:, :hidden] = dev(res)
    ex = torch.full((m, k), -1, dtype=torch.int32, device="cuda") if outs else None
    we = torch.full((m, k), -1.0, device="cuda") if outs else None
    n = q8d.q8d_moe_workspace_bytes(m, hidden, ffn, E, k)
    ws = torch.full((n // 4 + 4,), float("nan"), device="cuda")
    err = ints([0])
    d = [dev(w) for w in L]
    q8d.q8d_moe_ffn(X, ldx, d[0], d[1], d[2], d[3], R, ldy if in_place else hidden, Y, ldy, m, hidden, ffn, E, k,
                    int(norm), ex, we, ws, n, err, stream)
    torch.cuda.synchronize()
    assert err.item() == 0
    y = Y.cpu().numpy()
    assert np.all(y[:, hidden:] == -7.0)
    return y[:, :hidden], ex.cpu().numpy() if outs else None, we.cpu().numpy() if outs else None


def check(q8d, L, x, E, hidden, ffn, k, norm, res=None, **kw):
    y, ex, we = run(q8d, L, x, E, hidden, ffn, k, norm, res, **kw)
    at, w, ref, tol = plain(L, x, E, hidden, ffn, k, norm, res)
    if ex is not None:
        assert np.array_equal(ex, at)
        assert np.allclose(we, w, rtol=2 ** -22, atol=1e-30)
    assert np.all(np.abs(y - ref) <= tol), (np.abs(y - ref) / tol).max()


CASES = [  # m, hidden, ffn, E, k, norm, residual
    (1, 32, 32, 1, 1, False, False),
    (1, 64, 96, 8, 2, True, True),
    (2, 256, 256, 4, 4, False, True),
    (3, 96, 352, 5, 3, True, False),           # rows off every 16-byte boundary
    (1, 1024, 512, 32, 4, True, True),
    (5, 1056, 288, 60, 8, False, True),
    (8, 512, 544, 16, 6, True, False),
    (9, 2048, 128, 64, 8, True, True),
    (17, 288, 64, 8, 1, False, False),
    (31, 192, 96, 3, 2, True, True),
    (33, 320, 160, 128, 8, True, True),
    (64, 256, 128, 4, 2, True, True),          # every expert has many tokens
    (64, 128, 64, 512, 32, False, False),
    (1, 3584, 1184, 16, 6, False, False),
    (4, 8192, 64, 2, 1, True, False),
    (2, 64, 8192, 2, 2, True, False),
]


@pytest.mark.parametrize("m,hidden,ffn,E,k,norm,residual", CASES)
def test_parity(q8d, m, hidden, ffn, E, k, norm, residual):
    L = layer(m + hidden, E, hidden, ffn)
    x = synth.normal_f32(1, "moe.x", (m, hidden))
    res = synth.normal_f32(1, "moe.res", (m, hidden)) if residual else None
    check(q8d, L, x, E, hidden, ffn, k, norm, res)


@pytest.mark.parametrize("m", [2, 7, 8, 16, 24, 64])
def test_all_tokens_ask_the_same_experts(q8d, m):
    """Equal tokens: one expert has every token, the others none."""
    E, hidden, ffn, k = 6, 256, 160, 2
    L = layer(3, E, hidden, ffn)
    x = np.repeat(synth.normal_f32(3, "same.x", (1, hidden)), m, 0)
    x += synth.normal_f32(3, "same.d", (m, hidden)) * np.float32(1e-3)
    check(q8d, L, x, E, hidden, ffn, k, True)


def test_strides_outputs_and_in_place_residual(q8d):
    E, hidden, ffn, k, m = 8, 128, 96, 3, 5
    L = layer(4, E, hidden, ffn)
    x, res = synth.normal_f32(4, "str.x", (m, hidden)), synth.normal_f32(4, "str.r", (m, hidden))
    check(q8d, L, x, E, hidden, ffn, k, True, res, ldx=hidden + 12, ldy=hidden + 5, in_place=True)
    check(q8d, L, x, E, hidden, ffn, k, True, None, ldy=hidden + 3, outs=False)


def test_ties_go_to_the_lower_index(q8d):
    """Equal router rows, and a token of zeros: every logit equal."""
    E, hidden, ffn, k = 40, 64, 64, 5
    L = list(layer(5, E, hidden, ffn))
    L[0][7] = L[0][31] = L[0][39] = L[0][2]
    x = synth.normal_f32(5, "tie.x", (6, hidden))
    x[3] = 0
    x[4] = L[0][2] * 20  # the four equal experts come first
    check(q8d, L, x, E, hidden, ffn, k, False)


def test_neighbours_in_rank(q8d):
    """Logits that differ by less than an f32 sum's error are ranked as in
    f64."""
    E, hidden, ffn, k = 64, 1024, 32, 8
    L = list(layer(6, E, hidden, ffn))
    base = L[0][0].copy()
    for e in range(E):
        L[0][e] = base
        L[0][e, (e * 37) % hidden] = np.nextafter(base[(e * 37) % hidden], np.float32(np.inf if e % 2 else -np.inf))
    x = synth.normal_f32(6, "near.x", (12, hidden))
    check(q8d, L, x, E, hidden, ffn, k, True)


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 1e4])
def test_ranges_of_values(q8d, scale):
    """Tokens far from unit size, mixed within a batch and within a row."""
    E, hidden, ffn, k, m = 4, 256, 128, 2, 10
    L = layer(7, E, hidden, ffn)
    x = synth.normal_f32(7, "rng.x", (m, hidden))
    x[::2] *= np.float32(scale)
    x[1, :64] *= np.float32(1e-6)
    x[5] = 0
    check(q8d, L, x, E, hidden, ffn, k, True)


def test_nan_stays_in_its_token(q8d):
    E, hidden, ffn, k, m = 8, 128, 64, 2, 12
    L = layer(8, E, hidden, ffn)
    x = synth.normal_f32(8, "nan.x", (m, hidden))
    clean = x.copy()
    x[3, 17] = np.nan
    x[9, 5] = np.inf
    clean[3] = clean[9] = 0
    y, ex, we = run(q8d, L, x, E, hidden, ffn, k, True)
    at, w, ref, tol = plain(L, clean, E, hidden, ffn, k, True, None)
    for t in range(m):
        if t in (3, 9):
            assert not np.isfinite(y[t]).any()
            assert len(set(ex[t])) == k and ex[t].min() >= 0 and ex[t].max() < E
        else:
            assert np.array_equal(ex[t], at[t]) and np.all(np.abs(y[t] - ref[t]) <= tol[t])


def test_same_bits_every_time(q8d):
    E, hidden, ffn, k, m = 32, 512, 256, 4, 13
    L = layer(9, E, hidden, ffn)
    x = synth.normal_f32(9, "rep.x", (m, hidden))
    first = run(q8d, L, x, E, hidden, ffn, k, True)
    for _ in range(4):
        for a, b in zip(run(q8d, L, x, E, hidden, ffn, k, True), first):
            assert np.array_equal(a, b)


def test_back_to_back_calls_and_a_graph(q8d):
    """Three layers in a row on one stream over one workspace, each reading
    the one before, captured and replayed with new tokens."""
    E, hidden, ffn, k, m = 16, 256, 192, 3, 6
    layers = [layer(20 + i, E, hidden, ffn) for i in range(3)]
    d = [[dev(w) for w in L] for L in layers]
    bufs = [torch.zeros(m, hidden, device="cuda") for _ in range(4)]
    n = q8d.q8d_moe_workspace_bytes(m, hidden, ffn, E, k)
    ws, err = torch.empty(n, dtype=torch.uint8, device="cuda"), ints([0])

    def chain(st):
        for i in range(3):
            q8d.q8d_moe_ffn(bufs[i], hidden, d[i][0], d[i][1], d[i][2], d[i][3], bufs[i], hidden, bufs[i + 1],
                            hidden, m, hidden, ffn, E, k, 1, None, None, ws, n, err, st)

    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        chain(st)
    for turn in range(3):
        x = synth.normal_f32(turn, "chain.x", (m, hidden))
        bufs[0].copy_(dev(x))
        torch.cuda.synchronize()
        if turn == 1:
            chain(None)
        else:
            g.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for i in range(3):  # each layer against its own input, as the device computed it
            xi = bufs[i].cpu().numpy()
            _, _, ref, tol = plain(layers[i], xi, E, hidden, ffn, k, True, xi)
            y = bufs[i + 1].cpu().numpy()
            assert np.all(np.abs(y - ref) <= tol), (np.abs(y - ref) / tol).max()


# Widths by how their rows lie in memory: whole 16-byte lines or not, short
# rows, rows cut into slices; with one, few and many tokens an expert, enough
# units that a CTA's buffers are reused, a last unit of half the rows.
@pytest.mark.parametrize("hidden,ffn", [
    (32, 160), (160, 480), (480, 32), (1824, 608), (608, 1824), (3552, 96), (96, 3552), (2080, 4128), (544, 992),
    (1056, 800), (2048, 768), (2304, 1312), (1504, 1536),
])
@pytest.mark.parametrize("m,E,k", [(1, 3, 2), (3, 6, 1), (13, 7, 2), (40, 5, 3)])
def test_row_layouts(q8d, hidden, ffn, m, E, k):
    L = layer(hidden + ffn, E, hidden, ffn)
    check(q8d, L, synth.normal_f32(m, "rows.x", (m, hidden)), E, hidden, ffn, k, True)


@pytest.mark.parametrize("hidden,ffn,m,E,k", [
    (2336, 1376, 9, 40, 4), (1184, 1184, 24, 48, 6), (2048, 512, 30, 64, 4), (3488, 32, 16, 64, 8), (352, 96, 64, 300, 12),
])
def test_many_experts_a_block(q8d, hidden, ffn, m, E, k):
    """More items than buffers in every CTA."""
    L = layer(hidden + ffn, E, hidden, ffn)
    check(q8d, L, synth.normal_f32(m, "many.x", (m, hidden)), E, hidden, ffn, k, False)


@pytest.mark.parametrize("hidden,ffn,m,E,k", [
    (16384, 32, 3, 2, 1), (32, 16384, 3, 2, 2), (16384, 64, 64, 2, 2), (16352, 32, 20, 2, 1), (32, 16352, 20, 2, 2),
    (64, 32, 64, 32, 32), (96, 64, 64, 33, 32), (256, 128, 64, 1, 1),
])
def test_largest_sizes(q8d, hidden, ffn, m, E, k):
    """The longest rows, whole and off 16-byte lines; every token asking every
    expert."""
    L = layer(hidden + ffn, E, hidden, ffn)
    check(q8d, L, synth.normal_f32(m, "largest.x", (m, hidden)), E, hidden, ffn, k, True)
