"""Decode attention over the 4-bit cache through the C ABI against the f64
oracle, which reads the same cache's values as an f32 cache.

Tolerance 1e-5 * sum_t p_t |V_t| per output (the other caches' contract).
The kernel's error against it: a score's terms carry the split of q into two
f16 parts (2^-22 of each term) and f32 sums, so with scale * sum|q K| about
8 for these inputs a probability is off by at most about 12 * 2^-21 = 6e-6,
and the split of p * scale adds 2^-22."""
import math

import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
TOL = 1e-5
Q4, F32 = kp.Q4, kp.F32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def q4_cache(seed, name, cap, width, rows=None, noise=False):
    """One sequence's 4-bit cache of N(0,1) rows; rows past `rows` random
    bytes (scales among them NaN and inf) when noise."""
    n = kp.cache_bytes(Q4, cap * width)
    c = synth.stream(seed, name + ".noise").integers(0, 256, n, dtype=np.uint8) if noise else np.zeros(n, np.uint8)
    if noise:  # f16 scales of all ones bits: NaN
        c[cap * width // 2:] |= 0x7c
    rows = cap if rows is None else rows
    if rows:
        kp.store(c, Q4, width, cap, 0, synth.normal_f32(seed, name, (rows, width)))
    return c


def oracle_attn(orc, q, kc, vc, H, Hk, D, cap, L, scale, cells=None):
    width = Hk * D
    k, v = kp.values(kc, Q4, width, cap), kp.values(vc, Q4, width, cap)
    if cells is not None:
        k, v = k[cells], v[cells]
    return orc.gqa_decode_attn(q, np.ascontiguousarray(k), np.ascontiguousarray(v), F32, H, Hk, D, L, scale)


def run(q8d, q, kc, vc, H, Hk, D, lens, cap, scale, stride=None, k_new=None, v_new=None, runs=None,
        noalloc=False, out=None):
    batch = len(lens) if lens is not None else len(runs)
    out = torch.full((batch, H * D), -7.0, device="cuda") if out is None else out
    err = ints([0])
    if stride is None:  # (one sequence: the stride is not used)
        stride = cap * Hk * D if batch > 1 else 0
    if noalloc:
        q8d.q8d_gqa_decode_attn_noalloc(q, k_new, v_new, kc, vc, Q4, out, batch, H, Hk, D, cap, stride,
                                        ints(lens), scale, err)
    else:
        n = q8d.q8d_gqa_workspace_bytes(batch, H, Hk, D, cap)
        ws = torch.full((n // 4 + 4,), float("nan"), device="cuda")
        if runs is None:
            q8d.q8d_gqa_decode_attn(q, k_new, v_new, kc, vc, Q4, out, batch, H, Hk, D, cap, stride,
                                    ints(lens), scale, ws, n, err)
        else:
            q8d.q8d_gqa_decode_attn_window(q, k_new, v_new, kc, vc, Q4, out, batch, H, Hk, D, cap, stride,
                                           ints(runs), scale, ws, n, err)
    torch.cuda.synchronize()
    return out.cpu().numpy(), err.item()


def close(got, ref, ab, tol=TOL):
    assert np.all(np.abs(got - ref) <= tol * ab), (np.abs(got - ref) / ab).max()


CASES = [  # H, Hk, D, L, cap
    (1, 1, 64, 1, 1), (3, 1, 128, 2, 2), (16, 8, 128, 512, 512), (4, 2, 64, 9, 16),
    (14, 2, 64, 2048, 2048), (28, 4, 128, 2048, 8192), (28, 4, 128, 8191, 8192), (6, 2, 64, 129, 300),
    (16, 1, 128, 1000, 1000), (3, 3, 128, 77, 80), (8, 8, 64, 15, 15), (4, 1, 128, 17, 31),
    (5, 1, 64, 31, 64), (8, 1, 128, 33, 33), (9, 1, 64, 257, 257), (12, 1, 128, 143, 144),
    (32, 2, 128, 640, 641), (64, 8, 64, 127, 128),
]


@pytest.mark.parametrize("H,Hk,D,L,cap", CASES)
def test_parity(q8d, orc, H, Hk, D, L, cap):
    kc, vc = (q4_cache(0, f"q4.{x}", cap, Hk * D, L, noise=True) for x in "kv")
    q = synth.normal_f32(0, "q4.q", H * D)
    ref, ab = oracle_attn(orc, q, kc, vc, H, Hk, D, cap, L, 1 / math.sqrt(D))
    got, err = run(q8d, dev(q), dev(kc), dev(vc), H, Hk, D, [L], cap, 1 / math.sqrt(D))
    assert err == 0
    close(got[0], ref, ab)


def test_one_row_returns_v(q8d):
    """L = 1: the softmax is 1 whatever the score, so the output is V's row."""
    H, Hk, D, cap = 8, 2, 128, 4
    kc, vc = (q4_cache(1, f"one.{x}", cap, Hk * D, noise=True, rows=1) for x in "kv")
    got, err = run(q8d, dev(synth.normal_f32(1, "one.q", H * D)), dev(kc), dev(vc), H, Hk, D, [1], cap, 0.3)
    assert err == 0
    want = kp.values(vc, Q4, Hk * D, cap)[0].reshape(Hk, 1, D).repeat(H // Hk, 1).reshape(-1)
    assert np.allclose(got[0], want, rtol=2 ** -21, atol=0)


@pytest.mark.parametrize("batch", [2, 5, 33, 70])
@pytest.mark.parametrize("cap", [515, 400])
def test_ragged_batch(q8d, orc, batch, cap):
    """Unequal lengths, strides with a gap, refused sequences among them, with
    sequences cut into pieces and whole."""
    H, Hk, D = 12, 2, 64
    width = Hk * D
    stride = -(-cap * width // 256) * 256 + 512
    lens = [1 + (i * 7919) % cap for i in range(batch)]
    lens[-1] = cap
    lens[batch // 2] = [0, cap + 1, -3, 2 ** 31 - 1][batch % 4]
    n = kp.cache_bytes(Q4, stride)
    kc, vc = (np.zeros((batch, n), np.uint8) for _ in range(2))
    for s in range(batch):
        for c, x in ((kc, "k"), (vc, "v")):
            one = q4_cache(s, f"rag.{x}", cap, width, max(0, min(cap, lens[s])), noise=True)
            c[s, :one.size] = one
    q = synth.normal_f32(0, "rag.q", (batch, H * D))
    got, err = run(q8d, dev(q), dev(kc), dev(vc), H, Hk, D, lens, cap, 0.125, stride)
    assert err == q8d.Q8D_DERR_LEN_RANGE
    for s in range(batch):
        if not 1 <= lens[s] <= cap:
            assert np.isnan(got[s]).all()
            continue
        ref, ab = oracle_attn(orc, q[s], kc[s], vc[s], H, Hk, D, cap, lens[s], 0.125)
        close(got[s], ref, ab)


@pytest.mark.parametrize("H,Hk,D", [(28, 4, 128), (14, 2, 64), (16, 8, 128), (16, 1, 64)])
def test_append_in_the_call(q8d, orc, H, Hk, D):
    """The new rows are stored as q8d_kv_append stores them and attended to."""
    cap, width = 200, Hk * D
    stride = -(-cap * width // 256) * 256
    lens = [1, 130, 200]
    n = kp.cache_bytes(Q4, stride)
    kc, vc = (np.zeros((3, n), np.uint8) for _ in range(2))
    for s in range(3):
        for c, x in ((kc, "k"), (vc, "v")):
            one = q4_cache(s, f"app.{x}", cap, width, lens[s] - 1, noise=True)
            c[s, :one.size] = one
    q = synth.normal_f32(0, "app.q", (3, H * D))
    kn, vn = synth.normal_f32(0, "app.kn", (3, width)), synth.normal_f32(0, "app.vn", (3, width))
    dk, dv = dev(kc), dev(vc)
    got, err = run(q8d, dev(q), dk, dv, H, Hk, D, lens, cap, 0.1, stride, dev(kn), dev(vn))
    assert err == 0
    for s in range(3):
        kp.store(kc[s], Q4, width, cap, lens[s] - 1, kn[s:s + 1])
        kp.store(vc[s], Q4, width, cap, lens[s] - 1, vn[s:s + 1])
        ref, ab = oracle_attn(orc, q[s], kc[s], vc[s], H, Hk, D, cap, lens[s], 0.1)
        close(got[s], ref, ab)
    assert np.array_equal(dk.cpu().numpy(), kc) and np.array_equal(dv.cpu().numpy(), vc)


def test_windows(q8d, orc):
    """Spans and run maps over one shared cache; runs of every length around
    the tiles', an empty window and one outside the cache refused."""
    H, Hk, D, cap = 8, 2, 128, 700
    kc, vc = (q4_cache(5, f"win.{x}", cap, Hk * D) for x in "kv")
    runs = [
        [[0, 700], [0, 0], [0, 0], [0, 0]],
        [[3, 5], [100, 1], [690, 10], [0, 2]],
        [[0, 0], [50, 33], [0, 0], [10, 257]],
        [[699, 1], [0, 0], [0, 0], [0, 0]],
        [[0, 0], [0, 0], [0, 0], [0, 0]],
        [[0, 4], [698, 3], [0, 0], [0, 0]],
        [[1, 31], [64, 32], [128, 15], [300, 17]],
    ]
    q = synth.normal_f32(0, "win.q", (len(runs), H * D))
    got, err = run(q8d, dev(q), dev(kc), dev(vc), H, Hk, D, None, cap, 0.09, stride=0, runs=runs)
    assert err == q8d.Q8D_DERR_LEN_RANGE
    for s, r in enumerate(runs):
        if s in (4, 5):
            assert np.isnan(got[s]).all()
            continue
        cells = np.concatenate([np.arange(c, c + n) for c, n in r])
        ref, ab = oracle_attn(orc, q[s], kc, vc, H, Hk, D, cap, cells.size, 0.09, cells)
        close(got[s], ref, ab)


def test_window_append(q8d, orc):
    """New rows go to the last row of each sequence's last run."""
    H, Hk, D, cap, width = 4, 2, 64, 96, 128
    kc, vc = (np.stack([q4_cache(s, f"wapp.{x}", cap, width) for s in range(2)]) for x in "kv")
    runs = [[[5, 20], [60, 7], [0, 0], [0, 0]], [[80, 16], [0, 3], [0, 0], [0, 0]]]
    at = [66, 2]
    q = synth.normal_f32(0, "wapp.q", (2, H * D))
    kn, vn = synth.normal_f32(0, "wapp.kn", (2, width)), synth.normal_f32(0, "wapp.vn", (2, width))
    dk, dv = dev(kc), dev(vc)
    got, err = run(q8d, dev(q), dk, dv, H, Hk, D, None, cap, 0.125, k_new=dev(kn), v_new=dev(vn), runs=runs)
    assert err == 0
    for s in range(2):
        kp.store(kc[s], Q4, width, cap, at[s], kn[s:s + 1])
        kp.store(vc[s], Q4, width, cap, at[s], vn[s:s + 1])
        cells = np.concatenate([np.arange(c, c + n) for c, n in runs[s]])
        ref, ab = oracle_attn(orc, q[s], kc[s], vc[s], H, Hk, D, cap, cells.size, 0.125, cells)
        close(got[s], ref, ab)
    assert np.array_equal(dk.cpu().numpy(), kc) and np.array_equal(dv.cpu().numpy(), vc)


@pytest.mark.parametrize("q_scale,v_scale", [(1e-6, 1e-4), (300.0, 3e4), (1e4, 1.0), (0.0, 1.0), (1.0, 0.0)])
def test_ranges_of_values(q8d, orc, q_scale, v_scale):
    """Queries and V scales far from 1, scales of both signs that change from
    row to row by orders of magnitude, rows of zeros.  A large q makes the
    softmax one-hot: its error is bounded by the scores' own, 2^-21 of
    scale * sum|q K|, so those cases use scores below 64 through `scale`."""
    H, Hk, D, cap = 12, 2, 128, 300
    width = Hk * D
    x = synth.normal_f32(0, "range.v", (cap, width)) * np.float32(v_scale)
    x *= (10.0 ** -(np.arange(cap) % 5)).astype(np.float32)[:, None]
    x[7] = 0
    kc, vc = np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8), np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8)
    kp.store(kc, Q4, width, cap, 0, synth.normal_f32(0, "range.k", (cap, width)))
    kp.store(vc, Q4, width, cap, 0, x)
    q = synth.normal_f32(0, "range.q", H * D) * np.float32(q_scale)
    scale = 1 / math.sqrt(D) / max(1.0, q_scale)
    ref, ab = oracle_attn(orc, q, kc, vc, H, Hk, D, cap, cap, scale)
    got, err = run(q8d, dev(q), dev(kc), dev(vc), H, Hk, D, [cap], cap, scale)
    assert err == 0
    assert np.isfinite(got).all()
    close(got[0], ref, ab + 1e-30)


def test_same_result_every_time_and_without_a_workspace(q8d):
    """No order of arrival enters the result; the noalloc entry point gives
    the same bits."""
    H, Hk, D, cap = 28, 4, 128, 3000
    kc, vc = (dev(q4_cache(2, f"rep.{x}", cap, Hk * D)) for x in "kv")
    q = dev(synth.normal_f32(2, "rep.q", H * D))
    first, _ = run(q8d, q, kc, vc, H, Hk, D, [2999], cap, 0.09)
    for _ in range(5):
        again, _ = run(q8d, q, kc, vc, H, Hk, D, [2999], cap, 0.09)
        assert np.array_equal(again, first)
    other, err = run(q8d, q, kc, vc, H, Hk, D, [2999], cap, 0.09, noalloc=True)
    assert err == 0 and np.array_equal(other, first)


def test_captured_and_replayed_at_growing_lengths(q8d, orc):
    """One graph of the call with its append, replayed token by token across
    tile and chunk borders."""
    H, Hk, D, cap = 14, 2, 64, 140
    width = Hk * D
    kc = np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8)
    vc = kc.copy()
    dk, dv = dev(kc), dev(vc)
    q, kn, vn = (torch.zeros(n, device="cuda") for n in (H * D, width, width))
    lens, err, out = ints([1]), ints([0]), torch.zeros(H * D, device="cuda")
    n = q8d.q8d_gqa_workspace_bytes(1, H, Hk, D, cap)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        q8d.q8d_gqa_decode_attn(q, kn, vn, dk, dv, Q4, out, 1, H, Hk, D, cap, 0, lens, 0.125, ws, n, err, st)
    for L in range(1, cap + 1):
        hq, hk, hv = (synth.normal_f32(L, f"grow.{x}", m) for x, m in (("q", H * D), ("k", width), ("v", width)))
        for d, h in ((q, hq), (kn, hk), (vn, hv)):
            d.copy_(dev(h))
        lens.fill_(L)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        kp.store(kc, Q4, width, cap, L - 1, hk[None])
        kp.store(vc, Q4, width, cap, L - 1, hv[None])
        ref, ab = oracle_attn(orc, hq, kc, vc, H, Hk, D, cap, L, 0.125)
        close(out.cpu().numpy(), ref, ab)
    assert err.item() == 0
    assert np.array_equal(dk.cpu().numpy(), kc) and np.array_equal(dv.cpu().numpy(), vc)


def test_cache_past_2_to_the_32_bytes(q8d, orc):
    """The last sequence of a batch starts beyond 4 GiB."""
    H, Hk, D, cap, batch = 8, 8, 128, 131072, 72
    width = Hk * D
    stride = cap * width
    n = kp.cache_bytes(Q4, stride)  # 75 MB a sequence, 5.4 GB in all
    kc, vc = (torch.zeros(batch, n, dtype=torch.uint8, device="cuda") for _ in range(2))
    lens = [1] * batch
    lens[-1] = 300
    one = [np.zeros(n, np.uint8) for _ in range(2)]
    for c, o, x in ((kc, one[0], "k"), (vc, one[1], "v")):
        kp.store(o, Q4, width, cap, 0, synth.normal_f32(0, f"far.{x}", (300, width)))
        c[-1].copy_(dev(o))
    q = synth.normal_f32(0, "far.q", (batch, H * D))
    got, err = run(q8d, dev(q), kc, vc, H, Hk, D, lens, cap, 0.09)
    assert err == 0
    small = [np.concatenate([o[:300 * width // 2], o[cap * width // 2:cap * width // 2 + 300 * width // 16]]) for o in one]
    ref, ab = oracle_attn(orc, q[-1], small[0], small[1], H, Hk, D, 300, 300, 0.09)
    close(got[-1], ref, ab)
    assert np.all(got[0] == 0)


@pytest.mark.parametrize("cap", [512, 513])
def test_refused_alone(q8d, cap):
    """One sequence without rows: NaN, and nothing else is read."""
    H, Hk, D = 20, 2, 128
    kc, vc = (dev(q4_cache(4, f"ref.{x}", cap, Hk * D)) for x in "kv")
    q = dev(synth.normal_f32(4, "ref.q", H * D))
    for L in (0, -1, cap + 1):
        got, err = run(q8d, q, kc, vc, H, Hk, D, [L], cap, 0.1)
        assert err == q8d.Q8D_DERR_LEN_RANGE and np.isnan(got).all()


@pytest.mark.parametrize("H,Hk,D,cap,batch,kind", [
    (4, 2, 64, 6000, 40, "one long"), (3, 1, 128, 3000, 9, "one long"), (2, 2, 64, 128, 130, "short caches"),
    (96, 96, 64, 300, 7, "more heads than CTAs"), (160, 160, 64, 600, 3, "more heads than CTAs"),
    (200, 200, 64, 520, 1, "more heads than CTAs"), (16, 1, 64, 500, 35, "even"), (4, 4, 128, 130, 90, "two slots"),
    (8, 8, 64, 90, 2, "short caches"),
])
def test_batches_cut_into_pieces(q8d, orc, H, Hk, D, cap, batch, kind):
    """Pieces that hold many short sequences, sequences of many pieces among
    one-row ones, caches with a single workspace slot; nothing is written
    behind the workspace."""
    width = Hk * D
    stride = -(-cap * width // 256) * 256
    lens = [1 + (i * 613) % cap for i in range(batch)]
    if kind == "one long":
        lens = [1 + i % 3 for i in range(batch)]
        lens[batch // 3] = cap
    kc, vc = (np.zeros((batch, kp.cache_bytes(Q4, stride)), np.uint8) for _ in range(2))
    for s in range(batch):
        for c, x in ((kc, "k"), (vc, "v")):
            one = q4_cache(s, f"cut.{x}", cap, width, lens[s], noise=True)
            c[s, :one.size] = one
    q = synth.normal_f32(0, "cut.q", (batch, H * D))
    n = q8d.q8d_gqa_workspace_bytes(batch, H, Hk, D, cap)
    ws = torch.full((n // 4 + 1024,), 7.0, device="cuda")
    out, err = torch.full((batch, H * D), -7.0, device="cuda"), ints([0])
    q8d.q8d_gqa_decode_attn(dev(q), None, None, dev(kc), dev(vc), Q4, out, batch, H, Hk, D, cap, stride, ints(lens),
                            0.11, ws, n, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.all(ws[(n + 3) // 4:] == 7.0)
    for s in range(batch):
        ref, ab = oracle_attn(orc, q[s], kc[s], vc[s], H, Hk, D, cap, lens[s], 0.11)
        close(out[s].cpu().numpy(), ref, ab)
