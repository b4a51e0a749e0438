"""The 4-bit store inside the attention call where a block's largest magnitude
occurs with both signs: the first of them sets the scale, as in the other
stores.  Stored bytes have to be equal; the outputs keep the tolerance of
test_attn_q4kv_gpu.py."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev
from test_attn_q4kv_gpu import Q4, close, ints, oracle_attn, run

pytestmark = pytest.mark.gpu


def opposite_pairs(width, seed):
    """Rows of `width` whose blocks hold +a and -a at every pair of places, in
    both orders, among smaller elements."""
    pairs = [(i, j) for i in range(32) for j in range(32) if i != j]
    per = width // 32
    n = -(-len(pairs) // per)
    x = synth.stream(seed, "ties").uniform(-0.9, 0.9, (n * per, 32)).astype(np.float32)
    for b, (i, j) in enumerate(pairs):
        x[b, i], x[b, j] = 1.25, -1.25
    return x.reshape(n, width)


def to_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().float().numpy()


def rows_of(kind, width):
    if kind == "pairs":
        return opposite_pairs(width, 1), opposite_pairs(width, 2)[::-1]
    return tuple(to_bf16(synth.normal_f32(0, f"ties.{x}", (64, width))) for x in "kv")


@pytest.mark.parametrize("kind", ["pairs", "bf16"])
@pytest.mark.parametrize("H,Hk,D,cap", [(16, 8, 128, 40), (14, 2, 64, 40), (16, 1, 128, 520)])
def test_append_in_the_call_with_ties(q8d, orc, H, Hk, D, cap, kind):
    width = Hk * D
    kn, vn = (np.ascontiguousarray(x) for x in rows_of(kind, width))
    batch = kn.shape[0]
    stride = -(-cap * width // 256) * 256
    n = kp.cache_bytes(Q4, stride)
    lens = [1 + (7 * s) % cap for s in range(batch)]
    kc, vc = (np.zeros((batch, n), np.uint8) for _ in range(2))
    for c, x in ((kc, "k"), (vc, "v")):
        kp.store(c[0], Q4, width, cap, 0, synth.normal_f32(0, f"ties.c{x}", (cap, width)))
        c[1:] = c[0]
    q = synth.normal_f32(0, "ties.q", (batch, H * D))
    dk, dv, rk, rv = dev(kc), dev(vc), dev(kc), dev(vc)
    got, err = run(q8d, dev(q), dk, dv, H, Hk, D, lens, cap, 0.1, stride, dev(kn), dev(vn))
    assert err == 0
    e = ints([0])
    q8d.q8d_kv_append_rows(dev(kn), dev(vn), kp.F32, width, rk, rv, Q4, batch, 1, width, cap, stride,
                           ints([L - 1 for L in lens]), None, e)
    torch.cuda.synchronize()
    for s in range(batch):
        kp.store(kc[s], Q4, width, cap, lens[s] - 1, kn[s:s + 1])
        kp.store(vc[s], Q4, width, cap, lens[s] - 1, vn[s:s + 1])
    for d, r, c in ((dk, rk, kc), (dv, rv, vc)):
        assert np.array_equal(r.cpu().numpy(), c)
        assert np.array_equal(d.cpu().numpy(), c)
    for s in range(0, batch, 5):
        ref, ab = oracle_attn(orc, q[s], kc[s], vc[s], H, Hk, D, cap, lens[s], 0.1)
        close(got[s], ref, ab)


@pytest.mark.parametrize("kind", ["pairs", "bf16"])
def test_window_append_with_ties(q8d, kind):
    """The same through run maps: the row goes to the last row of the last run."""
    H, Hk, D, cap, width = 4, 2, 64, 96, 128
    kn, vn = (np.ascontiguousarray(x) for x in rows_of(kind, width))
    batch = kn.shape[0]
    kc, vc = (np.zeros((batch, kp.cache_bytes(Q4, cap * width)), np.uint8) for _ in range(2))
    runs = [[[5, 20], [60, 1 + s % 30], [0, 0], [0, 0]] for s in range(batch)]
    dk, dv = dev(kc), dev(vc)
    _, err = run(q8d, dev(synth.normal_f32(0, "ties.wq", (batch, H * D))), dk, dv, H, Hk, D, None, cap, 0.125,
                 stride=cap * width, k_new=dev(kn), v_new=dev(vn), runs=runs)
    assert err == 0
    for s in range(batch):
        kp.store(kc[s], Q4, width, cap, 60 + s % 30, kn[s:s + 1])
        kp.store(vc[s], Q4, width, cap, 60 + s % 30, vn[s:s + 1])
    assert np.array_equal(dk.cpu().numpy(), kc) and np.array_equal(dv.cpu().numpy(), vc)
