"""4-bit attention where the terms that make up an output lie far below others
of the same head: a token that takes the softmax but has no V, blocks of one
head whose scales lie far apart, a V that is zero in most dims.

Queries have one nonzero dim a head, and K's element there is its block's
largest (stored exactly), so a score is one product: off by the roundings of
scale * log2(e) and of q times it (2^-24 each, and 2^-24 of the constant), and
the split of the query into two f16 parts (2^-22), under 2^-21 of its
magnitude; a probability by that many nats.  The tolerance is the other
tests' 1e-5 sum_t p_t |V_t|, plus that."""
import numpy as np
import pytest

import kvplain as kp
import synth
from conftest import dev
from test_attn_q4kv_gpu import Q4, TOL, oracle_attn, run

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 128), (4, 4, 64), (7, 1, 128), (8, 1, 64), (16, 1, 128), (12, 1, 64)]
SINKS = slice(5, None, 32)  # one in every tile of 32 rows


def scores_cache(width, D, cap, score):
    """K with `score` at dim 0 of every head, smaller elements elsewhere."""
    x = synth.normal_f32(0, "wide.k", (cap, width)).clip(-3, 3) * np.float32(2 ** -6)
    for g in range(width // D):
        x[:, g * D] = score
        x[:, g * D + 1:g * D + 32] *= np.minimum(1, np.abs(score) * 4)[:, None]
    c = np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8)
    kp.store(c, Q4, width, cap, 0, x)
    v = kp.values(c, Q4, width, cap)
    assert np.array_equal(v[:, ::D], np.repeat(score[:, None], width // D, 1))
    return c


def check(q8d, orc, H, Hk, D, score, v):
    """score: nats above any constant, one a row."""
    cap, width = v.shape
    kc = scores_cache(width, D, cap, score)
    vc = np.zeros_like(kc)
    kp.store(vc, Q4, width, cap, 0, v)
    q = np.zeros((H, D), np.float32)
    q[:, 0] = 1 + np.arange(H, dtype=np.float32) / 64
    ref, ab = oracle_attn(orc, q.ravel(), kc, vc, H, Hk, D, cap, cap, 1.0)
    assert np.all(ab > 0)
    got, err = run(q8d, dev(q.ravel()), dev(kc), dev(vc), H, Hk, D, [cap], cap, 1.0)
    assert err == 0
    tol = TOL + 2.0 ** -21 * np.abs(score).max() * q.max()
    assert np.all(np.abs(got[0] - ref) <= tol * ab), (np.abs(got[0] - ref) / ab).max() / tol


def two_levels(cap, bits):
    """Scores of -1 .. 1 nats, and sinks `bits` doublings above them."""
    s = synth.stream(1, "wide.s").uniform(-1, 1, cap)
    s[SINKS] = bits * np.log(2)
    return (np.round(s * 32) / 32).astype(np.float32)  # (eighths of them are f16 values)


@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("bits", [10, 15, 20, 30, 60])
@pytest.mark.parametrize("cap", [300, 700])
def test_rows_that_take_the_softmax_without_a_v(q8d, orc, H, Hk, D, bits, cap):
    v = synth.normal_f32(2, "wide.v", (cap, Hk * D))
    v[SINKS] = 0
    check(q8d, orc, H, Hk, D, two_levels(cap, bits), v)


@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("bits", [10, 20, 30])
def test_rows_that_take_the_softmax_with_few_dims(q8d, orc, H, Hk, D, bits):
    """The sinks' V is one element a block; every other dim comes from rows of
    far smaller weight."""
    cap = 600
    v = synth.normal_f32(2, "wide.v", (cap, Hk * D))
    v[SINKS] = 0
    v[SINKS, ::32] = 1
    check(q8d, orc, H, Hk, D, two_levels(cap, bits), v)


@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("bits", [8, 14, 20, 26])
def test_blocks_of_a_head_far_apart(q8d, orc, H, Hk, D, bits):
    """Neighbouring blocks' scales `bits` doublings apart."""
    cap = 300
    v = synth.normal_f32(3, "wide.b", (cap, Hk * D)).reshape(cap, -1, 32)
    v[:, ::2] *= np.float32(2.0 ** 12)
    v[:, 1::2] *= np.float32(2.0 ** (12 - bits))
    check(q8d, orc, H, Hk, D, two_levels(cap, 1), v.reshape(cap, -1))


@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("bits", [8, 14, 20, 26])
def test_rows_far_apart(q8d, orc, H, Hk, D, bits):
    """The softmax lies on rows whose V is `bits` doublings below that of rows
    it leaves out."""
    cap = 300
    v = synth.normal_f32(3, "wide.b", (cap, Hk * D)) * np.float32(2.0 ** 12)
    v[SINKS] *= np.float32(2.0 ** -bits)
    check(q8d, orc, H, Hk, D, two_levels(cap, 60), v)
