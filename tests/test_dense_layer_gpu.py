"""A dense layer with 4-bit weights as a serving program runs it from calls:
norm, projections with biases, rotary positions and the cache, attention,
projection back into the stream, norm into 8 bits, gated projections, projection
back; prompts of unequal lengths, then tokens of the whole batch, eagerly and as
a captured graph.

Each operator is held against the f64 form of its own inputs as the device made
them, at its own contract (a rounding that tips a code would else change
everything after it)."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev
from test_q4_gpu import Matrix, q8_values
from test_rope_gpu import turn

pytestmark = pytest.mark.gpu

H, HK, D, ROT, CAP, HIDDEN, FFN, GROUP = 8, 2, 64, 32, 96, 384, 992, 64
WIDTH, BATCH, QKV = HK * D, 3, (H + 2 * HK) * D
STRIDE = -(-CAP * WIDTH // 256) * 256
PROMPTS = [40, 1, 0]
EPS = 1e-6
LDY = -(-HIDDEN // 256) * 256


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def host(t):
    return t.cpu().numpy()


class Layer:
    def __init__(self, q8d, kind, st=None):
        self.q8d, self.kind, self.st = q8d, kind, st
        self.qkv, self.o = Matrix(q8d, 70, QKV, HIDDEN, GROUP), Matrix(q8d, 71, HIDDEN, H * D, GROUP)
        self.g, self.u = Matrix(q8d, 72, FFN, HIDDEN, GROUP, 2.0), Matrix(q8d, 73, FFN, HIDDEN, GROUP)
        self.d = Matrix(q8d, 74, HIDDEN, FFN, GROUP)
        self.bias = (0.1 * synth.normal_f32(75, "dense.b", QKV)).astype(np.float32)
        self.w = [(1 + 0.1 * synth.normal_f32(76 + i, "dense.n", n)).astype(np.float32) for i, n in
                  enumerate((HIDDEN, HIDDEN, D, D))]
        self.dbias, self.dw = dev(self.bias), [dev(w) for w in self.w]
        self.table = torch.empty(CAP, ROT, device="cuda")
        q8d.q8d_rope_table(self.table, CAP, ROT, 1e4, q8d.Q8D_ROPE_PLAIN, 1.0, 0, 0, 0, 1.0)
        n = kp.cache_bytes(kind, STRIDE)
        self.kc, self.vc = (torch.zeros(BATCH, n, dtype=torch.uint8, device="cuda") for _ in range(2))
        rows = max(PROMPTS) * BATCH
        z = lambda *shape: torch.zeros(*shape, device="cuda")  # noqa: E731
        self.x, self.delta, self.h1, self.p = z(rows, HIDDEN), z(rows, HIDDEN), z(rows, HIDDEN), z(rows, QKV)
        self.q, self.a, self.x2, self.h = z(rows, H * D), z(BATCH, H * D), z(BATCH, HIDDEN), z(BATCH, FFN)
        self.h8 = torch.zeros(BATCH, LDY // 32 * 34, dtype=torch.uint8, device="cuda")
        self.pos, self.count, self.lens, self.err = ints([0] * BATCH), ints(PROMPTS), ints(PROMPTS), ints([0])
        self.ws = torch.empty(q8d.q8d_gqa_workspace_bytes(BATCH, H, HK, D, CAP), dtype=torch.uint8, device="cuda")
        self.desc = q8d.rope_desc(n_heads=H, n_kv_heads=HK, head_dim=D, rot_dim=ROT, layout=q8d.Q8D_ROPE_HALF, max_pos=CAP,
                                  row_dtype=kp.F32, q_dtype=kp.F32, kv_dtype=kind, cap=CAP, eps=EPS, ldq=QKV, ldkv=QKV,
                                  ldo=H * D, cache_batch_stride=STRIDE, table=self.table, q_norm=self.dw[2],
                                  k_norm=self.dw[3])
        torch.cuda.synchronize()

    def qkv_rows(self, rows, per_sequence, counts):
        """The first half of the layer on `rows` rows of the stream: norm of x, projections, positions, cache."""
        q8d, st = self.q8d, self.st
        q8d.q8d_rmsnorm_rows(self.x, None, None, kp.F32, HIDDEN, HIDDEN, HIDDEN, self.dw[0], EPS, self.h1, kp.F32, HIDDEN,
                             rows, HIDDEN, st)
        for r in range(0, rows, 16):
            m = min(16, rows - r)
            q8d.q8d_q4_matmul(self.h1[r:], kp.F32, HIDDEN, self.qkv.bytes, GROUP, self.dbias, None, 0, self.p[r:], QKV, m,
                              HIDDEN, QKV, st)
        q8d.q8d_rope_append_rows(self.desc, self.p, self.p[:, H * D:], self.p[:, H * D + WIDTH:], self.q, self.kc, self.vc,
                                 BATCH, per_sequence, self.pos, None, counts, self.err, st)

    def decode(self):
        """One token of every sequence: x becomes the layer's output."""
        q8d, st, m = self.q8d, self.st, BATCH
        self.qkv_rows(m, 1, None)
        q8d.q8d_gqa_decode_attn(self.q, None, None, self.kc, self.vc, self.kind, self.a, m, H, HK, D, CAP, STRIDE, self.lens,
                                0.125, self.ws, self.ws.numel(), self.err, st)
        q8d.q8d_q4_matmul(self.a, kp.F32, H * D, self.o.bytes, GROUP, None, None, 0, self.delta, HIDDEN, m, H * D, HIDDEN, st)
        # (the sum goes on as the stream, the norm of it into 8 bits)
        q8d.q8d_rmsnorm_rows(self.delta, self.x, self.x2, kp.F32, HIDDEN, HIDDEN, HIDDEN, self.dw[1], EPS, self.h8, kp.Q8_0,
                             LDY, m, HIDDEN, st)
        q8d.q8d_q4_gated(self.h8, kp.Q8_0, LDY, self.g.bytes, self.u.bytes, GROUP, self.h, FFN, m, HIDDEN, FFN, st)
        q8d.q8d_q4_matmul(self.h, kp.F32, FFN, self.d.bytes, GROUP, None, self.x2, HIDDEN, self.x2, HIDDEN, m, FFN, HIDDEN, st)


def near_product(got, x, W, tol=1e-5, more=0.0):
    x = x.astype(np.float64)
    assert np.all(np.abs(got - more - x @ W.values.T) <= tol * (np.abs(x) @ np.abs(W.values).T + np.abs(more)))


def norm_steps(x, w):
    x = x.astype(np.float32)
    inv = (1 / np.sqrt(np.square(x.astype(np.float64)).mean(-1, keepdims=True) + np.float64(np.float32(EPS))))
    return ((x * inv.astype(np.float32)).astype(np.float32) * w).astype(np.float32)


def head_steps(x, w, table):
    x = norm_steps(x.reshape(len(x), -1, D), w)
    t = table[:, None]
    return turn(x, t[..., :ROT // 2], t[..., ROT // 2:], ROT, 0, True).reshape(len(x), -1)


def check_stored(L, cache, s, first, rows):
    """Rows `rows` of the projection's output are the f32 steps' in the plain cache (updated), and q is theirs."""
    if len(rows) == 0:
        return
    p, table = host(L.p)[rows], host(L.table)[first:first + len(rows)]
    kp.store(cache[0][s], L.kind, WIDTH, CAP, first, head_steps(p[:, H * D:H * D + WIDTH], L.w[3], table))
    kp.store(cache[1][s], L.kind, WIDTH, CAP, first, p[:, H * D + WIDTH:])
    # (the f32 steps themselves: a factor may differ by one unit, so two of them and the products')
    q = head_steps(p[:, :H * D], L.w[2], table)
    assert np.all(np.abs(host(L.q)[rows] - q) <= 4 * 2.0 ** -24 * np.abs(q).max())


@pytest.mark.parametrize("kind", [kp.F16, kp.Q8_0, kp.Q4])
def test_prompt_then_tokens(q8d, orc, kind):
    L = Layer(q8d, kind)
    longest = max(PROMPTS)
    prompt = dev(synth.normal_f32(80, "dense.prompt", (BATCH * longest, HIDDEN)))
    L.x.copy_(prompt)
    torch.cuda.synchronize()
    L.qkv_rows(BATCH * longest, longest, L.count)
    torch.cuda.synchronize()
    cache = [np.zeros(tuple(L.kc.shape), np.uint8) for _ in range(2)]
    for s, n in enumerate(PROMPTS):
        check_stored(L, cache, s, 0, np.arange(s * longest, s * longest + n))
    assert np.array_equal(host(L.kc), cache[0]) and np.array_equal(host(L.vc), cache[1])
    inputs, outputs = [], []
    L.x[:BATCH].copy_(dev(synth.normal_f32(81, "dense.x", (BATCH, HIDDEN))))
    for step in range(20):
        L.pos.copy_(L.lens)
        L.lens.add_(1)
        torch.cuda.synchronize()
        L.decode()
        torch.cuda.synchronize()
        x, h1, p, q, a, delta, h8, h, x2 = (host(t)[:BATCH] for t in (L.x, L.h1, L.p, L.q, L.a, L.delta, L.h8, L.h, L.x2))
        assert np.array_equal(h1, norm_steps(x, L.w[0]))
        near_product(p, h1, L.qkv, more=L.bias.astype(np.float64))
        for s in range(BATCH):
            n = PROMPTS[s] + step + 1
            check_stored(L, cache, s, n - 1, np.array([s]))
            vals = [np.ascontiguousarray(kp.values(c[s], kind, WIDTH, CAP).astype(np.float32)) for c in cache]
            ref, ab = orc.gqa_decode_attn(q[s], vals[0], vals[1], kp.F32, H, HK, D, n, 0.125)
            assert np.all(np.abs(a[s] - ref) <= 1e-5 * ab)
        near_product(delta, a, L.o)
        stream = (delta + x).astype(np.float32)
        want8 = kp.q8_blocks(norm_steps(stream, L.w[1]).reshape(BATCH, -1, 32)).reshape(BATCH, -1)
        assert np.array_equal(h8[:, :HIDDEN // 32 * 34], want8)
        v = q8_values(want8)
        g, u = v @ L.g.values.T, v @ L.u.values.T
        gt, ut = (1e-5 * (np.abs(v) @ np.abs(W.values).T) for W in (L.g, L.u))
        silu = g / (1 + np.exp(-g))
        assert np.all(np.abs(h - silu * u) <= 1.1 * gt * (np.abs(u) + ut) + np.abs(silu) * ut + 2.0 ** -20 * np.abs(silu * u))
        near_product(x2, h, L.d, more=stream.astype(np.float64))
        inputs.append(x.copy())
        outputs.append(x2.copy())
        y = L.x2 / L.x2.square().mean(1, keepdim=True).sqrt()
        L.x[:BATCH].copy_(y)
    assert np.array_equal(host(L.kc), cache[0]) and np.array_equal(host(L.vc), cache[1])

    # the same tokens through one captured graph: the same bits
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    G = Layer(q8d, kind, st)
    G.x.copy_(prompt)
    torch.cuda.synchronize()
    G.qkv_rows(BATCH * longest, longest, G.count)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        G.decode()
    for x, y in zip(inputs, outputs):
        G.pos.copy_(G.lens)
        G.lens.add_(1)
        G.x[:BATCH].copy_(dev(x))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(G.x2), y)
    assert torch.equal(G.kc, L.kc) and torch.equal(G.vc, L.vc)
    assert L.err.item() == 0 and G.err.item() == 0


def test_two_layers_on_two_streams(q8d):
    """Two layers in turn on two streams give the bits each gives alone."""
    alone = Layer(q8d, kp.Q8_0)
    x = dev(synth.normal_f32(82, "dense.two", (BATCH, HIDDEN)))
    alone.x[:BATCH].copy_(x)
    alone.pos.copy_(ints([3, 0, 7]))
    alone.lens.copy_(ints([4, 1, 8]))
    torch.cuda.synchronize()
    alone.decode()
    torch.cuda.synchronize()
    pair = [Layer(q8d, kp.Q8_0, torch.cuda.Stream()) for _ in range(2)]
    for L in pair:
        L.x[:BATCH].copy_(x)
        L.pos.copy_(alone.pos)
        L.lens.copy_(alone.lens)
    torch.cuda.synchronize()
    for _ in range(20):
        for L in pair:
            L.decode()
    torch.cuda.synchronize()
    for L in pair:
        assert L.err.item() == 0
        assert torch.equal(L.x2, alone.x2) and torch.equal(L.kc, alone.kc) and torch.equal(L.vc, alone.vc)
