"""The 4-bit cache, its attention and the expert layer as a serving program
runs them: prompts of unequal lengths stored, then tokens decoded for the
whole batch, eagerly and as one captured graph, then a sequence moved to
another slot.

Each operator is held against the f64 form of its own inputs as the device
made them, at its own contract: 1e-5 of the sum of |terms| for a product and
for the attention, the expert layer's tolerance as in its own tests (a
rounding that tips a 4-bit quant or an expert's rank would else change
everything after it)."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev
from test_moe_gpu import dequant, ints, layer, plain

pytestmark = pytest.mark.gpu

H, HK, D, CAP, HIDDEN, FFN, E, TOP = 8, 2, 64, 96, 384, 160, 24, 4
WIDTH, BATCH = HK * D, 3
STRIDE = -(-CAP * WIDTH // 256) * 256
PROMPTS = [40, 1, 0]


class Layer:
    def __init__(self, q8d, st=None):
        self.q8d, self.st = q8d, st
        s = 1 / (73 * np.sqrt(HIDDEN))
        self.w = {n: synth.q8_matrix(60, "lay." + n, p, k, 0.5 * s, 1.5 * s)
                  for n, p, k in (("q", H * D, HIDDEN), ("k", WIDTH, HIDDEN), ("v", WIDTH, HIDDEN), ("o", HIDDEN, H * D))}
        self.experts = layer(61, E, HIDDEN, FFN)
        self.dw = {n: dev(w) for n, w in self.w.items()}
        self.de = [dev(w) for w in self.experts]
        n = kp.cache_bytes(kp.Q4, STRIDE)
        self.kc, self.vc = (torch.zeros(BATCH, n, dtype=torch.uint8, device="cuda") for _ in range(2))
        zeros = lambda *shape: torch.zeros(*shape, device="cuda")
        self.x, self.o, self.y = zeros(BATCH, HIDDEN), zeros(BATCH, HIDDEN), zeros(BATCH, HIDDEN)
        self.q, self.k, self.v, self.a = zeros(BATCH, H * D), zeros(BATCH, WIDTH), zeros(BATCH, WIDTH), zeros(BATCH, H * D)
        self.lens, self.err = ints(PROMPTS), ints([0])
        self.attn_ws = torch.empty(q8d.q8d_gqa_workspace_bytes(BATCH, H, HK, D, CAP), dtype=torch.uint8, device="cuda")
        self.moe_ws = torch.empty(q8d.q8d_moe_workspace_bytes(BATCH, HIDDEN, FFN, E, TOP), dtype=torch.uint8,
                                  device="cuda")

    def prompt(self):
        """The prompts' K and V rows, padded to the longest, stored at 0."""
        rows = max(PROMPTS)
        x = dev(synth.normal_f32(62, "lay.prompt", (BATCH * rows, HIDDEN)))
        k, v = (torch.empty(BATCH * rows, WIDTH, device="cuda") for _ in range(2))
        for dst, n in ((k, "k"), (v, "v")):
            for r in range(0, BATCH * rows, 64):
                m = min(64, BATCH * rows - r)
                self.q8d.q8d_matmul_small_m(x[r:], HIDDEN, self.dw[n], dst[r:], WIDTH, m, HIDDEN, WIDTH, self.st)
        self.q8d.q8d_kv_append_rows(k, v, kp.F32, WIDTH, self.kc, self.vc, kp.Q4, BATCH, rows, WIDTH, CAP, STRIDE,
                                    ints([0] * BATCH), ints(PROMPTS), self.err, self.st)
        torch.cuda.synchronize()
        return k.view(BATCH, rows, WIDTH), v.view(BATCH, rows, WIDTH)

    def decode(self):
        """One token of every sequence (lens: the lengths with it)."""
        m, st = BATCH, self.st
        mm = self.q8d.q8d_matmul_small_m
        for dst, n, p in ((self.q, "q", H * D), (self.k, "k", WIDTH), (self.v, "v", WIDTH)):
            mm(self.x, HIDDEN, self.dw[n], dst, p, m, HIDDEN, p, st)
        self.q8d.q8d_gqa_decode_attn(self.q, self.k, self.v, self.kc, self.vc, kp.Q4, self.a, m, H, HK, D, CAP, STRIDE,
                                     self.lens, 0.125, self.attn_ws, self.attn_ws.numel(), self.err, st)
        mm(self.a, H * D, self.dw["o"], self.o, HIDDEN, m, H * D, HIDDEN, st)
        self.q8d.q8d_moe_ffn(self.o, HIDDEN, *self.de, self.x, HIDDEN, self.y, HIDDEN, m, HIDDEN, FFN, E, TOP, 1, None,
                             None, self.moe_ws, self.moe_ws.numel(), self.err, st)


def host(t):
    return t.cpu().numpy()


def test_prompt_then_tokens(q8d, orc):
    L = Layer(q8d)
    kp_rows, vp_rows = L.prompt()
    cache = {}
    for n, d, rows in (("k", L.kc, kp_rows), ("v", L.vc, vp_rows)):
        want = np.zeros(tuple(d.shape), np.uint8)
        for s in range(BATCH):
            kp.store(want[s], kp.Q4, WIDTH, CAP, 0, host(rows)[s, :PROMPTS[s]])
        assert np.array_equal(host(d), want)
        cache[n] = want
    inputs, outputs = [], []
    L.x.copy_(dev(synth.normal_f32(63, "lay.x", (BATCH, HIDDEN))))
    for step in range(35):  # (across the borders of the 32-row tiles)
        L.lens.add_(1)
        torch.cuda.synchronize()
        L.decode()
        torch.cuda.synchronize()
        x, q, k, v, a, o, y = (host(t) for t in (L.x, L.q, L.k, L.v, L.a, L.o, L.y))
        inputs.append(x)
        outputs.append(y)
        for got, src, n, p, kk in ((q, x, "q", H * D, HIDDEN), (k, x, "k", WIDTH, HIDDEN), (o, a, "o", HIDDEN, H * D)):
            W = dequant(L.w[n], p, kk)
            assert np.all(np.abs(got - src.astype(np.float64) @ W.T) <= 1e-5 * (np.abs(src) @ np.abs(W).T))
        for s in range(BATCH):
            n = PROMPTS[s] + step + 1
            kp.store(cache["k"][s], kp.Q4, WIDTH, CAP, n - 1, k[s:s + 1])
            kp.store(cache["v"][s], kp.Q4, WIDTH, CAP, n - 1, v[s:s + 1])
            vals = [np.ascontiguousarray(kp.values(cache[c][s], kp.Q4, WIDTH, CAP)) for c in "kv"]
            ref, ab = orc.gqa_decode_attn(q[s], vals[0], vals[1], kp.F32, H, HK, D, n, 0.125)
            assert np.all(np.abs(a[s] - ref) <= 1e-5 * ab)
        _, _, ref, tol = plain(L.experts, o, E, HIDDEN, FFN, TOP, True, x)
        assert np.all(np.abs(y - ref) <= tol)
        L.x.copy_(L.y / L.y.square().mean(1, keepdim=True).sqrt())
    assert np.array_equal(host(L.kc), cache["k"]) and np.array_equal(host(L.vc), cache["v"])

    # the same tokens through one captured graph: the same bits
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    G = Layer(q8d, st)
    G.prompt()
    with torch.cuda.graph(g, stream=st):
        G.decode()
    for x, y in zip(inputs, outputs):
        G.lens.add_(1)
        G.x.copy_(dev(x))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(G.y), y)
    assert torch.equal(G.kc, L.kc) and torch.equal(G.vc, L.vc)
    assert L.err.item() == 0 and G.err.item() == 0

    # sequence 0 moves into slot 2 through f32 rows: 4-bit values come back to
    # the same bytes, and the next token is the same
    n = PROMPTS[0] + len(inputs)
    k, v = (torch.empty(1, n, WIDTH, device="cuda") for _ in range(2))
    q8d.q8d_kv_read_rows(L.kc, L.vc, kp.Q4, k, v, kp.F32, WIDTH, 1, n, WIDTH, CAP, STRIDE, ints([0]), None, L.err)
    q8d.q8d_kv_append_rows(k, v, kp.F32, WIDTH, L.kc[2], L.vc[2], kp.Q4, 1, n, WIDTH, CAP, STRIDE, ints([0]), None,
                           L.err)
    L.lens.copy_(ints([n + 1, n + 1, n + 1]))
    L.x[2].copy_(L.x[0])
    torch.cuda.synchronize()
    assert torch.equal(L.kc[0], L.kc[2]) and torch.equal(L.vc[0], L.vc[2])
    L.decode()
    torch.cuda.synchronize()
    assert L.err.item() == 0
    assert torch.equal(L.kc[0], L.kc[2])
    # (a batch's pieces cut its sequences in different places: equal to f32's accuracy)
    assert torch.allclose(L.a[0], L.a[2], rtol=1e-4, atol=1e-5)


def test_two_layers_on_two_streams(q8d):
    """Two layers with workspaces of their own, launched in turn on two
    streams, give the bits each gives alone."""
    alone = Layer(q8d)
    alone.prompt()
    x = dev(synth.normal_f32(64, "two.x", (BATCH, HIDDEN)))
    alone.x.copy_(x)
    alone.lens.add_(1)
    torch.cuda.synchronize()
    alone.decode()
    torch.cuda.synchronize()
    pair = [Layer(q8d, torch.cuda.Stream()) for _ in range(2)]
    for L in pair:
        L.prompt()
        L.x.copy_(x)
        L.lens.add_(1)
    torch.cuda.synchronize()
    for _ in range(20):  # (the same token again and again: it overwrites its own row)
        for L in pair:
            L.decode()
    torch.cuda.synchronize()
    for L in pair:
        assert L.err.item() == 0
        assert torch.equal(L.y, alone.y) and torch.equal(L.kc, alone.kc) and torch.equal(L.vc, alone.vc)
