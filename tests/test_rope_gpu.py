"""q8d_rope_table and q8d_rope_append_rows against the formulas: the table in
64 bits, q rows in 64 bits, and the caches byte by byte against the plain store
of rows worked out in f32 steps.

Tolerances: a table entry is rounded once, 2^-24 of its value (and angles in 64
bits: pos * f is off by 2^-53 pos f).  A rotated value is two products and a sum
of rounded factors: 2^-24 (|a cos| + |b sin|) for each of cosine's, product's and
sum's roundings; a norm before adds its 5 * 2^-24 of the terms, a bias 2^-24."""
import math

import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
F32, F16, Q8_0, Q4 = kp.F32, kp.F16, kp.Q8_0, kp.Q4
KINDS = [F32, F16, Q8_0, Q4]
NP = {F32: np.float32, F16: np.float16}
EPS = 1e-6
PLAIN, LINEAR, NTK, YARN = range(4)
HALF, PAIRS = 0, 1


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def frequencies(rot, theta, scaling, factor, orig, fast, slow):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == NTK:
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if scaling == LINEAR:
        return f / factor
    if scaling == YARN:
        at = lambda t: rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp)
    return f


def table64(max_pos, rot, mscale, *scaling):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * frequencies(rot, *scaling)
    return np.concatenate([np.cos(a), np.sin(a)], 1) * mscale


@pytest.mark.parametrize("max_pos,rot,mscale,scaling", [
    (1, 2, 1.0, (1e4, PLAIN, 1.0, 0, 0, 0)),
    (4097, 128, 1.0, (1e6, PLAIN, 1.0, 0, 0, 0)),
    (300, 20, 1.0, (1e4, LINEAR, 8.0, 0, 0, 0)),
    (2000, 64, 1.0, (1e4, NTK, 4.0, 0, 0, 0)),
    (131072, 128, 0.1 * math.log(4.0) + 1, (1e6, YARN, 4.0, 32768, 32.0, 1.0)),
    (5000, 32, 1.25, (1e4, YARN, 16.0, 256, 32.0, 1.0)),
])
def test_table(q8d, max_pos, rot, mscale, scaling):
    t = torch.full((max_pos * rot + 8,), 9.0, device="cuda")
    theta, kind, factor, orig, fast, slow = scaling
    q8d.q8d_rope_table(t, max_pos, rot, theta, kind, factor, orig, fast, slow, mscale)
    torch.cuda.synchronize()
    want = table64(max_pos, rot, mscale, *scaling)
    got = t[:max_pos * rot].view(max_pos, rot).cpu().numpy().astype(np.float64)
    # (frequencies by two pow functions: 2^-52 of them, times the position)
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -50 * max_pos * mscale + 2.0 ** -149)
    assert torch.all(t[max_pos * rot:] == 9)


def turn(x, cos, sin, rot, layout, step):
    """Heads [..., dim] turned; step: f32 steps, else 64 bits."""
    f = (lambda v: v.astype(np.float32)) if step else (lambda v: v)
    out = x.copy()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == HALF else (x[..., 0:rot:2], x[..., 1:rot:2])
    ya, yb = f(f(a * cos) - f(b * sin)), f(f(a * sin) + f(b * cos))
    if layout == HALF:
        out[..., :rot // 2], out[..., rot // 2:rot] = ya, yb
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = ya, yb
    return out


class Case:
    def __init__(self, q8d, H, HK, D, rot, layout, kind, batch, rows, cap, starts, counts, rope=None, src=F32, bias=False,
                 norm=False, fused=True, offset=0, qd=F32, max_pos=None, in_place=False):
        self.__dict__.update(locals())
        self.w, self.max_pos = HK * D, max_pos or cap
        rng = synth.stream(7, "rope.rows")
        self.q = rng.standard_normal((batch * rows, H * D)).astype(NP[src])
        self.k, self.v = (rng.standard_normal((batch * rows, self.w)).astype(NP[src]) for _ in range(2))
        self.b = [(0.1 * rng.standard_normal(n)).astype(np.float32) for n in (H * D, self.w, self.w)] if bias else [None] * 3
        self.g = [(1 + 0.1 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)] if norm else [None] * 2
        self.stride = -(-cap * self.w // 256) * 256
        self.before = rng.integers(0, 256, (2, batch, kp.cache_bytes(kind, self.stride)), dtype=np.uint8)
        self.scaling = (1e4, PLAIN, 1.0, 0, 0, 0)
        self.table = torch.empty(self.max_pos, max(rot, 2), device="cuda")
        if rot:
            q8d.q8d_rope_table(self.table, self.max_pos, rot, 1e4, PLAIN, 1.0, 0, 0, 0, 1.0)
        self.kc, self.vc = dev(self.before[0]), dev(self.before[1])
        if fused:
            ld = H * D + 2 * self.w
            both = np.concatenate([self.q, self.k, self.v], 1)
            buf = dev(np.concatenate([np.zeros(offset, NP[src]), both.reshape(-1)]))[offset:]
            dq, dk, dv, ldq, ldkv = buf, buf[H * D:], buf[H * D + self.w:], ld, ld
        else:
            dq, dk, dv, ldq, ldkv = dev(self.q), dev(self.k), dev(self.v), H * D, self.w
        self.ldo = ldq if in_place else H * D + 4
        self.out = dq if in_place else torch.full((batch * rows * self.ldo,), 3.0, device="cuda",
                                                  dtype=torch.float16 if qd == F16 else torch.float32)
        up = [None if a is None else dev(a) for a in self.b + self.g]
        self.desc = q8d.rope_desc(n_heads=H, n_kv_heads=HK, head_dim=D, rot_dim=rot, layout=layout, max_pos=self.max_pos,
                                  row_dtype=src, q_dtype=qd, kv_dtype=kind, cap=cap, eps=EPS, ldq=ldq, ldkv=ldkv, ldo=self.ldo,
                                  cache_batch_stride=self.stride, table=self.table if rot else None, bq=up[0], bk=up[1],
                                  bv=up[2], q_norm=up[3], k_norm=up[4])
        self.err = ints([0])
        self.args = (dq, dk, dv)
        self.call = lambda st=None: q8d.q8d_rope_append_rows(
            self.desc, dq, dk, dv, self.out, self.kc, self.vc, batch, rows, ints(starts), ints(rope), ints(counts), self.err, st)

    def head_rows(self, x, b, g, pos, step):
        f = (lambda v: v.astype(np.float32)) if step else (lambda v: v)
        x = x.astype(np.float32 if step else np.float64)
        if b is not None:
            x = f(x + b)
        if g is None and pos is None:
            return x
        x = x.reshape(len(x), x.shape[1] // self.D, self.D)
        if g is not None:
            inv = f(1 / np.sqrt(np.square(x.astype(np.float64)).mean(-1, keepdims=True) + np.float64(np.float32(EPS))))
            x = f(f(x * inv) * g)
        if self.rot:
            # (the table's own values: they have a test of their own)
            t = self.table.cpu().numpy()[pos][:, None].astype(x.dtype)
            x = turn(x, t[..., :self.rot // 2], t[..., self.rot // 2:], self.rot, self.layout, step)
        return x.reshape(len(x), x.shape[1] * self.D)

    def check(self):
        torch.cuda.synchronize()
        want = self.before.copy()
        out = self.out.cpu().numpy().astype(np.float64)
        H, D, rows = self.H, self.D, self.rows
        for s in range(self.batch):
            n = rows if self.counts is None else self.counts[s]
            at = slice(s * rows, s * rows + n)
            first = self.starts[s] if self.rope is None else self.rope[s]
            pos = np.arange(first, first + n)
            kp.store(want[0, s], self.kind, self.w, self.cap, self.starts[s],
                     self.head_rows(self.k[at], self.b[1], self.g[1], pos, True))
            v = self.v[at].astype(np.float32)
            kp.store(want[1, s], self.kind, self.w, self.cap, self.starts[s],
                     v if self.b[2] is None else (v + self.b[2]).astype(np.float32))
            ref = self.head_rows(self.q[at], self.b[0], self.g[0], pos, False)
            # the sum of |terms| of a rotated value: |a| + |b| of its pair covers cos and sin
            mag = np.abs(self.head_rows(self.q[at], self.b[0], self.g[0], None if self.g[0] is None else pos * 0, False))
            mag = mag.reshape(n, H, D)
            pair = mag.copy()
            r = self.rot
            if self.layout == HALF:
                pair[..., :r // 2] += mag[..., r // 2:r]
                pair[..., r // 2:r] += mag[..., :r // 2]
            else:
                pair[..., 0:r:2] += mag[..., 1:r:2]
                pair[..., 1:r:2] += mag[..., 0:r:2]
            pair = pair.reshape(n, H * D)
            if self.b[0] is not None:
                pair = pair + np.abs(self.q[at].astype(np.float64)) + np.abs(self.b[0])
            for i in range(n):
                got = out[(s * rows + i) * self.ldo:][:H * D]
                tol = 9 * 2.0 ** -24 * pair[i] + (2.0 ** -11 * np.abs(ref[i]) + 2.0 ** -24 if self.qd == F16 else 0)
                assert np.all(np.abs(got - ref[i]) <= tol), (s, i)
            if not self.in_place:
                rest = out[:self.batch * rows * self.ldo].reshape(self.batch * rows, self.ldo)
                assert np.all(rest[:, H * D:] == 3) and np.all(rest[s * rows + n:(s + 1) * rows] == 3)
        assert np.array_equal(self.kc.cpu().numpy(), want[0])
        assert np.array_equal(self.vc.cpu().numpy(), want[1])
        assert self.err.item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("H,HK,D,rot,batch,rows,cap,starts,counts", [
    (4, 2, 64, 64, 1, 1, 1, [0], None),
    (28, 4, 128, 128, 3, 2, 40, [38, 0, 7], [2, 1, 0]),
    (6, 2, 96, 96, 2, 5, 9, [4, 0], [5, 3]),
    (6, 2, 96, 24, 2, 5, 9, [4, 1], None),        # halves that cut a lane's elements
    (2, 1, 256, 128, 2, 3, 8, [5, 0], [3, 1]),
    (3, 3, 160, 20, 1, 4, 4, [0], None),
    (16, 8, 128, 64, 5, 1, 30, [29, 3, 0, 9, 1], None),
    (1, 1, 32, 0, 2, 2, 4, [2, 0], None),         # nothing turns
    (14, 2, 64, 32, 3, 700, 900, [200, 0, 111], [700, 1, 689]),
])
def test_rows(q8d, kind, layout, H, HK, D, rot, batch, rows, cap, starts, counts):
    c = Case(q8d, H, HK, D, rot, layout, kind, batch, rows, cap, starts, counts)
    c.call()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", [
    dict(bias=True), dict(norm=True), dict(bias=True, norm=True, src=F16), dict(src=F16, qd=F16), dict(fused=False),
    dict(offset=1), dict(offset=3, src=F16, norm=True), dict(rope=[90, 2], max_pos=128), dict(in_place=True),
    dict(in_place=True, offset=1, norm=True)])
@pytest.mark.parametrize("D,rot,layout", [(128, 128, HALF), (64, 16, PAIRS), (96, 40, HALF)])
def test_rows_options(q8d, kind, kw, D, rot, layout):
    c = Case(q8d, 5, 2, D, rot, layout, kind, 2, 6, 20, [14, 3], [6, 4], **kw)
    c.call()
    c.check()


@pytest.mark.parametrize("kind", [F32, F16])
@pytest.mark.parametrize("D,rot", [(8, 8), (24, 10), (40, 40), (200, 2)])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_of_narrow_heads(q8d, kind, D, rot, norm):
    c = Case(q8d, 9, 3, D, rot, HALF, kind, 2, 3, 5, [2, 0], None, norm=norm)
    c.call()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_refused_sequences(q8d, kind):
    """Bad counts, rows and positions: the bit is set, nothing of the sequence
    is stored, its q rows are NaN, the others are as ever."""
    starts, counts = [0, 5, -1, 18, 3, 2], [2, 3, 1, 3, -1, 0]
    c = Case(q8d, 4, 2, 64, 64, HALF, kind, 6, 3, 20, starts, counts)
    c.call()
    torch.cuda.synchronize()
    assert c.err.item() == q8d.Q8D_DERR_LEN_RANGE | q8d.Q8D_DERR_POS_RANGE
    out = c.out.view(6, 3, -1)[..., :256]
    assert torch.isnan(out[2:5]).all() and not torch.isnan(out[:2]).any() and torch.all(out[5] == 3)
    assert torch.equal(c.kc[2:], dev(c.before[0, 2:])) and torch.equal(c.vc[2:], dev(c.before[1, 2:]))
    assert not torch.equal(c.kc[1], dev(c.before[0, 1]))
    for rope, max_pos in ([0, 62], 64), ([-1, 0], 64):
        c = Case(q8d, 4, 2, 64, 64, HALF, kind, 2, 3, 20, [0, 1], None, rope=rope, max_pos=max_pos)
        c.call()
        torch.cuda.synchronize()
        bad = 1 if rope[0] == 0 else 0
        assert c.err.item() == q8d.Q8D_DERR_POS_RANGE
        assert torch.isnan(c.out.view(2, 3, -1)[bad, :, :256]).all()
        assert not torch.isnan(c.out.view(2, 3, -1)[1 - bad, :, :256]).any()
        assert torch.equal(c.kc[bad], dev(c.before[0, bad]))


def test_q_alone_and_k_alone(q8d):
    c = Case(q8d, 4, 2, 64, 64, HALF, F16, 2, 3, 20, [7, 0], None)
    c.call()
    d = Case(q8d, 4, 2, 64, 64, HALF, F16, 2, 3, 20, [7, 0], None)
    q, k, v = d.args
    q8d.q8d_rope_append_rows(d.desc, q, None, None, d.out, None, None, 2, 3, ints([7, 0]), None, None, d.err)
    torch.cuda.synchronize()
    assert torch.equal(d.out, c.out) and torch.equal(d.kc, dev(d.before[0]))
    d.out.fill_(3)
    q8d.q8d_rope_append_rows(d.desc, None, k, v, None, d.kc, d.vc, 2, 3, ints([7, 0]), None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(d.kc, c.kc) and torch.equal(d.vc, c.vc) and torch.all(d.out == 3)


def test_rows_in_a_graph(q8d):
    """Positions live on the device: a captured call serves every step."""
    c = Case(q8d, 4, 2, 64, 64, HALF, Q4, 2, 1, 20, [0, 3], None)
    pos, st, g = ints([0, 3]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q, k, v = c.args
    with torch.cuda.graph(g, stream=st):
        q8d.q8d_rope_append_rows(c.desc, q, k, v, c.out, c.kc, c.vc, 2, 1, pos, None, None, c.err, st)
    for step in range(5):
        g.replay()
        torch.cuda.synchronize()
        want = Case(q8d, 4, 2, 64, 64, HALF, Q4, 2, 1, 20, [step, 3 + step], None)
        want.call()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want.out)
        pos.add_(1)
    assert c.err.item() == 0


def test_more_sequences_than_a_grid_is_high(q8d):
    batch = 70_000
    c = Case(q8d, 1, 1, 8, 8, PAIRS, F16, batch, 1, 32, [i % 32 for i in range(batch)], None, max_pos=40)
    c.call()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    pos = np.arange(batch) % 32
    k = c.head_rows(c.k, None, None, pos, True).astype(np.float16)
    got = c.kc.view(torch.float16).view(batch, -1).cpu().numpy()[:, :32 * 8].reshape(batch, 32, 8)
    before = c.before[0].view(np.float16).reshape(batch, -1)[:, :32 * 8].reshape(batch, 32, 8).copy()
    before[np.arange(batch), pos] = k
    assert np.array_equal(got.view(np.uint16), before.view(np.uint16))
