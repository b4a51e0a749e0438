"""Operands that are columns of one buffer's rows: the numbers of operands that lie
apart, and nothing else of the buffer written."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev
from test_q4_gpu import Matrix

pytestmark = pytest.mark.gpu
F32, F16, Q8_0 = kp.F32, kp.F16, kp.Q8_0


@pytest.mark.parametrize("dtype,kind", [(torch.float32, F32), (torch.float16, F16)])
@pytest.mark.parametrize("rows,n,gap", [(1, 64, 0), (300, 128, 0), (40, 33, 1), (7, 100, 28), (513, 3584, 4)])
def test_norm(q8d, dtype, kind, rows, n, gap):
    """x | gap | y | gap | r (which becomes the sums) in one buffer."""
    ld = 3 * n + 2 * gap
    buf = dev(synth.normal_f32(1, "cols.x", (rows, ld))).to(dtype)
    w = dev((1 + 0.1 * synth.normal_f32(2, "cols.w", n)).astype(np.float32))
    x, y, r = 0, n + gap, 2 * (n + gap)
    apart = [buf[:, c:c + n].contiguous() for c in (x, r)]
    y0, s0 = (torch.empty(rows, n, dtype=dtype, device="cuda") for _ in range(2))
    q8d.q8d_rmsnorm_rows(apart[0], apart[1], s0, kind, n, n, n, w, 1e-6, y0, kind, n, rows, n)
    want = buf.clone()
    flat = buf.view(-1)
    q8d.q8d_rmsnorm_rows(flat, flat[r:], flat[r:], kind, ld, ld, ld, w, 1e-6, flat[y:], kind, ld, rows, n)
    torch.cuda.synchronize()
    want[:, y:y + n], want[:, r:r + n] = y0, s0
    assert torch.equal(buf, want)


@pytest.mark.parametrize("m", [1, 5, 16])
@pytest.mark.parametrize("p,n", [(48, 64), (1000, 3584)])
def test_product(q8d, m, p, n):
    """X | Y | residual in one buffer."""
    ld = n + 2 * (p + -p % 4)
    W = Matrix(q8d, 3, p, n, 32)
    buf = dev(synth.normal_f32(4, "cols.m", (m, ld)))
    Y, R = n, n + p + -p % 4
    x, res, y0 = buf[:, :n].contiguous(), buf[:, R:R + p].contiguous(), torch.empty(m, p, device="cuda")
    q8d.q8d_q4_matmul(x, F32, n, W.bytes, 32, None, res, p, y0, p, m, n, p)
    want = buf.clone()
    flat = buf.view(-1)
    q8d.q8d_q4_matmul(flat, F32, ld, W.bytes, 32, None, flat[R:], ld, flat[Y:], ld, m, n, p)
    torch.cuda.synchronize()
    want[:, Y:Y + p] = y0
    assert torch.equal(buf, want)


def test_rotary_rows(q8d):
    """q | k | v | turned q in one buffer."""
    H, HK, D, rows = 4, 2, 64, 37
    ld = (2 * H + 2 * HK) * D
    buf = dev(synth.normal_f32(5, "cols.q", (rows, ld)))
    table = torch.empty(rows, D, device="cuda")
    q8d.q8d_rope_table(table, rows, D, 1e4, 0, 1.0, 0.0, 0.0, 0.0, 1.0)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(out, ldo):
        kc, vc = (torch.zeros(rows, HK * D, device="cuda") for _ in range(2))
        desc = q8d.rope_desc(n_heads=H, n_kv_heads=HK, head_dim=D, rot_dim=D, layout=0, max_pos=rows, row_dtype=F32,
                             q_dtype=F32, kv_dtype=F32, cap=rows, eps=1e-6, ldq=ld, ldkv=ld, ldo=ldo,
                             cache_batch_stride=rows * HK * D, table=table)
        f = buf.view(-1)
        q8d.q8d_rope_append_rows(desc, f, f[H * D:], f[(H + HK) * D:], out, kc, vc, 1, rows, pos, None, None, None)
        return kc, vc
    apart = torch.empty(rows, H * D, device="cuda")
    k0, v0 = call(apart, H * D)
    want = buf.clone()
    at = (H + 2 * HK) * D
    want[:, at:] = apart
    k1, v1 = call(buf.view(-1)[at:], ld)
    torch.cuda.synchronize()
    assert torch.equal(buf, want) and torch.equal(k1, k0) and torch.equal(v1, v0)
