"""Operands whose byte or element offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
F32, F16, Q8_0, Q4 = kp.F32, kp.F16, kp.Q8_0, kp.Q4


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_norm_rows_far_apart(q8d):
    n, ld, rows = 256, 1 << 28, 12  # f16: rows 2^29 bytes apart, the last at 5.9 GB
    x = synth.normal_f32(90, "far.x", (rows, n)).astype(np.float16)
    buf = torch.empty((rows - 1) * ld + n, dtype=torch.float16, device="cuda")
    out = torch.empty_like(buf)
    view, oview = (torch.as_strided(t, (rows, n), (ld, 1)) for t in (buf, out))
    view.copy_(dev(x))
    w = dev(np.ones(n, np.float32))
    near = torch.empty(rows, n, dtype=torch.float16, device="cuda")
    q8d.q8d_rmsnorm_rows(buf, buf, buf, F16, ld, ld, ld, w, 1e-6, out, F16, ld, rows, n)
    q8d.q8d_rmsnorm_rows(dev(x), dev(x), None, F16, n, n, n, w, 1e-6, near, F16, n, rows, n)
    torch.cuda.synchronize()
    assert torch.equal(oview, near) and torch.equal(view, dev((x + x).astype(np.float16)))


@pytest.mark.parametrize("kind", [F16, Q8_0, Q4])
def test_cache_rows_far_out(q8d, kind):
    H, HK, D, cap, rows = 2, 8, 128, 4_300_000, 3  # 4.4e9 elements a cache
    w = HK * D
    nb = kp.cache_bytes(kind, cap * w)
    kc, vc = (torch.zeros(nb, dtype=torch.uint8, device="cuda") for _ in range(2))
    small = [torch.zeros(kp.cache_bytes(kind, 8 * w), dtype=torch.uint8, device="cuda") for _ in range(2)]
    p = dev(synth.normal_f32(91, "far.p", (rows, H * D + 2 * w)))
    table = torch.empty(16, D, device="cuda")
    q8d.q8d_rope_table(table, 16, D, 1e4, 0, 1.0, 0, 0, 0, 1.0)
    out = [torch.empty(rows, H * D, device="cuda") for _ in range(2)]
    read = [torch.empty(2, rows, w, device="cuda") for _ in range(2)]
    err = ints([0])
    for i, (c, first, caches) in enumerate(((cap, cap - rows, (kc, vc)), (8, 5, small))):
        desc = q8d.rope_desc(n_heads=H, n_kv_heads=HK, head_dim=D, rot_dim=D, layout=0, max_pos=16, row_dtype=F32, q_dtype=F32,
                             kv_dtype=kind, cap=c, eps=1e-6, ldq=p.stride(0), ldkv=p.stride(0), ldo=H * D,
                             cache_batch_stride=0, table=table)
        q8d.q8d_rope_append_rows(desc, p, p[:, H * D:], p[:, H * D + w:], out[i], *caches, 1, rows, ints([first]), ints([9]),
                                 None, err)
        q8d.q8d_kv_read_rows(*caches, kind, read[i][0], read[i][1], F32, w, 1, rows, w, c, 0, ints([first]), None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.equal(out[0], out[1]) and torch.equal(read[0], read[1]) and read[0].abs().sum() > 0


def tile_values(tile, group):
    """f64 [16, 128] of one tile's bytes, from the layout's definition."""
    out = np.zeros((16, 128))
    words = tile[:1024].view("<u4").reshape(2, 8, 4, 4)  # half, g, t, block of 32 columns
    scales = tile[1024:].view("<f2").reshape(8, 2, 128 // group).astype(np.float64)  # g, half
    for h in range(2):
        for g in range(8):
            for t in range(4):
                for b in range(4):
                    for e in range(8):
                        col = 32 * b + 8 * t + e
                        n = words[h, g, t, b] >> (4 * (e // 2 + 4 * (e % 2))) & 15
                        out[g + 8 * h, col] = scales[g, h, col // group] * (int(n) - 8)
    return out


@pytest.mark.parametrize("group", [32, 128])
def test_matrix_past_4_gb(q8d, group):
    """Rows behind the first 4 GB of a matrix, decoded here from the bytes."""
    p, n = 520_000, 16384
    rec = 1024 + 16 * (128 // group) * 2
    strips, tiles = -(-p // 16), n // 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    w = torch.randint(0, 256, (strips, tiles, rec), dtype=torch.uint8, device="cuda", generator=gen)
    assert w.numel() == q8d.q8d_q4_matrix_bytes(p, n, group) > 1 << 32
    scale = (0.005 + 0.01 * torch.rand(strips, tiles, (rec - 1024) // 2, device="cuda", generator=gen)).half()
    w[:, :, 1024:] = scale.view(torch.uint8)
    x = dev(synth.normal_f32(92, "far.xq", (2, n)))
    y = torch.empty(2, p, device="cuda")
    q8d.q8d_q4_matmul(x, F32, n, w, group, None, None, 0, y, p, 2, n, p)
    torch.cuda.synchronize()
    v = x.cpu().numpy().astype(np.float64)
    for s in (0, strips // 2, strips - 1):
        W = np.concatenate([tile_values(t, group) for t in w[s].cpu().numpy()], 1)
        got = y[:, 16 * s:16 * s + 16].cpu().numpy()
        assert np.all(np.abs(got - v @ W.T) <= 1e-5 * (np.abs(v) @ np.abs(W).T))


def test_output_rows_far_apart(q8d):
    p, n, m, ld = 40, 64, 3, 1 << 30
    w = torch.empty(q8d.q8d_q4_matrix_bytes(p, n, 32), dtype=torch.uint8, device="cuda")
    src = dev(synth.normal_f32(93, "far.w", (p, n)))
    q8d.q8d_q4_pack(src, F32, n, w, p, n, 32)
    x = dev(synth.normal_f32(94, "far.y", (m, n)))
    far = torch.empty((m - 1) * ld + p, device="cuda")
    near = torch.empty(m, p, device="cuda")
    q8d.q8d_q4_matmul(x, F32, n, w, 32, None, None, 0, far, ld, m, n, p)
    q8d.q8d_q4_matmul(x, F32, n, w, 32, None, None, 0, near, p, m, n, p)
    torch.cuda.synchronize()
    assert torch.equal(torch.as_strided(far, (m, p), (ld, 1)), near)
