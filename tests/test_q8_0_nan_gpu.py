"""Rows that hold a NaN or an infinity on their way into Q8_0 blocks: the block's
scale says so, the blocks and rows beside it keep their bytes, and a product that
reads such a row is no finite number."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev
from test_norm_gpu import rows_of, steps
from test_q4_gpu import Matrix

pytestmark = pytest.mark.gpu
F32, F16, Q8_0 = kp.F32, kp.F16, kp.Q8_0


def scales(b):
    return np.ascontiguousarray(b.reshape(len(b), -1, 34)[..., :2]).view(np.float16)[..., 0]


def same(got, rows):
    """Blocks without a NaN byte by byte, those with one by their scale."""
    x = rows.reshape(len(rows), -1, 32)
    bad = np.isnan(x).any(-1)
    want = kp.q8_blocks(np.where(bad[..., None], np.float32(0), x))
    got = got.reshape(want.shape)
    assert np.isnan(scales(got.reshape(len(got), -1))[bad]).all()
    assert np.array_equal(got[~bad], want[~bad])


@pytest.mark.parametrize("kind", [F32, F16])
@pytest.mark.parametrize("n,offset", [(32, 0), (160, 0), (160, 1), (3584, 0), (16384, 0)])
def test_norm(q8d, kind, n, offset):
    x = synth.normal_f32(1, "nan8.x", (9, n))
    for i, v in ((1, np.nan), (3, np.inf), (4, -np.inf)):
        x[i, n // 2] = v
    x[6, ::7] = np.nan
    x = x.astype(np.float32 if kind == F32 else np.float16)
    w = (1 + 0.1 * synth.normal_f32(2, "nan8.w", n)).astype(np.float32)
    y = torch.full((9, n // 32 * 34), 7, dtype=torch.uint8, device="cuda")
    q8d.q8d_rmsnorm_rows(rows_of(x, kind, n, offset), None, None, kind, n, 0, 0, dev(w), 1e-6, y, Q8_0, n, 9, n)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        _, want = steps(x, None, w, 1e-6)
    same(y.cpu().numpy(), want)
    # what reads them: rows of the product, and of the gated pair
    W, U = Matrix(q8d, 3, 40, n, 32), Matrix(q8d, 4, 40, n, 32)
    out, h = torch.zeros(9, 40, device="cuda"), torch.zeros(9, 40, device="cuda")
    q8d.q8d_q4_matmul(y, Q8_0, n, W.bytes, 32, None, None, 0, out, 40, 9, n, 40)
    q8d.q8d_q4_gated(y, Q8_0, n, W.bytes, U.bytes, 32, h, 40, 9, n, 40)
    torch.cuda.synchronize()
    broken = np.isnan(want).any(1)
    for o in (out, h):
        assert np.array_equal(~torch.isfinite(o).all(1).cpu().numpy(), broken)
        assert not torch.isfinite(o[torch.from_numpy(broken).cuda()]).any()


def test_norm_weights(q8d):
    """A NaN among the weights: its block of every row."""
    n = 96
    x, w = synth.normal_f32(5, "nan8.x", (4, n)), np.ones(n, np.float32)
    w[40] = np.nan
    y = torch.full((4, 102), 7, dtype=torch.uint8, device="cuda")
    q8d.q8d_rmsnorm_rows(dev(x), None, None, F32, n, 0, 0, dev(w), 1e-6, y, Q8_0, n, 4, n)
    torch.cuda.synchronize()
    same(y.cpu().numpy(), steps(x, None, w, 1e-6)[1])


@pytest.mark.parametrize("kind", [F32, F16])
def test_cache_rows(q8d, kind):
    """Rows into a packed cache, many at once and one by one: the same bytes."""
    w, cap = 128, 6
    k, v = (synth.normal_f32(6, s, (cap, w)).astype(np.float32 if kind == F32 else np.float16) for s in "kv")
    k[2, 70], v[3, 0], v[4, 31] = np.nan, np.nan, -np.nan
    kc, vc, k1, v1 = (torch.zeros(cap, w // 32 * 34, dtype=torch.uint8, device="cuda") for _ in range(4))
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    err = ints([0])
    q8d.q8d_kv_append_rows(dev(k), dev(v), kind, w, kc, vc, Q8_0, 1, cap, w, cap, cap * w, ints([0]), None, err)
    for i in range(cap):
        q8d.q8d_kv_append(dev(k[i].astype(np.float32)), dev(v[i].astype(np.float32)), k1, v1, Q8_0, w, cap, ints([i]), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for many, one, rows in ((kc, k1, k), (vc, v1, v)):
        same(many.cpu().numpy(), rows.astype(np.float32))
        assert torch.equal(many, one)
