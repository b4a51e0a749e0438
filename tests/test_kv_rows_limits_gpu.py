"""Rows at the limits of their widths and values."""
import numpy as np
import pytest
import torch

import kvplain as kp
from conftest import dev
from test_attn_q4kv_gpu import ints

pytestmark = pytest.mark.gpu
F16, F32, Q4 = kp.F16, kp.F32, kp.Q4


@pytest.mark.parametrize("kind", [F16, F32])
def test_the_widest_rows(q8d, kind):
    """One row of 2^31 - 1 halves each (4 GiB), stored and read back."""
    n = 2 ** 31 - 1
    gen = torch.Generator(device="cuda").manual_seed(0)
    rows = [torch.randint(0, 0x7c00, (n,), generator=gen, dtype=torch.int16, device="cuda") for _ in range(2)]
    size = q8d.q8d_kv_cache_bytes(kind, n, 1)
    guard = 256
    caches = [torch.full((size + guard,), 0x11, dtype=torch.uint8, device="cuda") for _ in range(2)]
    err, zero = ints([0]), ints([0])
    q8d.q8d_kv_append_rows(*rows, F16, n, *caches, kind, 1, 1, n, 1, 0, zero, None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for c, r in zip(caches, rows):
        assert torch.all(c[size:] == 0x11)
        if kind == F16:
            assert torch.equal(c[:size].view(torch.int16), r)
        else:
            for a in range(0, n, 1 << 28):
                got = c[4 * a:min(size, 4 * (a + (1 << 28)))].view(torch.float32)
                assert torch.equal(got, r[a:a + (1 << 28)].view(torch.float16).float())
    outs = [torch.full((n + 64,), -7, dtype=torch.int16, device="cuda") for _ in range(2)]
    q8d.q8d_kv_read_rows(*caches, kind, *outs, F16, n, 1, 1, n, 1, 0, zero, None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for o, r in zip(outs, rows):
        assert torch.equal(o[:n], r) and torch.all(o[n:] == -7)


@pytest.mark.parametrize("top,finite", [(524159.9, True), (524160.0, False), (524287.0, False)])
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_element_with_a_finite_scale(q8d, top, finite, sign):
    """A scale is the largest element / -8 as binary16: infinite from 65520 on."""
    width, cap = 64, 3
    x = np.ones((1, width), np.float32)
    x[0, 40] = sign * np.float32(top)
    kc, vc = (torch.zeros(kp.cache_bytes(Q4, cap * width), dtype=torch.uint8, device="cuda") for _ in range(2))
    err = ints([0])
    q8d.q8d_kv_append_rows(dev(x), dev(x), F32, width, kc, vc, Q4, 1, 1, width, cap, 0, ints([1]), None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    want = np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8)
    kp.store(want, Q4, width, cap, 1, x)
    assert np.array_equal(kc.cpu().numpy(), want) and np.array_equal(vc.cpu().numpy(), want)
    scale = kc.cpu().numpy()[cap * width // 2:].view(np.float16).reshape(cap, 2)[1, 1]
    assert np.isfinite(scale) == finite
