"""Attention calls over more rows than their kernels count: refused on the host
where the cache is too long, and by the device where run maps add up to too
many.  The caches here are a few rows long whatever `cap` says: nothing of a
refused sequence is read."""
import numpy as np
import pytest

BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from q8_block_quantized_matvec_gb300 import build
    build.build()
    import q8_block_quantized_matvec_gb300 as m
    m.lib()
    return m


def test_cache_of_more_rows_than_32_bits_hold(lib):
    A = 0x100000

    def attn(cap, kv):
        return lib.lib().q8d_gqa_decode_attn(A, None, None, A, A, kv, A, 1, 2, 2, 64, cap, 0, A, 0.125, A, 0, None, None)

    def window(cap, kv):
        return lib.lib().q8d_gqa_decode_attn_window(A, None, None, A, A, kv, A, 1, 2, 2, 64, cap, 0, A, 0.125, A, 0, None, None)

    for call in (attn, window):
        assert call(BIG + 1, 4) == lib.Q8D_EUNSUPPORTED
        assert call(2 ** 31 - 1, 4) == lib.Q8D_EUNSUPPORTED
        assert call(BIG, 4) == lib.Q8D_ERANGE       # (no workspace)
        assert call(2 ** 31 - 1, 1) == lib.Q8D_ERANGE  # other caches


@pytest.mark.gpu
@pytest.mark.parametrize("kv,cap,runs", [
    (4, BIG, [[0, BIG], [0, 1], [0, 0], [0, 0]]),
    (4, BIG, [[0, BIG], [0, BIG], [0, BIG], [0, BIG]]),                   # 2^32: wraps to 0
    (4, BIG // 2 + 9, [[0, BIG // 2 + 9], [9, BIG // 2], [0, 0], [0, 0]]),
    (0, BIG, [[0, BIG], [0, BIG], [0, 0], [0, 0]]),                       # 2^31
    (1, BIG + 64, [[0, BIG + 64]] * 4),                                   # wraps to 256
    (2, BIG + 64, [[0, BIG + 64]] * 4),
])
def test_windows_of_too_many_rows(q8d, kv, cap, runs):
    import torch
    H, Hk, D = 4, 2, 64
    kc, vc = (torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    out = torch.zeros(2, H * D, device="cuda")
    err, r = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0], [runs] * 2))
    n = q8d.q8d_gqa_workspace_bytes(2, H, Hk, D, cap)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    q8d.q8d_gqa_decode_attn_window(torch.ones(2, H * D, device="cuda"), None, None, kc, vc, kv, out, 2, H, Hk, D, cap, 0,
                                   r, 0.125, ws, n, err)
    torch.cuda.synchronize()
    assert err.item() == q8d.Q8D_DERR_LEN_RANGE
    assert np.isnan(out.cpu().numpy()).all()
    assert not kc.any() and not vc.any()
