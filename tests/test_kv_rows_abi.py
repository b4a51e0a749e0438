"""Refusals of the row store, the read-back and the 4-bit cache on the host:
every call here is rejected before anything touches a device."""
import pytest

A, B, C_, D_, E = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000  # fake, aligned addresses


@pytest.fixture(scope="module")
def q8d():
    from q8_block_quantized_matvec_gb300 import build
    build.build()
    import q8_block_quantized_matvec_gb300 as m
    m.lib()
    return m


def args(**kw):
    a = dict(k=A, v=B, row_dtype=0, ld=64, kc=C_, vc=D_, kv_dtype=4, batch=2, rows=4, width=64, cap=8,
             stride=512, pos=E, counts=None, err=None)
    a.update(kw)
    return a


def append(q8d, **kw):
    a = args(**kw)
    return q8d.lib().q8d_kv_append_rows(a["k"], a["v"], a["row_dtype"], a["ld"], a["kc"], a["vc"], a["kv_dtype"],
                                        a["batch"], a["rows"], a["width"], a["cap"], a["stride"], a["pos"],
                                        a["counts"], a["err"], None)


def read(q8d, **kw):
    a = args(**kw)
    return q8d.lib().q8d_kv_read_rows(a["kc"], a["vc"], a["kv_dtype"], a["k"], a["v"], a["row_dtype"], a["ld"],
                                      a["batch"], a["rows"], a["width"], a["cap"], a["stride"], a["pos"],
                                      a["counts"], a["err"], None)


@pytest.mark.parametrize("call", [append, read])
def test_row_refusals(q8d, call):
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    for nm in ("k", "v", "kc", "vc", "pos"):
        assert call(q8d, **{nm: None}) == EINVAL
    assert call(q8d, batch=0) == EINVAL
    assert call(q8d, rows=-1) == EINVAL
    assert call(q8d, width=0) == EINVAL
    assert call(q8d, cap=0) == EINVAL
    assert call(q8d, ld=63) == EINVAL
    assert call(q8d, stride=-256) == EINVAL
    assert call(q8d, stride=256) == EINVAL                        # sequences would overlap
    assert call(q8d, kv_dtype=3) == EUNS
    assert call(q8d, kv_dtype=-1) == EUNS
    assert call(q8d, row_dtype=2) == EUNS                         # rows are f32 or f16
    assert call(q8d, width=48, ld=48) == EUNS                     # whole blocks
    assert call(q8d, kv_dtype=2, width=48, ld=48) == EUNS
    assert call(q8d, stride=528) == EALIGN                        # no whole block
    assert call(q8d, stride=544) == EALIGN                        # starts off 16 bytes
    assert call(q8d, kc=C_ + 8) == EALIGN
    assert call(q8d, vc=D_ + 2) == EALIGN
    assert call(q8d, k=A + 2) == EALIGN
    assert call(q8d, v=B + 1, row_dtype=1) == EALIGN
    assert call(q8d, pos=E + 2) == EALIGN
    assert call(q8d, counts=E + 1) == EALIGN
    assert call(q8d, vc=C_ + 16) == EINVAL                        # the caches overlap
    assert call(q8d, kc=A + 64) == EINVAL                         # a cache overlaps the rows
    assert call(q8d, rows=0) == q8d.Q8D_OK


def test_read_outputs_must_not_share_values(q8d):
    assert read(q8d, k=A, v=A) == q8d.Q8D_EINVAL
    assert read(q8d, k=A, v=A + 128) == q8d.Q8D_EINVAL            # half a row on
    assert read(q8d, k=A + 4 * 96, v=A, ld=128) == q8d.Q8D_EINVAL  # runs into the next row's
    assert read(q8d, k=A, v=A + 4 * 64 * 7) == q8d.Q8D_EINVAL


def test_cache_bytes(q8d):
    n = q8d.q8d_kv_cache_bytes
    assert n(0, 33, 7) == 4 * 33 * 7 and n(1, 33, 7) == 2 * 33 * 7
    assert n(2, 1024, 100000) == 100000 * 32 * 34
    assert n(4, 1024, 10_000_000) == 10_000_000 * 32 * 18
    assert n(4, 48, 8) == 0 and n(2, 48, 8) == 0 and n(3, 64, 8) == 0 and n(4, 64, 0) == 0 and n(4, -32, 8) == 0


def test_q4_append_and_attention_refusals(q8d):
    L = q8d.lib()
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    assert L.q8d_kv_append(A, B, C_, D_, 4, 48, 8, E, None, None) == EUNS
    assert L.q8d_kv_append(A, B, C_ + 8, D_, 4, 64, 8, E, None, None) == EALIGN
    assert L.q8d_kv_append(A, B, C_, C_ + 272, 4, 64, 8, E, None, None) == EINVAL   # 288 bytes each
    ws = q8d.q8d_gqa_workspace_bytes(2, 8, 2, 64, 64)

    def attn(kc=C_, vc=D_, dim=64, stride=64 * 128, H=8, n=ws):
        return L.q8d_gqa_decode_attn(A, None, None, kc, vc, 4, B, 2, H, 2, dim, 64, stride, E, 0.125, A + 65536, n,
                                     None, None)
    assert attn(dim=96) == EUNS
    assert attn(H=34) == EUNS
    assert attn(kc=C_ + 8) == EALIGN
    assert attn(stride=64 * 128 + 16) == EALIGN
    assert attn(stride=64 * 128 + 32) == EALIGN
    assert attn(stride=64 * 64) == EINVAL
    assert attn(n=ws - 1) == q8d.Q8D_ERANGE


def test_q4_attention_counts_tiles_in_32_bits(q8d):
    """A batch whose tiles of 32 rows (and a sequence's fixed ones) pass 2^30
    is refused before anything else is looked at."""
    L, big = q8d.lib(), 1 << 62

    def attn(batch, cap, kv=4):
        return L.q8d_gqa_decode_attn(A, None, None, C_, D_, kv, B, batch, 2, 2, 64, cap, big, E, 0.125, A + 65536, 0, None, None)

    def window(batch, cap):
        return L.q8d_gqa_decode_attn_window(A, None, None, C_, D_, 4, B, batch, 2, 2, 64, cap, 0, E, 0.125, A + 65536, 0,
                                            None, None)

    for call, n, cap in ((attn, 32768, 1 << 20), (attn, 1 << 26, 1), (window, 8192, 1 << 20)):
        assert call(n, cap) == q8d.Q8D_EUNSUPPORTED
        assert call(n // 2, cap) == q8d.Q8D_ERANGE  # (no workspace)
    assert attn(32768, 1 << 20, 0) == q8d.Q8D_ERANGE  # other caches
