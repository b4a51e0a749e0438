"""Refusals of the norm, the rotary rows and the 4-bit matrices on the host:
every call here is rejected (or a no-op) before anything touches a device."""
import pytest

M = 1 << 28  # fake addresses, far apart


@pytest.fixture(scope="module")
def q8d():
    from q8_block_quantized_matvec_gb300 import build
    build.build()
    import q8_block_quantized_matvec_gb300 as m
    m.lib()
    return m


def norm(q8d, **kw):
    a = dict(x=1 * M, r=2 * M, s=3 * M, t=0, ldx=64, ldr=64, lds=64, w=4 * M, eps=1e-6, y=5 * M, yt=0, ldy=64, rows=3, n=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return q8d.lib().q8d_rmsnorm_rows(a["x"], a["r"], a["s"], a["t"], a["ldx"], a["ldr"], a["lds"], a["w"], a["eps"], a["y"],
                                      a["yt"], a["ldy"], a["rows"], a["n"], None)


def test_norm_refusals(q8d):
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(rows=-1), dict(n=0), dict(n=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=63), dict(ldr=63), dict(lds=63), dict(ldy=63),
                dict(ldx=1 << 30)):
        assert norm(q8d, **bad) == EINVAL, bad
    for bad in (dict(t=2), dict(t=3), dict(yt=4), dict(yt=3), dict(n=16385, ldx=16385, ldr=16385, lds=16385, ldy=16385),
                dict(yt=2, n=48)):
        assert norm(q8d, **bad) == EUNS, bad
    for bad in (dict(x=M + 2), dict(r=2 * M + 1), dict(s=3 * M + 3), dict(w=4 * M + 2), dict(y=5 * M + 2),
                dict(t=1, x=M + 1), dict(yt=1, y=5 * M + 1), dict(yt=2, y=5 * M + 1), dict(yt=2, ldy=80)):
        assert norm(q8d, **bad) == EALIGN, bad
    for bad in (dict(y=M), dict(y=M + 2 * 256), dict(y=2 * M + 256), dict(y=3 * M), dict(y=4 * M), dict(s=4 * M),
                dict(s=M + 256), dict(s=2 * M, lds=68), dict(s=M, ldx=80)):
        assert norm(q8d, **bad) == EINVAL, bad
    assert norm(q8d, rows=0) == q8d.Q8D_OK and norm(q8d, rows=0, x=None) == q8d.Q8D_OK


def test_table_refusals(q8d):
    def table(t=M, max_pos=8, rot=64, theta=1e4, kind=0, factor=1.0, orig=0.0, fast=0.0, slow=0.0, ms=1.0):
        return q8d.lib().q8d_rope_table(t, max_pos, rot, theta, kind, factor, orig, fast, slow, ms, None)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(t=None), dict(max_pos=0), dict(rot=0), dict(rot=-2), dict(theta=1.0), dict(theta=nan), dict(theta=inf),
                dict(factor=0.0), dict(factor=nan), dict(ms=inf), dict(kind=3), dict(kind=3, orig=8.0, fast=1.0),
                dict(kind=3, orig=inf, fast=1.0, slow=1.0), dict(kind=3, orig=8.0, fast=nan, slow=1.0)):
        assert table(**bad) == q8d.Q8D_EINVAL, bad
    for bad in (dict(rot=3), dict(rot=258), dict(kind=4), dict(kind=-1), dict(kind=2, rot=2)):
        assert table(**bad) == q8d.Q8D_EUNSUPPORTED, bad
    assert table(t=M + 8) == q8d.Q8D_EALIGN


def rope(q8d, **kw):
    d = dict(n_heads=4, n_kv_heads=2, head_dim=64, rot_dim=64, layout=0, max_pos=32, row_dtype=0, q_dtype=0, kv_dtype=1, cap=32,
             eps=1e-6, ldq=512, ldkv=512, ldo=256, cache_batch_stride=4096, table=9 * M, bq=None, bk=None, bv=None, q_norm=None,
             k_norm=None)
    a = dict(q=M, k=M + 4 * 256, v=M + 4 * 384, out=2 * M, kc=3 * M, vc=4 * M, batch=2, rows=3, pos=5 * M, rpos=None,
             counts=None, err=None)
    for name, value in kw.items():
        (d if name in d else a)[name] = value
    assert set(a) == {"q", "k", "v", "out", "kc", "vc", "batch", "rows", "pos", "rpos", "counts", "err"}
    return q8d.lib().q8d_rope_append_rows(q8d.rope_desc(**d), a["q"], a["k"], a["v"], a["out"], a["kc"], a["vc"], a["batch"],
                                          a["rows"], a["pos"], a["rpos"], a["counts"], a["err"], None)


def test_rope_refusals(q8d):
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    for bad in (dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(pos=None),
                dict(q=None, out=None, k=None, v=None, kc=None, vc=None), dict(batch=0), dict(rows=-1), dict(n_heads=0),
                dict(n_kv_heads=0), dict(head_dim=0), dict(cap=0), dict(max_pos=0), dict(eps=-1.0), dict(rot_dim=-2),
                dict(rot_dim=66), dict(table=None), dict(bq=6 * M), dict(bq=6 * M, bk=7 * M), dict(q_norm=6 * M),
                dict(ldq=255), dict(ldkv=127), dict(ldo=255), dict(cache_batch_stride=4095), dict(cache_batch_stride=-8)):
        assert rope(q8d, **bad) == EINVAL, bad
    assert q8d.lib().q8d_rope_append_rows(None, M, M, M, M, M, M, 1, 1, M, None, None, None, None) == EINVAL
    for bad in (dict(head_dim=60, rot_dim=60), dict(head_dim=264, rot_dim=64, ldq=2048, ldkv=2048, ldo=2048), dict(rot_dim=63),
                dict(layout=2), dict(row_dtype=2), dict(q_dtype=2), dict(kv_dtype=3), dict(kv_dtype=4, head_dim=48, rot_dim=48),
                dict(kv_dtype=2, head_dim=8, rot_dim=8), dict(batch=1 << 17, rows=1 << 15)):
        assert rope(q8d, **bad) == EUNS, bad
    for bad in (dict(q=M + 2), dict(k=M + 2), dict(v=M + 1), dict(out=2 * M + 2), dict(kc=3 * M + 8), dict(vc=4 * M + 2),
                dict(table=9 * M + 8), dict(pos=5 * M + 2), dict(rpos=5 * M + 1), dict(counts=5 * M + 2), dict(err=5 * M + 1),
                dict(kv_dtype=2, cache_batch_stride=4112), dict(cache_batch_stride=4097), dict(q_norm=6 * M + 2, k_norm=6 * M)):
        assert rope(q8d, **bad) == EALIGN, bad
    for bad in (dict(out=M), dict(out=3 * M), dict(kc=4 * M + 64), dict(kc=M), dict(vc=M + 2048), dict(out=9 * M),
                dict(kc=9 * M), dict(out=M, ldo=512, k=M + 64), dict(out=M, ldo=512, q_dtype=1),
                dict(out=M, ldo=512, v=M + 4 * 400)):
        assert rope(q8d, **bad) == EINVAL, bad
    assert rope(q8d, rows=0) == q8d.Q8D_OK


def q4(q8d, gated=False, **kw):
    a = dict(X=M, xt=0, ldx=64, w=2 * M, wu=3 * M, group=32, bias=4 * M, res=5 * M, ldr=48, Y=6 * M, ldy=48, m=3, n=64, p=48)
    assert set(kw) <= set(a)
    a.update(kw)
    L = q8d.lib()
    if gated:
        return L.q8d_q4_gated(a["X"], a["xt"], a["ldx"], a["w"], a["wu"], a["group"], a["Y"], a["ldy"], a["m"], a["n"], a["p"],
                              None)
    return L.q8d_q4_matmul(a["X"], a["xt"], a["ldx"], a["w"], a["group"], a["bias"], a["res"], a["ldr"], a["Y"], a["ldy"],
                           a["m"], a["n"], a["p"], None)


def test_q4_refusals(q8d):
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    for gated in (False, True):
        for bad in (dict(X=None), dict(w=None), dict(Y=None), dict(m=-1), dict(n=0), dict(n=-32), dict(p=-1), dict(ldx=32),
                    dict(ldy=47), dict(Y=M), dict(Y=M + 512), dict(Y=2 * M), dict(ldx=1 << 30)):
            assert q4(q8d, gated, **bad) == EINVAL, bad
        for bad in (dict(m=17), dict(n=48, ldx=48), dict(n=32800, ldx=32800), dict(group=16), dict(group=96), dict(group=256),
                    dict(xt=3), dict(xt=4), dict(p=(1 << 30) + 1, ldy=1 << 31, ldr=1 << 31)):
            assert q4(q8d, gated, **bad) == EUNS, bad
        for bad in (dict(X=M + 8), dict(ldx=66), dict(xt=1, ldx=68), dict(xt=2, X=M + 1), dict(xt=2, ldx=80), dict(w=2 * M + 8),
                    dict(Y=6 * M + 2)):
            assert q4(q8d, gated, **bad) == EALIGN, bad
        for noop in (dict(m=0), dict(p=0, ldy=0)):
            assert q4(q8d, gated, **noop) == q8d.Q8D_OK, noop
    assert q4(q8d, True, wu=None) == EINVAL and q4(q8d, True, wu=3 * M + 4) == EALIGN and q4(q8d, True, Y=3 * M) == EINVAL
    for bad in (dict(ldr=47), dict(Y=4 * M), dict(Y=5 * M, ldy=52), dict(Y=5 * M + 4)):
        assert q4(q8d, **bad) == EINVAL, bad
    assert q4(q8d, bias=4 * M + 2) == EALIGN and q4(q8d, res=5 * M + 1) == EALIGN


def test_q4_matrix_bytes_and_copies(q8d):
    n = q8d.q8d_q4_matrix_bytes
    assert n(1, 32, 32) == 1152 and n(16, 128, 64) == 1088 and n(17, 129 + 31, 128) == 4 * 1056
    assert n(0, 32, 32) == n(16, 48, 32) == n(16, 0, 32) == n(16, 128, 48) == n(-1, 32, 32) == n(1, 32800, 32) == 0
    assert n(151936, 896, 64) == 9496 * 7 * 1088
    L = q8d.lib()
    for f, pack in ((L.q8d_q4_pack, True), (L.q8d_q4_unpack, False)):
        def call(w=M, rows=2 * M, t=0, ld=64, p=5, k=64, group=32):
            return f(rows, t, ld, w, p, k, group, None) if pack else f(w, rows, t, ld, p, k, group, None)
        for bad in (dict(w=None), dict(rows=None), dict(p=-1), dict(k=0), dict(ld=63), dict(rows=M), dict(rows=M + 1136),
                    dict(ld=1 << 30)):
            assert call(**bad) == q8d.Q8D_EINVAL, bad
        for bad in (dict(k=33), dict(group=0), dict(t=3), dict(t=4), dict(k=32800, ld=32800), dict(p=(1 << 30) + 1)):
            assert call(**bad) == q8d.Q8D_EUNSUPPORTED, bad
        for bad in (dict(w=M + 8), dict(rows=2 * M + 2), dict(t=1, rows=2 * M + 1)):
            assert call(**bad) == q8d.Q8D_EALIGN, bad
        assert call(p=0, rows=None) == q8d.Q8D_OK
    assert L.q8d_q4_pack(2 * M, 2, 80, M, 5, 64, 32, None) == q8d.Q8D_EALIGN


def test_desc_fields(q8d):
    with pytest.raises(TypeError):
        q8d.rope_desc(heads=3)
