"""Refusals of q8d_moe_ffn on the host: every call here is rejected before
anything touches a device."""
import pytest

M = 1 << 24  # fake 16-byte aligned addresses, far apart
BASE = dict(X=1 * M, ldx=64, router=2 * M, wg=3 * M, wu=4 * M, wd=5 * M, residual=6 * M, ldr=64, Y=7 * M, ldy=64,
            m=3, hidden=64, ffn=96, E=8, k=2, norm=1, experts=8 * M, weights=9 * M, ws=10 * M, wsb=None, err=11 * M)


@pytest.fixture(scope="module")
def q8d():
    from q8_block_quantized_matvec_gb300 import build
    build.build()
    import q8_block_quantized_matvec_gb300 as m
    m.lib()
    return m


def call(q8d, **kw):
    a = dict(BASE)
    a.update(kw)
    n = q8d.q8d_moe_workspace_bytes(a["m"], a["hidden"], a["ffn"], a["E"], a["k"]) if a["wsb"] is None else a["wsb"]
    return q8d.lib().q8d_moe_ffn(a["X"], a["ldx"], a["router"], a["wg"], a["wu"], a["wd"], a["residual"], a["ldr"],
                                 a["Y"], a["ldy"], a["m"], a["hidden"], a["ffn"], a["E"], a["k"], a["norm"],
                                 a["experts"], a["weights"], a["ws"], n, a["err"], None)


def test_moe_refusals(q8d):
    EINVAL, EALIGN, EUNS = q8d.Q8D_EINVAL, q8d.Q8D_EALIGN, q8d.Q8D_EUNSUPPORTED
    for nm in ("X", "router", "wg", "wu", "wd", "Y", "ws"):
        assert call(q8d, **{nm: None}) == EINVAL, nm
    for bad in (dict(m=-1), dict(hidden=0), dict(ffn=-32), dict(E=0), dict(k=0), dict(k=9)):
        assert call(q8d, wsb=1 << 20, **bad) == EINVAL, bad
    for bad in (dict(m=65), dict(hidden=80, ldx=80, ldy=80, ldr=80), dict(ffn=100), dict(E=513, k=2),
                dict(E=64, k=33), dict(hidden=16416, ldx=16416, ldy=16416, ldr=16416), dict(ffn=16416)):
        assert call(q8d, wsb=1 << 30, **bad) == EUNS, bad
    assert call(q8d, ldx=60) == EINVAL and call(q8d, ldy=63) == EINVAL and call(q8d, ldr=63) == EINVAL
    for bad in (dict(X=M + 8), dict(ldx=66), dict(router=2 * M + 4), dict(wg=3 * M + 2), dict(wu=4 * M + 8),
                dict(wd=5 * M + 4), dict(ws=10 * M + 8), dict(Y=7 * M + 2), dict(residual=6 * M + 1),
                dict(experts=8 * M + 2), dict(weights=9 * M + 2), dict(err=11 * M + 2)):
        assert call(q8d, **bad) == EALIGN, bad
    n = q8d.q8d_moe_workspace_bytes(3, 64, 96, 8, 2)
    assert n > 0 and call(q8d, wsb=n - 1) == EINVAL
    # overlaps: outputs with inputs and with each other; Y with a shifted residual
    for bad in (dict(Y=M + 64), dict(Y=3 * M + 64), dict(Y=5 * M), dict(Y=2 * M), dict(residual=7 * M + 64),
                dict(residual=7 * M, ldr=68), dict(experts=7 * M + 4), dict(weights=8 * M), dict(ws=M),
                dict(ws=7 * M), dict(ws=4 * M + 16), dict(experts=6 * M + 16)):
        assert call(q8d, **bad) == EINVAL, bad
    assert call(q8d, m=0, wsb=0) == q8d.Q8D_OK


def test_moe_workspace_bytes(q8d):
    n = q8d.q8d_moe_workspace_bytes
    assert n(0, 64, 96, 8, 2) == 0 and n(65, 64, 96, 8, 2) == 0 and n(1, 65, 96, 8, 2) == 0
    assert n(1, 64, 96, 8, 9) == 0
    assert 0 < n(1, 2048, 768, 128, 8) < n(64, 2048, 768, 128, 8) < 64 << 20
