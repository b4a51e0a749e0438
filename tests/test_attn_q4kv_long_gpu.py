"""4-bit attention over V of one sign and many rows a warp, where sums that are
cut off instead of rounded drift.

Tolerance 1e-5 sum_t p_t V_t.  A warp adds up its tiles of 32 rows: 512 here.
Rounded additions are off by up to 2^-24 of the sum each, either way: six
standard deviations of 512 of them (each uniform over +- 2^-24) are 4.7e-6,
and of the weights' sums, per lane, the same; inside a tile at most eight
products are added on, off by 2^-23 of the tile's sum each, 1e-6; the scores'
part is 2^-21 sum |q K| with sum |q K| below 1 nat, 5e-7.  Not all at their
limits at once."""
import pytest
import torch

from test_attn_q4kv_gpu import Q4, TOL, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 7])
def test_long_sums_of_one_sign(q8d, G):
    """As many KV heads as leave a CTA a head: 16384 rows a warp."""
    Hk, D, L = 160, 64, 131072
    width, H = Hk * D, Hk * G
    gen = torch.Generator(device="cuda").manual_seed(1)
    plane = L * width // 2
    n = q8d.q8d_kv_cache_bytes(Q4, width, L)
    kc, vc = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[:plane] = torch.randint(0, 256, (plane,), generator=gen, dtype=torch.uint8, device="cuda")
    vc[:plane] = torch.randint(0, 256, (plane,), generator=gen, dtype=torch.uint8, device="cuda") & 0x77  # n - 8 < 0
    for c, s in ((kc, 0.25), (vc, -0.125)):
        c[plane:].view(torch.float16)[:] = torch.empty(L * width // 32, device="cuda").uniform_(0.5, 1, generator=gen) * s
    q = torch.randn(H * D, generator=gen, device="cuda") * 0.05
    out, err = torch.empty(H * D, device="cuda"), ints([0])
    m = q8d.q8d_gqa_workspace_bytes(1, H, Hk, D, L)
    q8d.q8d_gqa_decode_attn(q, None, None, kc, vc, Q4, out, 1, H, Hk, D, L, 0, ints([L]), 0.125,
                            torch.empty(m, dtype=torch.uint8, device="cuda"), m, err)
    assert err.item() == 0

    def head(c, g):
        b = c[:plane].view(L, width // 32, 16)[:, g * 2:g * 2 + 2]
        d = c[plane:].view(torch.float16).view(L, width // 32, 1)[:, g * 2:g * 2 + 2].double()
        return (torch.cat([b & 15, b >> 4], -1).double() - 8).mul(d).reshape(L, D)

    for g in (0, 77, 159):
        K, V = head(kc, g), head(vc, g)
        assert V.min() >= 0
        Q = q.view(H, D)[g * G:(g + 1) * G].double()
        assert (0.125 * Q.abs() @ K.abs().T).max() < 1
        p = torch.softmax(0.125 * (Q @ K.T), -1)
        ref = p @ V
        got = out.view(H, D)[g * G:(g + 1) * G].double()
        assert torch.all((got - ref).abs() <= TOL * ref), ((got - ref) / ref).abs().max().item()
