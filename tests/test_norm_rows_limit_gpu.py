"""The norm of as many rows as an int counts: every one of them is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_as_many_rows_as_an_int_counts(q8d):
    rows = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    # rows of one element: y = x / |x|
    x = torch.empty(rows, dtype=torch.float16, device="cuda")
    x.copy_(torch.tensor([0.5, -3.0, 2.0, -0.25, 7.0], dtype=torch.float16, device="cuda").repeat(2 ** 29)[:rows])
    y = torch.zeros(rows, dtype=torch.float16, device="cuda")
    w = torch.ones(1, device="cuda")
    q8d.q8d_rmsnorm_rows(x, None, None, 1, 1, 0, 0, w, 0.0, y, 1, 1, rows, 1)
    torch.cuda.synchronize()
    assert torch.equal(y, torch.sign(x))
