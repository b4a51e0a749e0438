"""Row calls of more items than their kernels number: refused on the host."""
import pytest

A, B, C_, D_, E = (i << 40 for i in range(1, 6))  # fake addresses, far apart


@pytest.mark.parametrize("call", ["q8d_kv_append_rows", "q8d_kv_read_rows"])
@pytest.mark.parametrize("rows,width", [((1 << 22) - 63, 4096), (2 ** 31 - 1, 8), (2 ** 31 - 1, 5)])
def test_more_rows_than_numbered(call, rows, width):
    """rows * ceil(width / 4) above 2^32 - 2^16, with items of four elements."""
    from q8_block_quantized_matvec_gb300 import build
    build.build()
    import q8_block_quantized_matvec_gb300 as q8d
    assert rows * -(-width // 4) > 2 ** 32 - 2 ** 16
    if call == "q8d_kv_append_rows":
        rc = q8d.lib().q8d_kv_append_rows(A, B, 0, width, C_, D_, 0, 1, rows, width, 4, 0, E, None, None, None)
    else:
        rc = q8d.lib().q8d_kv_read_rows(C_, D_, 0, A, B, 0, width, 1, rows, width, 4, 0, E, None, None, None)
    assert rc == q8d.Q8D_EUNSUPPORTED
