"""A captured call of q8d_rope_append_rows over the steps of a decode: positions live
on the device, and every replay stores k and v at its own cache rows and leaves those
of the steps before as they were."""
import numpy as np
import pytest
import torch

import kvplain as kp
from test_rope_gpu import F16, F32, HALF, KINDS, PAIRS, Case, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,norm,src", [(HALF, False, F32), (PAIRS, True, F16)])
@pytest.mark.parametrize("rows,counts", [(1, None), (3, [2, 0])])
def test_caches_of_every_replay(q8d, kind, layout, norm, src, rows, counts):
    starts = [0, 3]
    c = Case(q8d, 4, 2, 64, 32, layout, kind, 2, rows, 20, starts, counts, norm=norm, src=src)
    pos, d_counts, st, g = ints(starts), ints(counts), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q, k, v = c.args
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        q8d.q8d_rope_append_rows(c.desc, q, k, v, c.out, c.kc, c.vc, 2, rows, pos, None, d_counts, c.err, st)
    torch.cuda.synchronize()
    want = c.before.copy()
    assert np.array_equal(c.kc.cpu().numpy(), want[0])  # (nothing ran yet)
    for step in range(5):
        g.replay()
        torch.cuda.synchronize()
        for s in range(2):
            n, first = rows if counts is None else counts[s], starts[s] + step
            at = slice(s * rows, s * rows + n)
            kp.store(want[0, s], kind, c.w, c.cap, first, c.head_rows(c.k[at], None, c.g[1], np.arange(first, first + n), True))
            kp.store(want[1, s], kind, c.w, c.cap, first, c.v[at].astype(np.float32))
        assert np.array_equal(c.kc.cpu().numpy(), want[0]), step
        assert np.array_equal(c.vc.cpu().numpy(), want[1]), step
        pos.add_(1)
    assert c.err.item() == 0
