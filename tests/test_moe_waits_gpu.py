"""q8d_moe_ffn when a wait inside its products runs out: the error bit, NaN
where a result is missing, and calls afterwards as before.  Every way in which
rows come (whole lines, whole rows, rows in slices), one and many tokens."""
import numpy as np
import pytest
import torch

import synth
from conftest import dev
from test_moe_gpu import ints, layer, plain

pytestmark = pytest.mark.gpu

SHAPES = [  # m, hidden, ffn, E, k
    (1, 256, 256, 4, 2), (13, 256, 512, 7, 3), (40, 2048, 768, 16, 4), (64, 512, 256, 4, 2),
    (1, 96, 352, 4, 2), (13, 1056, 800, 7, 3), (64, 288, 160, 5, 2),
    (1, 2336, 2336, 3, 1), (13, 2336, 2400, 7, 2), (33, 4128, 96, 5, 3), (20, 96, 4128, 3, 2),
]


class Call:
    def __init__(self, q8d, m, hidden, ffn, E, k):
        self.q8d, self.shape = q8d, (m, hidden, ffn, E, k)
        self.L, self.x = layer(m + ffn, E, hidden, ffn), synth.normal_f32(m, "waits.x", (m, hidden))
        self.d, self.X = [dev(w) for w in self.L], dev(self.x)
        self.n = q8d.q8d_moe_workspace_bytes(m, hidden, ffn, E, k)
        self.ws = torch.zeros(self.n, dtype=torch.uint8, device="cuda")

    def __call__(self, polls):
        """(Y, error word) of a call with the wait limit `polls`."""
        m, hidden, ffn, E, k = self.shape
        Y, err = torch.full((m, hidden), -7.0, device="cuda"), ints([0])
        self.q8d.q8d_moe_set_wait_limit(polls)
        try:
            self.q8d.q8d_moe_ffn(self.X, hidden, *self.d, None, hidden, Y, hidden, m, hidden, ffn, E, k, 1, None, None,
                                 self.ws, self.n, err)
        finally:
            self.q8d.q8d_moe_set_wait_limit(0)
        torch.cuda.synchronize()
        return Y.cpu().numpy(), err.item()


@pytest.mark.parametrize("shape", SHAPES)
def test_no_wait_ends_in_time(q8d, shape):
    """Nothing is waited for: no number comes out, and the calls between keep
    their bits."""
    call = Call(q8d, *shape)
    first, err = call(0)
    _, _, ref, tol = plain(call.L, call.x, shape[3], shape[1], shape[2], shape[4], True, None)
    assert err == 0 and np.all(np.abs(first - ref) <= tol)
    for _ in range(4):
        y, err = call(1)
        assert err == q8d.Q8D_DERR_WAIT
        assert np.isnan(y).all()
        y, err = call(0)
        assert err == 0 and np.array_equal(y, first)


@pytest.mark.parametrize("shape", SHAPES)
def test_some_waits_end_in_time(q8d, shape):
    """Limits at which some waits succeed: each entry is right or NaN, and NaN
    comes with the error bit."""
    call = Call(q8d, *shape)
    first, err = call(0)
    assert err == 0
    for polls in (2, 3, 4, 6, 9, 14, 20, 40, 80, 160, 400):
        y, err = call(polls)
        bad = np.isnan(y)
        assert err in (0, q8d.Q8D_DERR_WAIT)
        assert err != 0 or not bad.any()
        assert np.array_equal(y[~bad], first[~bad])
    y, err = call(0)
    assert err == 0 and np.array_equal(y, first)


def test_limit_of_a_captured_call(q8d):
    """A graph keeps the limit it was captured with."""
    m, hidden, ffn, E, k = shape = (5, 256, 192, 6, 2)
    call = Call(q8d, *shape)
    first, _ = call(0)
    Y, err, st, g = torch.zeros(m, hidden, device="cuda"), ints([0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q8d.q8d_moe_set_wait_limit(1)
    try:
        with torch.cuda.graph(g, stream=st):
            q8d.q8d_moe_ffn(call.X, hidden, *call.d, None, hidden, Y, hidden, m, hidden, ffn, E, k, 1, None, None, call.ws,
                            call.n, err, st)
    finally:
        q8d.q8d_moe_set_wait_limit(0)
    g.replay()
    torch.cuda.synchronize()
    assert err.item() == q8d.Q8D_DERR_WAIT and torch.isnan(Y).all()
    y, e = call(0)
    assert e == 0 and np.array_equal(y, first)
