"""The 4-bit products when a wait for their weights runs out: NaN where a sum misses
a copy, and calls afterwards as before.  Whole CTAs and clusters of them, one and
several passes, every kind of rows."""
import pytest
import torch

import kvplain as kp
from test_q4_gpu import Matrix, activations

pytestmark = pytest.mark.gpu
F32, F16, Q8_0 = kp.F32, kp.F16, kp.Q8_0

CASES = [  # rows' kind, m, p, n, group, gated
    (F32, 1, 16, 32, 32, False), (F32, 1, 4608, 3584, 32, False), (F32, 2, 300, 18944, 128, False),
    (F32, 7, 5000, 896, 64, True), (F32, 16, 3584, 3584, 32, False), (F32, 16, 18944, 3584, 32, True),
    (F16, 3, 700, 1184, 32, True), (F16, 16, 100, 18944, 64, False), (Q8_0, 1, 3000, 640, 128, False),
    (Q8_0, 16, 4736, 3584, 64, True), (F32, 1, 900_001, 64, 32, False), (F32, 4, 250, 160, 64, True),
]


class Call:
    def __init__(self, q8d, kind, m, p, n, group, gated):
        self.q8d, self.m, self.p = q8d, m, p
        self.W = [Matrix(q8d, 50 + i, p, n, group) for i in range(2 if gated else 1)]
        self.x, _, self.ld = activations(52, m, n, kind)
        self.kind = kind

    def go(self, y, stream=None):
        W, q8d = self.W, self.q8d
        if len(W) == 2:
            q8d.q8d_q4_gated(self.x, self.kind, self.ld, W[0].bytes, W[1].bytes, W[0].group, y, self.p, self.m, W[0].n, self.p,
                             stream)
        else:
            q8d.q8d_q4_matmul(self.x, self.kind, self.ld, W[0].bytes, W[0].group, None, None, 0, y, self.p, self.m, W[0].n,
                              self.p, stream)

    def __call__(self, polls):
        y = torch.full((self.m, self.p), -7.0, device="cuda")
        self.q8d.q8d_q4_set_wait_limit(polls)
        try:
            self.go(y)
        finally:
            self.q8d.q8d_q4_set_wait_limit(0)
        torch.cuda.synchronize()
        return y


@pytest.mark.parametrize("case", CASES)
def test_no_wait_ends_in_time(q8d, case):
    """Nothing is waited for: no number comes out, and the calls between keep
    their bits."""
    call = Call(q8d, *case)
    first = call(0)
    assert torch.isfinite(first).all()
    for _ in range(4):
        assert torch.isnan(call(1)).all()
        assert torch.equal(call(0), first)


@pytest.mark.parametrize("case", CASES)
def test_some_waits_end_in_time(q8d, case):
    """Limits at which some waits succeed: each entry is right or NaN."""
    call = Call(q8d, *case)
    first = call(0)
    for polls in (2, 3, 4, 6, 9, 14, 20, 40, 80, 160, 400):
        y = call(polls)
        good = ~torch.isnan(y)
        assert torch.equal(y[good], first[good])
    assert torch.equal(call(0), first)


def test_limit_of_a_captured_call(q8d):
    """A graph keeps the limit it was captured with."""
    call = Call(q8d, F32, 3, 500, 416, 32, False)
    first = call(0)
    y, st, g = torch.zeros(3, 500, device="cuda"), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    q8d.q8d_q4_set_wait_limit(1)
    try:
        with torch.cuda.graph(g, stream=st):
            call.go(y, st)
    finally:
        q8d.q8d_q4_set_wait_limit(0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.isnan(y).all()
    assert torch.equal(call(0), first)
