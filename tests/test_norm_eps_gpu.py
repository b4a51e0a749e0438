"""The norm's factor is 1 / sqrt(mean + eps) in 64 bits rounded once, for every eps:
the bits of the f32 steps (tiny means and eps among them)."""
import numpy as np
import pytest
import torch

import synth
from conftest import dev
from test_norm_gpu import steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low,high", [(-45, -30), (-10, 10), (20, 30), (30, 36), (36, 38.5)])
def test_every_eps(q8d, low, high):
    n, w = 64, np.ones(64, np.float32)
    x = synth.normal_f32(1, "eps.x", (1, n))
    dx, dw = dev(x), dev(w)
    eps = (10.0 ** synth.stream(2, "eps.e").uniform(low, high, 400)).astype(np.float32)
    y = torch.empty(len(eps), n, device="cuda")
    for i, e in enumerate(eps):
        q8d.q8d_rmsnorm_rows(dx, None, None, 0, n, 0, 0, dw, float(e), y[i], 0, n, 1, n)
    torch.cuda.synchronize()
    want = np.concatenate([steps(x, None, w, e)[1] for e in eps])
    assert np.array_equal(y.cpu().numpy(), want)
