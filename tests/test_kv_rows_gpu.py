"""q8d_kv_append_rows / q8d_kv_read_rows and the 4-bit cache's store: every
stored byte and every value read back equals the plain numpy form, and
nothing else in the buffers changes."""
import numpy as np
import pytest
import torch

import kvplain as kp
import synth
from conftest import dev

pytestmark = pytest.mark.gpu
F32, F16, Q8_0, Q4 = kp.F32, kp.F16, kp.Q8_0, kp.Q4
KINDS = [F32, F16, Q8_0, Q4]
NP = {F32: np.float32, F16: np.float16}
TT = {F32: torch.float32, F16: torch.float16}


def stride_of(cap, width):
    return -(-cap * width // 256) * 256


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows_in(seed, name, batch, rows, width, src, ld, offset):
    """(device buffer view, f32 rows [batch, rows, width]) with rows `ld`
    values apart starting `offset` values into a buffer."""
    x = synth.normal_f32(seed, name, (batch, rows, width)).astype(np.float32)
    x *= (10.0 ** (np.arange(rows) % 7 - 3)).astype(np.float32)[None, :, None]
    if width >= 96:
        x[..., 32:64] = 0.0                                      # a block of zeros
        x[..., 64:96] = np.tile(np.array([8, -8, 2.5, -2.5, 0.5, -0.5, 127, -127], np.float32), 4)
    x = x.astype(NP[src])
    buf = np.zeros(offset + batch * rows * ld, NP[src])
    buf[offset:].reshape(batch * rows, ld)[:, :width] = x.reshape(batch * rows, width)
    return dev(buf)[offset:], x.astype(np.float32)


CASES = [  # width, cap, batch, rows, starts, counts, src type, ld, offset
    (32, 1, 1, 1, [0], None, F32, 32, 0),
    (32, 9, 3, 4, [0, 5, 2], [4, 0, 1], F32, 32, 0),
    (96, 7, 2, 7, [0, 0], [7, 3], F16, 96, 0),
    (512, 40, 1, 33, [7], None, F32, 4608, 0),        # columns of a fused projection
    (1024, 16, 5, 3, [13, 0, 1, 2, 9], [3, 2, 1, 0, 3], F16, 1024, 0),
    (128, 21, 2, 5, [16, 3], None, F32, 131, 1),      # rows off every 16-byte boundary
    (64, 300, 4, 257, [0, 43, 7, 1], [257, 256, 1, 100], F16, 65, 3),
    (2048, 6, 130, 1, [i % 6 for i in range(130)], [i % 2 for i in range(130)], F32, 2048, 0),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width,cap,batch,rows,starts,counts,src,ld,offset", CASES)
def test_append_rows_bytes(q8d, kind, width, cap, batch, rows, starts, counts, src, ld, offset):
    stride = stride_of(cap, width)
    nb = kp.cache_bytes(kind, stride)
    before = synth.stream(3, "rows.cache").integers(0, 256, (2, batch, nb), dtype=np.uint8)
    k, kx = rows_in(1, "rows.k", batch, rows, width, src, ld, offset)
    v, vx = rows_in(2, "rows.v", batch, rows, width, src, ld, offset)
    kc, vc, err = dev(before[0]), dev(before[1]), ints([0])
    q8d.q8d_kv_append_rows(k, v, src, ld, kc, vc, kind, batch, rows, width, cap, stride,
                           ints(starts), None if counts is None else ints(counts), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    want = before.copy()
    for s in range(batch):
        n = rows if counts is None else counts[s]
        kp.store(want[0, s], kind, width, cap, starts[s], kx[s, :n])
        kp.store(want[1, s], kind, width, cap, starts[s], vx[s, :n])
    assert np.array_equal(kc.cpu().numpy(), want[0])
    assert np.array_equal(vc.cpu().numpy(), want[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width,cap,batch,rows,starts,counts,dst,ld,offset", CASES)
def test_read_rows_values(q8d, kind, width, cap, batch, rows, starts, counts, dst, ld, offset):
    stride = stride_of(cap, width)
    caches = np.zeros((2, batch, kp.cache_bytes(kind, stride)), np.uint8)
    for i in range(2):
        for s in range(batch):
            kp.store(caches[i, s], kind, width, cap, 0,
                     synth.normal_f32(s, f"read.{i}", (cap, width)) * np.float32(3))
    outs = [torch.full((offset + batch * rows * ld,), -7.0, dtype=TT[dst], device="cuda") for _ in range(2)]
    err = ints([0])
    q8d.q8d_kv_read_rows(dev(caches[0]), dev(caches[1]), kind, outs[0][offset:], outs[1][offset:], dst,
                         ld, batch, rows, width, cap, stride, ints(starts),
                         None if counts is None else ints(counts), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for i in range(2):
        want = np.full(offset + batch * rows * ld, -7.0, NP[dst])
        grid = want[offset:].reshape(batch, rows, ld)
        for s in range(batch):
            n = rows if counts is None else counts[s]
            x = kp.values(caches[i, s], kind, width, cap)
            grid[s, :n, :width] = x[starts[s]:starts[s] + n].astype(NP[dst])
        assert np.array_equal(outs[i].cpu().numpy(), want)


@pytest.mark.parametrize("kind", [F32, F16])
@pytest.mark.parametrize("width", [1, 7, 33])
def test_rows_of_any_width(q8d, kind, width):
    """Element caches have no blocks: widths that are no multiple of anything."""
    cap, rows = 11, 6
    x = synth.normal_f32(0, "any", (2, rows, width))
    kc, vc = (torch.zeros(cap, width, dtype=TT[kind], device="cuda") for _ in range(2))
    out = [torch.zeros(rows, width, device="cuda") for _ in range(2)]
    err = ints([0])
    q8d.q8d_kv_append_rows(dev(x[0]), dev(x[1]), F32, width, kc, vc, kind, 1, rows, width, cap, 0,
                           ints([5]), None, err)
    q8d.q8d_kv_read_rows(kc, vc, kind, out[0], out[1], F32, width, 1, rows, width, cap, 0, ints([5]),
                         None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for i, c in enumerate((kc, vc)):
        want = np.zeros((cap, width), NP[kind])
        want[5:] = x[i].astype(NP[kind])
        assert np.array_equal(c.cpu().numpy(), want)
        assert np.array_equal(out[i].cpu().numpy(), want[5:].astype(np.float32))


@pytest.mark.parametrize("kind", KINDS)
def test_refused_sequences_write_nothing_and_read_nan(q8d, kind):
    """Bad counts and positions refuse their own sequence only; a count of 0
    is fine at any position."""
    width, cap, batch, rows = 64, 8, 6, 3
    starts, counts = [6, -1, 2, 5, 100, 0], [3, 1, 4, -1, 0, 3]
    good = [False, False, False, False, True, True]
    stride = stride_of(cap, width)
    nb = kp.cache_bytes(kind, stride)
    x = synth.normal_f32(0, "refused", (batch, rows, width))
    kc, vc = (torch.full((batch, nb), 17, dtype=torch.uint8, device="cuda") for _ in range(2))
    err = ints([0])
    q8d.q8d_kv_append_rows(dev(x), dev(x), F32, width, kc, vc, kind, batch, rows, width, cap, stride,
                           ints(starts), ints(counts), err)
    torch.cuda.synchronize()
    assert err.item() == q8d.Q8D_DERR_POS_RANGE | q8d.Q8D_DERR_LEN_RANGE
    want = np.full((batch, nb), 17, np.uint8)
    kp.store(want[5], kind, width, cap, 0, x[5])
    assert np.array_equal(kc.cpu().numpy(), want) and np.array_equal(vc.cpu().numpy(), want)
    ko, vo = (torch.full((batch, rows, width), 5.0, device="cuda") for _ in range(2))
    err.zero_()
    q8d.q8d_kv_read_rows(kc, vc, kind, ko, vo, F32, width, batch, rows, width, cap, stride, ints(starts),
                         ints(counts), err)
    torch.cuda.synchronize()
    assert err.item() == q8d.Q8D_DERR_POS_RANGE | q8d.Q8D_DERR_LEN_RANGE
    for o in (ko, vo):
        o = o.cpu().numpy()
        for s in range(batch):
            assert np.isnan(o[s]).all() != good[s]
        assert np.all(o[4] == 5.0)  # no rows asked: left as they were
        assert np.array_equal(o[5], kp.values(want[5], kind, width, cap)[:3])


def test_q4_single_row_append(q8d):
    """q8d_kv_append stores one row of a 4-bit cache."""
    for width, cap, pos in [(32, 3, 2), (128, 16, 0), (1024, 9, 7)]:
        x = synth.normal_f32(pos, "one", (2, width))
        want = np.full((2, kp.cache_bytes(Q4, cap * width)), 9, np.uint8)
        kc, vc, err = dev(want[0]), dev(want[1]), ints([0])
        q8d.q8d_kv_append(dev(x[0]), dev(x[1]), kc, vc, Q4, width, cap, ints([pos]), err)
        torch.cuda.synchronize()
        for i in range(2):
            kp.store(want[i], Q4, width, cap, pos, x[i:i + 1])
        assert err.item() == 0
        assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])
        for bad in (-1, cap):
            q8d.q8d_kv_append(dev(x[0]), dev(x[1]), kc, vc, Q4, width, cap, ints([bad]), err)
        torch.cuda.synchronize()
        assert err.item() == q8d.Q8D_DERR_POS_RANGE
        assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])


def test_q4_edges_of_the_quantizer(q8d):
    """Ties of the largest magnitude, denormal and tiny blocks, the largest
    finite scale, exact halves."""
    rows = np.zeros((8, 64), np.float32)
    rows[0, :32] = np.tile([3.0, -3.0], 16)
    rows[0, 32:] = np.tile([-3.0, 3.0], 16)
    rows[1] = np.float32(1e-45)
    rows[2] = np.linspace(-1, 1, 64).astype(np.float32) * np.float32(1e-38)
    rows[3] = np.linspace(-1, 1, 64).astype(np.float32) * np.float32(1e-7)
    rows[4] = np.linspace(-1, 1, 64).astype(np.float32) * np.float32(524031.0)
    rows[5, :32] = np.arange(-16, 16) / 2
    rows[5, 32:] = np.arange(16, -16, -1) / 2
    rows[6, 31] = -0.0
    rows[7, 0] = 1.0
    cap, width = 8, 64
    kc, vc = (torch.zeros(kp.cache_bytes(Q4, cap * width), dtype=torch.uint8, device="cuda") for _ in range(2))
    q8d.q8d_kv_append_rows(dev(rows), dev(-rows), F32, width, kc, vc, Q4, 1, 8, width, cap, 0, ints([0]),
                           None, None)
    torch.cuda.synchronize()
    for c, x in ((kc, rows), (vc, -rows)):
        want = np.zeros(kp.cache_bytes(Q4, cap * width), np.uint8)
        kp.store(want, Q4, width, cap, 0, x)
        assert np.array_equal(c.cpu().numpy(), want)


def test_rows_past_2_to_the_32_bytes(q8d):
    """A long f32 cache: rows whose byte offset does not fit 32 bits."""
    width, cap = 2048, 600_000  # 4.9 GB each
    kc, vc = (torch.empty(cap, width, device="cuda") for _ in range(2))
    x = synth.normal_f32(0, "far", (2, 3, width))
    out = [torch.zeros(3, width, device="cuda") for _ in range(2)]
    err = ints([0])
    kc[cap - 4].fill_(1.5)
    q8d.q8d_kv_append_rows(dev(x[0]), dev(x[1]), F32, width, kc, vc, F32, 1, 3, width, cap, 0,
                           ints([cap - 3]), None, err)
    q8d.q8d_kv_read_rows(kc, vc, F32, out[0], out[1], F32, width, 1, 3, width, cap, 0, ints([cap - 3]),
                         None, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert np.array_equal(kc[cap - 3:].cpu().numpy(), x[0]) and np.array_equal(vc[cap - 3:].cpu().numpy(), x[1])
    assert np.array_equal(out[0].cpu().numpy(), x[0]) and np.array_equal(out[1].cpu().numpy(), x[1])
    assert torch.all(kc[cap - 4] == 1.5)


def test_rows_on_another_stream_and_in_a_graph(q8d):
    """Append and read captured once and replayed with new rows, positions
    and counts."""
    width, cap, batch, rows = 256, 32, 3, 4
    k, v = (torch.zeros(batch * rows, width, device="cuda") for _ in range(2))
    kc, vc = (torch.zeros(batch, kp.cache_bytes(Q4, cap * width), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    ko, vo = (torch.zeros(batch * rows, width, device="cuda") for _ in range(2))
    pos, count, err = ints([0] * batch), ints([0] * batch), ints([0])

    def both(stream):
        q8d.q8d_kv_append_rows(k, v, F32, width, kc, vc, Q4, batch, rows, width, cap, cap * width, pos,
                               count, err, stream)
        q8d.q8d_kv_read_rows(kc, vc, Q4, ko, vo, F32, width, batch, rows, width, cap, cap * width, pos,
                             count, err, stream)

    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        both(st)
    want = np.zeros((batch, kp.cache_bytes(Q4, cap * width)), np.uint8)
    want_o = np.zeros((batch, rows, width), np.float32)
    for turn in range(3):
        x = synth.normal_f32(turn, "graph.rows", (batch, rows, width))
        starts, counts = [turn, 28, 3 * turn], [rows, 3, turn]
        k.copy_(dev(x.reshape(-1, width)))
        v.copy_(k)
        pos.copy_(ints(starts))
        count.copy_(ints(counts))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for s in range(batch):
            kp.store(want[s], Q4, width, cap, starts[s], x[s, :counts[s]])
            want_o[s, :counts[s]] = kp.values(want[s], Q4, width, cap)[starts[s]:starts[s] + counts[s]]
        assert err.item() == 0
        assert np.array_equal(kc.cpu().numpy(), want) and np.array_equal(vc.cpu().numpy(), want)
        assert np.array_equal(ko.cpu().numpy().reshape(want_o.shape), want_o)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rt", [F32, F16])
@pytest.mark.parametrize("width", [992, 1024])
def test_large_calls(q8d, kind, rt, width):
    """Calls large enough that a thread takes several groups: ragged ends
    inside a thread's groups, a sequence of one row, an empty and a refused
    one."""
    batch, rows, cap = 5, 2111, 2200
    stride = stride_of(cap, width)
    counts, starts = [2111, 1, 2109, 0, 2000], [89, 2199, 0, 5, 201]  # the last: past the end
    k, kx = rows_in(4, "large.k", batch, rows, width, rt, width, 0)
    v, vx = rows_in(5, "large.v", batch, rows, width, rt, width, 0)
    kc, vc = (torch.full((batch, kp.cache_bytes(kind, stride)), 0x11, dtype=torch.uint8, device="cuda") for _ in range(2))
    want = [c.cpu().numpy() for c in (kc, vc)]
    err = ints([0])
    q8d.q8d_kv_append_rows(k, v, rt, width, kc, vc, kind, batch, rows, width, cap, stride, ints(starts), ints(counts), err)
    torch.cuda.synchronize()
    assert err.item() == q8d.Q8D_DERR_POS_RANGE
    for s in range(4):
        for w, x in zip(want, (kx, vx)):
            kp.store(w[s], kind, width, cap, starts[s], x[s, :counts[s]])
    assert np.array_equal(kc.cpu().numpy(), want[0]) and np.array_equal(vc.cpu().numpy(), want[1])
    ko, vo = (torch.full((batch, rows, width), -7.0, dtype=TT[rt], device="cuda") for _ in range(2))
    q8d.q8d_kv_read_rows(kc, vc, kind, ko, vo, rt, width, batch, rows, width, cap, stride, ints(starts), ints(counts), err)
    torch.cuda.synchronize()
    for o, w in ((ko, want[0]), (vo, want[1])):
        o = o.cpu().numpy()
        for s in range(4):
            with np.errstate(over="ignore"):
                vals = kp.values(w[s], kind, width, cap)[starts[s]:starts[s] + counts[s]].astype(NP[rt])
            assert np.array_equal(o[s, :counts[s]], vals)
            assert np.all(o[s, counts[s]:] == -7.0)
        assert np.isnan(o[4]).all()
