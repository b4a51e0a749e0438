"""What the entry points launch, seen from the host: the library runs in a child
process behind a stand-in for the CUDA runtime (fake_cudart.c) that launches
nothing, counts, and fails where it is told to.  No GPU."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = """
import ctypes as C, sys
fake, L = C.CDLL(sys.argv[1]), C.CDLL(sys.argv[2])
vp, i32, i64, f32 = C.c_void_p, C.c_int, C.c_longlong, C.c_float
L.q8d_q4_matmul.argtypes = [vp, i32, i64, vp, i32, vp, vp, i64, vp, i64, i32, i32, i32, vp]
L.q8d_q4_gated.argtypes = [vp, i32, i64, vp, vp, i32, vp, i64, i32, i32, i32, vp]
L.q8d_rmsnorm_rows.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, f32, vp, i32, i64, i32, i32, vp]
M = 1 << 40  # addresses, far apart
"""


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    from q8_block_quantized_matvec_gb300 import build
    lib = build.build()
    fake = str(tmp_path_factory.mktemp("fake") / "libfake_cudart.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", fake, os.path.join(HERE, "fake_cudart.c")], check=True)

    def run(code):
        env = dict(os.environ, LD_PRELOAD=fake)
        r = subprocess.run([sys.executable, "-S", "-c", CHILD + code, fake, lib], env=env, capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, r.stderr
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    return run


GATED = "L.q8d_q4_gated(M, 0, 3584, 2 * M, 3 * M, 32, 4 * M, 18944, {m}, 3584, 18944, None)"


@pytest.mark.parametrize("m", [11, 16])
def test_nothing_is_launched_where_a_call_fails(child, m):
    """The two launches of 9 to 16 f32 rows: whichever call of the runtime fails,
    only a launch's own failure may leave one behind."""
    call = GATED.format(m=m)
    (rc, calls, launches), = child(f"fake.fake_reset(0)\nprint({call}, fake.fake_calls(), fake.fake_launches())")
    assert rc == 0 and launches == 2
    refused = 0
    for at in range(1, calls + 1):
        (rc, done, launch), = child(
            f"fake.fake_reset({at})\nprint({call}, fake.fake_launches(), fake.fake_failed_launch())")
        # (a number of SMs that is not to be had is no failure: one is taken)
        assert (rc == 0 and not launch) or (rc == -5 and (done == 0 or launch)), at
        refused += rc != 0 and not launch
    assert refused > 10


@pytest.mark.parametrize("n", [1, 7, 32, 100, 3584])
@pytest.mark.parametrize("rows", [1, 2 ** 31 - 40, 2 ** 31 - 31, 2 ** 31 - 1])
def test_blocks_of_a_norm(child, rows, n):
    """Every row has a block, up to the largest count of rows."""
    (rc, launches, x, y, z, _, per, _), = child(f"""
fake.fake_reset(0)
rc = L.q8d_rmsnorm_rows(M, None, None, 1, {n}, 0, 0, 64 * M, 1e-6, 128 * M, 1, {n}, {rows}, {n}, None)
print(rc, fake.fake_launches(), *(fake.fake_grid(0, i) for i in range(6)))""")
    # (a block is threads of a row by rows)
    assert rc == 0 and launches == 1 and (x, y, z) == (-(-rows // per), 1, 1)


def statuses(child, calls):
    lines = "".join(f"print({c})\n" for c in calls)
    return [rc for rc, in child("fake.fake_reset(0)\n" + lines)]


def test_columns_of_one_buffer(child):
    """Operands that lie beside each other in the rows of one buffer are taken, and
    refused by the first byte that they share."""
    # rows of 200 f32: x from column 0, y from column 64, the sums from column 128
    norm = "L.q8d_rmsnorm_rows(M + {x}, {r}, {s}, 0, {ldx}, 200, 200, 64 * M, 1e-6, M + {y}, {yt}, {ldy}, 5, 64, None)"

    def n(x=0, r=None, s=None, ldx=200, y=256, yt=0, ldy=200):
        at = lambda v: "None" if v is None else f"M + {v}"  # noqa: E731
        return norm.format(x=x, r=at(r), s=at(s), ldx=ldx, y=y, yt=yt, ldy=ldy)
    good = [n(), n(s=512), n(r=512, s=512), n(y=0, x=256), n(y=800 + 256), n(x=800, y=544), n(y=256, yt=1, ldy=400),
            n(x=0, y=544, s=256)]
    bad = [n(y=252), n(y=4), n(y=548), n(x=256, y=4), n(s=316), n(r=512, s=516), n(y=256, ldy=196), n(y=256, yt=1, ldy=200),
           n(y=800 + 252), n(y=800 - 252), n(x=800, y=548)]
    assert statuses(child, good) == [0] * len(good)
    assert statuses(child, bad) == [-1] * len(bad)
    # rows of 160 f32: X 64 wide, Y and its residual 48
    mul = "L.q8d_q4_matmul(M + {x}, 0, 160, 2 * M, 32, None, {r}, 160, M + {y}, {ldy}, 3, 64, 48, None)"
    good = [mul.format(x=0, r="None", y=256, ldy=160), mul.format(x=0, r="M + 448", y=256, ldy=160),
            mul.format(x=0, r="M + 256", y=256, ldy=160), mul.format(x=192, r="None", y=0, ldy=160),
            mul.format(x=0, r="None", y=640 + 256, ldy=160)]
    bad = [mul.format(x=0, r="None", y=252, ldy=160), mul.format(x=0, r="M + 444", y=256, ldy=160),
           mul.format(x=192, r="None", y=4, ldy=160), mul.format(x=0, r="None", y=256, ldy=156),
           mul.format(x=0, r="None", y=452, ldy=160)]
    assert statuses(child, good) == [0] * len(good)
    assert statuses(child, bad) == [-1] * len(bad)
