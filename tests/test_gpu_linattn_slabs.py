"""Linear attention in slabs of 64 of more than 64 columns, against the fp64
oracle (bounds as in test_gpu_linattn).  A launch takes them where its
workgroups would be more than 256 in slabs of 32 columns and are not in slabs
of 64; the shapes below meet that in the forward's walk, in the backward's
joined and single walks, and (cut) in the walks of the segments' states, with
whole and partial last slabs and every class of state rows."""

import pytest

import oracle
from gpu_util import log
from test_gpu_linattn import (BF16, F32, absolute, check, f64, make, run_bwd, run_fwd)

pytestmark = pytest.mark.gpu

ARGS = ("q", "k", "v", "log_decay", "s0")


def slabs_of_64(groups, N):
    return groups * -(-N // 32) > 256 >= groups * -(-N // 64)


def check_all(shape, dtype, seg):
    d, cu = make(*shape, dtype, do=True)
    f = f64(d)
    both = (f, absolute(f))
    n = shape[1] + max(shape[4:]) + 64
    fwd = [oracle.linattn_fwd(*(x[a] for a in ARGS)) for x in both]
    bwd = [oracle.linattn_bwd(*(x[a] for a in ARGS), x["do"], x["ds"]) for x in both]
    for name, g, r, a in zip(("o", "s_final"), run_fwd(d, cu, seg_chunks=seg), *fwd):
        check(name, g, r, a, dtype, n, state=name == "s_final")
    for name, g, r, a in zip(("dq", "dk", "dv", "ds0"), run_bwd(d, cu, seg_chunks=seg), *bwd):
        check(name, g, r, a, dtype, n, state=name == "ds0")


# B, T, H, Hq, dk, dv; (walks of a launch, columns) pairs that are in slabs of 64
WHOLE = [((2, 70, 60, 30, 16, 80), [(1, 80)]), ((2, 33, 60, 60, 32, 80), [(1, 80)]),
         ((1, 67, 80, 40, 64, 144), [(1, 144)]), ((1, 66, 60, 60, 128, 224), [(1, 224), (2, 128)]),
         ((1, 67, 40, 20, 128, 112), [(3, 128)]), ((1, 67, 60, 30, 128, 144), [(1, 144), (2, 128)]),
         ((1, 66, 80, 80, 16, 144), [(1, 144)])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,launches", WHOLE)
def test_whole(gpu_lib, shape, launches, dtype):
    log(f"[linattn slabs] {shape} {dtype}")
    assert all(slabs_of_64(shape[0] * shape[2] * n, N) for n, N in launches)
    check_all(shape, dtype, -1)


# two segments each: half the heads; the states' walks of the backward are two
CUT = [((1, 70, 60, 30, 32, 80), [(1, 80)]), ((1, 67, 40, 20, 64, 144), [(1, 144)]),
       ((1, 66, 30, 30, 128, 224), [(1, 224), (2, 128)]), ((1, 67, 20, 10, 128, 112), [(3, 128)]),
       ((1, 67, 30, 15, 128, 144), [(1, 144), (2, 128)]), ((1, 100, 20, 20, 16, 144), [(2, 144)]),
       ((1, 100, 30, 15, 128, 128), [(2, 128)])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,launches", CUT)
def test_cut(gpu_lib, shape, launches, dtype):
    log(f"[linattn slabs, cut] {shape} {dtype}")
    assert all(slabs_of_64(2 * shape[2] * n, N) for n, N in launches)
    check_all(shape, dtype, 1 if dtype == BF16 else 2)  # 64 tokens a segment
