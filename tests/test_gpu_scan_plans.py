"""The selective scan's kernels one by one: 16 and 8 states a lane with each
number of waves a channel, whole and padded, both types, gated or not, and the
step of a full batch.

How many states a lane has depends on the waves that a call fills: 16 from 512
waves on (8 or 4 where a channel has no more), halved below.  Segments of 16
tokens fill them with few tokens: groups of heads with rows of their own take a
wave each.  Bounds as in test_gpu_scan."""

import pytest
import torch

import gated_delta_rule_79_amd as gdn
from gpu_util import Padded, log
from test_gpu_scan import BF16, F32, Reference, gpu, make, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

# heads (each a group of its own), states -> states a lane, waves a channel, padded
PLANS = [(32, 16, (16, 1, False)), (32, 12, (16, 1, True)), (32, 32, (16, 2, False)),
         (32, 24, (16, 2, True)), (32, 20, (16, 2, True)), (32, 64, (16, 4, False)),
         (32, 48, (16, 4, True)), (32, 36, (16, 4, True)), (32, 8, (8, 1, False)),
         (20, 16, (8, 2, False)), (20, 12, (8, 2, True)), (10, 32, (8, 4, False)),
         (10, 28, (8, 4, True)), (10, 20, (8, 4, True))]


def plan(waves, dk):
    """States a lane, waves a channel, padded: the rule of the kernels' plan."""
    ns = 4 if dk <= 4 else 8 if dk <= 8 else 16
    split = lambda ns: next(w for w in (1, 2, 4, 8, 16) if w * ns >= dk)  # noqa: E731
    while ns > 4 and split(ns) < 8 and waves * split(ns) < 512:
        ns //= 2
    return ns, split(ns), dk != ns * split(ns)


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,dk,kind", PLANS)
def test_every_kernel(gpu_lib, H, dk, kind, dtype, gate):
    assert plan(17 * H, dk) == kind
    for cu in (None, [0, 5, 5, 100, 101, 267]):  # 17 segments of 16 tokens, the last one short
        log(f"[scan plan] {kind} {dtype} gate {gate} packed {cu is not None}")
        d = make(1, 267, H, H, dk, 5, dtype, cu=cu, gate=gate, s0=gate or cu is not None)
        ref, g = Reference(d, cu), gpu(d)
        ref.check_fwd(dtype, *run_fwd(g, cu, seg_chunks=1))
        ref.check_bwd(dtype, run_bwd(g, cu, seg_chunks=1), s0=d["s0"] is not None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [16, 24])
def test_groups_of_many_blocks(gpu_lib, dk, dtype):
    # 9 blocks of 64 channels in each of two groups, the last one of 8 channels;
    # 30 segments
    assert plan(30 * 18, dk) == ((16, 1, False) if dk == 16 else (16, 2, True))
    d = make(1, 470, 8, 2, dk, 130, dtype)
    ref, g = Reference(d, None), gpu(d)
    ref.check_fwd(dtype, *run_fwd(g, None, seg_chunks=1))
    ref.check_bwd(dtype, run_bwd(g, None, seg_chunks=1))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hb,dk", [(1, 16), (11, 24), (1, 64), (11, 4)])
def test_step_of_a_full_batch(gpu_lib, hb, dk, dtype, gate):
    # 132000 channels in all: four of them a thread
    N, H, dv = 300, 11, 40
    d = make(N, 1, H, hb, dk, dv, dtype, gate=gate)
    ref, g = Reference(d, None), gpu(d)
    one = {k: None if g[k] is None else g[k][:, 0].contiguous() for k in ("x", "dt", "b", "c", "z")}
    state = Padded(g["s0"].shape, F32)
    state.t.copy_(g["s0"])
    y = gdn.selective_scan_step(one["x"], one["dt"], g["a"], one["b"], one["c"], state.t, g["d"],
                                g["dt_bias"], one["z"])
    torch.cuda.synchronize()
    state.check("state")
    ref.check_fwd(dtype, y[:, None], state.t)
