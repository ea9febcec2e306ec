"""Packed batches of linear attention whose sequences are partly cut into
segments and partly walked whole, against the fp64 oracle (bounds as in
test_gpu_linattn)."""

import numpy as np
import pytest
import torch

import gated_delta_rule_79_amd as gdn
from gpu_util import log
from test_gpu_linattn import BF16, F32, check_bwd, check_fwd, make, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

# lengths of n sequences: short ones, and long ones at the borders of the 64
# lanes that look for them (long: more than six chunks, so cut by themselves)
def bounds(n, long_at, long, seed=3):
    length = np.random.default_rng(seed).integers(0, 6, n)
    length[list(long_at)] = long
    return np.concatenate([[0], np.cumsum(length)])


CASES = [(130, (0, 63, 64, 129), 500), (130, (128,), 450), (65, (63, 64), 385), (300, (), 0),
         (200, tuple(range(60, 70)), 129)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,long_at,long", CASES)
def test_long_among_short(gpu_lib, n, long_at, long, dtype):
    log(f"[linattn packed] {n} sequences, {long} tokens at {long_at} {dtype}")
    cu = bounds(n, long_at, long)
    d, cu = make(1, int(cu[-1]), 2, 1, 16, 16, dtype, cu=cu, do=True)
    for seg in (0, 2, -1):
        check_fwd(d, cu, dtype, *run_fwd(d, cu, seg_chunks=seg))
        check_bwd(d, cu, dtype, run_bwd(d, cu, seg_chunks=seg))


@pytest.mark.parametrize("dv", [48, 144])
def test_partly_cut_with_other_tiles(gpu_lib, dv):
    # dv's walk apart from the other two; states of whole sequences are taken
    # and left as matrices, those of cut ones in register order
    cu = bounds(70, (3, 69), 150)
    d, cu = make(1, int(cu[-1]), 4, 2, 128, dv, BF16, cu=cu, do=True)
    for seg in (1, 2):
        check_fwd(d, cu, BF16, *run_fwd(d, cu, seg_chunks=seg))
        check_bwd(d, cu, BF16, run_bwd(d, cu, seg_chunks=seg))


def test_partly_cut_without_states(gpu_lib):
    cu = bounds(70, (3, 69), 150)
    d, cu = make(1, int(cu[-1]), 2, 2, 32, 32, BF16, cu=cu, s0=False, do=True)
    for seg in (1, -1):
        o, sf = run_fwd(d, cu, seg_chunks=seg, output_final_state=False)
        assert sf is None
        check_fwd(d, cu, BF16, o, sf)
        check_bwd(d, cu, BF16, run_bwd(d, cu, seg_chunks=seg, need_ds0=False))


def test_whole_sequences_do_not_see_the_cut_ones(gpu_lib):
    # a short sequence's rows and state are those of a batch without the long one
    cu = bounds(40, (7,), 300)
    d, cu = make(1, int(cu[-1]), 2, 2, 32, 48, BF16, cu=cu, do=True)
    o, sf = run_fwd(d, cu, seg_chunks=1)
    g = run_bwd(d, cu, seg_chunks=1)
    keep = np.concatenate([np.arange(cu[7]), np.arange(cu[8], cu[-1])])
    others = np.delete(np.arange(40), 7)
    short = {k: t if t is None or k == "log_decay" else
             t[others] if k in ("s0", "ds") else t[:, keep] for k, t in d.items()}
    length = np.delete(np.diff(cu), 7)
    cu1 = np.concatenate([[0], np.cumsum(length)])
    o1, sf1 = run_fwd(short, cu1, seg_chunks=-1)
    g1 = run_bwd(short, cu1, seg_chunks=-1)
    assert torch.equal(o[:, keep], o1) and torch.equal(sf[others], sf1)
    for a, b in zip(g[:3], g1):
        assert torch.equal(a[:, keep], b)
    assert torch.equal(g[3][others], g1[3])


def test_partly_cut_captured_and_replayed(gpu_lib):
    cu = bounds(70, (3, 69), 150)
    d, cu = make(1, int(cu[-1]), 2, 2, 32, 32, BF16, cu=cu, do=True)
    x = {k: t.cuda() for k, t in d.items()}
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def step():
        kw = dict(cu_seqlens=cud, seg_chunks=1)
        a = (x["q"], x["k"], x["v"], x["log_decay"], x["s0"])
        return [*gdn.linear_attn_fwd(*a, **kw), *gdn.linear_attn_bwd(*a, x["do"], x["ds"], **kw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    rng = np.random.default_rng(8)
    for k in range(4):
        # other rows and, in the same buffers, other bounds: other sequences are cut
        x["q"].copy_(torch.randn_like(x["q"]))
        at = np.sort(rng.integers(0, cu[-1] + 1, 69))
        cud.copy_(torch.tensor(np.concatenate([[0], at, [cu[-1]]]), dtype=torch.int32))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k
