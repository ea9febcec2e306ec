"""GPU parity of linear attention with a decay per head against the fp64
oracle, element by element.

Bounds, derived from the arithmetic.  Write A for an output with every
operand and state replaced by its absolute value (the sum of the magnitudes
of all terms of the exact expression).  u = 2^-24 is an fp32 half step, each
accumulated term passes at most n additions (n: rows of the contraction plus
tokens plus a few), so fp32 arithmetic is off by at most n u A.  With bf16
rows the copy of the state that multiplies them, x y^T and the weighted rows
that enter the state go in two operand parts each (2^-17 of a value left), the
state that is handed out keeps the fp32 value of each term in three, and the
result is rounded once (half a step, 2^-8 |out|).  The bounds here are wider:
2^-8 A besides, as one rounding of the state's copy and of x y^T would need;
test_gpu_linattn_rounding holds the outputs to one rounding of their own."""

import numpy as np
import pytest
import torch

import gated_delta_rule_79_amd as gdn
import oracle
from gpu_util import Padded, log, np64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def make(B, T, H, Hq, dk, dv, dtype, cu=None, s0=True, seed=1, decay="span", do=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    la = {"span": torch.log1p(-torch.exp2(-torch.linspace(1, 9, H))), "none": None,
          "zero": torch.full((H,), -float("inf")), "hard": torch.full((H,), -60.0),
          "one": torch.zeros(H)}[decay]
    d = dict(q=r(B, T, Hq, dk) / dk ** 0.5, k=r(B, T, Hq, dk), v=r(B, T, H, dv), log_decay=la,
             s0=torch.randn(n, H, dk, dv, generator=g) if s0 else None)
    if do:
        d["do"] = r(B, T, H, dv)
        d["ds"] = torch.randn(n, H, dk, dv, generator=g) if s0 else None
    cu = None if cu is None else np.asarray(cu)
    return d, cu


def f64(d):
    return {k: None if t is None else t.double().numpy() for k, t in d.items()}


def gpu(d):
    return {k: None if t is None else t.cuda() for k, t in d.items()}


def absolute(d):
    return {k: None if t is None else (t if k == "log_decay" else np.abs(t)) for k, t in d.items()}


def check(name, got, ref, mag, dtype, n, state=False):
    got = np64(got)
    tol = n * U * mag
    if dtype == BF16 and state:
        tol = tol + 2.0 ** -26 * mag
    if dtype == BF16 and not state:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -6) * mag + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got - ref)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    log(f"    {name}: worst error / bound {worst:.3f}")
    assert np.all(np.isfinite(got)) and np.all(err <= tol + 1e-30), name


def check_fwd(d, cu, dtype, o, sf):
    f = f64(d)
    args = ("q", "k", "v", "log_decay", "s0")
    ro, rs = oracle.linattn_fwd(*(f[a] for a in args), cu)
    m = absolute(f)
    mo, ms = oracle.linattn_fwd(*(m[a] for a in args), cu)
    n = d["q"].shape[1] + d["q"].shape[-1] + 64
    check("o", o, ro, mo, dtype, n)
    if sf is not None:
        check("s_final", sf, rs, ms, dtype, n, state=True)


def check_bwd(d, cu, dtype, got):
    f = f64(d)
    args = ("q", "k", "v", "log_decay", "s0", "do", "ds")
    ref = oracle.linattn_bwd(*(f[a] for a in args), cu)
    m = absolute(f)
    mag = oracle.linattn_bwd(*(m[a] for a in args), cu)
    n = d["q"].shape[1] + max(d["q"].shape[-1], d["v"].shape[-1]) + 64
    for name, g, r, a in zip(("dq", "dk", "dv", "ds0"), got, ref, mag):
        if g is not None:
            check(name, g, r, a, dtype, n, state=name == "ds0")


def run_fwd(d, cu, **kw):
    x = gpu(d)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, sf = gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], cu_seqlens=cud,
                                **kw)
    torch.cuda.synchronize()
    return o, sf


def run_bwd(d, cu, **kw):
    x = gpu(d)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], x["do"], x["ds"],
                              cu_seqlens=cud, **kw)
    torch.cuda.synchronize()
    return out


SHAPES = [  # B, T, H, Hq, dk, dv
    (1, 1, 1, 1, 16, 16), (2, 64, 2, 2, 16, 16), (1, 65, 3, 1, 32, 48), (2, 130, 4, 2, 64, 80),
    (1, 257, 2, 2, 128, 128), (1, 100, 6, 2, 128, 144), (1, 333, 2, 1, 64, 256),
    (3, 31, 2, 2, 128, 32), (1, 200, 2, 2, 32, 112)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(gpu_lib, shape, dtype):
    log(f"[linattn fwd] {shape} {dtype}")
    d, cu = make(*shape, dtype)
    for seg in (0, 1, 2, -1):
        o, sf = run_fwd(d, cu, seg_chunks=seg)
        check_fwd(d, cu, dtype, o, sf)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(gpu_lib, shape, dtype):
    log(f"[linattn bwd] {shape} {dtype}")
    d, cu = make(*shape, dtype, do=True)
    for seg in (0, 1, 2, -1):
        check_bwd(d, cu, dtype, run_bwd(d, cu, seg_chunks=seg))


# Enough heads that slabs are 128 columns wide (fewer workgroups than CUs take
# 64 or 32): every size class of rows and columns, partial slabs among them.
WIDE = [(2, 70, 66, 33, 128, 128), (1, 67, 88, 88, 64, 144), (1, 66, 70, 35, 128, 224),
        (2, 70, 66, 66, 32, 112), (2, 70, 66, 66, 16, 80)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", WIDE)
def test_many_heads(gpu_lib, shape, dtype):
    log(f"[linattn many heads] {shape} {dtype}")
    d, cu = make(*shape, dtype, do=True)
    f = f64(d)
    m = absolute(f)
    args = ("q", "k", "v", "log_decay", "s0")
    n = shape[1] + max(shape[4:]) + 64
    fwd = [oracle.linattn_fwd(*(x[a] for a in args)) for x in (f, m)]
    bwd = [oracle.linattn_bwd(*(x[a] for a in args), x["do"], x["ds"]) for x in (f, m)]
    for seg in (-1, 1):
        for name, g, r, a in zip(("o", "s_final"), run_fwd(d, cu, seg_chunks=seg), *fwd):
            check(name, g, r, a, dtype, n, state=name == "s_final")
        for name, g, r, a in zip(("dq", "dk", "dv", "ds0"), run_bwd(d, cu, seg_chunks=seg), *bwd):
            check(name, g, r, a, dtype, n, state=name == "ds0")


CUTS = [[0, 0, 1, 64, 64, 129, 300], [0, 300], [0, 150, 150], [0, 63, 127, 300], [0, 1, 2, 3]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", CUTS)
def test_packed(gpu_lib, cu, dtype):
    log(f"[linattn packed] {cu} {dtype}")
    d, cu = make(1, cu[-1], 4, 2, 64, 48, dtype, cu=cu, do=True)
    for seg in (0, 1, 2, -1):
        check_fwd(d, cu, dtype, *run_fwd(d, cu, seg_chunks=seg))
        check_bwd(d, cu, dtype, run_bwd(d, cu, seg_chunks=seg))


def test_many_sequences(gpu_lib):
    # more sequences than lanes of a wave, with empty ones at the borders
    rng = np.random.default_rng(2)
    n = rng.integers(0, 9, 200)
    n[[0, 63, 64, 127, 199]] = 0
    n[70] = 200
    cu = np.concatenate([[0], np.cumsum(n)])
    d, cu = make(1, int(cu[-1]), 2, 2, 32, 16, BF16, cu=cu, do=True)
    for seg in (0, 1, -1):
        check_fwd(d, cu, BF16, *run_fwd(d, cu, seg_chunks=seg))
        check_bwd(d, cu, BF16, run_bwd(d, cu, seg_chunks=seg))


@pytest.mark.parametrize("decay", ["none", "zero", "hard", "one"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decays(gpu_lib, decay, dtype):
    d, cu = make(1, 200, 2, 2, 32, 32, dtype, do=True, decay=decay)
    for seg in (1, -1):
        check_fwd(d, cu, dtype, *run_fwd(d, cu, seg_chunks=seg))
        check_bwd(d, cu, dtype, run_bwd(d, cu, seg_chunks=seg))


def test_without_states(gpu_lib):
    d, cu = make(2, 150, 2, 1, 64, 64, BF16, s0=False, do=True)
    o, sf = run_fwd(d, cu, output_final_state=False)
    assert sf is None
    check_fwd(d, cu, BF16, o, sf)
    got = run_bwd(d, cu, need_ds0=False)
    assert got[3] is None
    check_bwd(d, cu, BF16, got)


def test_empty_batch_keeps_the_state(gpu_lib):
    for cu in (None, [0, 0, 0]):
        d, cu = make(1, 0, 2, 2, 32, 48, BF16, cu=cu, do=True)
        _, sf = run_fwd(d, cu)
        assert torch.equal(sf.cpu(), d["s0"])
        assert torch.equal(run_bwd(d, cu)[3].cpu(), d["ds"])


@pytest.mark.parametrize("grouped", [False, True])
def test_outputs_stay_in_their_bounds(gpu_lib, grouped):
    # rows behind the last sequence are left alone, nothing outside is written
    T, used = 300, 211
    d, cu = make(1, T, 4, 2 if grouped else 4, 64, 80, BF16, cu=[0, 100, used], do=True)
    x = gpu(d)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for name in ("q", "k", "v", "do"):
        x[name][:, used:] = float("nan")
    pads = {n: Padded(t.shape, t.dtype) for n, t in
            (("o", d["v"]), ("sf", d["s0"]), ("dq", d["q"]), ("dk", d["k"]), ("dv", d["v"]),
             ("ds0", d["s0"]))}
    for p in pads.values():
        p.t.fill_(7.0)
    gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], cu_seqlens=cud,
                        o=pads["o"].t, s_final=pads["sf"].t, seg_chunks=1)
    gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], x["do"], x["ds"],
                        cu_seqlens=cud, seg_chunks=1,
                        out=tuple(pads[n].t for n in ("dq", "dk", "dv", "ds0")))
    torch.cuda.synchronize()
    for n, p in pads.items():
        p.check(n)
        if n in ("o", "dq", "dk", "dv"):
            assert bool((p.t[:, used:] == 7.0).all()), n
            assert bool(torch.isfinite(p.t[:, :used].float()).all()), n
    short = {n: (t[:, :used] if n in ("q", "k", "v", "do") else t) for n, t in d.items()}
    check_fwd(short, cu, BF16, pads["o"].t[:, :used], pads["sf"].t)
    check_bwd(short, cu, BF16, (pads["dq"].t[:, :used], pads["dk"].t[:, :used],
                                pads["dv"].t[:, :used], pads["ds0"].t))


def test_a_bad_sequence_stays_alone(gpu_lib):
    d, cu = make(1, 192, 2, 2, 32, 32, BF16, cu=[0, 50, 120, 192], do=True)
    clean = run_fwd(d, cu, seg_chunks=1), run_bwd(d, cu, seg_chunks=1)
    bad = dict(d)
    for n in ("q", "k", "v", "do"):
        bad[n] = d[n].clone()
        bad[n][:, 50:120] = float("inf")
    dirty = run_fwd(bad, cu, seg_chunks=1), run_bwd(bad, cu, seg_chunks=1)
    for a, b in zip([*clean[0], *clean[1]], [*dirty[0], *dirty[1]]):
        if a.shape[0] == 3:  # states
            assert torch.equal(a[[0, 2]], b[[0, 2]])
        else:
            assert torch.equal(a[:, :50], b[:, :50]) and torch.equal(a[:, 120:], b[:, 120:])


def test_runs_are_equal(gpu_lib):
    d, cu = make(1, 700, 4, 2, 128, 128, BF16, do=True)
    a = [*run_fwd(d, cu), *run_bwd(d, cu)]
    b = [*run_fwd(d, cu), *run_bwd(d, cu)]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_long_state_keeps_fp32(gpu_lib):
    # 4096 tokens under a slow decay: the state's error stays that of fp32
    # sums (the bound's n u A), not of bf16 products
    d, cu = make(1, 4096, 2, 2, 32, 32, BF16, decay="one")
    d["log_decay"] = torch.tensor([-1e-4, -1e-6])
    for seg in (0, 8):
        o, sf = run_fwd(d, cu, seg_chunks=seg)
        check_fwd(d, cu, BF16, o, sf)
        f = f64(d)
        _, rs = oracle.linattn_fwd(f["q"], f["k"], f["v"], f["log_decay"], f["s0"])
        rel = np.linalg.norm(np64(sf) - rs) / np.linalg.norm(rs)
        assert rel < 2e-6, rel  # sqrt(4096 roundings) u = 3.8e-6 of the largest partial sum


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 4, 2, 32, 48), (5, 6, 3, 64, 80),
                                   (2, 2, 2, 128, 256)])
def test_decode(gpu_lib, shape, dtype):
    N, H, Hq, dk, dv = shape
    d, _ = make(N, 3, H, Hq, dk, dv, dtype)
    x = gpu(d)
    state = x["s0"].clone()
    outs = [gdn.linear_attn_decode_step(x["q"][:, t].contiguous(), x["k"][:, t].contiguous(),
                                        x["v"][:, t].contiguous(), x["log_decay"], state)
            for t in range(3)]
    torch.cuda.synchronize()
    f = f64(d)
    args = ("q", "k", "v", "log_decay", "s0")
    ro, rs = oracle.linattn_fwd(*(f[a] for a in args))
    m = absolute(f)
    mo, ms = oracle.linattn_fwd(*(m[a] for a in args))
    n = dk + 8  # all fp32: only o's rounding is coarser
    err = np.abs(np64(torch.stack(outs, 1)) - ro)
    assert np.all(err <= n * U * mo + (2.0 ** -8 * np.abs(ro) if dtype == BF16 else 0))
    assert np.all(np.abs(np64(state) - rs) <= n * U * ms)


def test_prefill_then_decode_equals_longer_prefill(gpu_lib):
    d, cu = make(2, 97, 4, 2, 64, 64, F32)
    x = gpu(d)
    o_all, s_all = run_fwd(d, cu)
    cut = {k: (t[:, :96].contiguous() if k in "qkv" else t) for k, t in x.items()}
    _, s = gdn.linear_attn_fwd(cut["q"], cut["k"], cut["v"], x["log_decay"], x["s0"])
    o = gdn.linear_attn_decode_step(x["q"][:, 96].contiguous(), x["k"][:, 96].contiguous(),
                                    x["v"][:, 96].contiguous(), x["log_decay"], s)
    torch.cuda.synchronize()
    f = f64(d)
    m = absolute(f)
    mo, ms = oracle.linattn_fwd(*(m[a] for a in ("q", "k", "v", "log_decay", "s0")))
    # two fp32 evaluations of the same sums: twice the bound of one
    assert np.all(np.abs(np64(o) - np64(o_all[:, 96])) <= 2 * 225 * U * mo[:, 96])
    assert np.all(np.abs(np64(s) - np64(s_all)) <= 2 * 225 * U * ms)


def test_training_block(gpu_lib):
    """A retention block's core as a training step runs it: attention, group
    norm under a SiLU gate, and both backwards, against the oracle's chain."""
    B, T, H, dk, dv = 1, 150, 4, 32, 64
    d, cu = make(B, T, H, 2, dk, dv, F32, s0=False, do=True)
    g = torch.Generator().manual_seed(9)
    z, dy = torch.randn(B, T, H, dv, generator=g), torch.randn(B, T, H, dv, generator=g)
    w, b = torch.randn(H, dv, generator=g), torch.randn(H, dv, generator=g)
    x = gpu(d)
    o, _ = gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"])
    y = gdn.group_norm_fwd(o, w.cuda(), b.cuda(), z.cuda())
    do, dz, dw, db = gdn.group_norm_bwd(o, dy.cuda(), w.cuda(), b.cuda(), z.cuda())
    dq, dk_, dv_, _ = gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], None, do,
                                          need_ds0=False)
    torch.cuda.synchronize()
    f = f64(d)
    ro, _ = oracle.linattn_fwd(f["q"], f["k"], f["v"], f["log_decay"])
    n64 = [t.double().numpy() for t in (w, b, z, dy)]
    ry = oracle.group_norm_fwd(ro, *n64[:3])
    rdo, rdz, rdw, rdb = oracle.group_norm_bwd(ro, n64[3], *n64[:3])
    rq, rk, rv, _ = oracle.linattn_bwd(f["q"], f["k"], f["v"], f["log_decay"], None, rdo)
    # fp32 throughout: the attention's sums (T + dk terms, conditioned by
    # |terms| / |sum| <= 2^6 here) and the norm's division by the row's scale
    for name, a, r in (("y", y, ry), ("dz", dz, rdz), ("dw", dw, rdw), ("db", db, rdb),
                       ("dq", dq, rq), ("dk", dk_, rk), ("dv", dv_, rv)):
        rel = np.linalg.norm(np64(a) - r) / np.linalg.norm(r)
        log(f"    {name}: {rel:.2e}")
        assert rel < (T + dk) * U * 2 ** 6, name


@pytest.mark.parametrize("seg", [-1, 1])
def test_captured_and_replayed(gpu_lib, seg):
    d, cu = make(1, 300, 4, 2, 64, 64, BF16, cu=[0, 100, 300], do=True)
    x = gpu(d)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def step():
        o, sf = gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"],
                                    cu_seqlens=cud, seg_chunks=seg)
        g = gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], x["do"], x["ds"],
                                cu_seqlens=cud, seg_chunks=seg)
        return [o, sf, *g]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x["q"].copy_(torch.randn_like(x["q"]))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k


def test_offsets_past_four_gigabytes(gpu_lib):
    # the last sequence's rows lie behind 2^32 bytes of every tensor
    T, H, d = 600_000, 32, 128
    cu = [0, T - 130, T]
    x = {n: torch.zeros(1, T, H, d, dtype=BF16, device="cuda") for n in ("q", "k", "v", "do")}
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in x.values():
        t[:, cu[1]:] = torch.randn(130, H, d, generator=g, device="cuda").to(BF16)
    la = torch.log1p(-torch.exp2(-torch.linspace(1, 9, H))).cuda()
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    tail = {n: t[:, cu[1]:].contiguous() for n, t in x.items()}
    host = dict({n: t.cpu() for n, t in tail.items()}, log_decay=la.cpu(), s0=None)
    for seg in (-1, 4096):
        o, sf = gdn.linear_attn_fwd(x["q"], x["k"], x["v"], la, cu_seqlens=cud, seg_chunks=seg)
        o1, s1 = gdn.linear_attn_fwd(tail["q"], tail["k"], tail["v"], la, seg_chunks=-1)
        torch.cuda.synchronize()
        # Not cut, both walks are the same arithmetic.  Cut, the state that
        # multiplies q holds two operand parts of each product where the
        # other holds three: 2^-17 apart, an output's rounding may fall on
        # either side, so only the bounds above hold.
        if seg == -1:
            assert torch.equal(o[:, cu[1]:], o1) and torch.equal(sf[1], s1[0])
        check_fwd(host, None, BF16, o[:, cu[1]:], sf[1:])
        assert not sf[0].any()
    del o
    got = gdn.linear_attn_bwd(x["q"], x["k"], x["v"], la, None, x["do"], cu_seqlens=cud,
                              need_ds0=False, seg_chunks=-1)
    one = gdn.linear_attn_bwd(tail["q"], tail["k"], tail["v"], la, None, tail["do"],
                              need_ds0=False, seg_chunks=-1)
    torch.cuda.synchronize()
    for a, b in zip(got[:3], one[:3]):
        assert torch.equal(a[:, cu[1]:], b)


def test_overlapping_bounds_stay_in_range(gpu_lib):
    # malformed bounds are the caller's fault, but reach no memory outside
    d, _ = make(1, 300, 2, 2, 32, 32, BF16, cu=[0, 1, 2, 3, 4], do=True)
    x = gpu(d)
    cud = torch.tensor([0, 300, 0, 300, 0], dtype=torch.int32, device="cuda")
    need = gdn._bytes
    pads = {n: Padded(t.shape, t.dtype) for n, t in
            (("o", d["v"]), ("sf", d["s0"]), ("dq", d["q"]), ("dk", d["k"]), ("dv", d["v"]),
             ("ds0", d["s0"]))}
    p, hq, _ = gdn._linattn_problem(x["q"], x["k"], x["v"], x["log_decay"], cud, 1, 2)
    ws = Padded((need(gpu_lib.gdn_linear_attn_bwd_workspace, p, hq),), torch.uint8)
    gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], cu_seqlens=cud,
                        o=pads["o"].t, s_final=pads["sf"].t, seg_chunks=1, workspace=ws.t)
    gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], x["do"], x["ds"],
                        cu_seqlens=cud, seg_chunks=1, workspace=ws.t,
                        out=tuple(pads[n].t for n in ("dq", "dk", "dv", "ds0")))
    torch.cuda.synchronize()
    ws.check("workspace")
    for n, q in pads.items():
        q.check(n)


def test_two_streams_at_once(gpu_lib):
    jobs = [make(1, 500, 4, 4, 64, 64, BF16, seed=s, do=True)[0] for s in (1, 2)]
    want = [[*run_fwd(d, None), *run_bwd(d, None)] for d in jobs]
    xs = [gpu(d) for d in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(3):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                o, sf = gdn.linear_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"])
                g = gdn.linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], x["do"],
                                        x["ds"])
                got[i].append([o, sf, *g])
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_refusals(gpu_lib):
    d, _ = make(1, 20, 4, 2, 32, 32, BF16)
    x = gpu(d)
    q, k, v, la, s0 = (x[n] for n in ("q", "k", "v", "log_decay", "s0"))
    bad = [dict(k=k[:, :10].contiguous()), dict(k=k.float()), dict(v=v[:, :19].contiguous()),
           dict(v=v.float()), dict(la=la[:2]), dict(la=la.double()), dict(la=la.cpu()),
           dict(s0=s0[:, :2].contiguous()), dict(s0=s0.bfloat16()), dict(q=q.transpose(1, 2)),
           dict(v=v[..., ::2])]
    for kw in bad:
        a = dict(q=q, k=k, v=v, la=la, s0=s0)
        a.update(kw)
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.linear_attn_fwd(a["q"], a["k"], a["v"], a["la"], a["s0"])
    with pytest.raises(ValueError):
        gdn.linear_attn_fwd(q, k, v, la, s0, cu_seqlens=torch.tensor([0, 20], device="cuda"))
    with pytest.raises(ValueError):
        gdn.linear_attn_fwd(q, k, v, la, s0, cu_seqlens=torch.zeros(1, dtype=torch.int32,
                                                                    device="cuda"))
    with pytest.raises(TypeError):
        gdn.linear_attn_fwd(q.half(), k.half(), v.half(), la, s0)
    with pytest.raises(gdn.GdnError):
        gdn.linear_attn_fwd(q[..., :24].contiguous(), k[..., :24].contiguous(), v, la)
    with pytest.raises(gdn.GdnError):  # 3 q heads do not divide 4
        q3 = torch.zeros(1, 20, 3, 32, device="cuda", dtype=BF16)
        gdn.linear_attn_fwd(q3, q3, v, la)
    with pytest.raises(ValueError):
        gdn.linear_attn_bwd(q, k, v, la, s0, v.float())
    # outputs of another shape, type, layout or memory
    for kw in (dict(o=torch.empty_like(v, device="cpu")), dict(o=v.float()),
               dict(o=torch.empty(1, 4, 20, 32, device="cuda", dtype=BF16).transpose(1, 2)),
               dict(s_final=s0.cpu()), dict(s_final=s0[:, :2].contiguous()),
               dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            gdn.linear_attn_fwd(q, k, v, la, s0, **kw)
    for i, t in ((0, q.cpu()), (1, k.float()), (2, v[:, :4].contiguous()), (3, s0.cpu())):
        out = [None] * 4
        out[i] = t
        with pytest.raises(ValueError):
            gdn.linear_attn_bwd(q, k, v, la, s0, v, out=out)
    with pytest.raises(ValueError):
        gdn.linear_attn_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                    v[:, 0].contiguous(), la, s0.bfloat16())
