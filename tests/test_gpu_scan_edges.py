"""The selective scan where its contract has edges: rows outside every
sequence, gates and steps at the ends of their range, rates of -inf."""

import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_79_amd as gdn
from gated_delta_rule_79_amd import _lib
from gpu_util import log, np64
from test_gpu_scan import BF16, F32, U, Reference, dev_cu, gpu, make, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

ROWS = ("x", "dt", "b", "c", "z", "dy")


def bwd_into(g, cu, seg, fill):
    """The backward's C entry point on outputs that hold `fill` and a workspace
    of NaN."""
    lib = _lib.load()
    p, hb, _ = gdn._scan_problem(g["x"], g["dt"], g["a"], g["b"], g["c"], g["d"], g["dt_bias"],
                                 g["z"], cu, seg, 2)
    need = gdn._bytes(lib.gdn_selective_scan_bwd_workspace, p, hb)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    ins = [g[k] for k in ("x", "dt", "a", "b", "c", "d", "dt_bias", "z", "s0")]
    out = [torch.full_like(t, fill) for t in ins]
    gdn._launch(lib.gdn_selective_scan_bwd, g["x"].device, ctypes.byref(p), hb, 1,
                *(gdn._ptr(t) for t in (*ins, g["dy"], g["ds"], *out, ws)), need)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", [[0, 20, 37], [5, 20, 20, 41], [16, 16, 16]])
def test_rows_outside_the_sequences_are_left_alone(gpu_lib, cu, dtype):
    # in front of the first and behind the last; nothing of the workspace that
    # no walk has written reaches them
    d = make(1, 60, 2, 2, 16, 40, dtype, cu=cu)
    lo, hi = cu[0], cu[-1]
    for k in ROWS:
        d[k][:, :lo], d[k][:, hi:] = float("nan"), float("nan")
    inside = {k: t[:, lo:hi].contiguous() if k in ROWS else t for k, t in d.items()}
    ref, g = Reference(inside, [n - lo for n in cu]), gpu(d)
    rows = dict(zip((0, 1, 3, 4, 7), ("dx", "ddt", "db", "dc", "dz")))
    for seg in (0, 1, -1):
        y, sf = run_fwd(g, cu, seg_chunks=seg, y=torch.full_like(g["x"], 7.0))
        grads = bwd_into(g, dev_cu(cu), seg, 7.0)
        for name, t in (("y", y), *((rows[i], grads[i]) for i in rows)):
            assert bool((t[:, :lo] == 7.0).all()) and bool((t[:, hi:] == 7.0).all()), (name, seg)
        ref.check_fwd(dtype, y[:, lo:hi], sf)
        ref.check_bwd(dtype, [t[:, lo:hi] if i in rows else t for i, t in enumerate(grads)])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_of_the_lowest_value(gpu_lib, dtype):
    # silu and its slope are zero there (z times the zero of its sigmoid), and
    # so is all that such a token gives on: as behind a gate of -1000
    d = make(2, 37, 2, 1, 16, 40, dtype)
    off = torch.rand(2, 37, 2, 40, generator=torch.Generator().manual_seed(5)) < 0.3
    runs = []
    for low in (torch.finfo(dtype).min, -1000.0):
        d["z"] = torch.where(off, low, d["z"].float()).to(dtype)
        g = gpu(d)
        for seg in (1, -1):
            y, sf = run_fwd(g, None, seg_chunks=seg)
            grads = run_bwd(g, None, seg_chunks=seg)
            assert not y.cpu()[off].any() and not grads[7].cpu()[off].any()
            runs.append([y, sf, *grads])
        one = {k: g[k][:, 0].contiguous() for k in ("x", "dt", "b", "c", "z")}
        y = gdn.selective_scan_step(one["x"], one["dt"], g["a"], one["b"], one["c"],
                                    g["s0"].clone(), g["d"], g["dt_bias"], one["z"])
        assert not y.cpu()[off[:, 0]].any()
    for a, b in zip(runs[:2], runs[2:]):
        assert all(torch.equal(s, t) and bool(s.isfinite().all()) for s, t in zip(a, b))


def test_steps_over_their_whole_range(gpu_lib):
    # one token, one state that c reads with a one: y is delta itself, off by
    # at most 12 u of itself as the bounds of the other tests take it
    v = torch.cat([torch.linspace(-82.9, -20.0, 3001), torch.linspace(-20.0, 20.0, 8001),
                   torch.linspace(20.0, 90.0, 501)])
    n = v.numel()
    b = torch.tensor([1.0, 0.0, 0.0, 0.0]).view(1, 1, 1, 4).cuda()
    y, _ = gdn.selective_scan_fwd(torch.ones(1, 1, 1, n, device="cuda"), v.view(1, 1, 1, n).cuda(),
                                  torch.full((1, 4, n), -1.0, device="cuda"), b, b)
    want = np.logaddexp(v.double().numpy(), 0.0)
    err = np.abs(np64(y).reshape(-1) - want) / want / U
    at = int(err.argmax())
    log(f"    worst error {err[at]:.2f} u at {float(v[at]):.3f}")
    assert err.max() <= 12.0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_step_that_is_nan_is_seen(gpu_lib, dtype):
    # from its token on, in its channel; nothing in front of it
    d = make(1, 40, 1, 1, 8, 24, dtype)
    d["dt"][0, 13, 0, 7] = float("nan")
    g = gpu(d)
    for seg in (1, -1):
        y, sf = run_fwd(g, None, seg_chunks=seg)
        bad = y.isnan().cpu()[0, :, 0]
        assert bool(bad[13:, 7].all()) and not bad[:13].any() and not bad[:, :7].any()
        assert bool(sf.isnan()[0, 0, :, 7].all()) and int(sf.isnan().sum()) == 8


@pytest.mark.parametrize("shift", [-60.0, -82.0, -84.0, -88.0, -120.0, -1e30])
def test_rates_of_minus_infinity_and_hardly_a_step(gpu_lib, shift):
    # exp(delta a) of such a rate is zero however small delta is: the oracle
    # has a rate that even the least of them takes to zero.  (Its own steps are
    # zero from e^-746 down, which would keep what the rate takes: it has e^-600
    # there, both far below the bounds.)
    for cu in (None, [0, 37, 38, 70]):
        d = make(1 if cu else 2, 70, 2, 1, 16, 40, F32, cu=cu)
        d["dt_bias"] = torch.full_like(d["dt_bias"], max(shift, -600.0))
        gone = torch.rand(d["a"].shape, generator=torch.Generator().manual_seed(8)) < 0.25
        d["a"] = d["a"].double()
        d["a"][gone] = -1e300
        ref = Reference(d, cu)
        d["a"], d["dt_bias"] = d["a"].float(), torch.full_like(d["dt_bias"], shift)
        assert bool((d["a"][gone] == -float("inf")).all())
        g = gpu(d)
        for seg in (0, 1, -1):
            ref.check_fwd(F32, *run_fwd(g, cu, seg_chunks=seg))
            ref.check_bwd(F32, run_bwd(g, cu, seg_chunks=seg))
        one = {k: g[k][:, 0].contiguous() for k in ("x", "dt", "b", "c", "z")}
        state = g["s0"][:one["x"].shape[0]].clone()
        gdn.selective_scan_step(one["x"], one["dt"], g["a"], one["b"], one["c"], state, g["d"],
                                g["dt_bias"], one["z"])
        # (its token's write alone, delta x b with delta < 1e-25)
        assert float(state.cpu()[:, gone].abs().max()) < 1e-22


def test_rates_of_minus_infinity_and_steps_as_given(gpu_lib):
    # the least step that leaves nothing, and none, which leaves all
    H, dk, dv = 1, 4, 8
    one = lambda v: torch.full((1, 1, H, dv), v, device="cuda")  # noqa: E731
    b = torch.zeros(1, 1, 1, dk, device="cuda")
    a = torch.full((H, dk, dv), -float("inf"), device="cuda")
    s0 = torch.randn(1, H, dk, dv, generator=torch.Generator().manual_seed(1)).cuda()
    for step, left in ((4.4e-37, 0.0), (1e-30, 0.0), (1.0, 0.0), (0.0, 1.0)):
        _, sf = gdn.selective_scan_fwd(one(1.0), one(step), a, b, b, s0=s0, softplus=False)
        assert torch.equal(sf, s0 * left), step


def test_outputs_that_overlap_are_refused(gpu_lib):
    # also b and c, which have y's shape where each head has rows of its own,
    # and any part of a tensor
    H, n = 2, 16
    g = gpu(make(1, 10, H, H, n, n, F32))
    ins = {k: g[k] for k in ("x", "dt", "a", "b", "c")}
    buf = torch.zeros(3 * g["x"].numel(), device="cuda")
    size = g["x"].numel()
    part = lambda at, like: buf[at:at + like.numel()].view(like.shape)  # noqa: E731
    states = torch.zeros(2 * g["s0"].numel(), device="cuda")
    shared = states[H * n:H * n + g["s0"].numel()].view(g["s0"].shape)
    shared.copy_(g["s0"])
    bad = [dict(y=g["b"]), dict(y=g["c"]), dict(y=g["x"]), dict(y=g["z"], z=g["z"]),
           dict(x=part(0, g["x"]), y=part(8 * n, g["x"])),
           dict(b=part(size, g["x"]), y=part(size - 4, g["x"])),
           dict(s0=shared, s_final=states[:g["s0"].numel()].view(g["s0"].shape)),
           dict(a=g["s0"][0], s_final=g["s0"]),
           dict(y=states[:size].view(g["x"].shape), s_final=shared)]
    for kw in bad:
        with pytest.raises(ValueError):
            gdn.selective_scan_fwd(**{**ins, **kw})
    # parts that only touch are fine
    want, _ = gdn.selective_scan_fwd(**ins)
    x, y = part(0, g["x"]), part(size, g["x"])
    x.copy_(g["x"])
    gdn.selective_scan_fwd(**{**ins, "x": x}, y=y)
    assert torch.equal(y, want)
    one = {k: t[:, 0].contiguous() if k != "a" else t for k, t in ins.items()}
    for other in ("b", "c"):
        with pytest.raises(ValueError):
            gdn.selective_scan_step(**one, state=g["s0"].clone(), y=one[other])
    s = g["s0"].clone()
    with pytest.raises(ValueError):
        gdn.selective_scan_step(**one, state=s, y=s.view(-1)[:one["x"].numel()].view(1, H, n))
    # the step's own rows may be its output
    z = g["z"][:, 0].contiguous()
    want = gdn.selective_scan_step(**one, state=g["s0"].clone(), z=z)
    for k in ("x", "dt", "z"):
        rows = {n: t.clone() for n, t in {**one, "z": z}.items()}
        gdn.selective_scan_step(**rows, state=g["s0"].clone(), y=rows[k])
        assert torch.equal(rows[k], want), k


@pytest.mark.parametrize("cu", [None, [3, 20, 37]])
def test_preallocated_gradients(gpu_lib, cu):
    d = make(1 if cu else 2, 45, 2, 2, 16, 40, BF16, cu=cu)
    g = gpu(d)
    want = run_bwd(g, cu)
    lo, hi = (0, 45) if cu is None else (cu[0], cu[-1])
    out = [torch.full_like(t, 7.0) for t in want]
    got = run_bwd(g, cu, out=out)
    for i, (a, o, b) in enumerate(zip(got, out, want)):
        assert a is o
        if i in (0, 1, 3, 4, 7):
            assert bool((a[:, :lo] == 7.0).all()) and bool((a[:, hi:] == 7.0).all())
            a, b = a[:, lo:hi], b[:, lo:hi]
        assert torch.equal(a, b), i
    # some of them, and none of what is not there
    part = [torch.empty_like(out[0]), *[None] * 8]
    got = run_bwd({**g, "d": None, "z": None}, cu, out=part)
    assert got[0] is part[0] and got[5] is None and got[7] is None
    ins = [g[k] for k in ("x", "dt", "a", "b", "c", "dy", "d", "dt_bias", "z", "s0", "ds")]
    for bad in (out[:8], [out[0][:, :9], *out[1:]], [g["x"], *out[1:]], [g["dy"], *out[1:]],
                [out[0], out[0], *out[2:]], [*out[:3], out[0][..., :16], *out[4:]],
                [*out[:2], out[2].to(BF16), *out[3:]], [*out[:8], g["ds"]]):
        with pytest.raises(ValueError):
            gdn.selective_scan_bwd(*ins, cu_seqlens=dev_cu(cu), out=bad)
    with pytest.raises(ValueError):
        run_bwd({**g, "z": None}, cu, out=out)
