"""GPU parity of the short convolution with a history (forward, backward,
step) against the fp64 oracle, element by element.

Bounds (u = 2^-24).  The sum p of W products and a bias is off by (W + 2) u P,
P the sum of their magnitudes.  An activation's slope and its derivative's
slope are at most 1.1, and both take 8 roundings and an exponential that is
off by 2 u (1 + |p|) (twice that in bf16): y is off by u (1.1 (W + 2) P +
(8 + 4 (1 + |p|)) |p|), e = dy act'(p) by u |dy| (1.1 (W + 2) P + 16 (1 +
|p|)).  Gradients are sums of e with taps or inputs: that error in place of
each e, plus one rounding a term.  bf16 outputs add one rounding, 2^-8 of the
value; the kept inputs are copies."""

import numpy as np
import pytest
import torch

import gated_delta_rule_79_amd as gdn
import oracle
from gated_delta_rule_79_amd import _lib
from gpu_util import Padded, log, np64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def make(B, T, H, d, W, dtype, cu=None, bias=True, s0=True, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    return dict(x=r(B, T, H, d).to(dtype), taps=r(H, d, W) / W ** 0.5,
                bias=r(H, d) * 0.3 if bias else None,
                s0=r(n, W - 1, H, d).to(dtype) if s0 else None, dy=r(B, T, H, d).to(dtype),
                ds=r(n, W - 1, H, d).to(dtype) if s0 else None)


def dev_cu(cu):
    return None if cu is None else torch.tensor(np.asarray(cu), dtype=torch.int32, device="cuda")


def compare(name, got, ref, tol, dtype):
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(ref)
    err = np.abs(np64(got) - ref)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    log(f"    {name}: worst error / bound {worst:.3f}")
    assert np.all(err <= tol + 1e-30), name


def check(d, cu, act, dtype, y, sf, grads, rows=slice(None)):
    f = {k: None if t is None else t.double().numpy() for k, t in d.items()}
    W = f["taps"].shape[-1]
    kw = dict(act=act, cu_seqlens=cu)
    ry, rs = oracle.conv_fwd(f["x"], f["taps"], f["bias"], f["s0"], **kw)
    m = {k: None if t is None else np.abs(t) for k, t in f.items()}
    P, _ = oracle.conv_fwd(m["x"], m["taps"], m["bias"], m["s0"], act="none", cu_seqlens=cu)
    p = np.abs(oracle.conv_fwd(f["x"], f["taps"], f["bias"], f["s0"], act="none", cu_seqlens=cu)[0])
    compare("y", y[:, rows], ry[:, rows],
            U * (1.1 * (W + 2) * P + (8 + 4 * (1 + p)) * p)[:, rows], dtype)
    if sf is not None:
        assert np.array_equal(np64(sf), rs), "s_final"
    if grads is None:
        return
    ref = oracle.conv_bwd(f["x"], f["taps"], f["dy"], f["bias"], f["s0"], f["ds"], **kw)
    off = U * m["dy"] * (1.1 * (W + 2) * P + 16 * (1 + p))
    wide = oracle.conv_bwd(f["x"], f["taps"], off, None, f["s0"], None, act="none", cu_seqlens=cu,
                           absolute=True)
    mag = oracle.conv_bwd(f["x"], f["taps"], f["dy"], f["bias"], f["s0"], f["ds"], act=act,
                          cu_seqlens=cu, absolute=True)
    n = f["x"].shape[0] * f["x"].shape[1]
    for name, g, r, w, a, k, dt in zip(("dx", "dtaps", "dbias", "ds0"), grads, ref, wide, mag,
                                       (W + 2, n + 2, n + 2, W + 2), (dtype, F32, F32, dtype)):
        if g is None:
            assert d[{"dbias": "bias", "ds0": "s0"}[name]] is None
            continue
        at = (slice(None), rows) if name == "dx" else (slice(None),)
        compare(name, g[at], r[at], (w + k * U * a)[at], dt)


def run(d, cu, act="silu", **kw):
    g = {k: None if t is None else t.cuda() for k, t in d.items()}
    c = dev_cu(cu)
    y, sf = gdn.short_conv_fwd(g["x"], g["taps"], g["bias"], g["s0"], act=act, cu_seqlens=c, **kw)
    grads = gdn.short_conv_bwd(g["x"], g["taps"], g["dy"], g["bias"], g["s0"], g["ds"], act=act,
                               cu_seqlens=c)
    torch.cuda.synchronize()
    return y, sf, grads


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("shape", [(2, 37, 3, 16), (1, 70, 2, 5), (3, 2, 1, 264)])
def test_dense(gpu_lib, shape, W, dtype):
    log(f"[short conv] {shape} W {W} {dtype}")
    d = make(*shape, W, dtype)
    check(d, None, "silu", dtype, *run(d, None))


PACKED = [[0, 40], [0, 0, 16, 16, 48, 48], [0, 1, 2, 3, 4, 5], [0, 15, 16, 17, 33, 100, 100],
          [0, 0, 0, 63, 64, 130], list(range(0, 80, 2))]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", PACKED)
def test_packed(gpu_lib, cu, dtype):
    for W, s0, bias in ((4, True, True), (4, False, True), (8, True, False), (2, True, True)):
        log(f"[short conv packed] {cu} W {W} {dtype}")
        d = make(1, cu[-1], 2, 24, W, dtype, cu=cu, s0=s0, bias=bias)
        check(d, cu, "silu", dtype, *run(d, cu))


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_activations(gpu_lib, act):
    for dtype in (F32, BF16):
        d = make(2, 50, 2, 40, 4, dtype, seed=7)
        d["x"][0, :5] *= 20
        check(d, None, act, dtype, *run(d, None, act))


def test_many_runs(gpu_lib):
    # more rows than the workgroups of a launch have at 16 tokens each
    d = make(1, 70000, 1, 8, 4, F32, cu=[0, 12345, 12346, 70000])
    check(d, [0, 12345, 12346, 70000], "silu", F32, *run(d, [0, 12345, 12346, 70000]))


def test_empty_sequences_keep_their_history(gpu_lib):
    for cu in (None, [0, 0, 0]):
        d = make(1 if cu else 2, 0, 2, 16, 4, BF16, cu=cu)
        y, sf, g = run(d, cu)
        assert y.numel() == 0 and torch.equal(sf.cpu(), d["s0"])
        assert torch.equal(g[3].cpu(), d["ds"]) and not g[1].any() and not g[2].any()


def test_rows_behind_the_last_sequence(gpu_lib):
    cu = [0, 20, 37]
    d = make(1, 60, 2, 16, 4, F32, cu=cu)
    d["x"][:, 37:] = float("nan")
    d["dy"][:, 37:] = float("nan")
    y = torch.full((1, 60, 2, 16), 7.0, device="cuda")
    y, sf, g = run(d, cu, y=y)
    assert bool((y[:, 37:] == 7.0).all())
    d["x"][:, 37:] = 0
    d["dy"][:, 37:] = 0
    check(d, cu, "silu", F32, y, sf, g, rows=slice(0, 37))


def test_bounds_out_of_order_stay_in_range(gpu_lib):
    d = make(1, 90, 2, 20, 4, F32, cu=[0] * 6)
    g = {k: t.cuda() for k, t in d.items()}
    for cu in ([0, 50, 20, 400, -7, 90], [5, 5, 1000, 3, 90, 10], [90, 0, 90, 0, 90, 0]):
        y, sf = Padded(d["x"].shape, F32), Padded(d["s0"].shape, F32)
        gdn.short_conv_fwd(g["x"], g["taps"], g["bias"], g["s0"], cu_seqlens=dev_cu(cu), y=y.t,
                           s_final=sf.t)
        gdn.short_conv_bwd(g["x"], g["taps"], g["dy"], g["bias"], g["s0"], g["ds"],
                           cu_seqlens=dev_cu(cu))
        torch.cuda.synchronize()
        y.check("y")
        sf.check("s_final")


def test_a_bad_sequence_stays_alone(gpu_lib):
    cu = [0, 13, 30, 64]
    d = make(1, 64, 2, 16, 4, F32, cu=cu)
    good = run(d, cu)
    d["x"][0, 28] = float("nan")
    d["dy"][0, 15] = float("inf")
    y, sf, g = run(d, cu)
    for lo, hi in ((0, 13), (30, 64)):
        assert torch.equal(y[:, lo:hi], good[0][:, lo:hi])
        assert torch.equal(g[0][:, lo:hi], good[2][0][:, lo:hi])
    assert torch.equal(sf[[0, 2]], good[1][[0, 2]]) and torch.equal(g[3][[0, 2]], good[2][3][[0, 2]])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("N,H,d", [(1, 1, 1), (5, 3, 16), (300, 2, 24), (33, 2, 7)])
def test_step(gpu_lib, N, H, d, W, dtype):
    i = make(N, 1, H, d, W, dtype)
    x = i["x"][:, 0].contiguous().cuda()
    state = Padded(i["s0"].shape, dtype)
    state.t.copy_(i["s0"])
    args = (i["taps"].cuda(), state.t, i["bias"].cuda())
    y = gdn.short_conv_step(x, *args)
    torch.cuda.synchronize()
    state.check("state")
    check(i, None, "silu", dtype, y[:, None], state.t, None)
    # the output in the input's place
    again = state.t.clone()
    want = gdn.short_conv_step(x, args[0], again.clone(), args[2])
    gdn.short_conv_step(x, args[0], again, args[2], y=x)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


def test_prefill_then_steps_equal_a_longer_prefill(gpu_lib):
    d = make(3, 20, 2, 16, 4, BF16)
    g = {k: t.cuda() for k, t in d.items()}
    whole, end = gdn.short_conv_fwd(g["x"], g["taps"], g["bias"], g["s0"])
    y, state = gdn.short_conv_fwd(g["x"][:, :2].contiguous(), g["taps"], g["bias"], g["s0"])
    ys = [y]
    for t in range(2, 20):
        ys.append(gdn.short_conv_step(g["x"][:, t].contiguous(), g["taps"], state, g["bias"])[:, None])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ys, 1), whole) and torch.equal(state, end)


def test_without_history_is_the_prologue(gpu_lib):
    d = make(2, 33, 2, 16, 4, F32, bias=False, s0=False)
    y, _ = gdn.short_conv_fwd(d["x"].cuda(), d["taps"].cuda(), output_final_state=False)
    p = gdn.prologue_fwd(d["x"].cuda(), d["taps"].cuda(), False)
    assert torch.allclose(y, p, rtol=1e-6, atol=1e-6)


def test_captured_and_replayed(gpu_lib):
    d = make(1, 100, 2, 32, 4, BF16, cu=[0, 40, 100])
    g = {k: t.cuda() for k, t in d.items()}
    cu = dev_cu([0, 40, 100])
    step = torch.randn(2, 2, 32, device="cuda").to(BF16)
    state = g["s0"].clone()

    def work():
        return [*gdn.short_conv_fwd(g["x"], g["taps"], g["bias"], g["s0"], cu_seqlens=cu),
                *gdn.short_conv_bwd(g["x"], g["taps"], g["dy"], g["bias"], g["s0"], g["ds"],
                                    cu_seqlens=cu),
                gdn.short_conv_step(step, g["taps"], state, g["bias"])]
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        g["x"].copy_(torch.randn(g["x"].shape, generator=torch.Generator().manual_seed(k)))
        state.copy_(g["s0"])
        graph.replay()
        torch.cuda.synchronize()
        after = state.clone()
        state.copy_(g["s0"])
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(after, state)


def test_offsets_past_four_gigabytes(gpu_lib):
    T, d = 270000, 8192
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, T, 1, d, generator=gen, device="cuda", dtype=BF16)
    taps = torch.randn(1, d, 4, generator=gen, device="cuda")
    y, sf = gdn.short_conv_fwd(x, taps)
    grads = gdn.short_conv_bwd(x, taps, x)
    tail = x[:, T - 100:].contiguous()
    y1, sf1 = gdn.short_conv_fwd(tail, taps)
    g1 = gdn.short_conv_bwd(tail, taps, tail)
    assert torch.equal(y[:, T - 97:], y1[:, 3:]) and torch.equal(sf, sf1)
    assert torch.equal(grads[0][:, T - 97:], g1[0][:, 3:])


def test_refusals(gpu_lib):
    d = {k: t.cuda() for k, t in make(2, 10, 2, 16, 4, F32).items()}
    bad = [dict(taps=d["taps"].double()), dict(taps=d["taps"][:1]), dict(x=d["x"].cpu()),
           dict(bias=d["bias"][:, :8]), dict(s0=d["s0"][:1]), dict(s0=d["s0"].to(BF16)),
           dict(act="relu"), dict(x=d["x"].half()), dict(x=d["x"][0]), dict(y=d["x"][:1]),
           dict(s_final=d["s0"], s0=d["s0"]), dict(taps=torch.zeros(2, 16, 9, device="cuda")),
           dict(x=d["x"].transpose(1, 2)),
           dict(cu_seqlens=torch.tensor([0], dtype=torch.int32, device="cuda"))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.short_conv_fwd(**{**dict(x=d["x"], taps=d["taps"]), **kw})
    for kw in (dict(dy=None), dict(dy=d["dy"][:1]), dict(dy=d["dy"], ds_final=d["s0"][:1])):
        with pytest.raises(ValueError):
            gdn.short_conv_bwd(d["x"], d["taps"], **kw)
    for state in (None, d["s0"][:, :1]):
        with pytest.raises(ValueError):
            gdn.short_conv_step(d["x"][:, 0].contiguous(), d["taps"], state)
    assert _lib.load()


def test_outputs_that_are_inputs_are_refused(gpu_lib):
    d = {k: t.cuda() for k, t in make(2, 10, 2, 16, 4, F32).items()}
    with pytest.raises(ValueError):
        gdn.short_conv_fwd(d["x"], d["taps"], y=d["x"])


def test_outputs_that_overlap_are_refused(gpu_lib):
    d = {k: t.cuda() for k, t in make(2, 10, 2, 16, 4, F32).items()}
    n = d["x"].numel()
    buf = torch.zeros(2 * n, device="cuda")
    x = buf[:n].view(d["x"].shape)
    kept = buf[n - 16:n - 16 + d["s0"].numel()].view(d["s0"].shape)
    for kw in (dict(x=x, y=buf[32:n + 32].view(x.shape)), dict(x=x, s_final=kept),
               dict(x=d["x"], s0=d["s0"], y=d["x"]),
               dict(x=d["x"], y=buf[:n].view(x.shape), s_final=kept)):
        with pytest.raises(ValueError):
            gdn.short_conv_fwd(taps=d["taps"], **kw)
    one = buf[:64].view(2, 2, 16)
    state = torch.zeros(2, 3, 2, 16, device="cuda")
    for kw in (dict(y=buf[16:80].view(2, 2, 16)), dict(y=state.view(-1)[:64].view(2, 2, 16))):
        with pytest.raises(ValueError):
            gdn.short_conv_step(one, d["taps"], state, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", [[0, 20, 37], [5, 20, 20, 41], [16, 16, 16]])
def test_gradients_outside_the_sequences_are_left_alone(gpu_lib, cu, dtype):
    # in front of the first and behind the last; the workspace holds NaN
    d = make(1, 60, 2, 16, 4, dtype, cu=cu)
    lo, hi = cu[0], cu[-1]
    for k in ("x", "dy"):
        d[k][:, :lo], d[k][:, hi:] = float("nan"), float("nan")
    g = {k: t.cuda() for k, t in d.items()}
    out = [torch.full_like(g[k], 7.0) for k in ("x", "taps", "bias", "s0")]
    ws = torch.full((1 << 20,), float("nan"), device="cuda")
    y = torch.full_like(g["x"], 7.0)
    y, sf = gdn.short_conv_fwd(g["x"], g["taps"], g["bias"], g["s0"], cu_seqlens=dev_cu(cu), y=y)
    got = gdn.short_conv_bwd(g["x"], g["taps"], g["dy"], g["bias"], g["s0"], g["ds"],
                             cu_seqlens=dev_cu(cu), workspace=ws, out=out)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(got, out))
    for t in (y, got[0]):
        assert bool((t[:, :lo] == 7.0).all()) and bool((t[:, hi:] == 7.0).all())
    inside = {k: t[:, lo:hi].contiguous() if k in ("x", "dy") else t for k, t in d.items()}
    check(inside, [n - lo for n in cu], "silu", dtype, y[:, lo:hi], sf,
          (got[0][:, lo:hi], *got[1:]))


def test_preallocated_gradients_are_checked(gpu_lib):
    d = {k: t.cuda() for k, t in make(2, 10, 2, 16, 4, F32).items()}
    out = [torch.empty_like(d[k]) for k in ("x", "taps", "bias", "s0")]
    ins = (d["x"], d["taps"], d["dy"], d["bias"], d["s0"], d["ds"])
    for bad in (out[:3], [out[0][:1], *out[1:]], [d["dy"], *out[1:]], [*out[:3], d["ds"]],
                [out[0], out[1].to(BF16), *out[2:]]):
        with pytest.raises(ValueError):
            gdn.short_conv_bwd(*ins, out=bad)
    with pytest.raises(ValueError):
        gdn.short_conv_bwd(*ins[:3], None, *ins[4:], out=out)
    got = gdn.short_conv_bwd(*ins, out=[None, out[1], None, None])
    assert got[1] is out[1] and got[3] is not None
