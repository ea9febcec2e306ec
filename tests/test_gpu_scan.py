"""GPU parity of the selective scan (forward, backward, step) against the fp64
oracle, element by element.

Bounds, derived from the arithmetic (all of it fp32; u = 2^-24).  Write A for
an output with every operand replaced by its absolute value (the sum of the
magnitudes of all terms), A' for the same with a halved.  delta is off by at
most 12 u of itself (an exponential, a quotient and eight terms), the decay's
exponent delta a by two more roundings, the exponential by 2 u: a decay is off
by (14 |delta a| + 2) u, and a term that passes T of them and as many
multiply-adds by (14 s + 3 T) u with s the sum of its |delta a|.  Where a
segment's decay is taken from the sum of its delta, that sum is off by at most
T u of itself, s T u.  s e^{-s} < e^{-s/2}, so what goes with s is at most
(T + 14) u A'.  A sum of n terms adds n u A, the gate, the skip and the step's
derivative 64 u A.  Gradients pass two such walks and multiply by |a| (halved
in A'): twice the counts, four times A'.  bf16 outputs add one rounding,
2^-8 of the value."""

import ctypes

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
NAMES = ("x", "dt", "a", "b", "c", "d", "dt_bias", "z", "s0", "dy", "ds")


def make(B, T, H, hb, dk, dv, dtype, cu=None, gate=True, s0=True, affine=True, seed=1, rate=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    step = torch.exp(torch.rand(H, dv, generator=g) * 4.6 - 6.9)  # 0.001 .. 0.1
    return dict(
        x=r(B, T, H, dv).to(dtype), dt=(r(B, T, H, dv) * 0.5).to(dtype),
        a=-torch.exp(0.2 * r(H, dk, dv)) * torch.arange(1, dk + 1).view(1, dk, 1) * rate,
        b=r(B, T, hb, dk).to(dtype), c=r(B, T, hb, dk).to(dtype),
        d=r(H, dv) if affine else None,
        dt_bias=torch.log(torch.expm1(step)) if affine else None,
        z=r(B, T, H, dv).to(dtype) if gate else None,
        s0=r(n, H, dk, dv) if s0 else None,
        dy=r(B, T, H, dv).to(dtype), ds=r(n, H, dk, dv) if s0 else None)


def gpu(d):
    return {k: None if t is None else t.cuda() for k, t in d.items()}


def dev_cu(cu):
    return None if cu is None else torch.tensor(np.asarray(cu), dtype=torch.int32, device="cuda")


def run_fwd(g, cu, **kw):
    out = gdn.selective_scan_fwd(g["x"], g["dt"], g["a"], g["b"], g["c"], g["d"], g["dt_bias"],
                                 g["z"], g["s0"], cu_seqlens=dev_cu(cu), **kw)
    torch.cuda.synchronize()
    return out


def run_bwd(g, cu, **kw):
    out = gdn.selective_scan_bwd(g["x"], g["dt"], g["a"], g["b"], g["c"], g["dy"], g["d"],
                                 g["dt_bias"], g["z"], g["s0"], g["ds"], cu_seqlens=dev_cu(cu),
                                 **kw)
    torch.cuda.synchronize()
    return out


class Reference:
    """The oracle's outputs and the magnitudes behind their bounds."""

    def __init__(self, d, cu, softplus=True):
        f = {k: None if t is None else t.double().numpy() for k, t in d.items()}
        self.T = d["x"].shape[1]
        self.tokens = self.T * d["x"].shape[0]
        self.group = d["x"].shape[2] * d["x"].shape[3] // d["b"].shape[2]
        self.dk = d["a"].shape[1]
        ins = ("x", "dt", "a", "b", "c")
        opt = dict(d=f["d"], dt_bias=f["dt_bias"], z=f["z"], s0=f["s0"], softplus=softplus,
                   cu_seqlens=cu)
        self.fwd = oracle.scan_fwd(*(f[k] for k in ins), **opt)
        self.bwd = oracle.scan_bwd(*(f[k] for k in ins), f["dy"], ds_final=f["ds"], **opt)
        m = {k: None if t is None else np.abs(t) for k, t in f.items()}
        m["dt"] = np.abs(oracle.scan_delta(f["dt"], f["dt_bias"], softplus))
        self.mag = []
        for scale in (1.0, 0.5):
            opt = dict(d=m["d"], z=m["z"], s0=m["s0"], softplus=False, cu_seqlens=cu)
            args = (m["x"], m["dt"], f["a"] * scale, m["b"], m["c"])
            grads = list(oracle.scan_bwd(*args, m["dy"], ds_final=m["ds"], absolute=True, **opt))
            grads[6] = None if f["dt_bias"] is None else grads[1].sum((0, 1))
            self.mag.append((oracle.scan_fwd(*args, **opt), grads))

    def check(self, names, got, want, mag, half, dtypes, times, n):
        for name, g, r, m, h, dt in zip(names, got, want, mag, half, dtypes):
            if r is None or g is None:
                assert g is None, name
                continue
            count = n.get(name, self.dk)
            tol = U * (times * (3 * self.T + 64) + count) * m + U * times * times * (self.T + 14) * h
            if dt == BF16:
                tol = tol + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(r)
            x = np64(g)
            err = np.abs(x - r)
            worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
            log(f"    {name}: worst error / bound {worst:.3f}")
            assert np.all(np.isfinite(x)) and np.all(err <= tol + 1e-30), name

    def check_fwd(self, dtype, y, sf):
        self.check(("y", "s_final"), (y, sf), (self.fwd[0], None if sf is None else self.fwd[1]),
                   self.mag[0][0], self.mag[1][0], (dtype, F32), 1, {})

    def check_bwd(self, dtype, got, s0=True):
        names = ("dx", "ddt", "da", "db", "dc", "dd", "ddt_bias", "dz", "ds0")
        want = list(self.bwd)
        if not s0:
            want[8] = None
        types = (dtype, dtype, F32, dtype, dtype, F32, F32, dtype, F32)
        n = dict(da=self.tokens, dd=self.tokens, ddt_bias=self.tokens + self.dk, db=self.group,
                 dc=self.group)
        self.check(names, got, want, self.mag[0][1], self.mag[1][1], types, 2, n)


SHAPES = [  # B, T, H, hb, dk, dv
    (1, 1, 1, 1, 4, 1), (2, 64, 2, 1, 16, 16), (1, 65, 3, 3, 8, 48), (2, 130, 4, 2, 12, 5),
    (1, 257, 2, 1, 16, 128), (1, 100, 6, 2, 24, 44), (3, 31, 2, 2, 64, 32), (1, 150, 2, 1, 32, 70),
    (1, 90, 1, 1, 48, 130), (2, 40, 3, 1, 20, 33)]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_dense(gpu_lib, shape, dtype, gate):
    d = make(*shape, dtype, gate=gate)
    ref, g = Reference(d, None), gpu(d)
    for seg in (0, 1, 2, -1):
        log(f"[scan] {shape} {dtype} gate {gate} segments {seg}")
        ref.check_fwd(dtype, *run_fwd(g, None, seg_chunks=seg))
        ref.check_bwd(dtype, run_bwd(g, None, seg_chunks=seg))


PACKED = [[0, 40], [0, 0, 16, 16, 48, 48], [0, 1, 2, 3, 4, 5], [0, 15, 16, 17, 33, 100, 100],
          [0, 0, 0, 63, 64, 130], [0, 7, 7, 7, 90]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", PACKED)
def test_packed(gpu_lib, cu, dtype):
    for hb, dk, dv, seed in ((2, 16, 20, 3), (1, 24, 70, 4)):
        d = make(1, cu[-1], 2, hb, dk, dv, dtype, cu=cu, seed=seed)
        ref, g = Reference(d, cu), gpu(d)
        for seg in (0, 1, 2, -1):
            log(f"[scan packed] {cu} {dtype} dk {dk} segments {seg}")
            ref.check_fwd(dtype, *run_fwd(g, cu, seg_chunks=seg))
            ref.check_bwd(dtype, run_bwd(g, cu, seg_chunks=seg))


def test_many_sequences(gpu_lib):
    cu = np.concatenate([[0], np.cumsum(np.random.default_rng(5).integers(0, 9, 130))])
    d = make(1, int(cu[-1]), 2, 1, 8, 24, F32, cu=cu)
    ref, g = Reference(d, cu), gpu(d)
    for seg in (0, 1, 4):
        ref.check_fwd(F32, *run_fwd(g, cu, seg_chunks=seg))
        ref.check_bwd(F32, run_bwd(g, cu, seg_chunks=seg))


def test_without_options(gpu_lib):
    for cu in (None, [0, 5, 5, 70]):
        d = make(1 if cu else 2, 70, 2, 1, 16, 40, F32, cu=cu, gate=False, s0=False, affine=False)
        ref, g = Reference(d, cu), gpu(d)
        for seg in (1, -1):
            y, sf = run_fwd(g, cu, seg_chunks=seg, output_final_state=False)
            assert sf is None
            ref.check_fwd(F32, y, sf)
            ref.check_fwd(F32, *run_fwd(g, cu, seg_chunks=seg))
            ref.check_bwd(F32, run_bwd(g, cu, seg_chunks=seg), s0=False)


def test_steps_as_given(gpu_lib):
    # without the softplus; steps are positive
    d = make(2, 50, 2, 2, 16, 30, F32)
    d["dt"], d["dt_bias"] = d["dt"].abs() * 0.1, d["dt_bias"].exp()
    ref, g = Reference(d, None, softplus=False), gpu(d)
    for seg in (1, -1):
        ref.check_fwd(F32, *run_fwd(g, None, seg_chunks=seg, softplus=False))
        ref.check_bwd(F32, run_bwd(g, None, seg_chunks=seg, softplus=False))


@pytest.mark.parametrize("shift,rate", [(-30.0, 1.0), (-8.0, 0.01), (20.0, 1.0), (60.0, 3.0)])
def test_tiny_and_huge_steps(gpu_lib, shift, rate):
    # states that hardly move, hardly decay, or vanish within a token
    d = make(1, 70, 2, 1, 16, 16, F32, rate=rate)
    d["dt_bias"] = torch.full_like(d["dt_bias"], shift)
    ref, g = Reference(d, None), gpu(d)
    for seg in (1, -1):
        ref.check_fwd(F32, *run_fwd(g, None, seg_chunks=seg))
        ref.check_bwd(F32, run_bwd(g, None, seg_chunks=seg))


@pytest.mark.parametrize("packed", [False, True])
def test_empty_sequences_keep_the_state(gpu_lib, packed):
    cu = [0, 0, 0, 0] if packed else None
    d = make(1 if packed else 3, 0, 2, 1, 16, 20, BF16, cu=cu)
    g = gpu(d)
    y, sf = run_fwd(g, cu)
    got = run_bwd(g, cu)
    assert y.numel() == 0 and torch.equal(sf, g["s0"]) and torch.equal(got[8], g["ds"])
    for i in (2, 5, 6):
        assert not got[i].any()


def call(g, cu, bwd, pad):
    """The C entry point on outputs and a workspace that are watched."""
    lib = _lib.load()
    p, hb, states = gdn._scan_problem(g["x"], g["dt"], g["a"], g["b"], g["c"], g["d"],
                                      g["dt_bias"], g["z"], cu, pad.get("seg", 0), 2)
    need = gdn._bytes(getattr(lib, f"gdn_selective_scan_{'bwd' if bwd else 'fwd'}_workspace"), p,
                      hb)
    ws = Padded((max(need, 1),), torch.uint8)
    if bwd:
        like = [g[k] for k in ("x", "dt", "a", "b", "c", "d", "dt_bias", "z", "s0")]
        outs = [Padded(t.shape, t.dtype) for t in like]
        extra = [gdn._ptr(g["dy"]), gdn._ptr(g["ds"])]
        fn = lib.gdn_selective_scan_bwd
    else:
        outs = [Padded(g["x"].shape, g["x"].dtype), Padded(states, F32)]
        extra, fn = [], lib.gdn_selective_scan_fwd
    ins = [gdn._ptr(g[k]) for k in ("x", "dt", "a", "b", "c", "d", "dt_bias", "z", "s0")]
    st = fn(ctypes.byref(p), hb, 1, *ins, *extra, *(o.t.data_ptr() for o in outs),
            ws.t.data_ptr(), need, gdn._stream(g["x"].device))
    assert st == _lib.GDN_OK
    torch.cuda.synchronize()
    for i, o in enumerate([*outs, ws]):
        o.check(f"output {i}")
    return [o.t for o in outs]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dk,dv", [(16, 70), (12, 33), (40, 64), (8, 5)])
def test_outputs_stay_in_their_bounds(gpu_lib, dk, dv, packed):
    cu = [0, 3, 3, 50, 77] if packed else None
    d = make(1 if packed else 2, 77, 4, 2, dk, dv, BF16, cu=cu)
    g = gpu(d)
    for seg in (0, 1, -1):
        a = call(g, dev_cu(cu), False, dict(seg=seg))
        b = run_fwd(g, cu, seg_chunks=seg)
        assert all(torch.equal(s, t) for s, t in zip(a, b))
        a = call(g, dev_cu(cu), True, dict(seg=seg))
        b = run_bwd(g, cu, seg_chunks=seg)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_rows_behind_the_last_sequence(gpu_lib):
    cu = [0, 20, 37]
    d = make(1, 60, 2, 1, 16, 40, F32, cu=cu)
    for k in ("x", "dt", "b", "c", "z", "dy"):
        d[k][:, 37:] = float("nan")
    g = gpu(d)
    short = {k: (t[:, :37].contiguous() if k in ("x", "dt", "b", "c", "z", "dy") else t)
             for k, t in d.items()}
    ref = Reference(short, cu)
    for seg in (0, 1, -1):
        y = torch.full_like(g["x"], 7.0)
        y, sf = run_fwd(g, cu, seg_chunks=seg, y=y)
        assert bool((y[:, 37:] == 7.0).all())
        ref.check_fwd(F32, y[:, :37], sf)
        got = list(run_bwd(g, cu, seg_chunks=seg))
        for i in (0, 1, 3, 4, 7):
            got[i] = got[i][:, :37]
        ref.check_bwd(F32, got)


def test_a_bad_sequence_stays_alone(gpu_lib):
    cu = [0, 13, 30, 47, 64]
    d = make(1, 64, 2, 1, 16, 40, F32, cu=cu)
    ref = Reference(d, cu)
    for bad in (float("nan"), float("inf")):
        for k in ("x", "dt", "b", "c", "z", "dy"):
            e = {n: None if t is None else t.clone() for n, t in d.items()}
            e[k][0, 20] = bad
            g = gpu(e)
            for seg in (1, -1):
                y, sf = run_fwd(g, cu, seg_chunks=seg)
                got = run_bwd(g, cu, seg_chunks=seg)
                for lo, hi, n in ((0, 13, 0), (30, 47, 2), (47, 64, 3)):
                    for t, r in ((y, ref.fwd[0]), (got[0], ref.bwd[0]), (got[3], ref.bwd[3]),
                                 (got[4], ref.bwd[4]), (got[7], ref.bwd[7])):
                        assert np.allclose(np64(t)[:, lo:hi], r[:, lo:hi], rtol=1e-3, atol=1e-3)
                    assert np.allclose(np64(sf)[n], ref.fwd[1][n], rtol=1e-3, atol=1e-3)
                    assert np.allclose(np64(got[8])[n], ref.bwd[8][n], rtol=1e-3, atol=1e-3)


@pytest.mark.parametrize("token", [5, 60, 200, 399])
def test_a_bad_sequence_passes_no_segment_of_another(gpu_lib, token):
    # every sequence lies in several segments and ends inside one, so that the
    # states (and, backwards, the gradients) of a bad one meet the next one's
    # where the segments are chained
    cu = [0, 40, 70, 300, 360, 400]
    d = make(1, 400, 2, 1, 16, 40, F32, cu=cu)
    ref = Reference(d, cu)
    sick = int(np.searchsorted(cu, token, side="right")) - 1
    for bad in (float("nan"), float("inf")):
        e = {n: None if t is None else t.clone() for n, t in d.items()}
        for k in ("x", "dy"):
            e[k][0, token] = bad
        g = gpu(e)
        for seg in (0, 1, 2, -1):
            y, sf = run_fwd(g, cu, seg_chunks=seg)
            got = run_bwd(g, cu, seg_chunks=seg)
            for n in (i for i in range(5) if i != sick):
                lo, hi = cu[n], cu[n + 1]
                for t, r in ((y, ref.fwd[0]), (got[0], ref.bwd[0]), (got[1], ref.bwd[1]),
                             (got[3], ref.bwd[3]), (got[4], ref.bwd[4]), (got[7], ref.bwd[7])):
                    assert np.allclose(np64(t)[:, lo:hi], r[:, lo:hi], rtol=1e-3, atol=1e-3)
                assert np.allclose(np64(sf)[n], ref.fwd[1][n], rtol=1e-3, atol=1e-3)
                assert np.allclose(np64(got[8])[n], ref.bwd[8][n], rtol=1e-3, atol=1e-3)


def test_rates_of_minus_infinity(gpu_lib):
    # such a state holds its token's write alone: what a rate too large for any
    # step gives
    for cu in (None, [0, 37, 38, 70]):
        d = make(1 if cu else 2, 70, 2, 1, 16, 40, F32, cu=cu)
        gone = torch.rand(d["a"].shape, generator=torch.Generator().manual_seed(8)) < 0.25
        d["a"][gone] = -1e30
        ref = Reference(d, cu)
        d["a"][gone] = -float("inf")
        g = gpu(d)
        for seg in (0, 1, -1):
            ref.check_fwd(F32, *run_fwd(g, cu, seg_chunks=seg))
            ref.check_bwd(F32, run_bwd(g, cu, seg_chunks=seg))


def test_bounds_out_of_order_stay_in_range(gpu_lib):
    d = make(1, 90, 2, 1, 16, 40, F32, cu=[0] * 6)
    g = gpu(d)
    for cu in ([0, 50, 20, 400, -7, 90], [5, 5, 1000, 3, 90, 10], [90, 0, 90, 0, 90, 0]):
        for seg in (0, 1, -1):
            call(g, dev_cu(cu), False, dict(seg=seg))
            call(g, dev_cu(cu), True, dict(seg=seg))


def test_runs_are_equal(gpu_lib):
    d = make(2, 300, 4, 2, 16, 64, BF16)
    g = gpu(d)
    first = [*run_fwd(g, None), *run_bwd(g, None)]
    for _ in range(3):
        again = [*run_fwd(g, None), *run_bwd(g, None)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------- step ---

@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 4, 1), (3, 2, 1, 16, 64), (5, 6, 3, 24, 44),
                                   (40, 2, 2, 64, 30), (300, 3, 1, 8, 12)])
def test_step(gpu_lib, shape, dtype, gate):
    N, H, hb, dk, dv = shape
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


def test_prefill_then_steps_equal_a_longer_prefill(gpu_lib):
    d = make(2, 40, 4, 2, 16, 24, F32)
    ref, g = Reference(d, None), gpu(d)
    rows = ("x", "dt", "b", "c", "z")
    head = {k: (t[:, :33].contiguous() if k in rows else t) for k, t in g.items()}
    y, state = run_fwd(head, None)
    ys = [y]
    for t in range(33, 40):
        one = {k: g[k][:, t].contiguous() for k in rows}
        ys.append(gdn.selective_scan_step(one["x"], one["dt"], g["a"], one["b"], one["c"], state,
                                          g["d"], g["dt_bias"], one["z"])[:, None])
    torch.cuda.synchronize()
    ref.check_fwd(F32, torch.cat(ys, 1), state)


# ------------------------------------------------- graphs, streams, offsets ---

@pytest.mark.parametrize("seg", [0, -1])
def test_captured_and_replayed(gpu_lib, seg):
    d = make(1, 200, 2, 1, 16, 64, BF16, cu=[0, 90, 200])
    g = gpu(d)
    cu = dev_cu([0, 90, 200])
    fwd = lambda: gdn.selective_scan_fwd(  # noqa: E731
        g["x"], g["dt"], g["a"], g["b"], g["c"], g["d"], g["dt_bias"], g["z"], g["s0"],
        cu_seqlens=cu, seg_chunks=seg)
    bwd = lambda: gdn.selective_scan_bwd(  # noqa: E731
        g["x"], g["dt"], g["a"], g["b"], g["c"], g["dy"], g["d"], g["dt_bias"], g["z"], g["s0"],
        g["ds"], cu_seqlens=cu, seg_chunks=seg)
    fwd(), bwd()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [*fwd(), *bwd()]
    for k in range(4):
        for n in ("x", "dt", "dy", "s0"):
            g[n].copy_(torch.randn(g[n].shape, generator=torch.Generator().manual_seed(10 * k + 1)))
        graph.replay()
        torch.cuda.synchronize()
        want = [*fwd(), *bwd()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_two_streams_at_once(gpu_lib):
    sets = [gpu(make(1, 500, 2, 1, 16, 96, BF16, seed=s)) for s in (1, 2)]
    want = [[*run_fwd(g, None), *run_bwd(g, None)] for g in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got = []
        for g, s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append([
                    *gdn.selective_scan_fwd(g["x"], g["dt"], g["a"], g["b"], g["c"], g["d"],
                                            g["dt_bias"], g["z"], g["s0"]),
                    *gdn.selective_scan_bwd(g["x"], g["dt"], g["a"], g["b"], g["c"], g["dy"],
                                            g["d"], g["dt_bias"], g["z"], g["s0"], g["ds"])])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_offsets_past_four_gigabytes(gpu_lib):
    # a state that is forgotten within tens of tokens: the last tokens of a
    # long sequence are those of a short one
    T, H, dv, dk, last = 525312, 16, 256, 4, 600
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    x, dy = r(1, T, H, dv), r(1, T, H, dv)
    dt = torch.zeros(1, T, H, dv, device="cuda", dtype=BF16)
    b, c = r(1, T, 1, dk), r(1, T, 1, dk)
    a = torch.full((H, dk, dv), -1.0, device="cuda")
    assert x.numel() * 2 > 1 << 32
    tail = lambda t: t[:, T - last:].contiguous()  # noqa: E731
    y, sf = gdn.selective_scan_fwd(x, dt, a, b, c)
    y1, sf1 = gdn.selective_scan_fwd(tail(x), tail(dt), a, tail(b), tail(c))
    half = last // 2
    assert torch.allclose(y[:, T - half:].float(), y1[:, half:].float(), rtol=2.0 ** -7, atol=1e-4)
    assert torch.allclose(sf, sf1, rtol=1e-5, atol=1e-5)
    del y, sf
    g = gdn.selective_scan_bwd(x, dt, a, b, c, dy)
    g1 = gdn.selective_scan_bwd(tail(x), tail(dt), a, tail(b), tail(c), tail(dy))
    torch.cuda.synchronize()
    for i in (0, 1, 3, 4):
        assert torch.allclose(g[i][:, T - half:].float(), g1[i][:, half:].float(),
                              rtol=2.0 ** -7, atol=1e-3), i


def test_refusals(gpu_lib):
    d = make(2, 10, 4, 2, 16, 24, F32)
    g = gpu(d)
    ok = dict(x=g["x"], dt=g["dt"], a=g["a"], b=g["b"], c=g["c"])
    bad = [dict(dt=g["dt"][:, :9]), dict(a=g["a"].double()), dict(b=g["b"].to(BF16)),
           dict(c=g["c"][..., :8]), dict(x=g["x"].cpu()), dict(a=g["a"][:, :8]),
           dict(x=g["x"].transpose(1, 2)), dict(d=g["dt"]), dict(dt_bias=g["d"].cpu()),
           dict(z=g["x"].to(BF16)), dict(s0=g["s0"][:1]), dict(y=g["x"][:1]),
           dict(s_final=g["s0"].double()),
           dict(cu_seqlens=torch.tensor([0], dtype=torch.int32, device="cuda")),
           dict(cu_seqlens=torch.tensor([0, 10], device="cuda"))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.selective_scan_fwd(**{**ok, **kw})
    with pytest.raises(gdn.GdnError):  # packed rows of two sequences
        gdn.selective_scan_fwd(**ok, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32,
                                                             device="cuda"))
    for kw in (dict(dy=g["dy"][:1]), dict(dy=None), dict(dy=g["dy"], ds_final=g["s0"][:1])):
        with pytest.raises(ValueError):
            gdn.selective_scan_bwd(**ok, **kw)
    one = {k: v[:, 0].contiguous() if k != "a" else v for k, v in ok.items()}
    for state in (None, g["s0"][:1], g["s0"].double()):
        with pytest.raises(ValueError):
            gdn.selective_scan_step(**one, state=state)
    odd = make(1, 4, 1, 1, 8, 8, F32)
    odd["a"], odd["b"], odd["c"] = odd["a"][:, :6].contiguous(), *(odd[k][..., :6].contiguous() for k in "bc")
    with pytest.raises(gdn.GdnError):
        gdn.selective_scan_fwd(*(odd[k].cuda() for k in ("x", "dt", "a", "b", "c")))


def test_outputs_that_are_inputs_are_refused(gpu_lib):
    g = gpu(make(1, 10, 2, 1, 16, 24, F32))
    ins = (g["x"], g["dt"], g["a"], g["b"], g["c"])
    for kw in (dict(y=g["x"]), dict(y=g["dt"]), dict(y=g["z"], z=g["z"]),
               dict(s0=g["s0"], s_final=g["s0"])):
        with pytest.raises(ValueError):
            gdn.selective_scan_fwd(*ins, **kw)
