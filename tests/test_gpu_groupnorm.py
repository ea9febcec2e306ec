"""GPU parity of the causal group norm and its backward against the fp64
oracle, element by element.

Bounds.  All arithmetic is fp32 with at most 128 roundings along any path (8
additions a lane, 5 over the lanes of a row, twice, and some tens of
products, exponentials and quotients), each 2^-24 of magnitudes that are, for
a row with kappa = max|x| / sqrt(var + eps), at most (1 + kappa) times the
row's largest output before the activation: 2^-17 (1 + kappa) of that row's
magnitude M.  The exponential in bf16 runs adds |z| 2^-23, below the same
count for |z| < 32.  bf16 outputs add one half step, 2^-8 |y|."""

import numpy as np
import pytest
import torch

import gated_delta_rule_79_amd as gdn
import oracle
from gpu_util import Padded, log, np64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(B, T, H, d, dtype, affine="group", gate=True, seed=3, mean=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shape = {"group": (H, d), "shared": (d,), "none": None}[affine]
    return dict(x=(r(B, T, H, d) + mean).to(dtype), gate=r(B, T, H, d).to(dtype) if gate else None,
                weight=None if shape is None else r(*shape),
                bias=None if shape is None else r(*shape), dy=r(B, T, H, d).to(dtype))


def f64(t):
    return None if t is None else t.double().numpy()


def dev(t):
    return None if t is None else t.cuda()


def kappa(x, eps, center):
    c = x - x.mean(-1, keepdims=True) if center else x
    return 1 + np.abs(x).max(-1, keepdims=True) / np.sqrt((c * c).mean(-1, keepdims=True) + eps)


def check(name, got, ref, mag, dtype):
    err = np.abs(np64(got) - ref)
    tol = 2.0 ** -17 * mag + (2.0 ** -8 * np.abs(ref) if dtype == BF16 else 0)
    log(f"    {name}: worst error / bound {float(np.max(err / np.maximum(tol, 1e-300))):.3f}")
    assert np.all(err <= tol), name


def check_all(d, dtype, act, center, eps=1e-5, run=None):
    p = {k: f64(t) for k, t in d.items()}
    kw = dict(weight=p["weight"], bias=p["bias"], gate=p["gate"], kind=act, eps=eps, center=center)
    g = {k: dev(t) for k, t in d.items()}
    gkw = dict(weight=g["weight"], bias=g["bias"], gate=g["gate"], act=act, eps=eps, center=center)
    y = gdn.group_norm_fwd(g["x"], **gkw)
    got = gdn.group_norm_bwd(g["x"], g["dy"], **gkw)
    torch.cuda.synchronize()
    x = p["x"]
    k = kappa(x, eps, center)
    w = 1.0 if p["weight"] is None else np.abs(p["weight"])
    b = 0.0 if p["bias"] is None else np.abs(p["bias"])
    c = x - x.mean(-1, keepdims=True) if center else x
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = np.abs(c * r) * w + b + w           # largest |n|, and its condition
    top = lambda t: t.max(-1, keepdims=True)  # noqa: E731
    f = np.ones_like(x) if p["gate"] is None else 1 + np.abs(p["gate"])  # |act|, |act'| <= this
    if p["gate"] is None:
        f = 1 + n                           # act, act' at n: slopes up to 1.1, values up to |n|
    check("y", y, oracle.group_norm_fwd(x, **kw), top(n * f) * k, dtype)
    ref = oracle.group_norm_bwd(x, p["dy"], **kw)
    dyf = np.abs(p["dy"]) * f
    # each gradient's own magnitude; errors of n move act' by up to 1.1 times
    lead = top(dyf * (w + 0 * x) * (n if p["gate"] is None else 1.0)) * k
    check("dx", got[0], ref[0], 4 * r * lead * top(1 + n), dtype)
    if p["gate"] is not None:
        check("dz", got[1], ref[1], top(np.abs(p["dy"]) * n * f) * k, dtype)
    else:
        assert got[1] is None
    if p["weight"] is not None:
        # sums over tokens: each term's bound, plus the additions (at most one
        # per row on any path) at 2^-24 of the terms' magnitudes
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        over = (0, 1) if p["weight"].ndim == 2 else (0, 1, 2)
        for name, a, rr, term in (("dw", got[2], ref[2], dyf * (1 + n) * (1 + np.abs(c * r))),
                                  ("db", got[3], ref[3], dyf * (1 + n))):
            mag = (top(term) * k + 0 * x).sum(over)
            err = np.abs(np64(a) - rr)
            assert np.all(err <= (2.0 ** -17 + rows * 2.0 ** -24) * mag), name
    else:
        assert got[2] is None and got[3] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_kinds(gpu_lib, dtype, act, gate, center):
    for affine in ("group", "shared", "none"):
        check_all(make(1, 37, 3, 64, dtype, affine, gate), dtype, act, center)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16 * i for i in range(1, 17)])
def test_widths(gpu_lib, dtype, d):
    for H in (1, 5, 16):
        check_all(make(2, 11, H, d, dtype), dtype, "silu", True)


@pytest.mark.parametrize("B,T,H,d", [(1, 1, 1, 16), (1, 1, 7, 128), (3, 700, 2, 32),
                                     (1, 5000, 3, 16), (1, 2, 300, 48)])
def test_sizes(gpu_lib, B, T, H, d):
    for affine in ("group", "shared"):
        check_all(make(B, T, H, d, BF16, affine), BF16, "silu", True)


def test_flat_rows(gpu_lib):
    # a row without variance: the eps alone scales it, nothing overflows
    d = make(1, 6, 2, 64, F32)
    d["x"][:, 2] = 0.0
    d["x"][:, 3] = 3.0
    d["x"][:, 4] = 1e-20
    for center in (True, False):
        check_all(d, F32, "silu", center, eps=1e-3)


def test_a_bad_token_stays_alone(gpu_lib):
    d = {k: dev(t) for k, t in make(1, 40, 4, 80, BF16).items()}
    call = lambda x: (gdn.group_norm_fwd(x, d["weight"], d["bias"], d["gate"]),  # noqa: E731
                      gdn.group_norm_bwd(x, d["dy"], d["weight"], d["bias"], d["gate"])[0])
    clean = call(d["x"])
    x = d["x"].clone()
    x[:, 7, 1] = float("nan")
    x[:, 8, 2, 3] = float("inf")
    for a, b in zip(clean, call(x)):
        same = torch.ones(a.shape[:3], dtype=torch.bool, device="cuda")
        same[:, 7, 1] = same[:, 8, 2] = False
        assert torch.equal(a[same], b[same])


def test_no_tokens(gpu_lib):
    d = {k: dev(t) for k, t in make(1, 0, 3, 32, BF16).items()}
    assert gdn.group_norm_fwd(d["x"], d["weight"], d["bias"], d["gate"]).shape == d["x"].shape
    _, _, dw, db = gdn.group_norm_bwd(d["x"], d["dy"], d["weight"], d["bias"], d["gate"])
    assert not dw.any() and not db.any()


def test_outputs_stay_in_their_bounds_and_in_place(gpu_lib):
    d = {k: dev(t) for k, t in make(1, 33, 5, 80, BF16).items()}
    want = gdn.group_norm_fwd(d["x"], d["weight"], d["bias"], d["gate"])
    y = Padded(d["x"].shape, BF16)
    gdn.group_norm_fwd(d["x"], d["weight"], d["bias"], d["gate"], y=y.t)
    x = d["x"].clone()
    gdn.group_norm_fwd(x, d["weight"], d["bias"], d["gate"], y=x)
    z = d["gate"].clone()
    gdn.group_norm_fwd(d["x"], d["weight"], d["bias"], z, y=z)
    torch.cuda.synchronize()
    y.check("y")
    assert torch.equal(y.t, want) and torch.equal(x, want) and torch.equal(z, want)


def test_runs_are_equal_and_replayed(gpu_lib):
    d = {k: dev(t) for k, t in make(1, 3000, 4, 128, BF16, "shared").items()}

    def step():
        kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"])
        return [gdn.group_norm_fwd(d["x"], **kw), *gdn.group_norm_bwd(d["x"], d["dy"], **kw)]

    a, b = step(), step()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        d["x"].copy_(torch.randn_like(d["x"]))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want)), k


def test_normalises_the_gated_delta_forward(gpu_lib):
    # the output stage of a gated delta block, from the library's own forward
    from gated_delta_rule_79_amd import synth
    inp = synth.make_inputs(1, 100, 2, 32, 48, dtype=F32, chunk=16, seed=4).to("cuda")
    o, _ = gdn.chunk_fwd(inp.q, inp.k, inp.v, inp.beta, inp.log_alpha, chunk=16)
    z = torch.randn(o.shape, device="cuda")
    w = torch.rand(48, device="cuda") + 0.5
    y = gdn.group_norm_fwd(o, w, gate=z, center=False)
    torch.cuda.synchronize()
    x = np64(o)
    ref = oracle.group_norm_fwd(x, np64(w), None, np64(z), center=False)
    mag = (np.abs(ref) + np64(w) * (1 + np.abs(np64(z)))).max(-1, keepdims=True)
    check("y", y, ref, mag * kappa(x, 1e-5, False), F32)


def test_refusals(gpu_lib):
    d = {k: dev(t) for k, t in make(1, 9, 2, 32, BF16).items()}
    x, w = d["x"], d["weight"]
    for kw in (dict(weight=w[:1]), dict(weight=w.bfloat16()), dict(bias=w.cpu()),
               dict(weight=w, bias=w[0].contiguous()), dict(gate=x.float()),
               dict(gate=x[:, :3].contiguous()), dict(act="gelu"), dict(weight=w.t()),
               dict(y=x.float()), dict(y=x.cpu())):
        with pytest.raises(ValueError):
            gdn.group_norm_fwd(x, **kw)
    with pytest.raises(gdn.GdnError):
        gdn.group_norm_fwd(x, eps=0.0)
    with pytest.raises(gdn.GdnError):
        gdn.group_norm_fwd(x[..., :24].contiguous())
    with pytest.raises(ValueError):
        gdn.group_norm_fwd(x.transpose(1, 2))
    with pytest.raises(ValueError):
        gdn.group_norm_bwd(x, d["dy"].float())
