"""Pins of the linear-attention and group-norm oracle (CPU)."""

import numpy as np
import pytest

import oracle


def rows(rng, *shape):
    return rng.standard_normal(shape)


def problem(seed=3, B=2, T=9, H=4, Hq=2, dk=5, dv=3, cu=None):
    rng = np.random.default_rng(seed)
    n = B if cu is None else len(cu) - 1
    return dict(q=rows(rng, B, T, Hq, dk), k=rows(rng, B, T, Hq, dk), v=rows(rng, B, T, H, dv),
                log_decay=-rng.uniform(0.0, 1.0, H), s0=rows(rng, n, H, dk, dv), cu_seqlens=cu)


def test_is_the_erase_free_limit_of_the_decoupled_rule():
    p = problem(Hq=4)
    B, T, H = p["v"].shape[:3]
    la = np.broadcast_to(p["log_decay"], (B, T, H))
    o, s = oracle.gdn2_fwd(p["q"], p["k"], p["v"], np.zeros((B, T, H)), np.ones((B, T, H)), la,
                           p["s0"], "scalar")
    o2, s2 = oracle.linattn_fwd(**p)
    assert np.allclose(o, o2, rtol=0, atol=1e-12) and np.allclose(s, s2, rtol=0, atol=1e-12)


def test_no_decay_is_the_masked_product():
    p = problem(Hq=2)
    p["log_decay"] = p["s0"] = None
    o, s = oracle.linattn_fwd(**p)
    k, q = np.repeat(p["k"], 2, 2), np.repeat(p["q"], 2, 2)
    P = np.tril(np.einsum("bihd,bjhd->bhij", q, k))
    assert np.allclose(o, np.einsum("bhij,bjhv->bihv", P, p["v"]), atol=1e-12)
    assert np.allclose(s, np.einsum("bjhd,bjhv->bhdv", k, p["v"]), atol=1e-12)


def test_zero_decay_factor_keeps_only_the_token():
    p = problem()
    p["log_decay"] = np.full(4, -np.inf)
    o, _ = oracle.linattn_fwd(**p)
    qk = np.repeat((p["q"] * p["k"]).sum(-1), 2, 2)
    assert np.allclose(o, qk[..., None] * p["v"], atol=1e-12)


def test_packed_is_separate_and_resumable():
    cu = np.array([0, 4, 4, 9])
    p = problem(B=1, cu=cu)
    o, s = oracle.linattn_fwd(**p)
    for n in range(3):
        lo, hi = cu[n], cu[n + 1]
        part = {x: p[x][:, lo:hi] for x in ("q", "k", "v")}
        on, sn = oracle.linattn_fwd(**part, log_decay=p["log_decay"], s0=p["s0"][n:n + 1])
        assert np.allclose(o[:, lo:hi], on, atol=1e-12) and np.allclose(s[n], sn[0], atol=1e-12)
    st = p["s0"][:1]
    for t in range(4):
        ot, st = oracle.linattn_decode(p["q"][:, t], p["k"][:, t], p["v"][:, t], p["log_decay"], st)
        assert np.allclose(ot, o[:, t], atol=1e-12)
    assert np.allclose(st[0], s[0], atol=1e-12)


def differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        g[i] = (up - f()) / (2 * h)
        x[i] = old
    return g


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 7]])
def test_backward_matches_differences(cu):
    cu = None if cu is None else np.array(cu)
    p = problem(B=1, T=7, dk=3, dv=2, cu=cu)
    rng = np.random.default_rng(8)
    do, ds = rows(rng, *p["v"].shape), rows(rng, *p["s0"].shape)

    def loss():
        o, s = oracle.linattn_fwd(**p)
        return (do * o).sum() + (ds * s).sum()

    got = oracle.linattn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["s0"], do, ds, cu)
    for name, g in zip(("q", "k", "v", "s0"), got):
        # central differences of a multilinear function: only rounding is left
        assert np.allclose(g, differences(loss, p[name]), rtol=0, atol=1e-7), name


@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_backward_matches_differences(kind, gated, center, shared):
    rng = np.random.default_rng(5)
    x = rows(rng, 1, 3, 2, 6)
    w, b = ((rows(rng, 6), rows(rng, 6)) if shared else (rows(rng, 2, 6), rows(rng, 2, 6)))
    z = rows(rng, *x.shape) if gated else None
    dy = rows(rng, *x.shape)
    kw = dict(weight=w, bias=b, gate=z, kind=kind, center=center)
    got = oracle.group_norm_bwd(x, dy, **kw)
    loss = lambda: (dy * oracle.group_norm_fwd(x, **kw)).sum()  # noqa: E731
    for name, t, g in zip(("x", "gate", "weight", "bias"), (x, z, w, b), got):
        if t is None:
            assert g is None
        else:
            assert np.allclose(g, differences(loss, t), rtol=0, atol=1e-7), name


def test_norm_rows_have_unit_scale():
    x = rows(np.random.default_rng(1), 2, 3, 4, 64) * 7 + 5
    n = oracle.group_norm_fwd(x, kind="none", eps=0.0)
    assert np.allclose(n.mean(-1), 0, atol=1e-12) and np.allclose((n ** 2).mean(-1), 1, atol=1e-12)
    r = oracle.group_norm_fwd(x, kind="none", eps=0.0, center=False)
    assert np.allclose((r ** 2).mean(-1), 1, atol=1e-12)
    assert np.allclose(r / x, (r / x)[..., :1], atol=1e-12)
