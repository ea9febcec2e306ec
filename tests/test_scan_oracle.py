"""Pins of the fp64 oracle of the selective scan, the short convolution with a
history and draft acceptance, and planted mistakes that the pins catch."""

import numpy as np
import pytest

import oracle
from oracle import scan_oracle


def scan_inputs(B=2, T=7, H=4, dk=4, dv=3, hb=2, seed=0, nseq=None):
    r = np.random.default_rng(seed)
    n = nseq or B
    return dict(x=r.normal(size=(B, T, H, dv)), dt=r.normal(size=(B, T, H, dv)),
                a=-np.exp(r.normal(size=(H, dk, dv)) * 0.3), b=r.normal(size=(B, T, hb, dk)),
                c=r.normal(size=(B, T, hb, dk)), d=r.normal(size=(H, dv)),
                dt_bias=r.normal(size=(H, dv)), z=r.normal(size=(B, T, H, dv)),
                s0=r.normal(size=(n, H, dk, dv)))


def test_one_decay_for_all_is_linear_attention():
    i = scan_inputs(hb=2)
    # a and delta constant in a head: decay exp(delta a), k = b, v = delta x, q = c
    delta, rate = np.array([0.3, 0.7, 1.1, 0.2]), -np.array([0.5, 0.1, 1.0, 2.0])
    dt = np.broadcast_to(delta[:, None], i["x"].shape)
    a = np.broadcast_to(rate[:, None, None], i["a"].shape)
    y, sf = oracle.scan_fwd(i["x"], dt, a, i["b"], i["c"], s0=i["s0"], softplus=False)
    o, so = oracle.linattn_fwd(i["c"], i["b"], dt * i["x"], delta * rate, i["s0"])
    assert np.abs(y - o).max() < 1e-12 and np.abs(sf - so).max() < 1e-12


def test_packed_is_separate_and_resumed():
    i = scan_inputs(B=1, T=9, nseq=3)
    cu = [0, 4, 4, 9]
    y, sf = oracle.scan_fwd(**i, cu_seqlens=cu)
    one = {k: v for k, v in i.items() if k in ("a", "d", "dt_bias")}
    for n in range(3):
        part = {k: i[k][:, cu[n]:cu[n + 1]] for k in ("x", "dt", "b", "c", "z")}
        yn, sn = oracle.scan_fwd(**part, **one, s0=i["s0"][n:n + 1])
        assert np.array_equal(y[:, cu[n]:cu[n + 1]], yn) and np.array_equal(sf[n:n + 1], sn)
    assert np.array_equal(sf[1], i["s0"][1])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_are_differences(packed, softplus):
    cu = [0, 3, 3, 7] if packed else None
    i = scan_inputs(B=1 if packed else 2, nseq=3 if packed else None, seed=2)
    if not softplus:  # steps are positive: states shrink
        i["dt"], i["dt_bias"] = np.abs(i["dt"]), np.abs(i["dt_bias"])
    r = np.random.default_rng(3)
    dy, ds = r.normal(size=i["x"].shape), r.normal(size=i["s0"].shape)

    def loss(k):
        y, sf = oracle.scan_fwd(**k, softplus=softplus, cu_seqlens=cu)
        return (y * dy).sum() + (sf * ds).sum()

    names = ("x", "dt", "a", "b", "c", "d", "dt_bias", "z", "s0")
    got = dict(zip(names, oracle.scan_bwd(dy=dy, ds_final=ds, softplus=softplus, cu_seqlens=cu,
                                          **i)))
    for k in names:
        v = r.normal(size=i[k].shape)
        h = 1e-6
        diff = (loss({**i, k: i[k] + h * v}) - loss({**i, k: i[k] - h * v})) / (2 * h)
        want = (got[k] * v).sum()
        assert abs(diff - want) < 1e-6 * max(1.0, abs(want)), k


def test_convolution_without_a_history_is_the_short_convolution():
    r = np.random.default_rng(5)
    x, taps = r.normal(size=(2, 9, 3, 4)), r.normal(size=(3, 4, 4))
    y, _ = oracle.conv_fwd(x, taps, act="none")
    assert np.abs(y - oracle.short_conv(x, taps)).max() < 1e-13


@pytest.mark.parametrize("W", [1, 2, 4, 8])
def test_convolution_resumed_is_whole(W):
    r = np.random.default_rng(6)
    x, taps, bias = r.normal(size=(1, 12, 2, 3)), r.normal(size=(2, 3, W)), r.normal(size=(2, 3))
    whole, end = oracle.conv_fwd(x, taps, bias)
    s, parts = None, []
    for lo, hi in ((0, 2), (2, 2), (2, 3), (3, 12)):
        y, s = oracle.conv_fwd(x[:, lo:hi], taps, bias, s)
        parts.append(y)
    assert np.abs(np.concatenate(parts, 1) - whole).max() < 1e-13 and np.array_equal(s, end)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 9]])
def test_convolution_gradients_are_differences(act, cu):
    r = np.random.default_rng(7)
    W, n = 4, 2 if cu is None else 3
    i = dict(x=r.normal(size=(2 if cu is None else 1, 9, 2, 3)), taps=r.normal(size=(2, 3, W)),
             bias=r.normal(size=(2, 3)), s0=r.normal(size=(n, W - 1, 2, 3)))
    dy, ds = r.normal(size=i["x"].shape), r.normal(size=i["s0"].shape)

    def loss(k):
        y, sf = oracle.conv_fwd(**k, act=act, cu_seqlens=cu)
        return (y * dy).sum() + (sf * ds).sum()

    got = dict(zip(("x", "taps", "bias", "s0"),
                   oracle.conv_bwd(dy=dy, ds_final=ds, act=act, cu_seqlens=cu, **i)))
    for k in i:
        v = r.normal(size=i[k].shape)
        h = 1e-6
        diff = (loss({**i, k: i[k] + h * v}) - loss({**i, k: i[k] - h * v})) / (2 * h)
        assert abs(diff - (got[k] * v).sum()) < 1e-6 * max(1.0, abs(diff)), k


# the next token's distribution is the target's, whatever the draft's
P = np.array([0.5, 0.3, 0.2])
Q = np.array([0.2, 0.1, 0.7])


def emitted(accept, parent, drafts):
    """Distribution of the first emitted token over an even grid of m uniforms
    (a probability is off by at most 1 / 2m there); drafts: [(weight, tokens)]."""
    m = 20
    grid = (np.arange(m) + 0.5) / m
    out = np.zeros(3)
    for weight, tokens in drafts:
        n = len(tokens)
        rows = np.stack([P] + [P] * n)
        qs = np.stack([Q] * (n + 1))
        for k in np.ndindex(*[m] * (n + 1)):
            cur, length, nxt = accept(tokens, rows, qs, grid[list(k)], parent)
            first = tokens[cur if parent is not None else 0] if length else nxt
            out[first] += weight / m ** (n + 1)
    return out


CHAIN = [(Q[i], [i]) for i in range(3)]
PAIR = [(Q[i] * Q[j], [i, j]) for i in range(3) for j in range(3)]


def test_accepted_tokens_follow_the_target():
    assert np.abs(emitted(oracle.accept, None, CHAIN) - P).max() < 1 / 40
    # two children of the root, drawn from the draft independently
    assert np.abs(emitted(oracle.accept, [-1, -1], PAIR) - P).max() < 1 / 40


def test_planted_mistakes_in_acceptance_are_caught(monkeypatch):
    import inspect
    src = inspect.getsource(scan_oracle.accept)
    wrong = [("left = np.maximum(r / Z - q, 0.0)", "left = r"),
             ("float(uniform[i]) * q[x] * Z < r[x]", "float(uniform[i]) < r[x]"),
             ("r, Z = left, left.sum()", "r, Z = left, 1.0")]
    for old, new in wrong:
        assert old in src
        space = {"np": np}
        exec(src.replace(old, new), space)
        far = max(np.abs(emitted(space["accept"], None, CHAIN) - P).max(),
                  np.abs(emitted(space["accept"], [-1, -1], PAIR) - P).max())
        assert far > 0.03, new


def test_acceptance_paths():
    V = 4
    sure = lambda t: np.eye(V)[t]  # noqa: E731
    # a path of certain tokens is followed to its end, siblings are tried in order
    parent = [-1, -1, 1, 1, 2]
    tokens = [0, 1, 2, 3, 3]
    target = np.stack([sure(1), sure(0), sure(2), sure(3), sure(0), sure(2)])
    u = np.full(6, 0.5)
    assert oracle.accept(tokens, target, None, u, parent) == (4, 3, 2)
    # certain drafts that are wrong: the residual leaves the token out
    assert oracle.accept([0], np.array([[0.25, 0.75, 0, 0], sure(0)]), None, [0.9, 0.0]) == (-1, 0, 1)
    # no drafts: a draw from the first row
    assert oracle.accept([], np.array([[0.25, 0.25, 0.5, 0]]), None, [0.5]) == (-1, 0, 2)
    # tokens outside the vocabulary end a chain and are passed over in a tree
    assert oracle.accept([-1, 1], np.stack([sure(1)] * 3), None, u[:3]) == (-1, 0, 1)
    assert oracle.accept([9, 1], np.stack([sure(1)] * 3), None, u[:3], [-1, -1]) == (1, 1, 1)
