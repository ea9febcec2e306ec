"""How exact bf16 linear attention is: every output is the 64-bit result
rounded once, but for terms two operand parts leave behind.

Bound.  Write A for an output with every operand and state replaced by its
absolute value.  A bf16 part keeps 8 significant bits, so one part leaves
2^-8 of a value, two leave 2^-17 (the rest after the first is a value of its
own, half a step of it is 2^-8 of at most 2^-9) and three leave nothing of an
fp32 value.  The copy of the state that multiplies the rows, the weighted
rows that enter the state and the weighted x y^T each take two parts: the
first two stand behind the state's share of A, the third behind the rest of
it, so together they leave at most 2^-16 A.  Sums run in fp32, u = 2^-24 an
addition: a term passes at most 2 T additions on its way through the state
(two parts), 2 d in the product with the row, 2 * 64 in the chunk's own
product, and some tens of products, decays and quotients.  The result is
rounded to bf16, half a step of 2^-8 of its value."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import log, np64
from test_gpu_linattn import BF16, U, absolute, f64, make, run_bwd, run_fwd


def bound(ref, mag, T, d):
    wide = (2.0 ** -16 + (2 * T + 2 * d + 2 * 64 + 64) * U) * (1 + 2.0 ** -6) * mag
    return wide + 2.0 ** -8 * (np.abs(ref) + wide)


def check(name, got, ref, mag, T, d):
    err, tol = np.abs(got - ref), bound(ref, mag, T, d)
    worst = float(np.max(err / np.maximum(tol, 1e-300)))
    log(f"    {name}: worst error / bound {worst:.3f}")
    assert worst <= 1.0, (name, worst)


ARGS = ("q", "k", "v", "log_decay", "s0")


def fwd_both(d, cu):
    return [oracle.linattn_fwd(*(x[a] for a in ARGS), cu)[0] for x in (f64(d), absolute(f64(d)))]


# ------------------------------------------------------- the bound, on the CPU

def parts(x, n):
    """x as the sum of n bf16 operand parts (0: x itself)."""
    left, out = x, np.zeros_like(x)
    for _ in range(n):
        p = torch.from_numpy(left).to(BF16).double().numpy()
        out, left = out + p, left - p
    return out if n else x


def rounded_fwd(d, copy, own, C=64):
    """The forward in chunks, the state's copy and x y^T in that many parts."""
    f = f64(d)
    q, k, v = f["q"], f["k"], f["v"]
    B, T, H = v.shape[:3]
    grp = H // q.shape[2]
    out = np.zeros_like(v)
    for b in range(B):
        for h in range(H):
            a = np.exp(f["log_decay"][h])
            S = np.zeros((k.shape[-1], v.shape[-1])) if f["s0"] is None else f["s0"][b, h]
            for t in range(0, T, C):
                x, y, z = q[b, t:t + C, h // grp], k[b, t:t + C, h // grp], v[b, t:t + C, h]
                n = len(x)
                i = np.arange(n)
                P = np.tril(x @ y.T * a ** np.abs(i[:, None] - i[None, :]))
                o = (a ** (i + 1))[:, None] * (x @ parts(S, copy)) + parts(P, own) @ z
                out[b, t:t + C, h] = torch.from_numpy(o).to(BF16).double().numpy()
                S = a ** n * S + (y * (a ** (n - 1 - i))[:, None]).T @ z
    return out


SHAPES = [(1, 130, 2, 2, 64, 64), (2, 65, 4, 2, 32, 48), (1, 200, 2, 1, 16, 32),
          (1, 100, 2, 2, 128, 80), (3, 31, 2, 2, 128, 256)]


@pytest.mark.parametrize("shape", SHAPES)
def test_the_bound_tells_parts_apart(shape):
    d, _ = make(*shape, BF16)
    T, dk = shape[1], shape[4]
    ref, mag = fwd_both(d, None)
    check("two parts", rounded_fwd(d, 2, 2), ref, mag, T, dk)
    for copy, own in ((1, 2), (2, 1)):
        with pytest.raises(AssertionError):
            check(f"{copy}, {own}", rounded_fwd(d, copy, own), ref, mag, T, dk)


def test_what_parts_leave():
    # the shares named above are met but not passed, and three parts are whole
    r = np.random.default_rng(5)
    x = (r.standard_normal(1 << 18) * 2.0 ** r.integers(-30, 30, 1 << 18)).astype(np.float32)
    x = np.concatenate([x, np.nextafter(np.float32(1), np.float32(2)) + np.float32(2.0 ** -8),
                        np.float32(2) - np.float32(2.0 ** -23)], axis=None).astype(np.float64)
    for n, most in ((1, 2.0 ** -8), (2, 2.0 ** -17), (3, 0.0)):
        left = np.abs(x - parts(x, n)) / np.abs(x)
        assert left.max() <= most, n
        assert n == 3 or left.max() > most / 2, n


# ------------------------------------------------------------------ the kernels

@pytest.mark.gpu
@pytest.mark.parametrize("s0", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_rounds_once(gpu_lib, shape, s0):
    d, _ = make(*shape, BF16, s0=s0)
    ref, mag = fwd_both(d, None)
    for seg in (-1, 1):
        o, _ = run_fwd(d, None, seg_chunks=seg)
        check(f"o seg {seg}", np64(o), ref, mag, shape[1], shape[4])


@pytest.mark.gpu
@pytest.mark.parametrize("s0", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_rounds_once(gpu_lib, shape, s0):
    d, _ = make(*shape, BF16, s0=s0, do=True)
    ref, mag = (oracle.linattn_bwd(*(x[a] for a in ARGS), x["do"], x["ds"])
                for x in (f64(d), absolute(f64(d))))
    wide = max(shape[4:]) + shape[2] // shape[3]  # the rows' sum, and the shared heads'
    for seg in (-1, 1):
        got = run_bwd(d, None, seg_chunks=seg)
        for name, g, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
            check(f"{name} seg {seg}", np64(g), r, m, shape[1], wide)


@pytest.mark.gpu
def test_packed_rounds_once(gpu_lib):
    cu = [0, 0, 1, 64, 129, 300]
    d, cu = make(1, cu[-1], 4, 2, 64, 48, BF16, cu=cu, do=True)
    ref, mag = fwd_both(d, cu)
    gref, gmag = (oracle.linattn_bwd(*(x[a] for a in ARGS), x["do"], x["ds"], cu)
                  for x in (f64(d), absolute(f64(d))))
    for seg in (0, 1, -1):
        check(f"o seg {seg}", np64(run_fwd(d, cu, seg_chunks=seg)[0]), ref, mag, 171, 64)
        for name, g, r, m in zip(("dq", "dk", "dv"), run_bwd(d, cu, seg_chunks=seg), gref, gmag):
            check(f"{name} seg {seg}", np64(g), r, m, 171, 66)
