"""fp64 oracle of the selective state space scan, the short convolution with a
carried history and the acceptance of drafted tokens (test infrastructure, as
the rest of the package).

Token by token, from the definitions:

    delta_t = softplus(dt_t + dt_bias)
    S_t[n, j] = exp(delta_t[j] a[n, j]) S_{t-1}[n, j] + delta_t[j] x_t[j] b_t[n]
    y_t[j] = (sum_n c_t[n] S_t[n, j] + d[j] x_t[j]) silu(z_t[j])

    y_t = act(bias + sum_j taps[j] x_{t-j})     (x_{-1}, .. the history's rows)

None of them has a source page; the pins tie the scan to ``linattn_fwd`` (one
decay for all channels and states) and to its own finite differences, the
convolution to ``short_conv``, the acceptance to the target's distribution.
"""

from __future__ import annotations

import numpy as np


def _runs(B, T, cu_seqlens):
    if cu_seqlens is None:
        return [(b, 0, T, b) for b in range(B)]
    cu = np.asarray(cu_seqlens)
    return [(0, int(cu[n]), int(cu[n + 1]), n) for n in range(len(cu) - 1)]


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def scan_delta(dt, dt_bias=None, softplus=True):
    pre = dt if dt_bias is None else dt + dt_bias
    return np.logaddexp(pre, 0.0) if softplus else pre


def scan_fwd(x, dt, a, b, c, d=None, dt_bias=None, z=None, s0=None, softplus=True,
             cu_seqlens=None):
    """(y [B,T,H,dv], s_final [nseq,H,dk,dv])."""
    B, T, H, dv = x.shape
    dk = b.shape[-1]
    grp = H // b.shape[2]
    delta = scan_delta(dt, dt_bias, softplus)
    runs = _runs(B, T, cu_seqlens)
    y = np.zeros(x.shape)
    sf = np.zeros((len(runs), H, dk, dv))
    for i, lo, hi, n in runs:
        S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0[n], dtype=np.float64)
        for t in range(lo, hi):
            bt, ct = np.repeat(b[i, t], grp, 0), np.repeat(c[i, t], grp, 0)
            S = (np.exp(delta[i, t][:, None] * a) * S
                 + bt[:, :, None] * (delta[i, t] * x[i, t])[:, None])
            y[i, t] = np.einsum("hkv,hk->hv", S, ct)
        sf[n] = S
    if d is not None:
        y = y + d * x
    return (y if z is None else y * z * _sigmoid(z)), sf


def scan_bwd(x, dt, a, b, c, dy, d=None, dt_bias=None, z=None, s0=None, ds_final=None,
             softplus=True, cu_seqlens=None, absolute=False):
    """(dx, ddt, da, db, dc, dd, ddt_bias, dz, ds0) of <dy, y> + <ds_final,
    s_final>.  absolute: every term's magnitude in place of the term (the
    inputs' magnitudes are the caller's)."""
    B, T, H, dv = x.shape
    hb, dk = b.shape[2:]
    grp = H // hb
    delta = scan_delta(dt, dt_bias, softplus)
    mag = np.abs if absolute else (lambda v: v)
    runs = _runs(B, T, cu_seqlens)
    dx, ddelta, ys = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    db, dc = np.zeros((B, T, H, dk)), np.zeros((B, T, H, dk))
    da, ds0 = np.zeros(a.shape), np.zeros((len(runs), H, dk, dv))
    gate = 1.0 if z is None else z * _sigmoid(z)
    g0 = dy * gate  # the gradient in front of the gate
    for i, lo, hi, n in runs:
        S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0[n], dtype=np.float64)
        hist = [S]
        for t in range(lo, hi):
            bt = np.repeat(b[i, t], grp, 0)
            S = (np.exp(delta[i, t][:, None] * a) * S
                 + bt[:, :, None] * (delta[i, t] * x[i, t])[:, None])
            hist.append(S)
        g = np.zeros((H, dk, dv)) if ds_final is None else np.array(ds_final[n], dtype=np.float64)
        for t in reversed(range(lo, hi)):
            bt, ct = np.repeat(b[i, t], grp, 0), np.repeat(c[i, t], grp, 0)
            S, before = hist[t - lo + 1], hist[t - lo]
            e = np.exp(delta[i, t][:, None] * a)
            ys[i, t] = np.einsum("hkv,hk->hv", S, ct)
            g = g + ct[:, :, None] * g0[i, t][:, None]
            dc[i, t] = np.einsum("hkv,hv->hk", S, g0[i, t])
            db[i, t] = np.einsum("hkv,hv->hk", g, delta[i, t] * x[i, t])
            gb = np.einsum("hkv,hk->hv", g, bt)
            w = g * e * before
            dx[i, t] = delta[i, t] * gb
            ddelta[i, t] = x[i, t] * gb + (mag(a) * w).sum(1)
            da += w * delta[i, t][:, None]
            g = g * e
        ds0[n] = g
    if d is not None:
        dx = dx + d * g0
        ys = ys + d * x
    pre = dt if dt_bias is None else dt + dt_bias
    ddt = ddelta * _sigmoid(pre) if softplus else ddelta
    share = lambda t: t.reshape(B, T, hb, grp, dk).sum(3)  # noqa: E731
    dz = None
    if z is not None:
        s = _sigmoid(z)
        dz = dy * ys * s * (1 + z * (1 - s))
    return (dx, ddt, da, share(db), share(dc), None if d is None else (g0 * x).sum((0, 1)),
            None if dt_bias is None else ddt.sum((0, 1)), dz, ds0)


_ACT = {"none": lambda p: p, "silu": lambda p: p * _sigmoid(p), "sigmoid": _sigmoid}
_ACT_GRAD = {"none": np.ones_like, "sigmoid": lambda p: _sigmoid(p) * (1 - _sigmoid(p)),
             "silu": lambda p: _sigmoid(p) * (1 + p * (1 - _sigmoid(p)))}


def _rows(x, s0, W, i, lo, hi, n):
    old = np.zeros((W - 1, *x.shape[2:])) if s0 is None else np.asarray(s0[n], dtype=np.float64)
    return np.concatenate([old, x[i, lo:hi]])


def conv_fwd(x, taps, bias=None, s0=None, act="silu", cu_seqlens=None):
    """(y [B,T,H,d], the sequences' last W - 1 inputs [nseq,W-1,H,d])."""
    B, T = x.shape[:2]
    W = taps.shape[-1]
    runs = _runs(B, T, cu_seqlens)
    y, sf = np.zeros(x.shape), np.zeros((len(runs), W - 1, *x.shape[2:]))
    for i, lo, hi, n in runs:
        row = _rows(x, s0, W, i, lo, hi, n)
        p = sum(taps[..., j] * row[W - 1 - j:len(row) - j] for j in range(W))
        y[i, lo:hi] = _ACT[act](p if bias is None else p + bias)
        sf[n] = row[len(row) - (W - 1):]
    return y, sf


def conv_bwd(x, taps, dy, bias=None, s0=None, ds_final=None, act="silu", cu_seqlens=None,
             absolute=False):
    """(dx, dtaps, dbias, ds0) of <dy, y> + <ds_final, s_final>.  absolute: the
    magnitudes of the terms of dtaps, dx, ..., the activation's derivative
    taken at the signed p."""
    B, T = x.shape[:2]
    W = taps.shape[-1]
    mag = np.abs if absolute else (lambda v: v)
    runs = _runs(B, T, cu_seqlens)
    dx, dtaps = np.zeros(x.shape), np.zeros(taps.shape)
    dbias, ds0 = np.zeros(taps.shape[:-1]), np.zeros((len(runs), W - 1, *x.shape[2:]))
    for i, lo, hi, n in runs:
        row = _rows(x, s0, W, i, lo, hi, n)
        p = sum(taps[..., j] * row[W - 1 - j:len(row) - j] for j in range(W))
        p = p if bias is None else p + bias
        e = mag(dy[i, lo:hi] * _ACT_GRAD[act](p))
        g = np.zeros(row.shape)
        for j in range(W):
            part = row[W - 1 - j:len(row) - j]
            g[W - 1 - j:len(row) - j] += mag(taps[..., j]) * e
            dtaps[..., j] += (e * mag(part)).sum(0)
        dbias += e.sum(0)
        if ds_final is not None:
            g[len(row) - (W - 1):] += mag(np.asarray(ds_final[n], dtype=np.float64))
        dx[i, lo:hi], ds0[n] = g[W - 1:], g[:W - 1]
    return dx, dtaps, dbias, ds0


def accept(tokens, target, draft, uniform, parent=None):
    """One tree: (last accepted node or -1, accepted nodes, next token).
    tokens [n], target and draft [n + 1, V] (draft None: certain), uniform
    [n + 1], parent [n] or None (a chain)."""
    n, V = len(tokens), target.shape[1]
    r, Z, cur, length = target[0].astype(np.float64), 1.0, -1, 0
    for i in range(n):
        p = i - 1 if parent is None else int(parent[i])
        if (p if -1 <= p < i else -1) != cur or not 0 <= tokens[i] < V:
            if parent is None and cur == i - 1:
                break
            continue
        x = int(tokens[i])
        if draft is None:
            q = np.zeros(V)
            q[x] = 1.0
        else:
            q = draft[cur + 1].astype(np.float64)
        if float(uniform[i]) * q[x] * Z < r[x]:
            cur, length, r, Z = i, length + 1, target[i + 1].astype(np.float64), 1.0
            continue
        left = np.maximum(r / Z - q, 0.0)
        if left.sum() > 0:
            r, Z = left, left.sum()
    run = np.cumsum(r)
    over = np.nonzero((run > float(uniform[n]) * run[-1]) & (r > 0))[0]
    some = np.nonzero(r > 0)[0]
    return cur, length, int(over[0] if len(over) else some[-1] if len(some) else V - 1)
