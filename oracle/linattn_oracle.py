"""fp64 oracle of linear attention with a constant decay per head and of the
causal group norm (test infrastructure, as the rest of the package).

Token by token, from the definitions:

    S_t = a_h S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a_h = exp(log_decay[h])

v head h reads q, k head h // (H // Hq).  The decay has no source page of its
own: it is gated linear attention (the gated delta rule's erase-free limit)
with one gate per head for all tokens, and the pins tie it to
``gdn2_fwd`` with erase = 0.
"""

from __future__ import annotations

import numpy as np


def _runs(B, T, cu_seqlens):
    if cu_seqlens is None:
        return [(b, 0, T, b) for b in range(B)]
    cu = np.asarray(cu_seqlens)
    return [(0, int(cu[n]), int(cu[n + 1]), n) for n in range(len(cu) - 1)]


def _decays(log_decay, H):
    return np.ones(H) if log_decay is None else np.exp(np.asarray(log_decay, dtype=np.float64))


def linattn_fwd(q, k, v, log_decay=None, s0=None, cu_seqlens=None):
    """(o [B,T,H,dv], s_final [nseq,H,dk,dv])."""
    B, T, Hq, dk = q.shape
    H, dv = v.shape[2:]
    grp = H // Hq
    a = _decays(log_decay, H)[:, None, None]
    runs = _runs(B, T, cu_seqlens)
    o = np.zeros((B, T, H, dv))
    sf = np.zeros((len(runs), H, dk, dv))
    for b, lo, hi, n in runs:
        S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0[n], dtype=np.float64)
        for t in range(lo, hi):
            kt, qt = np.repeat(k[b, t], grp, 0), np.repeat(q[b, t], grp, 0)
            S = a * S + kt[:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.einsum("hkv,hk->hv", S, qt)
        sf[n] = S
    return o, sf


def linattn_decode(q, k, v, log_decay, state):
    """One token per sequence: (o [N,H,dv], new state)."""
    o, s = linattn_fwd(q[:, None], k[:, None], v[:, None], log_decay, state)
    return o[:, 0], s


def linattn_bwd(q, k, v, log_decay, s0, do, ds_final=None, cu_seqlens=None):
    """Gradients (dq, dk, dv, ds0) of <do, o> + <ds_final, s_final>."""
    B, T, Hq, dk = q.shape
    H, dv = v.shape[2:]
    grp = H // Hq
    a = _decays(log_decay, H)[:, None, None]
    runs = _runs(B, T, cu_seqlens)
    gq, gk, gv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    gs = np.zeros((len(runs), H, dk, dv))
    share = lambda d: d.reshape(Hq, grp, dk).sum(1)  # noqa: E731
    for b, lo, hi, n in runs:
        S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0[n], dtype=np.float64)
        for t in range(lo, hi):
            kt = np.repeat(k[b, t], grp, 0)
            S = a * S + kt[:, :, None] * v[b, t][:, None, :]
            gq[b, t] = share(np.einsum("hkv,hv->hk", S, do[b, t]))
        D = np.zeros((H, dk, dv)) if ds_final is None else np.array(ds_final[n], dtype=np.float64)
        for t in range(hi - 1, lo - 1, -1):
            kt, qt = np.repeat(k[b, t], grp, 0), np.repeat(q[b, t], grp, 0)
            D = D + qt[:, :, None] * do[b, t][:, None, :]
            gk[b, t] = share(np.einsum("hkv,hv->hk", D, v[b, t]))
            gv[b, t] = np.einsum("hkv,hk->hv", D, kt)
            D = a * D
        gs[n] = D
    return gq, gk, gv, gs


def _sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def act(x, kind):
    return {"none": x, "silu": x * _sigmoid(x), "sigmoid": _sigmoid(x)}[kind]


def act_grad(x, kind):
    s = _sigmoid(x)
    return {"none": np.ones_like(x), "silu": s + x * s * (1 - s), "sigmoid": s * (1 - s)}[kind]


def group_norm_fwd(x, weight=None, bias=None, gate=None, kind="silu", eps=1e-5, center=True):
    """y [B,T,H,d]; weight, bias [H,d] or [d]."""
    c = x - x.mean(-1, keepdims=True) if center else x
    n = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = n * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return act(n, kind) if gate is None else n * act(gate, kind)


def group_norm_bwd(x, dy, weight=None, bias=None, gate=None, kind="silu", eps=1e-5, center=True):
    """(dx, dgate, dweight, dbias) of <dy, y>, None where the input is."""
    d = x.shape[-1]
    c = x - x.mean(-1, keepdims=True) if center else x
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    w = np.ones(d) if weight is None else weight
    n = c * r * w + (0.0 if bias is None else bias)
    dn = dy * act_grad(n, kind) if gate is None else dy * act(gate, kind)
    dz = None if gate is None else dy * n * act_grad(gate, kind)
    # n depends on c directly and through r: dr = -r^3 <c, dc> / d
    dc = dn * w * r - c * r ** 3 * (dn * w * c).sum(-1, keepdims=True) / d
    dx = dc - dc.mean(-1, keepdims=True) if center else dc
    over = lambda t, p: None if p is None else t.sum((0, 1) if p.ndim == 2 else (0, 1, 2))  # noqa: E731
    return dx, dz, over(dn * c * r, weight), over(dn, bias)
