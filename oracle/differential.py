"""fp64 forms of the differential softmax anchor and of the block norms, with
their gradients (test infrastructure, like the rest of this package).

Differential anchor, per batch and head, q and k columns in two halves:
    P_m = softmax over s < key_lens[b] of scale q_m . k_m
    A = P_1 v - lambda P_2 v,  out = A * sigmoid(g)
Block norms, per token:
    h' = res_scale h + gate_b * (Norm(o) w_post)
    u = Norm(h') w_pre (1 + scale_b) + shift_b
"""
from __future__ import annotations

import math

import numpy as np

from . import _f64, merge_heads, sigmoid, split_heads


def _maps(q, k, scale, n):
    """P_1, P_2 [N, keys] of one head (q, k [., d]); keys at or behind n have no weight."""
    m = q.shape[1] // 2
    out = []
    for c in (slice(0, m), slice(m, 2 * m)):
        p = np.zeros((q.shape[0], k.shape[0]))
        if n > 0:
            s = scale * (q[:, c] @ k[:n, c].T)
            e = np.exp(s - s.max(axis=1, keepdims=True))
            p[:, :n] = e / e.sum(axis=1, keepdims=True)
        out.append(p)
    return out


def _lambda(lam, B, N, H, raw):
    """lambda [B, H, N] of logits (or values) [B, N, H] or [H]"""
    x = _f64(lam)
    x = np.broadcast_to(x, (B, N, H)) if x.ndim == 1 else x
    return (x if raw else sigmoid(x)).transpose(0, 2, 1)


def diff_anchor(q, k, v, g, lam, H, key_lens=None, raw=False, scale=None, dout=None):
    """dict of out, o1, o2, lse [2, B, H, N], and, with dout, dq, dk, dv, dgate, dlam.
    Rows of k and v behind key_lens are never touched."""
    qh, kh, vh = (split_heads(x, H) for x in (q, k, v))
    B, _, N, d = qh.shape
    keys = kh.shape[2]
    gh = None if g is None else split_heads(g, H)
    scale = 1.0 / math.sqrt(d // 2) if scale is None else scale
    lam_h = _lambda(lam, B, N, H, raw)
    lens = [keys] * B if key_lens is None else [max(0, min(keys, int(n))) for n in key_lens]
    out, o1, o2, dq, dg = (np.zeros_like(qh) for _ in range(5))
    dk, dv = np.zeros_like(kh), np.zeros_like(vh)
    lse = np.full((2, B, H, N), -np.inf)
    dlam = np.zeros((B, H, N))
    dyh = None if dout is None else split_heads(dout, H)
    for b in range(B):
        n = lens[b]
        for h in range(H):
            Q, K, V = qh[b, h], np.where(np.arange(keys)[:, None] < n, kh[b, h], 0.0), \
                np.where(np.arange(keys)[:, None] < n, vh[b, h], 0.0)
            L = lam_h[b, h][:, None]
            P = _maps(Q, K, scale, n)
            o1[b, h], o2[b, h] = P[0] @ V, P[1] @ V
            A = o1[b, h] - L * o2[b, h]
            s = 1.0 if gh is None else sigmoid(gh[b, h])
            out[b, h] = A * s
            m = d // 2
            halves = (slice(0, m), slice(m, d))
            if n:
                for i, c in enumerate(halves):
                    z = scale * (Q[:, c] @ K[:n, c].T)
                    top = z.max(axis=1)
                    lse[i, b, h] = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
            if dyh is None:
                continue
            dA = dyh[b, h] * s
            if gh is not None:
                dg[b, h] = dyh[b, h] * A * s * (1 - s)
            dv[b, h] = (P[0] - L * P[1]).T @ dA
            dlam[b, h] = -(dA * o2[b, h]).sum(axis=1)
            dP = dA @ V.T
            for i, (c, w) in enumerate(zip(halves, (1.0, -L))):
                # softmax's Jacobian, written out: dS = P (dP - sum_s P dP), the map's weight in front
                dS = w * P[i] * (dP - (P[i] * dP).sum(axis=1, keepdims=True))
                dq[b, h][:, c] = scale * (dS @ K[:, c])
                dk[b, h][:, c] = scale * (dS.T @ Q[:, c])
    res = dict(out=merge_heads(out), o1=merge_heads(o1), o2=merge_heads(o2), lse=lse)
    if dout is not None:
        if not raw:
            dlam = dlam * lam_h * (1 - lam_h)
        res.update(dq=merge_heads(dq), dk=merge_heads(dk), dv=merge_heads(dv),
                   dgate=merge_heads(dg),
                   dlam=dlam.sum(axis=(0, 2)) if np.ndim(lam) == 1 else dlam.transpose(0, 2, 1))
    return res


def _norm(x, layer, eps):
    c = x - x.mean(axis=-1, keepdims=True) if layer else x
    return c / np.sqrt((c * c).mean(axis=-1, keepdims=True) + eps)


def _norm_grad(dy, x, layer, eps):
    """Gradient of sum(dy * Norm(x)) by x, from the quotient rule on c / sqrt(mean c^2 + eps)."""
    c = x - x.mean(axis=-1, keepdims=True) if layer else x
    v = (c * c).mean(axis=-1, keepdims=True) + eps
    dc = dy / np.sqrt(v) - c * (dy * c).mean(axis=-1, keepdims=True) / v ** 1.5
    return dc - dc.mean(axis=-1, keepdims=True) if layer else dc


def block_norm(h, o=None, w_post=None, gate=None, w_pre=None, scale=None, shift=None, pre=True,
               layer=False, eps=1e-6, res_scale=1.0, dh_out=None, du=None):
    """dict of h_out, u and, with dh_out or du, dh, do, dw_post, dgate, dw_pre, dscale, dshift."""
    def row(x, default):
        return default if x is None else _f64(x)[:, None, :]

    h = _f64(h)
    D = h.shape[-1]
    wq = np.ones(D) if w_post is None else _f64(w_post)
    wp = np.ones(D) if w_pre is None else _f64(w_pre)
    gt, sc, sh = row(gate, 1.0), 1.0 + row(scale, 0.0), row(shift, 0.0)
    res = {}
    hp = h
    if o is not None:
        on = _norm(_f64(o), layer, eps)
        hp = res["h_out"] = res_scale * h + gt * (on * wq)
    if pre:
        hn = _norm(hp, layer, eps)
        res["u"] = hn * wp * sc + sh
    if dh_out is None and du is None:
        return res
    dh = np.zeros_like(h) if dh_out is None else _f64(dh_out)
    if pre:
        du = _f64(du)
        res["dshift"] = du.sum(axis=1)
        res["dscale"] = (du * hn * wp).sum(axis=1)
        res["dw_pre"] = (du * hn * sc).sum(axis=(0, 1))
        dh = dh + _norm_grad(du * wp * sc, hp, layer, eps)
    if o is not None:
        res["dgate"] = (dh * on * wq).sum(axis=1)
        res["dw_post"] = (dh * on * gt).sum(axis=(0, 1))
        res["do"] = _norm_grad(dh * gt * wq, _f64(o), layer, eps)
        dh = res_scale * dh
    res["dh"] = dh
    return res
