"""Attention within each molecule and layer norm, forward and backward, of the
oracle in float64.  Test infrastructure only.

All pairs inside a molecule, the dense counterpart of oracle/attention.py:

    x_ij = q_i . k_j / sqrt(dk),  s_ij = f(x_ij) - slope |r_i - r_j|,
    f(x) = x or cap tanh(x / cap),  a_ij = softmax_j(s_ij),  m_i = sum_j a_ij h'_j

and for an upstream gradient G of m, with dP_ij = G_i . h'_j (per head):

    dS_ij = a_ij (dP_ij - sum_j a_ij dP_ij),   dx_ij = dS_ij f'(x_ij) / sqrt(dk)
    dq_i = sum_j dx_ij k_j,  dk_j = sum_i dx_ij q_i,  dh'_j = sum_i a_ij G_i
    dslope = -sum_ij dS_ij d_ij,  dr_i = -sum_jh slope dS_ij (r_i - r_j) / d_ij  (dr_j its negative)

Both functions also return, for each output, the same sum over the magnitudes
of its terms: what a relative error of the terms can move the output by.

Pins (tests/test_oracle_molecule.py): hand values, differences of the forward
for every gradient, torch's own softmax and layer norm in float64.
"""
from __future__ import annotations

import numpy as np


def _heads(x, H):
    """[n, D, C] -> [H, n, D * C / H]."""
    n, D, C = x.shape
    return x.reshape(n, D, H, C // H).transpose(2, 0, 1, 3).reshape(H, n, -1)


def _unheads(x, D, C):
    H, n, _ = x.shape
    return x.reshape(H, n, D, C // H).transpose(1, 2, 0, 3).reshape(n, D, C)


def _scores(q, k, cap, pos_q, pos_k, slope):
    dk = q.shape[2]
    x = q.transpose(1, 0, 2) @ k.transpose(1, 2, 0) / np.sqrt(dk)
    s = cap * np.tanh(x / cap) if cap else x
    if slope is None:
        return x, s, None, None
    diff = pos_q[:, None] - pos_k[None]
    d = np.sqrt((diff ** 2).sum(2))
    return x, s - slope[:, None, None] * d, d, diff


def molecule_attention(q, k, hp, q_ptr, k_ptr=None, cap=0.0, pos_q=None, pos_k=None, slope=None, grad=None):
    """dict of m, lse (and with grad: dq, dk, dhp, dpos_q, dpos_k, dslope), float64, and of the
    magnitude sums under the same names with an "abs_" in front; "score" is the largest sum of magnitudes in
    an x_ij, "dist" the largest slope d_ij.  k_ptr None: the self form, where dpos_q is the whole dL/dr."""
    q, k, hp = (np.asarray(a, np.float64) for a in (q, k, hp))
    self_form = k_ptr is None
    if self_form:
        k_ptr, pos_k = q_ptr, pos_q
    nq, H, dk = q.shape
    nk, D, C = hp.shape
    o = {"m": np.zeros((nq, D, C)), "lse": np.full((nq, H), -np.inf), "abs_m": np.zeros((nq, D, C)),
         "score": 0.0, "dist": 0.0}
    if slope is not None:
        slope, pos_q, pos_k = (np.asarray(a, np.float64) for a in (slope, pos_q, pos_k))
    if grad is not None:
        grad = np.asarray(grad, np.float64)
        for p in ("", "abs_"):
            o[p + "dq"], o[p + "dk"], o[p + "dhp"] = np.zeros_like(q), np.zeros_like(k), np.zeros_like(hp)
            if slope is not None:
                o[p + "dpos_q"], o[p + "dpos_k"], o[p + "dslope"] = np.zeros((nq, 3)), np.zeros((nk, 3)), np.zeros(H)
    for b in range(len(q_ptr) - 1):
        i, j = slice(q_ptr[b], q_ptr[b + 1]), slice(k_ptr[b], k_ptr[b + 1])
        if i.start >= i.stop or j.start >= j.stop:
            continue
        args = (pos_q[i], pos_k[j], slope) if slope is not None else (None, None, None)
        x, s, d, diff = _scores(q[i], k[j], cap, *args)
        o["score"] = max(o["score"], (np.abs(q[i]).transpose(1, 0, 2) @ np.abs(k[j]).transpose(1, 2, 0)).max() / np.sqrt(dk))
        if d is not None:
            o["dist"] = max(o["dist"], np.abs(slope).max() * d.max())
        top = s.max(2, keepdims=True)
        w = np.exp(s - top)
        o["lse"][i] = (top[..., 0] + np.log(w.sum(2))).T
        a = w / w.sum(2, keepdims=True)
        V = _heads(hp[j], H)
        o["m"][i] = _unheads(a @ V, D, C)
        o["abs_m"][i] = _unheads(a @ np.abs(V), D, C)
        if grad is None:
            continue
        G = _heads(grad[i], H)
        dP = G @ V.transpose(0, 2, 1)
        dS = a * (dP - (a * dP).sum(2, keepdims=True))
        # magnitudes: each |a_ij| (|dP_ij| + |delta_i|) with dP's own terms in magnitude
        aP = np.abs(G) @ np.abs(V).transpose(0, 2, 1)
        aS = a * (aP + (a * aP).sum(2, keepdims=True))
        o["dhp"][j] = _unheads(a.transpose(0, 2, 1) @ G, D, C)
        o["abs_dhp"][j] = _unheads(a.transpose(0, 2, 1) @ np.abs(G), D, C)
        # 1 - tanh^2 = 1 / cosh^2, without the cancellation
        fx = (np.cosh(x / cap) ** -2 if cap else 1.0) / np.sqrt(dk)
        for p, S, qq, kk in (("", dS * fx, q, k), ("abs_", aS * fx, np.abs(q), np.abs(k))):
            o[p + "dq"][i] = (S @ kk[j].transpose(1, 0, 2)).transpose(1, 0, 2)
            o[p + "dk"][j] = (S.transpose(0, 2, 1) @ qq[i].transpose(1, 0, 2)).transpose(1, 0, 2)
        if slope is None:
            continue
        u = np.divide(diff, d[..., None], out=np.zeros_like(diff), where=d[..., None] > 0)
        for p, S, sl, uu, sg in (("", -dS, slope, u, -1), ("abs_", aS, np.abs(slope), np.abs(u), 1)):
            o[p + "dslope"] += (S * d).sum((1, 2))
            f = (S * sl[:, None, None]).sum(0)[..., None] * uu
            o[p + "dpos_q"][i] += f.sum(1)
            o[p + "dpos_k"][j] += sg * f.sum(0)
    if grad is not None and slope is not None and self_form:
        for p in ("", "abs_"):
            o[p + "dpos_q"] = o[p + "dpos_q"] + o.pop(p + "dpos_k")
    return o


def layer_norm(x, weight=None, bias=None, eps=1e-5, grad=None):
    """dict of y, mu, rstd (and with grad: dx, dweight, dbias and their magnitude sums), float64."""
    x = np.asarray(x, np.float64)
    W = x.shape[1]
    w = np.ones(W) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(W) if bias is None else np.asarray(bias, np.float64)
    mu = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    z = (x - mu) * rstd
    o = {"y": z * w + b, "mu": mu[:, 0], "rstd": rstd[:, 0], "z": z}
    if grad is not None:
        g = np.asarray(grad, np.float64)
        t = g * w
        o["dx"] = rstd * (t - t.mean(1, keepdims=True) - z * (t * z).mean(1, keepdims=True))
        o["abs_dx"] = rstd * (np.abs(t) + np.abs(t).mean(1, keepdims=True)
                              + np.abs(z) * np.abs(t * z).mean(1, keepdims=True))
        o["dweight"], o["dbias"] = (g * z).sum(0), g.sum(0)
        o["abs_dweight"], o["abs_dbias"] = np.abs(g * z).sum(0), np.abs(g).sum(0)
    return o
