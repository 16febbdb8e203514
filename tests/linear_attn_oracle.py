"""Plain fp64 definitions of the linear-attention operators, token by token, on the CPU.

Each returns, next to a value, the sum of the absolute values of the products it is made of (``mag``): a
kernel that rounds products or partial sums to a relative 2^-k is off by at most 2^-k * mag.
"""
import numpy as np
import torch


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def scan(q, k, v, log_decay, scale, S):
    """One sequence: q [L, H, Dk], k [L, H, Dk], v [L, H, Dv], S [H, Dk, Dv] -> o, S."""
    a = np.exp(log_decay)[:, None, None]
    o = np.zeros((q.shape[0], q.shape[1], v.shape[2]))
    S = S.copy()
    for t in range(q.shape[0]):
        S = a * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
    return o, S


def scan_grads(q, k, v, log_decay, scale, S0, do, dS):
    """Adjoint of ``scan``: gradients of sum(do * o) + sum(dS * S_last), token by token."""
    a = np.exp(log_decay)[:, None, None]
    states, S = [], S0.copy()
    for t in range(q.shape[0]):
        S = a * S + k[t][:, :, None] * v[t][:, None, :]
        states.append(S)
    dq, dk, dv, G = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), dS.copy()
    for t in range(q.shape[0] - 1, -1, -1):
        dq[t] = scale * np.einsum("hkv,hv->hk", states[t], do[t])
        G = G + scale * q[t][:, :, None] * do[t][:, None, :]
        dk[t] = np.einsum("hkv,hv->hk", G, v[t])
        dv[t] = np.einsum("hkv,hk->hv", G, k[t])
        G = a * G
    return dq, dk, dv, G


def _sequences(x, spans):
    return [x[a:b] for a, b in spans]


def _spans(shape, cu):
    if cu is None:
        return [(b * shape[1], (b + 1) * shape[1]) for b in range(shape[0])]
    return list(zip(cu[:-1], cu[1:]))


def _rows(t, cu):
    x = _np(t)
    return x.reshape((-1,) + x.shape[2:]) if cu is None else x


def prefill(q, k, v, log_decay, scale, init=None, cu=None):
    """(o, S, mag_o, mag_S) of a batch [B, L, H, D] or packed rows [T, H, D] with offsets ``cu``; rows outside
    every sequence are NaN."""
    spans, H, group = _spans(q.shape, cu), q.shape[-2], q.shape[-2] // k.shape[-2]
    ld = _np(log_decay)
    out = []
    for f in (lambda x: x, np.abs):
        Q, K, V = (f(_rows(t, cu)) for t in (q, k, v))
        K, V = K.repeat(group, 1), V.repeat(group, 1)
        o = np.full((Q.shape[0], H, V.shape[2]), np.nan)
        S = np.zeros((len(spans), H, Q.shape[2], V.shape[2])) if init is None else f(_np(init)).copy()
        for i, (a, b) in enumerate(spans):
            o[a:b], S[i] = scan(Q[a:b], K[a:b], V[a:b], ld, abs(scale) if f is np.abs else scale, S[i])
        out += [o.reshape(q.shape[:-1] + (V.shape[2],)), S]
    return out[0], out[1], out[2], out[3]


def backward(q, k, v, log_decay, scale, do, init=None, d_final=None, cu=None):
    """Two dicts (gradients, mags) with the keys q, k, v, init_state."""
    spans, H, group = _spans(q.shape, cu), q.shape[-2], q.shape[-2] // k.shape[-2]
    ld = _np(log_decay)
    got = []
    for f in (lambda x: x, np.abs):
        Q, K, V, DO = (f(_rows(t, cu)) for t in (q, k, v, do))
        K, V = K.repeat(group, 1), V.repeat(group, 1)
        shape = (len(spans), H, Q.shape[2], V.shape[2])
        S0 = np.zeros(shape) if init is None else f(_np(init))
        dS = np.zeros(shape) if d_final is None else f(_np(d_final))
        dq, dk, dv, d0 = (np.full(Q.shape, np.nan), np.full(K.shape, np.nan), np.full(V.shape, np.nan),
                          np.zeros(shape))
        for i, (a, b) in enumerate(spans):
            dq[a:b], dk[a:b], dv[a:b], d0[i] = scan_grads(Q[a:b], K[a:b], V[a:b], ld,
                                                         abs(scale) if f is np.abs else scale, S0[i], DO[a:b], dS[i])
        dk, dv = (x.reshape(x.shape[0], -1, group, x.shape[2]).sum(2) for x in (dk, dv))
        got.append({"q": dq.reshape(tuple(q.shape)), "k": dk.reshape(tuple(k.shape)), "v": dv.reshape(tuple(v.shape)),
                    "init_state": d0})
    return got


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """x [..., H, D] -> y."""
    x, w = _np(x), _np(w)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    angle = np.asarray(positions.cpu(), dtype=np.float64)[..., None, None] * _np(inv_freq)
    c, s, half = np.cos(angle), np.sin(angle), angle.shape[-1]
    y = n.copy()
    ia, ib = ((np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved
              else (np.arange(half), np.arange(half) + half))
    y[..., ia] = n[..., ia] * c - n[..., ib] * s
    y[..., ib] = n[..., ib] * c + n[..., ia] * s
    return y


def norm_rope_grads(x, w, positions, inv_freq, eps, interleaved, dy):
    """(dx, dw) and their magnitudes (of the terms that each sums)."""
    x, w, dy = _np(x), _np(w), _np(dy)
    angle = np.asarray(positions.cpu(), dtype=np.float64)[..., None, None] * _np(inv_freq)
    c, s, half = np.cos(angle), np.sin(angle), angle.shape[-1]
    ia, ib = ((np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved
              else (np.arange(half), np.arange(half) + half))
    dn, mn = dy.copy(), np.abs(dy)
    dn[..., ia] = dy[..., ia] * c + dy[..., ib] * s
    dn[..., ib] = dy[..., ib] * c - dy[..., ia] * s
    mn[..., ia] = np.abs(dy[..., ia] * c) + np.abs(dy[..., ib] * s)
    mn[..., ib] = np.abs(dy[..., ib] * c) + np.abs(dy[..., ia] * s)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dh, mh = dn * w, mn * np.abs(w)
    dx = r * (dh - xh * (dh * xh).mean(-1, keepdims=True))
    mx = r * (mh + np.abs(xh) * (mh * np.abs(xh)).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dn * xh).sum(lead), mx, (mn * np.abs(xh)).sum(lead)


def torch64(x):
    return torch.from_numpy(np.ascontiguousarray(x))
