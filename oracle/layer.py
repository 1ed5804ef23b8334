"""fp64 numpy references of the operators around and beside the plain
attention: norm and rotation of queries and keys, attention with a causal
window and sinks, their gradients, and the single-token form.  Every score
matrix is materialised; nothing here is shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch


def f64(t):
    return t.detach().cpu().double().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, np.float64)


# ------------------------------------------------------- norm and rotation

def angles(max_pos, rot, base=10000.0, scaling="none", factor=1.0, original_max_pos=0):
    """(cos, sin) [max_pos, rot / 2] by the scaling's own definition, pair by pair."""
    inv, mul = [], 1.0
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            # pair index at which a wavelength fits `t` times into the original context
            at = {t: rot / 2 * math.log(original_max_pos / (2 * math.pi * t)) / math.log(base)
                  for t in (32, 1)}
            lo, hi = max(math.floor(at[32]), 0), min(math.ceil(at[1]), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f = f * (1 - ramp) + f / factor * ramp
            mul = 1 + 0.1 * math.log(factor)
        inv.append(f)
    a = np.arange(max_pos, dtype=np.float64)[:, None] * np.array(inv)[None, :]
    return np.cos(a) * mul, np.sin(a) * mul


def pair_columns(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotation_matrices(cos, sin, positions, d, interleaved):
    """[B, N, d, d]: the rotation of each token as a dense matrix."""
    cos, sin = f64(cos), f64(sin)
    B, N = positions.shape
    a, b = pair_columns(2 * cos.shape[1], interleaved)
    R = np.tile(np.eye(d), (B, N, 1, 1))
    c, s = cos[positions], sin[positions]
    R[:, :, a, a], R[:, :, b, b] = c, c
    R[:, :, a, b], R[:, :, b, a] = -s, s
    return R


def norm_rope(x, w, cos, sin, positions, eps, interleaved):
    """[B, H, N, d] -> (result, the sum of the moduli of each element's terms)."""
    x = f64(x)
    R = rotation_matrices(cos, sin, positions, x.shape[-1], interleaved)
    y = x if w is None else x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * f64(w)
    return (np.einsum("bnij,bhnj->bhni", R, y), np.einsum("bnij,bhnj->bhni", np.abs(R), np.abs(y)))


def norm_rope_bwd(dy, x, w, cos, sin, positions, eps, interleaved):
    """(dx, dw, moduli of dx's terms, moduli of dw's terms); dw None without a norm."""
    dy, x = f64(dy), f64(x)
    d = x.shape[-1]
    R = rotation_matrices(cos, sin, positions, d, interleaved)
    g = np.einsum("bnij,bhni->bhnj", R, dy)
    ga = np.einsum("bnij,bhni->bhnj", np.abs(R), np.abs(dy))
    if w is None:
        return g, None, ga, None
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    n, w = x * r, f64(w)
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdims=True))
    dxa = r * (ga * np.abs(w) + np.abs(n) * (ga * np.abs(w * n)).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1, 2)), dxa, (ga * np.abs(n)).sum((0, 1, 2))


# ------------------------------------------------- window and sinks

def visible(n, window, sinks):
    """[n, n]: key j visible from query i iff j <= i and (i - j <= window or j < sinks)."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((window < 0) | (i - j <= window) | (j < sinks))


def sinks_probs(q, k, window, sinks, scale):
    """(P [B, H, N, N], LSE [B, H, N]) with k's heads shared by H / Hk query heads."""
    q, k = f64(q), np.repeat(f64(k), q.shape[1] // k.shape[1], axis=1)
    s = np.einsum("bhid,bhjd->bhij", q, k) * scale
    s = np.where(visible(q.shape[2], window, sinks), s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    return p / l, (m + np.log(l))[..., 0]


def sinks_fwd(q, k, v, window, sinks, scale):
    p, lse = sinks_probs(q, k, window, sinks, scale)
    return p @ np.repeat(f64(v), q.shape[1] // v.shape[1], axis=1), lse


def sinks_bwd(q, k, v, dout, window, sinks, scale, u=0.0):
    """(dQ, dK, dV) and, for a relative rounding u of P, dS and O, the bounds
    of the three results' errors."""
    B, H, N, d = q.shape
    Hk = k.shape[1]
    G = H // Hk
    p, _ = sinks_probs(q, k, window, sinks, scale)
    qd, g = f64(q), f64(dout)
    kd, vd = (np.repeat(f64(t), G, axis=1) for t in (k, v))
    o = p @ vd
    dp = g @ vd.swapaxes(-1, -2)
    D = (g * o).sum(-1, keepdims=True)
    ds = p * (dp - D)
    E = p * (2 * u * np.abs(dp - D) + u * np.abs(g * o).sum(-1, keepdims=True))

    def heads(t):  # sum over the query heads that share a key head
        return t.reshape(B, Hk, G, N, d).sum(2)

    grads = (scale * ds @ kd, scale * heads(ds.swapaxes(-1, -2) @ qd), heads(p.swapaxes(-1, -2) @ g))
    bounds = (scale * E @ np.abs(kd), scale * heads(E.swapaxes(-1, -2) @ np.abs(qd)),
              u * heads(p.swapaxes(-1, -2) @ np.abs(g)))
    return grads, bounds


def sinks_decode(q, k, v, lens, window, sinks, scale):
    """q [B, H, d] against the first lens[b] cached rows of k, v [B, Hk, S, d];
    (O, LSE, sum_j P |v_j|).  Rows no query sees are not read."""
    q = f64(q)
    B, H, d = q.shape
    Hk = k.shape[1]
    o, a, lse = np.zeros((B, H, d)), np.zeros((B, H, d)), np.full((B, H), -np.inf)
    for b in range(B):
        n = int(lens[b])
        j = [x for x in range(n) if window < 0 or x >= n - 1 - window or x < sinks]
        if not j:
            continue
        kb, vb = f64(k[b][:, j]), f64(v[b][:, j])
        for h in range(H):
            c = h // (H // Hk)
            s = kb[c] @ q[b, h] * scale
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + math.log(p.sum())
            p /= p.sum()
            o[b, h], a[b, h] = p @ vb[c], p @ np.abs(vb[c])
    return o, lse, a
