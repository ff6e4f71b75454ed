"""fp64 oracle of the gated delta rule, layer norm and dropout (numpy, token
by token and element by element from the definitions in
``include/selscan.h``; shares no code with the HIP path)."""
from __future__ import annotations

import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def _lengths(lengths, batch, L):
    if lengths is None:
        return [L] * batch
    return [min(max(int(n), 0), L) for n in lengths]


def delta(q, k, v, g, beta, scale=None, lengths=None, h0=None):
    """(y [B, L, H, P], last_state [B, H, P, N]) of the recurrence."""
    q, k, v, g, beta, h0 = map(_f64, (q, k, v, g, beta, h0))
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    S = np.zeros((B, H, P, N)) if h0 is None else h0.copy()
    y = np.zeros((B, L, H, P))
    for b, n in enumerate(_lengths(lengths, B, L)):
        for t in range(n):
            for h in range(H):
                kt, qt = k[b, t, h // (H // G)], q[b, t, h // (H // G)]
                Sa = np.exp(g[b, t, h]) * S[b, h]
                u = beta[b, t, h] * (v[b, t, h] - Sa @ kt)
                S[b, h] = Sa + np.outer(u, kt)
                y[b, t, h] = scale * (S[b, h] @ qt)
    return y, S


def delta_bwd(q, k, v, g, beta, dout, scale=None, lengths=None, h0=None, dlast=None):
    """Gradients by reverse mode through the recurrence, every state kept."""
    q, k, v, g, beta, dout, h0, dlast = map(_f64, (q, k, v, g, beta, dout, h0, dlast))
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    r = H // G
    scale = N ** -0.5 if scale is None else scale
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g),
           "dbeta": np.zeros_like(beta), "dh0": np.zeros((B, H, P, N))}
    for b, n in enumerate(_lengths(lengths, B, L)):
        for h in range(H):
            S = np.zeros((P, N)) if h0 is None else h0[b, h].copy()
            hist = []
            for t in range(n):
                Sa = np.exp(g[b, t, h]) * S
                e = v[b, t, h] - Sa @ k[b, t, h // r]
                S = Sa + np.outer(beta[b, t, h] * e, k[b, t, h // r])
                hist.append((Sa, e, S))
            D = np.zeros((P, N)) if dlast is None else dlast[b, h].copy()
            for t in reversed(range(n)):
                Sa, e, St = hist[t]
                kt, qt, bt = k[b, t, h // r], q[b, t, h // r], beta[b, t, h]
                dy = scale * dout[b, t, h]
                out["dq"][b, t, h // r] += dy @ St
                D = D + np.outer(dy, qt)
                du = D @ kt
                out["dk"][b, t, h // r] += (bt * e) @ D - (bt * du) @ Sa
                out["dv"][b, t, h] = bt * du
                out["dbeta"][b, t, h] = du @ e
                X = D - np.outer(bt * du, kt)
                out["dg"][b, t, h] = np.sum(X * Sa)
                D = np.exp(g[b, t, h]) * X
            out["dh0"][b, h] = D
    return out


def philox(counter, key):
    """Philox4x32-10 of one counter (four words) and key (two words)."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def keep(n, p, seed, offset):
    """Truth of the n elements that dropout keeps."""
    m = 0xFFFFFFFF
    words = []
    for i in range((n + 3) // 4):
        words += philox((i & m, i >> 32, offset & m, offset >> 32), (seed & m, seed >> 32))
    return np.asarray(words[:n], dtype=np.uint64) >= int(p * 2.0 ** 32)


def dropout(x, p, seed, offset=0):
    x = _f64(x)
    if p == 0.0:
        return x
    return np.where(keep(x.size, p, seed, offset).reshape(x.shape), x / (1.0 - p) if p < 1.0 else 0.0, 0.0)


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5, p=0.0, seed=0, offset=0):
    """(y, s, mean, rstd)."""
    s = dropout(x, p, seed, offset)
    if residual is not None:
        s = s + _f64(residual)
    mean = s.mean(-1)
    rstd = 1.0 / np.sqrt(((s - mean[..., None]) ** 2).mean(-1) + eps)
    y = (s - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, s, mean, rstd


def layer_norm_bwd(dy, s, weight, mean, rstd, dresidual=None, p=0.0, seed=0, offset=0):
    dy, s, weight, mean, rstd, dresidual = map(_f64, (dy, s, weight, mean, rstd, dresidual))
    dim = s.shape[-1]
    xh = (s - mean[..., None]) * rstd[..., None]
    w = dy if weight is None else dy * weight
    ds = rstd[..., None] * (w - w.mean(-1, keepdims=True) - xh * (w * xh).mean(-1, keepdims=True))
    if dresidual is not None:
        ds = ds + dresidual
    return {"dx": dropout(ds, p, seed, offset), "dresidual": ds, "dweight": (dy * xh).reshape(-1, dim).sum(0),
            "dbias": dy.reshape(-1, dim).sum(0)}
