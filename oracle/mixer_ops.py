"""fp64 oracle of the short convolution, the Mamba-2 mixer with it in front, and
RMS norm: the definitions, token by token, in plain torch on the CPU.

Each function returns values and, for tolerances, magnitudes: the same sums
with every term's absolute value, which is what a rounding inside is relative
to.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def _d(t):
    return None if t is None else t.detach().cpu().to(F64)


def _lengths(lengths, batch, L):
    return [L] * batch if lengths is None else [min(max(int(n), 0), L) for n in lengths]


def _act(pre, silu):
    return pre * torch.sigmoid(pre) if silu else pre


def _slope(pre, silu):
    s = torch.sigmoid(pre)
    return s * (1.0 + pre * (1.0 - s)) if silu else torch.ones_like(pre)


def conv(x, weight, bias=None, silu=True, lengths=None, state=None):
    """(y, last_state, magnitude of y) of x [B, L, D]."""
    x, w, b, s0 = _d(x), _d(weight), _d(bias), _d(state)
    B, L, D = x.shape
    K = w.shape[1]
    y, mag = torch.zeros(B, L, D, dtype=F64), torch.zeros(B, L, D, dtype=F64)
    last = torch.zeros(B, K - 1, D, dtype=F64)
    for i, n in enumerate(_lengths(lengths, B, L)):
        rows = torch.cat([s0[i] if s0 is not None else torch.zeros(K - 1, D, dtype=F64), x[i, :n]])
        for t in range(n):
            pre = (rows[t:t + K] * w.t()).sum(0) + (0 if b is None else b)
            y[i, t] = _act(pre, silu)
            mag[i, t] = (rows[t:t + K] * w.t()).abs().sum(0) + (0 if b is None else b.abs())
        last[i] = rows[n:n + K - 1]
    return y, last, mag


def conv_bwd(x, weight, bias, dout, silu=True, lengths=None, state=None, dlast=None):
    """Gradients and their magnitudes, as two dicts."""
    x, w, b, s0, dy, dl = _d(x), _d(weight), _d(bias), _d(state), _d(dout), _d(dlast)
    B, L, D = x.shape
    K = w.shape[1]
    zero = lambda *s: torch.zeros(*s, dtype=F64)
    g = {"dx": zero(B, L, D), "dweight": zero(D, K), "dbias": zero(D), "dstate": zero(B, K - 1, D)}
    m = {k: torch.zeros_like(v) for k, v in g.items()}
    for i, n in enumerate(_lengths(lengths, B, L)):
        rows = torch.cat([s0[i] if s0 is not None else zero(K - 1, D), x[i, :n]])
        drows, mrows = zero(n + K - 1, D), zero(n + K - 1, D)
        for t in range(n):
            terms = rows[t:t + K] * w.t()
            pre = terms.sum(0) + (0 if b is None else b)
            size = terms.abs().sum(0) + (0 if b is None else b.abs())
            gt = dy[i, t] * _slope(pre, silu)
            gm = dy[i, t].abs() * (1.0 + size)
            for k in range(K):
                drows[t + k] += w[:, k] * gt
                mrows[t + k] += w[:, k].abs() * gm
                g["dweight"][:, k] += gt * rows[t + k]
                m["dweight"][:, k] += gm * rows[t + k].abs()
            g["dbias"] += gt
            m["dbias"] += gm
        if dl is not None:
            drows[n:] += dl[i]
            mrows[n:] += dl[i].abs()
        g["dstate"][i], m["dstate"][i] = drows[:K - 1], mrows[:K - 1]
        g["dx"][i, :n], m["dx"][i, :n] = drows[K - 1:], mrows[K - 1:]
    return g, m


def mixer(xbc, dt, weight, bias, A, D, dt_bias, ngroups, dstate, lengths=None, h0=None, conv_state=None):
    """(y, last_state, last_conv_state) and the magnitudes of the first two."""
    v, last_conv, vm = conv(xbc, weight, bias, True, lengths, conv_state)
    A, D, dtb, dt = _d(A), _d(D), _d(dt_bias), _d(dt)
    B, L, H = dt.shape
    G, N = ngroups, dstate
    P = (v.shape[2] - 2 * G * N) // H
    head = torch.arange(H) // (H // G)

    def parts(t):
        x, b, c = t.split([H * P, G * N, G * N], -1)
        return x.reshape(B, L, H, P), b.reshape(B, L, G, N)[:, :, head], c.reshape(B, L, G, N)[:, :, head]

    (x, b, c), (xm, bm, cm) = parts(v), parts(vm)
    step = dt + (0 if dtb is None else dtb)
    step = torch.where(step > 30, step, torch.log1p(torch.exp(step.clamp(max=30))))
    S = _d(h0).clone() if h0 is not None else torch.zeros(B, H, P, N, dtype=F64)
    Sm = S.abs()
    y, ym = torch.zeros(B, L, H, P, dtype=F64), torch.zeros(B, L, H, P, dtype=F64)
    for i, n in enumerate(_lengths(lengths, B, L)):
        for t in range(n):
            a, s = torch.exp(step[i, t] * A)[:, None, None], step[i, t][:, None, None]
            S[i] = a * S[i] + s * x[i, t][:, :, None] * b[i, t][:, None]
            Sm[i] = a * Sm[i] + s * xm[i, t][:, :, None] * bm[i, t][:, None]
            y[i, t] = (S[i] * c[i, t][:, None]).sum(-1)
            ym[i, t] = (Sm[i] * cm[i, t][:, None]).sum(-1)
            if D is not None:
                y[i, t] += D[:, None] * x[i, t]
                ym[i, t] += D.abs()[:, None] * xm[i, t]
    return (y, S, last_conv), (ym, Sm)


def rms(x, weight=None, residual=None, gate=None, groups=1, eps=1e-5):
    """(y, s, rstd [rows, groups]) of x [rows, dim], and the magnitude of y."""
    x, w, r, z = _d(x), _d(weight), _d(residual), _d(gate)
    s, sm = x, x.abs()
    if z is not None:
        s = x * z * torch.sigmoid(z)
        sm = s.abs()
    if r is not None:
        s, sm = x + r, x.abs() + r.abs()
    R, D = s.shape
    rstd = 1.0 / torch.sqrt(s.reshape(R, groups, -1).square().mean(-1) + eps)
    by = rstd.repeat_interleave(D // groups, 1) * (1.0 if w is None else w)
    return s * by, s, rstd, sm * by.abs()


def rms_bwd(dy, s, weight, rstd, gate=None, groups=1, dresidual=None):
    """Gradients and their magnitudes, as two dicts; with a gate s is x."""
    dy, x, w, z, dr = _d(dy), _d(s), _d(weight), _d(gate), _d(dresidual)
    R, D = x.shape
    a = None if z is None else torch.sigmoid(z)
    s = x if z is None else x * z * a
    r = _d(rstd).reshape(R, groups).repeat_interleave(D // groups, 1)
    xh = s * r
    v = dy if w is None else dy * w
    mean = lambda t: t.reshape(R, groups, -1).mean(-1).repeat_interleave(D // groups, 1)
    ds = r * (v - xh * mean(v * xh))
    dm = r * (v.abs() + xh.abs() * mean((v * xh).abs()))
    g, m = {"dweight": (dy * xh).sum(0)}, {"dweight": (dy * xh).abs().sum(0)}
    if z is not None:
        slope = a * (1.0 + z * (1.0 - a))
        g["dx"], g["dgate"] = ds * z * a, ds * x * slope
        m["dx"], m["dgate"] = dm * (z * a).abs(), dm * x.abs() * (a * (1.0 + (z * (1.0 - a)).abs()))
        return g, m
    if dr is not None:
        ds, dm = ds + dr, dm + dr.abs()
    g["dx"] = g["dresidual"] = ds
    m["dx"] = m["dresidual"] = dm
    return g, m
