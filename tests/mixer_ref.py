"""Plain 64-bit forms of linear attention with a decay per head and of the norm and
rotation of its queries and keys, and of their gradients, in torch on the CPU.  Tests and
magnitudes only; nothing here is shared with the kernels.

Every function takes `mag`: with it, each factor enters by its absolute value, so that
the result is the sum of the absolute values of the terms.
"""
from __future__ import annotations

import torch

from tests.layer_ref import _abs, d64, held

F64 = torch.float64


def power(g, d):
    """exp(g d) for [H] rates and whole distances, 1 at distance 0 whatever the rate: [H, *d]."""
    x = g.view(-1, *[1] * d.dim()) * d
    return torch.where(d == 0, torch.ones((), dtype=F64), torch.exp(x))


def attention(q, k, v, log_decay, h0=None, scale=None, lengths=None, mag=False, dy=None, dh_final=None):
    """y, h and, with dy, dq, dk, dv, dh0.  Rows behind the lengths are zero here."""
    q, k, v, g, h0, dy, dh = (d64(t) for t in (q, k, v, log_decay, h0, dy, dh_final))
    Bt, L, H, K = q.shape
    Hk, V = v.shape[2:]
    per, scale = H // Hk, K ** -0.5 if scale is None else scale
    out = dict(y=torch.zeros(Bt, L, H, V, dtype=F64), h=torch.zeros(Bt, H, K, V, dtype=F64))
    if dy is not None:
        out.update(dq=torch.zeros(Bt, L, H, K, dtype=F64), dk=torch.zeros(Bt, L, Hk, K, dtype=F64),
                   dv=torch.zeros(Bt, L, Hk, V, dtype=F64), dh0=torch.zeros(Bt, H, K, V, dtype=F64))
    for b, n in enumerate(held(lengths, Bt, L)):
        def heads(x, many):
            x = _abs(x[b, :n].transpose(0, 1), mag)  # [heads, n, .]
            return x.repeat_interleave(many, 0)

        zero = torch.zeros(H, K, V, dtype=F64)
        S0 = zero if h0 is None else _abs(h0[b], mag)
        qb, kb, vb = heads(q, 1), heads(k, per), heads(v, per)
        i = torch.arange(n, dtype=F64)
        w = torch.tril(power(g, (i[:, None] - i).clamp(min=0)))
        ahead, left = power(g, i + 1)[..., None], power(g, n - 1 - i)[..., None]
        whole = power(g, torch.tensor(float(n), dtype=F64))[:, None, None]
        s = abs(scale) if mag else scale
        out["y"][b, :n] = (s * ((qb @ kb.mT * w) @ vb + ahead * (qb @ S0))).transpose(0, 1)
        out["h"][b] = whole * S0 + (kb * left).mT @ vb
        if dy is None:
            continue
        db = heads(dy, 1)
        D = zero if dh is None else _abs(dh[b], mag)
        dP = db @ vb.mT * w  # [H, t, j]
        P = qb @ kb.mT * w
        out["dq"][b, :n] = (s * (dP @ kb + ahead * (db @ S0.mT))).transpose(0, 1)
        dk = s * (dP.mT @ qb) + left * (vb @ D.mT)
        dv = s * (P.mT @ db) + left * (kb @ D)
        out["dk"][b, :n] = dk.view(Hk, per, n, K).sum(1).transpose(0, 1)
        out["dv"][b, :n] = dv.view(Hk, per, n, V).sum(1).transpose(0, 1)
        out["dh0"][b] = whole * D + s * ((qb * ahead).mT @ db)
    return out


def _turn(x, cos, sin, R, adjacent, mag):
    """The first R elements in pairs: y0 = x0 cos - x1 sin, y1 = x1 cos + x0 sin."""
    if R == 0:
        return x
    y = x.clone()
    lo = slice(0, R, 2) if adjacent else slice(0, R // 2)
    hi = slice(1, R, 2) if adjacent else slice(R // 2, R)
    x0, x1 = x[..., lo], x[..., hi]
    if mag:
        c, s = cos.abs(), sin.abs()
        y[..., lo], y[..., hi] = x0 * c + x1 * s, x1 * c + x0 * s
    else:
        y[..., lo], y[..., hi] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    return y


def rope(x, w=None, freqs=None, positions=None, start=0, lengths=None, eps=1e-6, norm=True, adjacent=False, mag=False, dy=None):
    """y and, with dy, dx and dw, for one of the two tensors.  Rows behind the lengths
    are zero here."""
    x, w, freqs, dy = (d64(t) for t in (x, w, freqs, dy))
    Bt, L, H, D = x.shape
    R = 0 if freqs is None else 2 * len(freqs)
    at = torch.arange(L).expand(Bt, L) + start if positions is None else positions.cpu()
    ns = torch.tensor(held(lengths, Bt, L))
    ok = (torch.arange(L)[None] < ns[:, None])[..., None, None]
    x = torch.where(ok, x, torch.zeros((), dtype=F64))
    angle = at.to(F64)[..., None, None] * (freqs if R else torch.zeros(1, dtype=F64))
    cos, sin = torch.cos(angle), torch.sin(angle)
    gain = torch.ones(D, dtype=F64) if w is None else w
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if norm else torch.ones((), dtype=F64)
    n = _abs(x, mag) * r
    out = dict(y=torch.where(ok, _turn(n * _abs(gain, mag), cos, sin, R, adjacent, mag), torch.zeros((), dtype=F64)))
    if dy is None:
        return out
    dy = torch.where(ok, _abs(dy, mag), torch.zeros((), dtype=F64))
    d = _turn(dy, cos, -sin, R, adjacent, mag)
    out["dw"] = (d * n).sum((0, 1, 2))
    e = d * _abs(gain, mag)
    if norm:
        m = n * (e * n).mean(-1, keepdim=True)
        e = r * (e + m if mag else e - m)
    out["dx"] = torch.where(ok, e, torch.zeros((), dtype=F64))
    return out
