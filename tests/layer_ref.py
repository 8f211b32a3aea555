"""Plain 64-bit forms of the layer operators (causal convolution, selective
scan, gated and residual norms) and of their gradients, token by token in torch
on the CPU.  Tests and magnitudes only; nothing here is shared with the kernels.

Every function takes `mag`: with it, each factor enters by its absolute value,
so that the result is the sum of the absolute values of the terms.  A sum of
products computed in fp32 with at most k roundings on any path from an input to
the result is off by at most about k 2^-24 times that magnitude; an output type
adds half a step of its own.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def d64(t):
    return None if t is None else t.detach().to("cpu", F64)


def _abs(t, mag):
    return t.abs() if mag and t is not None else t


def sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def silu(v, mag=False):
    return _abs(v, mag) * sigmoid(v)


def dsilu(v, mag=False):
    g = sigmoid(v)
    return g * (1 + _abs(v, mag) * (1 - g))


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def held(lengths, Bt, L):
    if lengths is None:
        return [L] * Bt
    return [max(0, min(L, int(n))) for n in lengths]


# ---------------------------------------------------------------- convolution
def conv(x, w, bias=None, state=None, lengths=None, act=True, mag=False, dy=None):
    """y, state and, with dy, dx, dw, dbias, dstate.  Rows of y behind the
    lengths are zero here."""
    x, w, bias, state, dy = (d64(t) for t in (x, w, bias, state, dy))
    Bt, L, D = x.shape
    W = w.shape[1]
    out = dict(y=torch.zeros_like(x), state=torch.zeros(Bt, W - 1, D, dtype=F64))
    if dy is not None:
        out.update(dx=torch.zeros_like(x), dw=torch.zeros_like(w), dbias=torch.zeros(D, dtype=F64),
                   dstate=torch.zeros(Bt, W - 1, D, dtype=F64))
    wm = _abs(w, mag)
    for b, n in enumerate(held(lengths, Bt, L)):
        first = state[b] if state is not None else torch.zeros(W - 1, D, dtype=F64)
        xs = torch.cat([first, x[b, :n]])
        out["state"][b] = xs[n:n + W - 1]
        true = torch.zeros(n, D, dtype=F64) + (bias if bias is not None else 0)
        for k in range(W):
            true = true + w[:, k] * xs[k:k + n]
        xs = _abs(xs, mag)
        pre = torch.zeros(n, D, dtype=F64) + (_abs(bias, mag) if bias is not None else 0)
        for k in range(W):
            pre = pre + wm[:, k] * xs[k:k + n]
        # magnitude of act: |act'| <= 1.1 on the argument's own magnitude
        out["y"][b, :n] = (pre if mag else silu(pre)) if act else pre
        if dy is None:
            continue
        dp = _abs(dy[b, :n], mag) * (dsilu(true, mag) if act else 1.0)
        if mag and act:  # |act''| <= 0.5 on the argument's own magnitude
            dp = dp + 0.5 * dy[b, :n].abs() * pre
        dxs = torch.zeros(n + W - 1, D, dtype=F64)
        for k in range(W):
            dxs[k:k + n] += wm[:, k] * dp
            out["dw"][:, k] += (dp * xs[k:k + n]).sum(0)
        out["dbias"] += dp.sum(0)
        out["dx"][b, :n] = dxs[W - 1:]
        out["dstate"][b] = dxs[:W - 1]
    return out


# ---------------------------------------------------------------- selective scan
def scan(x, dt, A, B, C, D=None, z=None, h0=None, lengths=None, dt_softplus=False, dt_bias=None, mag=False, dy=None,
         dh_final=None):
    """y, h and, with dy, every gradient.  Rows of y behind the lengths are zero
    here."""
    x, dt, A, B, C, D, z, h0, dt_bias, dy, dh_final = (d64(t) for t in (x, dt, A, B, C, D, z, h0, dt_bias, dy, dh_final))
    Bt, L, Dm = x.shape
    G, N = B.shape[-2:]
    per = Dm // G
    ns = torch.tensor(held(lengths, Bt, L))
    ok = (torch.arange(L)[None] < ns[:, None])[..., None]
    zero = torch.zeros((), dtype=F64)
    x, dt = torch.where(ok, x, zero), torch.where(ok, dt, zero)
    z = None if z is None else torch.where(ok, z, zero)
    B, C = torch.where(ok[..., None], B, zero), torch.where(ok[..., None], C, zero)
    raw = dt + dt_bias if dt_bias is not None else dt
    delta = torch.where(ok, softplus(raw) if dt_softplus else raw, zero)
    x, B, C, D, h0, dh_final = (_abs(t, mag) for t in (x, B, C, D, h0, dh_final))
    Am = _abs(A, mag)
    dm = _abs(delta, mag)
    Bw, Cw = B.repeat_interleave(per, 2), C.repeat_interleave(per, 2)  # [Bt, L, Dm, N]
    skip = D if D is not None else torch.zeros(Dm, dtype=F64)
    h = h0 if h0 is not None else torch.zeros(Bt, Dm, N, dtype=F64)
    a = torch.exp(delta[..., None] * A)
    u = dm * x
    hs, before, o = [], [], []
    for t in range(L):
        before.append(h)
        h = a[:, t] * h + u[:, t, :, None] * Bw[:, t]
        hs.append(h)
        o.append((h * Cw[:, t]).sum(-1) + skip * x[:, t])
    o = torch.stack(o, 1)
    gate = silu(z, mag) if z is not None else torch.ones_like(x)
    out = dict(y=torch.where(ok, o * gate, zero), h=h)
    if dy is None:
        return out
    dy = torch.where(ok, _abs(dy, mag), zero)
    do = dy * gate
    out["dz"] = None if z is None else dy * o * dsilu(z, mag)
    out["dD"] = None if D is None else (do * x).sum((0, 1))
    g = dh_final if dh_final is not None else torch.zeros(Bt, Dm, N, dtype=F64)
    dx, ddt = torch.zeros_like(x), torch.zeros_like(x)
    dB, dC, dA = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A)
    for t in reversed(range(L)):
        g = g + Cw[:, t] * do[:, t, :, None]
        dC[:, t] = (do[:, t, :, None] * hs[t]).view(Bt, G, per, N).sum(2)
        dB[:, t] = (g * u[:, t, :, None]).view(Bt, G, per, N).sum(2)
        gB = (g * Bw[:, t]).sum(-1)
        q = g * a[:, t] * before[t]
        dx[:, t] = skip * do[:, t] + dm[:, t] * gB
        dd = x[:, t] * gB + (q * Am).sum(-1)
        ddt[:, t] = dd * sigmoid(raw[:, t]) if dt_softplus else dd
        dA += (q * dm[:, t, :, None]).sum(0)
        g = a[:, t] * g
    out.update(dx=torch.where(ok, dx, zero), ddt=torch.where(ok, ddt, zero), dA=dA, dB=torch.where(ok[..., None], dB, zero),
               dC=torch.where(ok[..., None], dC, zero), dh0=g)
    out["ddt_bias"] = None if dt_bias is None else out["ddt"].sum((0, 1))
    out["steepest"] = float((delta[..., None] * A).abs().max())
    return out


# ---------------------------------------------------------------- norms
def gated_norm(x, z=None, w=None, groups=1, eps=1e-6, gate_first=True, mag=False, dy=None):
    x, z, w, dy = (d64(t) for t in (x, z, w, dy))
    lead, width = x.shape[:-1], x.shape[-1]
    x = x.reshape(-1, width)
    z = None if z is None else z.reshape(-1, width)
    gate = silu(z) if z is not None else torch.ones_like(x)
    wv = w if w is not None else torch.ones(width, dtype=F64)
    v = x * gate if gate_first else x
    r = (v.view(-1, groups, width // groups).square().mean(-1, keepdim=True) + eps) ** -0.5
    r = r.expand(-1, groups, width // groups).reshape(v.shape)
    n = v * r
    out = dict(y=(n * wv if gate_first else n * wv * gate).reshape(*lead, width))
    if mag:
        out["y"] = out["y"].abs()
    if dy is None:
        return out
    dy = dy.reshape(-1, width)
    up = dy if gate_first else dy * gate
    e = up * wv

    def mean(q):
        m = q.view(-1, groups, width // groups).mean(-1, keepdim=True)
        return m.expand(-1, groups, width // groups).reshape(v.shape)

    if mag:
        x, gate, n, up, e, wv, dy = (q.abs() for q in (x, gate, n, up, e, wv, dy))
        dv = r * (e + n * mean(e * n))
        dg = dsilu(z, True) if z is not None else None
    else:
        dv = r * (e - n * mean(e * n))
        dg = dsilu(z) if z is not None else None
    out["dx"] = (dv * gate if gate_first else dv).reshape(*lead, width)
    out["dz"] = None if z is None else ((dv * x if gate_first else dy * n * wv) * dg).reshape(*lead, width)
    out["dw"] = None if w is None else (up * n).sum(0)
    return out


def residual_norm(x, residual=None, w=None, scale=None, eps=1e-6, mag=False):
    x, residual, w, scale = (d64(t) for t in (x, residual, w, scale))
    sx = x * (scale if scale is not None else 1.0)
    h = sx + (residual if residual is not None else 0.0)
    r = (h.square().mean(-1, keepdim=True) + eps) ** -0.5
    m = sx.abs() + (residual.abs() if residual is not None else 0.0) if mag else h
    return dict(residual=m, y=m * r * (_abs(w, mag) if w is not None else 1.0))


def residual_norm_backward(h, x=None, w=None, scale=None, dy=None, dresidual=None, eps=1e-6, mag=False):
    h, x, w, scale, dy, dresidual = (d64(t) for t in (h, x, w, scale, dy, dresidual))
    r = (h.square().mean(-1, keepdim=True) + eps) ** -0.5
    h, x, w, scale, dy, dresidual = (_abs(t, mag) for t in (h, x, w, scale, dy, dresidual))
    n = h * r
    e = dy * (w if w is not None else 1.0)
    m = n * (e * n).mean(-1, keepdim=True)
    dh = r * (e + m if mag else e - m) + (dresidual if dresidual is not None else 0.0)
    rows = tuple(range(h.dim() - 1))
    return dict(dresidual=dh, dx=dh * (scale if scale is not None else 1.0), dw=None if w is None else (dy * n).sum(rows),
                dscale=None if scale is None else (dh * x).sum(rows))
