"""Timing and accuracy cases of the layer operators around a selective state-space
core: the short causal convolution, the selective scan (A per channel and state),
the gated group norm after it and the residual norm before the next block; each for
prompts, for training (backward) and, where it differs, for single tokens.

`run` computes a case either in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with `own` set, through the library's entry
points; `exact` computes it from the definitions in 64 bits, token by token.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the convolution in front of the core over whole prompts: x is one half of the
        # input projection's rows (strided), the last W - 1 inputs are kept for decoding
        dict(name="conv_prompt", op="conv", Bt=8, L=4096, D=2048, W=4, dtype="bf16", ragged=False),
        # the same convolution in a training step: gradients of inputs, taps and bias
        dict(name="conv_training", op="conv_backward", Bt=8, L=4096, D=2048, W=4, dtype="bf16", ragged=False),
        # one token of one sequence: nothing but latency
        dict(name="conv_token", op="conv_step", Bt=1, D=2048, W=4, dtype="bf16"),
        # the scan over a batch of prompts, gated, with the state kept for decoding
        dict(name="scan_prompt", op="scan", Bt=8, L=4096, D=2048, N=16, G=1, dtype="bf16", ragged=False),
        # one long document: few channels to share the work, a long token axis
        dict(name="scan_long", op="scan", Bt=1, L=16384, D=2048, N=16, G=1, dtype="bf16", ragged=False),
        # a padded batch of uneven requests (one empty, one of a single token), odd sizes,
        # two groups of B and C, full precision
        dict(name="scan_ragged", op="scan", Bt=5, L=1537, D=1000, N=24, G=2, dtype="fp32", ragged=True),
        # the scan's gradients in a training step
        dict(name="scan_training", op="scan_backward", Bt=8, L=2048, D=2048, N=16, G=1, dtype="bf16", ragged=False),
        # one token for each of 256 sequences against the resident states
        dict(name="scan_token", op="scan_step", Bt=256, D=2048, N=16, G=1, dtype="bf16"),
        # the gated group norm behind the core over whole prompts, the gate strided
        dict(name="gated_prompt", op="gated_norm", M=32768, D=2048, G=8, gate_first=True, dtype="bf16"),
        # its gradients in a training step
        dict(name="gated_training", op="gated_norm_backward", M=32768, D=2048, G=8, gate_first=True, dtype="bf16"),
        # residual sum and norm in front of the next block, one token for each of 256
        # sequences, the residual stream kept in fp32
        dict(name="residual_tokens", op="residual_norm", M=256, D=2048, dtype="bf16", res_dtype="fp32"),
        # its gradients in a training step, with a scale per channel on the block's output
        dict(name="residual_training", op="residual_norm_backward", M=32768, D=2048, dtype="bf16", res_dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_backward", "conv_step", "scan", "scan", "scan_backward", "scan_backward", "scan_step",
                     "gated_norm", "gated_norm_backward", "residual_norm", "residual_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D = _log(rng, 48, 4096)
    if rng.random() < 0.6:  # widths are mostly multiples of 64, but not all of them
        D = max(64, D // 64 * 64)
    if op in ("conv", "conv_backward"):
        L = _log(rng, 1, 8192)
        Bt = _log(rng, 1, max(1, min(64, (1 << 25) // (L * D))))
        return dict(op=op, Bt=Bt, L=L, D=D, W=rng.choice([2, 3, 4]), dtype=dtype, ragged=rng.random() < 0.3)
    if op == "conv_step":
        return dict(op=op, Bt=_log(rng, 1, 512), D=D, W=rng.choice([2, 3, 4]), dtype=dtype)
    if op in ("scan", "scan_backward", "scan_step"):
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 2])
        D = max(2, D // G) * G
        if op == "scan_step":
            return dict(op=op, Bt=_log(rng, 1, 256), D=D, N=N, G=G, dtype=dtype)
        L = _log(rng, 1, 8192)
        most = (1 << 29) if op == "scan" else (1 << 28)
        L = max(1, min(L, most // (D * N)))
        Bt = _log(rng, 1, max(1, min(32, most // (L * D * N))))
        return dict(op=op, Bt=Bt, L=L, D=D, N=N, G=G, dtype=dtype, ragged=rng.random() < 0.3)
    M = _log(rng, 1, max(1, min(65536, (1 << 26) // D)))
    if op in ("gated_norm", "gated_norm_backward"):
        G = rng.choice([1, 1, 2, 4, 8])
        D = max(8, D // G) * G
        return dict(op=op, M=M, D=D, G=G, gate_first=rng.random() < 0.6, dtype=dtype)
    return dict(op=op, M=M, D=D, dtype=dtype, res_dtype=rng.choice([dtype, "fp32"]))


# ---------------------------------------------------------------- inputs
def _lengths(c, gen):
    """Request lengths in a padded batch: one empty, one of a single token, one full."""
    if not c["ragged"]:
        return None
    n = torch.randint(0, c["L"] + 1, (c["Bt"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = c["L"]
    if c["Bt"] > 1:
        n[1] = 0
    if c["Bt"] > 2:
        n[2] = 1
    return n


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = DTYPES[c["dtype"]]

    def normal(*shape, dtype=t, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    f32 = torch.float32
    op, D = c["op"], c["D"]
    s = {"case": c}
    if op.startswith("conv"):
        W = c["W"]
        s["w"] = normal(D, W, dtype=f32, scale=W ** -0.5)
        s["bias"] = normal(D, dtype=f32, scale=0.1)
        if op == "conv_step":
            s["x"] = normal(c["Bt"], 2 * D)[:, :D]
            s["state"] = normal(c["Bt"], W - 1, D)
            s["state_out"] = torch.zeros_like(s["state"])
            return s
        Bt, L = c["Bt"], c["L"]
        s["x"] = normal(Bt, L, 2 * D)[:, :, :D]
        s["lengths"] = _lengths(c, gen)
        if op == "conv":
            s["state"] = normal(Bt, W - 1, D)
            s["y"] = torch.zeros((Bt, L, D), device="cuda", dtype=t)
        else:
            s["dy"] = normal(Bt, L, D)
        return s
    if op.startswith("scan"):
        N, G, Bt = c["N"], c["G"], c["Bt"]
        step = op == "scan_step"
        lead = (Bt,) if step else (Bt, c["L"])
        s["x"] = normal(*lead, D)
        s["dt"] = normal(*lead, D)
        s["z"] = normal(*lead, 2 * D)[..., D:]
        # B and C are slices of one projection's rows, behind the part that makes dt
        proj = normal(*lead, 64 + 2 * G * N)
        s["B"] = proj[..., 64:64 + G * N].unflatten(-1, (G, N))
        s["C"] = proj[..., 64 + G * N:].unflatten(-1, (G, N))
        s["A"] = -torch.exp(torch.rand((D, N), generator=gen, device="cuda") * math.log(16.0))
        s["D"] = normal(D, dtype=f32, shift=1.0, scale=0.1)
        s["dt_bias"] = normal(D, dtype=f32, shift=-4.0)
        s["h0"] = normal(Bt, D, N, dtype=f32, scale=0.1)
        if step:
            s["h_out"] = torch.zeros_like(s["h0"])
            return s
        s["lengths"] = _lengths(c, gen)
        if op == "scan":
            s["y"] = torch.zeros((*lead, D), device="cuda", dtype=t)
        else:
            s["dy"] = normal(*lead, D)
            s["dh_final"] = normal(Bt, D, N, dtype=f32, scale=0.1)
        return s
    M = c["M"]
    s["w"] = normal(D, dtype=f32, shift=1.0, scale=0.1)
    s["x"] = normal(M, D)
    if op.startswith("gated"):
        s["z"] = normal(M, 2 * D)[:, D:]
    else:
        s["scale"] = normal(D, dtype=f32, shift=0.5, scale=0.1)
        s["residual"] = normal(M, D, dtype=DTYPES[c["res_dtype"]], scale=2.0)
    if op.endswith("backward"):
        s["dy"] = normal(M, D)
        if op.startswith("residual"):
            s["dresidual"] = normal(M, D, dtype=DTYPES[c["res_dtype"]])
    return s


# ---------------------------------------------------------------- plain forms
def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    g = torch.sigmoid(v)
    return g * (1.0 + v * (1.0 - g))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _valid(s, L):
    """[Bt, L, 1] truth values: the token lies within its request."""
    if s["lengths"] is None:
        return None
    return (torch.arange(L, device="cuda")[None, :] < s["lengths"][:, None])[:, :, None]


def _conv_inputs(s):
    """fp32 inputs with the W - 1 tokens before the first in front: [Bt, W - 1 + L, D]."""
    x = s["x"].float()
    Bt, L, D = x.shape
    W = s["w"].shape[1]
    before = s["state"].float() if "state" in s else x.new_zeros((Bt, W - 1, D))
    return torch.cat([before, x], 1)


def _plain_conv(s):
    xs = _conv_inputs(s)
    L, W, t = s["x"].shape[1], s["w"].shape[1], s["x"].dtype
    pre = s["bias"] + sum(xs[:, k:k + L] * s["w"][:, k] for k in range(W))
    y = _silu(pre)
    ok = _valid(s, L)
    n = torch.full((xs.shape[0],), L, device="cuda") if ok is None else s["lengths"].long()
    if ok is not None:
        y = torch.where(ok, y, torch.zeros_like(y))
    at = n[:, None] + torch.arange(W - 1, device="cuda")  # the W - 1 inputs that end with the last token
    state = torch.gather(xs, 1, at[:, :, None].expand(-1, -1, xs.shape[2]))
    return {"y": y.to(t), "state": state.to(t)}


def _plain_conv_backward(s):
    x, w = s["x"].float(), s["w"]
    L, W, t = x.shape[1], w.shape[1], s["x"].dtype
    ok = _valid(s, L)
    if ok is not None:
        x = torch.where(ok, x, torch.zeros_like(x))
    xs = torch.cat([x.new_zeros((x.shape[0], W - 1, x.shape[2])), x], 1)
    pre = s["bias"] + sum(xs[:, k:k + L] * w[:, k] for k in range(W))
    dpre = s["dy"].float() * _dsilu(pre)
    if ok is not None:
        dpre = torch.where(ok, dpre, torch.zeros_like(dpre))
    dxs = torch.zeros_like(xs)
    dw = []
    for k in range(W):
        dxs[:, k:k + L] += dpre * w[:, k]
        dw.append((dpre * xs[:, k:k + L]).double().sum((0, 1)))
    return {"dx": dxs[:, W - 1:].to(t), "dw": torch.stack(dw, 1).float(), "dbias": dpre.double().sum((0, 1)).float()}


def _plain_conv_step(s):
    t, W = s["x"].dtype, s["w"].shape[1]
    xs = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    pre = s["bias"] + sum(xs[:, k] * s["w"][:, k] for k in range(W))
    return {"y": _silu(pre).to(t), "state": xs[:, 1:].to(t)}


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 by doubling, h before the first token 0; both are overwritten."""
    step, L = 1, a.shape[1]
    while step < L:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _scan_inputs(s):
    """fp32 tensors with the channels as [G, D / G]: delta, u = delta x, x, B, C, A, and the valid mask."""
    x, G, N = s["x"].float(), s["B"].shape[-2], s["B"].shape[-1]
    raw = s["dt"].float() + s["dt_bias"]
    delta = _softplus(raw)
    B, C = s["B"].float(), s["C"].float()
    ok = _valid(s, x.shape[1]) if "lengths" in s else None
    if ok is not None:
        zero = torch.zeros((), device="cuda")
        delta, x = torch.where(ok, delta, zero), torch.where(ok, x, zero)
        B, C = torch.where(ok[..., None], B, zero), torch.where(ok[..., None], C, zero)
    return dict(x=x, raw=raw, delta=delta.unflatten(-1, (G, -1)), u=(delta * x).unflatten(-1, (G, -1)), B=B[..., None, :],
                C=C[..., None, :], A=s["A"].view(G, -1, N), ok=ok)


def _states(q, h0):
    """States after every token, [Bt, L, G, D / G, N], and the decays."""
    a = torch.exp(q["delta"][..., None] * q["A"])
    b = q["u"][..., None] * q["B"]
    b[:, 0] += a[:, 0] * h0.view(b[:, 0].shape)
    return _recurrence(a.clone(), b), a


def _plain_scan(s):
    q = _scan_inputs(s)
    t = s["x"].dtype
    h, a = _states(q, s["h0"])
    del a
    o = (h * q["C"]).sum(-1).flatten(-2) + s["D"] * q["x"]
    y = o * _silu(s["z"].float())
    if q["ok"] is not None:
        y = torch.where(q["ok"], y, torch.zeros_like(y))
    return {"y": y.to(t), "h": h[:, -1].reshape(s["h0"].shape).clone()}


def _plain_scan_step(s):
    q = _scan_inputs(s)
    t = s["x"].dtype
    h = torch.exp(q["delta"][..., None] * q["A"]) * s["h0"].view(q["u"].shape + (-1,)) + q["u"][..., None] * q["B"]
    o = (h * q["C"]).sum(-1).flatten(-2) + s["D"] * q["x"]
    return {"y": (o * _silu(s["z"].float())).to(t), "h": h.reshape(s["h0"].shape)}


def _plain_scan_backward(s):
    q = _scan_inputs(s)
    t, z, dy = s["x"].dtype, s["z"].float(), s["dy"].float()
    if q["ok"] is not None:
        zero = torch.zeros((), device="cuda")
        z, dy = torch.where(q["ok"], z, zero), torch.where(q["ok"], dy, zero)
    Bt, L, D = z.shape
    G = q["A"].shape[0]
    h, a = _states(q, s["h0"])
    o = (h * q["C"]).sum(-1).flatten(-2) + s["D"] * q["x"]
    do = dy * _silu(z)
    dz = dy * o * _dsilu(z)
    dog = do.unflatten(-1, (G, -1))[..., None]
    dC = (dog * h).sum(-2)
    # a_t h_{t-1}: the state before each token times its decay
    hb = torch.cat([s["h0"].view(h[:, :1].shape), h[:, :-1]], 1)
    del h
    ah = a * hb
    del hb
    # reverse recurrence g_t = C_t do_t + a_{t+1} g_{t+1}, by flipping the token axis
    g = (dog * q["C"]).flip(1)
    g[:, 0] += s["dh_final"].view(g[:, 0].shape)
    ar = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    g = _recurrence(ar, g).flip(1)
    del ar
    dh0 = (a[:, 0] * g[:, 0]).reshape(s["h0"].shape)
    del a
    dB = (g * q["u"][..., None]).sum(-2)
    gB = (g * q["B"]).sum(-1).flatten(-2)
    ah *= g
    ddelta = q["x"] * gB + (ah * q["A"]).sum(-1).flatten(-2)
    dA = (ah * q["delta"][..., None]).double().sum((0, 1)).float().reshape(D, -1)
    delta = q["delta"].flatten(-2)
    dx = s["D"] * do + delta * gB
    ddt = ddelta * torch.sigmoid(q["raw"])
    if q["ok"] is not None:
        ddt = torch.where(q["ok"], ddt, zero)
    return {"dx": dx.to(t), "ddt": ddt.to(t), "dA": dA, "dB": dB.to(t), "dC": dC.to(t),
            "dD": (do * q["x"]).double().sum((0, 1)).float(), "dz": dz.to(t), "ddt_bias": ddt.double().sum((0, 1)).float(), "dh0": dh0}


def _plain_gated_norm(s):
    c, x, z = s["case"], s["x"].float(), s["z"].float()
    v = x * _silu(z) if c["gate_first"] else x
    vg = v.view(c["M"], c["G"], -1)
    n = (vg * torch.rsqrt(vg.square().mean(-1, keepdim=True) + EPS)).view(v.shape) * s["w"]
    return (n if c["gate_first"] else n * _silu(z)).to(s["x"].dtype)


def _plain_gated_norm_backward(s):
    c, x, z, dy, t = s["case"], s["x"].float(), s["z"].float(), s["dy"].float(), s["x"].dtype
    first, shape = c["gate_first"], (c["M"], c["G"], -1)
    gate = _silu(z)
    v = (x * gate if first else x).view(shape)
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    n = (v * r).view(x.shape)
    dn = dy if first else dy * gate
    dw = (dn * n).double().sum(0).float()
    dn = (dn * s["w"]).view(shape)
    dv = (r * (dn - n.view(shape) * (dn * n.view(shape)).mean(-1, keepdim=True))).view(x.shape)
    dx, dz = (dv * gate, dv * x * _dsilu(z)) if first else (dv, dy * n * s["w"] * _dsilu(z))
    return {"dx": dx.to(t), "dz": dz.to(t), "dw": dw}


def _plain_residual_norm(s):
    h = s["residual"].float() + s["scale"] * s["x"].float()
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"]
    return {"y": n.to(s["x"].dtype), "residual": h.to(s["residual"].dtype)}


def _plain_residual_norm_backward(s):
    h, x, dy = s["residual"].float(), s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * r
    dn = dy * s["w"]
    dh = s["dresidual"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": (s["scale"] * dh).to(s["x"].dtype), "dresidual": dh.to(s["residual"].dtype),
            "dw": (dy * n).double().sum(0).float(), "dscale": (dh * x).double().sum(0).float()}


PLAIN = {"conv": _plain_conv, "conv_backward": _plain_conv_backward, "conv_step": _plain_conv_step, "scan": _plain_scan,
         "scan_step": _plain_scan_step, "scan_backward": _plain_scan_backward, "gated_norm": _plain_gated_norm,
         "gated_norm_backward": _plain_gated_norm_backward, "residual_norm": _plain_residual_norm,
         "residual_norm_backward": _plain_residual_norm_backward}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from state_space_sequence_ssm_amd import ops

    c, op = s["case"], s["case"]["op"]
    if op == "conv":
        return ops.m3_causal_conv(s["x"], s["w"], s["bias"], s["state"], lengths=s["lengths"], silu=True, y=s["y"], want_state=True)
    if op == "conv_backward":
        r = ops.m3_causal_conv_backward(s["x"], s["w"], s["bias"], dy=s["dy"], lengths=s["lengths"], silu=True)
        return {k: r[k] for k in ("dx", "dw", "dbias")}
    if op == "conv_step":
        y = ops.m3_causal_conv_step(s["state"], s["x"], s["w"], s["bias"], silu=True, state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if op == "scan":
        return ops.m3_selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["h0"], lengths=s["lengths"],
                                     dt_softplus=True, dt_bias=s["dt_bias"], y=s["y"])
    if op == "scan_backward":
        return ops.m3_selective_scan_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["h0"], dy=s["dy"],
                                              dh_final=s["dh_final"], lengths=s["lengths"], dt_softplus=True,
                                              dt_bias=s["dt_bias"], want_carry_grads=True)
    if op == "scan_step":
        y = ops.m3_selective_scan_step(s["h0"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], dt_softplus=True,
                                       dt_bias=s["dt_bias"], h_out=s["h_out"])
        return {"y": y, "h": s["h_out"]}
    if op == "gated_norm":
        return ops.m3_gated_norm(s["x"], s["z"], s["w"], groups=c["G"], eps=EPS, gate_first=c["gate_first"])
    if op == "gated_norm_backward":
        return ops.m3_gated_norm_backward(s["x"], s["z"], s["w"], dy=s["dy"], groups=c["G"], eps=EPS, gate_first=c["gate_first"])
    if op == "residual_norm":
        return ops.m3_residual_norm(s["x"], s["residual"], s["w"], s["scale"], eps=EPS)
    return ops.m3_residual_norm_backward(s["residual"], s["x"], s["w"], s["scale"], dy=s["dy"], dresidual=s["dresidual"], eps=EPS)


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- cost
def work(case):
    """Bytes of every input read once and every output written once, and the
    operations of the definition (a multiply-add counts two, exp and the like one)."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op, D = c["op"], c["D"]
    if op.startswith("conv"):
        W = c["W"]
        rows = c["Bt"] * c.get("L", 1)
        edge = c["Bt"] * (W - 1) * D * e
        par = D * (W + 1) * 4
        if op == "conv_backward":
            return {"bytes": 3 * rows * D * e + 2 * par, "flops": rows * D * (6 * W + 12)}
        return {"bytes": 2 * rows * D * e + 2 * edge + par, "flops": rows * D * (2 * W + 4)}
    if op.startswith("scan"):
        N, G = c["N"], c["G"]
        rows = c["Bt"] * c.get("L", 1)
        state = c["Bt"] * D * N * 4
        par = D * (N + 2) * 4
        if op == "scan_backward":
            return {"bytes": (4 + 3) * rows * D * e + 4 * rows * G * N * e + 3 * state + 2 * par, "flops": rows * D * (21 * N + 30)}
        return {"bytes": 4 * rows * D * e + 2 * rows * G * N * e + 2 * state + par, "flops": rows * D * (7 * N + 12)}
    n = c["M"] * D
    if op == "gated_norm":
        return {"bytes": 3 * n * e + 4 * D, "flops": n * 9}
    if op == "gated_norm_backward":
        return {"bytes": 5 * n * e + 8 * D, "flops": n * 22}
    q = 2 if c["res_dtype"] == "bf16" else 4
    if op == "residual_norm":
        return {"bytes": n * (2 * e + 2 * q) + 8 * D, "flops": n * 6}
    return {"bytes": n * (3 * e + 3 * q) + 16 * D, "flops": n * 15}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}

    def sig(v):
        return 1 / (1 + torch.exp(-v))

    if op == "conv_step":
        pre = d["bias"] + d["x"] * d["w"][:, -1] + (d["state"] * d["w"][:, :-1].T).sum(1)
        return {"y": pre * sig(pre), "state": torch.cat([d["state"][:, 1:], d["x"][:, None]], 1)}
    if op == "conv":
        W, L = c["W"], c["L"]
        hist = [d["state"][:, k] for k in range(W - 1)]
        y = torch.zeros_like(d["y"])
        n = s["lengths"] if s["lengths"] is not None else torch.full((c["Bt"],), L, device="cuda")
        for t in range(L):
            on = (n > t)[:, None]
            taps = hist + [d["x"][:, t]]
            pre = d["bias"].clone()
            for k in range(W):
                pre = pre + d["w"][:, k] * taps[k]
            y[:, t] = torch.where(on, pre * sig(pre), torch.zeros_like(pre))
            hist = [torch.where(on, new, old) for new, old in zip(taps[1:], hist)]
        return {"y": y, "state": torch.stack(hist, 1)}
    if op == "conv_backward":
        W, L = c["W"], c["L"]
        dx, dw, dbias = torch.zeros_like(d["dy"]), torch.zeros_like(d["w"]), torch.zeros_like(d["bias"])
        for b in range(c["Bt"]):
            n = L if s["lengths"] is None else int(s["lengths"][b])
            x, dy = d["x"][b, :n], d["dy"][b, :n]
            pre = d["bias"].expand(n, -1).clone()
            for lag in range(min(W, n)):
                pre[lag:] += d["w"][:, W - 1 - lag] * x[:n - lag]
            dpre = dy * (sig(pre) + pre * sig(pre) * (1 - sig(pre)))
            dbias += dpre.sum(0)
            for lag in range(min(W, n)):
                dx[b, :n - lag] += d["w"][:, W - 1 - lag] * dpre[lag:]
                dw[:, W - 1 - lag] += (dpre[lag:] * x[:n - lag]).sum(0)
        return {"dx": dx, "dw": dw, "dbias": dbias}
    if op.startswith("scan"):
        return _exact_scan(s, d, sig)
    if op.startswith("gated"):
        G, M = c["G"], c["M"]
        gate = d["z"] * sig(d["z"])
        v = d["x"] * gate if c["gate_first"] else d["x"]
        var = (v.view(M, G, -1) ** 2).mean(-1, keepdim=True) + EPS
        inv = (var ** -0.5).expand(M, G, v.shape[1] // G).reshape(v.shape)
        if op == "gated_norm":
            out = v * inv * d["w"]
            return out if c["gate_first"] else out * gate
        up = d["dy"] if c["gate_first"] else d["dy"] * gate
        e = up * d["w"]
        mean = (e * v).view(M, G, -1).mean(-1, keepdim=True).expand(M, G, v.shape[1] // G).reshape(v.shape)
        dv = inv * e - v * mean * inv ** 3
        dgate = sig(d["z"]) * (1 + d["z"] * (1 - sig(d["z"])))
        if c["gate_first"]:
            return {"dx": dv * gate, "dz": dv * d["x"] * dgate, "dw": (up * v * inv).sum(0)}
        return {"dx": dv, "dz": d["dy"] * v * inv * d["w"] * dgate, "dw": (up * v * inv).sum(0)}
    if op == "residual_norm":
        h = d["residual"] + d["scale"] * d["x"]
        return {"y": h / ((h ** 2).mean(-1, keepdim=True) + EPS) ** 0.5 * d["w"], "residual": h}
    h = d["residual"]
    inv = ((h ** 2).mean(-1, keepdim=True) + EPS) ** -0.5
    e = d["dy"] * d["w"]
    dh = d["dresidual"] + inv * e - h * inv ** 3 * (e * h).mean(-1, keepdim=True)
    return {"dx": d["scale"] * dh, "dresidual": dh, "dw": (d["dy"] * h * inv).sum(0), "dscale": (dh * d["x"]).sum(0)}


def _exact_scan(s, d, sig):
    """The recurrence and its reverse, token by token in 64 bits."""
    c, op = s["case"], s["case"]["op"]
    Bt, D, N, G = c["Bt"], c["D"], c["N"], c["G"]
    L = c.get("L", 1)
    if op == "scan_step":
        for k in ("x", "dt", "z", "B", "C"):
            d[k] = d[k][:, None]
    n = s.get("lengths")
    n = torch.full((Bt,), L, device="cuda") if n is None else n
    per = D // G

    def wide(v):  # [Bt, G, N] -> [Bt, D, N]: each group's row for its channels
        return v[:, :, None, :].expand(Bt, G, per, N).reshape(Bt, D, N)

    def delta(t):
        return torch.nn.functional.softplus(d["dt"][:, t] + d["dt_bias"], threshold=100.0)

    h, y, kept = d["h0"], torch.zeros((Bt, L, D), dtype=torch.float64, device="cuda"), []
    back = op == "scan_backward"
    for t in range(L):
        on = (n > t)[:, None, None]
        dl = delta(t)
        new = torch.exp(dl[..., None] * d["A"]) * h + (dl * d["x"][:, t])[..., None] * wide(d["B"][:, t])
        if back:
            kept.append(h)
        h = torch.where(on, new, h)
        o = (h * wide(d["C"][:, t])).sum(-1) + d["D"] * d["x"][:, t]
        if back:
            y[:, t] = o
        else:
            y[:, t] = torch.where(on[..., 0], o * d["z"][:, t] * sig(d["z"][:, t]), torch.zeros_like(o))
    if op == "scan_step":
        return {"y": y[:, 0], "h": h}
    if op == "scan":
        return {"y": y, "h": h}
    g = d["dh_final"].clone()  # gradient of the state after token t
    out = {k: torch.zeros((Bt, L, D), dtype=torch.float64, device="cuda") for k in ("dx", "ddt", "dz")}
    out["dB"], out["dC"] = (torch.zeros((Bt, L, G, N), dtype=torch.float64, device="cuda") for _ in range(2))
    out["dA"] = torch.zeros_like(d["A"])
    out["dD"], out["ddt_bias"] = torch.zeros_like(d["D"]), torch.zeros_like(d["D"])
    for t in reversed(range(L)):
        on = (n > t)[:, None]
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        x, z, dy, dl = d["x"][:, t], d["z"][:, t], torch.where(on, d["dy"][:, t], zero), delta(t)
        B, C, hp = wide(d["B"][:, t]), wide(d["C"][:, t]), kept.pop()
        a = torch.exp(dl[..., None] * d["A"])
        hn = a * hp + (dl * x)[..., None] * B
        do = dy * z * sig(z)
        out["dz"][:, t] = dy * y[:, t] * (sig(z) + z * sig(z) * (1 - sig(z)))
        gt = torch.where(on[..., None], g + do[..., None] * C, zero)
        out["dC"][:, t] = (do[..., None] * hn).view(Bt, G, per, N).sum(2)
        out["dB"][:, t] = (gt * (dl * x)[..., None]).view(Bt, G, per, N).sum(2)
        gB = (gt * B).sum(-1)
        out["dx"][:, t] = d["D"] * do + dl * gB
        da = gt * hp * a
        draw_ = (x * gB + (da * d["A"]).sum(-1)) * sig(d["dt"][:, t] + d["dt_bias"])
        out["ddt"][:, t] = draw_
        out["ddt_bias"] += draw_.sum(0)
        out["dA"] += (da * dl[..., None]).sum(0)
        out["dD"] += (do * x).sum(0)
        g = torch.where(on[..., None], gt * a, g)
    out["dh0"] = g
    return out
