"""Timing and accuracy cases of linear attention with a decay per head and of the norm and
rotation of its queries and keys: each for prompts, for training (backward) and for single
tokens.

`run` computes a case either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with `own` set, through the library's entry points; `exact`
computes it from the definitions in 64 bits, token by token.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a batch of whole prompts, the states kept for decoding
        dict(name="attention_prompt", op="attention", Bt=8, L=4096, H=16, Hk=16, K=128, V=128, dtype="bf16", ragged=False),
        # one long document: 16 heads over 4 shared ones, a long token axis
        dict(name="attention_long", op="attention", Bt=1, L=16384, H=16, Hk=4, K=128, V=128, dtype="bf16", ragged=False),
        # a padded batch of uneven requests (one empty, one of a single token), odd sizes, full precision
        dict(name="attention_ragged", op="attention", Bt=5, L=1537, H=6, Hk=3, K=80, V=100, dtype="fp32", ragged=True),
        # the gradients in a training step
        dict(name="attention_training", op="attention_backward", Bt=8, L=2048, H=16, Hk=16, K=128, V=128, dtype="bf16",
             ragged=False),
        # the same over a padded batch with shared heads, full precision
        dict(name="attention_training_ragged", op="attention_backward", Bt=3, L=1000, H=8, Hk=2, K=64, V=64, dtype="fp32",
             ragged=True),
        # one token for each of 256 sequences against the resident states
        dict(name="attention_token", op="attention_step", Bt=256, H=16, Hk=16, K=128, V=128, dtype="bf16"),
        # one token of one sequence: nothing but latency
        dict(name="attention_one", op="attention_step", Bt=1, H=16, Hk=4, K=64, V=64, dtype="bf16"),
        # norm and rotation of whole prompts' queries and keys, slices of one projection's rows
        dict(name="rotation_prompt", op="rotation", Bt=8, L=4096, H=16, Hk=16, D=128, R=128, adjacent=False, dtype="bf16",
             ragged=False, far=False),
        # a padded batch, odd sizes, a part of each head rotated in adjacent pairs, full precision
        dict(name="rotation_ragged", op="rotation", Bt=5, L=1537, H=6, Hk=3, D=80, R=40, adjacent=True, dtype="fp32",
             ragged=True, far=False),
        # the gradients in a training step, with shared key heads
        dict(name="rotation_training", op="rotation_backward", Bt=8, L=4096, H=16, Hk=4, D=128, R=128, adjacent=False,
             dtype="bf16", ragged=False, far=False),
        # its smallest training step: one short sequence
        dict(name="rotation_training_short", op="rotation_backward", Bt=1, L=128, H=8, Hk=8, D=64, R=64, adjacent=False,
             dtype="fp32", ragged=False, far=False),
        # one token for each of 256 sequences, far positions
        dict(name="rotation_tokens", op="rotation", Bt=256, L=1, H=16, Hk=4, D=128, R=64, adjacent=False, dtype="bf16",
             ragged=False, far=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_backward", "attention_backward", "attention_step", "rotation",
                     "rotation_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    Hk = _log(rng, 1, 32)
    H = Hk * rng.choice([1, 1, 2, 4])
    if op.startswith("attention"):
        K, V = (rng.choice([32, 64, 64, 128, 128, 256, rng.randint(8, 200)]) for _ in range(2))
        if op == "attention_step":
            return dict(op=op, Bt=_log(rng, 1, max(1, min(512, (1 << 26) // (H * K * V)))), H=H, Hk=Hk, K=K, V=V, dtype=dtype)
        most, values = (1 << 32, 1 << 25) if op == "attention" else (1 << 31, 3 << 22)
        L = max(1, min(_log(rng, 1, 16384), most // (H * K * V), values // (H * max(K, V))))
        Bt = _log(rng, 1, max(1, min(32, most // (L * H * K * V), values // (L * H * max(K, V)), values // (H * K * V))))
        return dict(op=op, Bt=Bt, L=L, H=H, Hk=Hk, K=K, V=V, dtype=dtype, ragged=rng.random() < 0.3)
    D = rng.choice([64, 64, 128, 128, 256, 2 * rng.randint(8, 100)])
    R = rng.choice([D, D, D // 4 * 2])
    L = max(1, min(_log(rng, 1, 8192), (1 << 24) // (H * D)))
    Bt = _log(rng, 1, max(1, min(256, (1 << 24) // (L * H * D))))
    return dict(op=op, Bt=Bt, L=L, H=H, Hk=Hk, D=D, R=R, adjacent=rng.random() < 0.4, dtype=dtype, ragged=rng.random() < 0.3,
                far=rng.random() < 0.3)


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
    t, f32 = DTYPES[c["dtype"]], torch.float32

    def normal(*shape, dtype=t, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    op, H, Hk = c["op"], c["H"], c["Hk"]
    s = {"case": c}
    if op.startswith("attention"):
        Bt, K, V = c["Bt"], c["K"], c["V"]
        step = op == "attention_step"
        lead = (Bt,) if step else (Bt, c["L"])
        # a head's memory spans 32 tokens in the first and 4096 in the last
        reach = torch.linspace(5.0, 12.0, H, device="cuda")
        s["log_decay"] = torch.log1p(-torch.exp2(-reach))
        s["q"], s["k"] = normal(*lead, H, K), normal(*lead, Hk, K)
        # the values are a slice of the projection's rows, behind as many other columns
        s["v"] = normal(*lead, 2 * Hk * V)[..., Hk * V:].unflatten(-1, (Hk, V))
        s["h0"] = normal(Bt, H, K, V, dtype=f32)
        if step:
            s["h_out"] = torch.zeros_like(s["h0"])
            return s
        s["lengths"] = _lengths(c, gen)
        if op == "attention":
            s["y"] = torch.zeros((*lead, H, V), device="cuda", dtype=t)
        else:
            s["dy"] = normal(*lead, H, V)
            s["dh_final"] = normal(Bt, H, K, V, dtype=f32)
        return s
    Bt, L, D, R = c["Bt"], c["L"], c["D"], c["R"]
    proj = normal(Bt, L, (H + 2 * Hk) * D)
    s["q"] = proj[..., :H * D].unflatten(-1, (H, D))
    s["k"] = proj[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D))
    s["q_w"], s["k_w"] = (normal(D, dtype=f32, shift=1.0, scale=0.1) for _ in range(2))
    s["freqs"] = torch.exp(torch.arange(R // 2, device="cuda", dtype=f32) * (-math.log(10000.0) / max(1, R // 2)))
    s["positions"] = None
    if c["far"]:  # sequences that go on behind up to a million tokens
        start = torch.randint(0, 1 << 20, (Bt, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["positions"] = start + torch.arange(L, device="cuda", dtype=torch.int32)
    s["lengths"] = _lengths(c, gen)
    if op == "rotation":
        s["q_out"], s["k_out"] = torch.zeros((Bt, L, H, D), device="cuda", dtype=t), torch.zeros((Bt, L, Hk, D), device="cuda", dtype=t)
    else:
        s["dq"], s["dk"] = normal(Bt, L, H, D), normal(Bt, L, Hk, D)
    return s


# ---------------------------------------------------------------- plain forms
def _valid(s, L):
    """[Bt, L, 1, 1] truth values: the token lies within its request."""
    if s["lengths"] is None:
        return None
    return (torch.arange(L, device="cuda")[None, :] < s["lengths"][:, None])[:, :, None, None]


def _heads_first(s, name, H, ok):
    """[Bt, H, L, .] in fp32, shared heads repeated, zeros behind the lengths."""
    x = s[name].float()
    if ok is not None:
        x = torch.where(ok, x, torch.zeros((), device="cuda"))
    return x.repeat_interleave(H // x.shape[2], 2).transpose(1, 2).contiguous()


def _recurrence(a, b):
    """h_c = a_c h_{c-1} + b_c along axis 2 by doubling, h before the first 0; both are overwritten."""
    step, n = 1, b.shape[2]
    while step < n:
        b[:, :, step:] += a[:, :, step:] * b[:, :, :-step]
        a[:, :, step:] = a[:, :, step:] * a[:, :, :-step]
        step *= 2
    return b


def _decayed(g, steps):
    """exp(g steps) with the heads in front: [H, *steps]."""
    return torch.exp(g.view(-1, *[1] * steps.dim()) * steps)


def _attend(a, b, c, g):
    """sum_{j <= t} exp(g (t - j)) (a_t . b_j) c_j over [Bt, H, L, .], by chunks."""
    Bt, H, L, _ = a.shape
    C = min(64, L)
    pad = -L % C
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, pad)).unflatten(2, (-1, C)) for x in (a, b, c))
    i = torch.arange(C, device="cuda", dtype=torch.float32)
    apart = i[:, None] - i
    w = torch.where(apart >= 0, _decayed(g, apart.clamp(min=0)), torch.zeros((), device="cuda"))
    out = torch.matmul(torch.matmul(a, b.transpose(-1, -2).contiguous()) * w[:, None], c)
    ends = torch.matmul((b * _decayed(g, C - 1 - i)[:, None, :, None]).transpose(-1, -2).contiguous(), c)
    if ends.shape[2] > 1:
        whole = _decayed(g, torch.full((ends.shape[2],), float(C), device="cuda"))[None, :, :, None, None].expand(Bt, -1, -1, 1, 1)
        states = _recurrence(whole.clone(), ends)
        out[:, :, 1:] += _decayed(g, i + 1)[:, None, :, None] * torch.matmul(a[:, :, 1:], states[:, :, :-1])
    return out.flatten(2, 3)[:, :, :L]


def _tokens_first(y, ok, t):
    y = y.transpose(1, 2)
    return (y if ok is None else torch.where(ok, y, torch.zeros((), device="cuda"))).to(t).contiguous()


def _ends(s, L):
    """Each item's length, and every token's distance from its item's last one: [Bt], [Bt, L]."""
    Bt = s["q"].shape[0]
    n = torch.full((Bt,), float(L), device="cuda") if s["lengths"] is None else s["lengths"].float()
    return n, (n[:, None] - 1 - torch.arange(L, device="cuda")).clamp(min=0)


def _plain_attention(s):
    g, H, L, t = s["log_decay"], s["case"]["H"], s["q"].shape[1], s["q"].dtype
    ok = _valid(s, L)
    q, k, v = (_heads_first(s, x, H, ok) for x in "qkv")
    scale = q.shape[-1] ** -0.5
    n, left = _ends(s, L)
    i = torch.arange(L, device="cuda", dtype=torch.float32)
    y = _attend(q, k, v, g) + _decayed(g, i + 1)[..., None] * torch.matmul(q, s["h0"])
    kw = k * _decayed(g, left).transpose(0, 1)[..., None]
    h = _decayed(g, n).T[..., None, None] * s["h0"] + torch.matmul(kw.transpose(-1, -2).contiguous(), v)
    return {"y": _tokens_first(scale * y, ok, t), "h": h}


def _plain_attention_backward(s):
    g, H, Hk, L, t = s["log_decay"], s["case"]["H"], s["case"]["Hk"], s["q"].shape[1], s["q"].dtype
    ok = _valid(s, L)
    q, k, v, dy = (_heads_first(s, x, H, ok) for x in ("q", "k", "v", "dy"))
    scale = q.shape[-1] ** -0.5
    dh = s["dh_final"]
    n, left = _ends(s, L)
    i = torch.arange(L, device="cuda", dtype=torch.float32)
    ahead = _decayed(g, i + 1)[..., None]
    behind = _decayed(g, left).transpose(0, 1)[..., None]
    dq = _attend(dy, v, k, g) + ahead * torch.matmul(dy, s["h0"].transpose(-1, -2).contiguous())
    qr, kr, vr, dyr = (x.flip(2) for x in (q, k, v, dy))
    dk = scale * _attend(vr, dyr, qr, g).flip(2) + behind * torch.matmul(v, dh.transpose(-1, -2).contiguous())
    dv = scale * _attend(kr, qr, dyr, g).flip(2) + behind * torch.matmul(k, dh)
    dh0 = _decayed(g, n).T[..., None, None] * dh + scale * torch.matmul((q * ahead).transpose(-1, -2).contiguous(), dy)
    dk, dv = (x.unflatten(1, (Hk, H // Hk)).sum(2) for x in (dk, dv))
    return {"dq": _tokens_first(scale * dq, ok, t), "dk": _tokens_first(dk, ok, t), "dv": _tokens_first(dv, ok, t), "dh0": dh0}


def _plain_attention_step(s):
    H, t = s["case"]["H"], s["q"].dtype
    q, k, v = (s[x].float().repeat_interleave(H // s[x].shape[1], 1) for x in "qkv")
    h = torch.exp(s["log_decay"])[:, None, None] * s["h0"] + k[..., None] * v[..., None, :]
    return {"y": (q.shape[-1] ** -0.5 * (q[..., None] * h).sum(-2)).to(t), "h": h}


def _angles(s):
    """cos and sin of position times rate, [Bt, L, 1, R / 2]; the angles in 64 bits."""
    Bt, L = s["q"].shape[:2]
    at = s["positions"] if s["positions"] is not None else torch.arange(L, device="cuda").expand(Bt, L)
    angle = at.double()[:, :, None, None] * s["freqs"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, R, adjacent):
    """The first R elements of each head rotated in pairs."""
    if adjacent:
        x0, x1 = x[..., 0:R:2], x[..., 1:R:2]
        both = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    else:
        x0, x1 = x[..., :R // 2], x[..., R // 2:R]
        both = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    return torch.cat([both, x[..., R:]], -1)


def _plain_rotation(s):
    c, t = s["case"], s["q"].dtype
    ok = _valid(s, c["L"])
    cos, sin = _angles(s)
    out = {}
    for name in "qk":
        x = s[name].float()
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[name + "_w"]
        y = _turn(n, cos, sin, c["R"], c["adjacent"])
        out[name] = (y if ok is None else torch.where(ok, y, torch.zeros((), device="cuda"))).to(t)
    return out


def _plain_rotation_backward(s):
    c, t = s["case"], s["q"].dtype
    ok = _valid(s, c["L"])
    cos, sin = _angles(s)
    out = {}
    for name in "qk":
        x, dy, w = s[name].float(), s["d" + name].float(), s[name + "_w"]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dn = _turn(dy, cos, -sin, c["R"], c["adjacent"])
        if ok is not None:
            dn = torch.where(ok, dn, torch.zeros((), device="cuda"))
        out["d" + name + "_w"] = (dn * n).double().sum((0, 1, 2)).float()
        dn = dn * w
        out["d" + name] = (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(t)
    return out


PLAIN = {"attention": _plain_attention, "attention_backward": _plain_attention_backward, "attention_step": _plain_attention_step,
         "rotation": _plain_rotation, "rotation_backward": _plain_rotation_backward}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from state_space_sequence_ssm_amd import ops

    c, op = s["case"], s["case"]["op"]
    if op == "attention":
        return ops.m3_linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["h0"], lengths=s["lengths"], y=s["y"])
    if op == "attention_backward":
        return ops.m3_linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["h0"], dy=s["dy"], dh_final=s["dh_final"],
                                                lengths=s["lengths"], want_carry_grads=True)
    if op == "attention_step":
        y = ops.m3_linear_attention_step(s["h0"], s["q"], s["k"], s["v"], s["log_decay"], h_out=s["h_out"])
        return {"y": y, "h": s["h_out"]}
    how = dict(freqs=s["freqs"], positions=s["positions"], lengths=s["lengths"], eps=EPS, adjacent=c["adjacent"])
    if op == "rotation":
        return ops.m3_qk_norm_rope(s["q"], s["k"], s["q_w"], s["k_w"], q_out=s["q_out"], k_out=s["k_out"], **how)
    return ops.m3_qk_norm_rope_backward(s["q"], s["k"], s["q_w"], s["k_w"], dq_out=s["dq"], dk_out=s["dk"], **how)


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- cost
def work(case):
    """Bytes of every input read once and every output written once, and the operations of
    the recurrence token by token (a multiply-add counts two)."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    rows = c["Bt"] * c.get("L", 1)
    H, Hk = c["H"], c["Hk"]
    if c["op"].startswith("attention"):
        K, V = c["K"], c["V"]
        state = c["Bt"] * H * K * V * 4
        once = rows * (H * K + Hk * (K + V)) * e
        if c["op"] == "attention_backward":
            return {"bytes": 2 * once + rows * H * V * e + 3 * state + 4 * H, "flops": rows * H * (13 * K * V)}
        return {"bytes": once + rows * H * V * e + 2 * state + 4 * H, "flops": rows * H * 5 * K * V}
    D, R = c["D"], c["R"]
    n = rows * (H + Hk) * D
    extra = 2 * D * 4 + R * 2 + (rows * 4 if c["far"] else 0)
    if c["op"] == "rotation":
        return {"bytes": 2 * n * e + extra, "flops": n * 8}
    return {"bytes": 3 * n * e + extra + 2 * D * 4, "flops": n * 16}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op.startswith("attention"):
        return _exact_attention(c, s, d)
    pos = s["positions"] if s["positions"] is not None else torch.arange(c["L"], device="cuda").repeat(c["Bt"], 1)
    R, half = c["R"], c["R"] // 2
    lo = torch.arange(half, device="cuda") * (2 if c["adjacent"] else 1)
    hi = lo + (1 if c["adjacent"] else half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[..., None, None] * d["freqs"])
    held = torch.ones_like(pos, dtype=torch.bool)
    if s["lengths"] is not None:
        held = torch.arange(c["L"], device="cuda") < s["lengths"][:, None].long()
    held = held[..., None, None].double()
    out = {}
    for name in "qk":
        x, w = d[name], d[name + "_w"]
        inv = 1 / ((x * x).sum(-1, keepdim=True) / c["D"] + EPS) ** 0.5
        if op == "rotation":
            y = x * inv * w
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
            out[name] = y * held
            continue
        e = d["d" + name] * held
        z = torch.complex(e[..., lo], e[..., hi]) * turn.conj()
        e[..., lo], e[..., hi] = z.real, z.imag
        out["d" + name + "_w"] = (e * x * inv).sum((0, 1, 2))
        e = e * w
        out["d" + name] = inv * e - x * inv ** 3 * (e * x).sum(-1, keepdim=True) / c["D"]
    return out


def _exact_attention(c, s, d):
    """The recurrence and, for the gradients, its reverse, token by token in 64 bits."""
    Bt, H, Hk, K, V = c["Bt"], c["H"], c["Hk"], c["K"], c["V"]
    per, scale, L = H // Hk, 1 / math.sqrt(c["K"]), c.get("L", 1)
    if c["op"] == "attention_step":
        for x in "qkv":
            d[x] = d[x][:, None]
    n = s.get("lengths")
    n = torch.full((Bt,), L, device="cuda") if n is None else n
    lam = torch.exp(d["log_decay"])[None, :, None, None]
    back = c["op"] == "attention_backward"

    def head(name, t):
        """[Bt, H, .]: row h of a shared input is that of its group."""
        x = d[name][:, t]
        return x[:, torch.arange(H, device="cuda") // (H // x.shape[1])]

    h = d["h0"].clone()
    y = torch.zeros((Bt, L, H, K if back else V), dtype=torch.float64, device="cuda")
    for t in range(L):
        on = (n > t)[:, None, None]
        new = lam * h + head("k", t)[..., :, None] * head("v", t)[..., None, :]
        h = torch.where(on[..., None], new, h)
        if back:  # the gradient of q is the state times dy
            o = scale * (h * head("dy", t)[..., None, :]).sum(-1)
        else:
            o = scale * (h * head("q", t)[..., :, None]).sum(-2)
        y[:, t] = torch.where(on, o, torch.zeros_like(o))
    if c["op"] == "attention_step":
        return {"y": y[:, 0], "h": h}
    if not back:
        return {"y": y, "h": h}
    g = d["dh_final"].clone()  # gradient of the state after token t
    dk = torch.zeros((Bt, L, Hk, K), dtype=torch.float64, device="cuda")
    dv = torch.zeros((Bt, L, Hk, V), dtype=torch.float64, device="cuda")
    for t in reversed(range(L)):
        on = (n > t)[:, None, None]
        gt = g + scale * head("q", t)[..., :, None] * head("dy", t)[..., None, :]
        gk = (gt * head("v", t)[..., None, :]).sum(-1).view(Bt, Hk, per, K).sum(2)
        gv = (gt * head("k", t)[..., :, None]).sum(-2).view(Bt, Hk, per, V).sum(2)
        dk[:, t] = torch.where(on, gk, torch.zeros_like(gk))
        dv[:, t] = torch.where(on, gv, torch.zeros_like(gv))
        g = torch.where(on[..., None], lam * gt, g)
    return {"dq": y, "dk": dk, "dv": dv, "dh0": g}
