"""Layer operators together and in use: a whole mixer block over a prompt, token
by token and in a training step; graphs captured and replayed; other streams;
repeated calls; tensors past 32-bit offsets; values that must stay where they are."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref as ref  # noqa: E402
from tests.test_gpu_layers import BF, F32, NAN, Maker, ilen, wide  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


def rel(got, want):
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    return float((got - want).norm() / want.norm())


# ---------------------------------------------------------------- a mixer block
E, D, N, G, R, W = 24, 48, 16, 2, 4, 4  # model width, channels, states, groups, rank of dt, taps


def _params(m):
    return dict(w_in=m(E, 2 * D, scale=E ** -0.5), w_x=m(D, R + 2 * G * N, scale=D ** -0.5), w_dt=m(R, D, scale=R ** -0.5),
                w_out=m(D, E, scale=D ** -0.5), conv_w=m(D, W, scale=0.5), conv_b=m(D, scale=0.1),
                A=-torch.exp(torch.rand(D, N, generator=m.g) * 2.0).cuda(), skip=m(D), dt_bias=m(D, shift=-2.0),
                norm_w=m(E, shift=1.0, scale=0.1), scale=m(E, shift=1.0, scale=0.1), gate_w=m(D, shift=1.0, scale=0.1))


def _reference(p, x, res, lengths=None):
    """The block in the inputs' own precision, by torch operations that
    differentiate: the residual stream and the block's output."""
    h = res + p["scale"] * x
    u = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * p["norm_w"]
    xz = u @ p["w_in"]
    xc, z = xz[..., :D], xz[..., D:]
    pad = torch.cat([xc.new_zeros(xc.shape[0], W - 1, D), xc], 1)
    L = xc.shape[1]
    xc = torch.nn.functional.silu(p["conv_b"] + sum(p["conv_w"][:, k] * pad[:, k:k + L] for k in range(W)))
    proj = xc @ p["w_x"]
    dt = torch.nn.functional.softplus(proj[..., :R] @ p["w_dt"] + p["dt_bias"])
    B, C = (proj[..., R + i * G * N:R + (i + 1) * G * N].unflatten(-1, (G, N)).repeat_interleave(D // G, 2) for i in (0, 1))
    state, ys = xc.new_zeros(xc.shape[0], D, N), []
    for t in range(L):
        state = torch.exp(dt[:, t, :, None] * p["A"]) * state + (dt[:, t] * xc[:, t])[..., None] * B[:, t]
        ys.append((state * C[:, t]).sum(-1) + p["skip"] * xc[:, t])
    v = torch.stack(ys, 1) * torch.nn.functional.silu(z)
    vg = v.unflatten(-1, (G, -1))
    y = (vg * (vg.square().mean(-1, keepdim=True) + 1e-5).rsqrt()).flatten(-2) * p["gate_w"]
    return h, y @ p["w_out"], state


def _prompt(ops, p, x, res, lengths=None, keep=None):
    r = ops.m3_residual_norm(x, res, p["norm_w"], p["scale"], eps=1e-5)
    xz = r["y"] @ p["w_in"]
    c = ops.m3_causal_conv(xz[..., :D], p["conv_w"], p["conv_b"], lengths=lengths, want_state=True,
                           y=torch.zeros_like(xz[..., :D].contiguous()))
    proj = c["y"] @ p["w_x"]
    dt = proj[..., :R] @ p["w_dt"]
    B, C = (proj[..., R + i * G * N:R + (i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
    s = ops.m3_selective_scan(c["y"], dt, p["A"], B, C, p["skip"], None, lengths=lengths, dt_softplus=True, dt_bias=p["dt_bias"],
                              y=torch.zeros_like(c["y"]))
    y = ops.m3_gated_norm(s["y"], xz[..., D:], p["gate_w"], groups=G, eps=1e-5)
    if keep is not None:
        keep.update(u=r["y"], xz=xz, xc=c["y"], proj=proj, dt=dt, B=B, C=C, s=s["y"], y=y)
    return r["residual"], y @ p["w_out"], dict(conv=c["state"], h=s["h"])


def _token(ops, p, x, res, st):
    r = ops.m3_residual_norm(x, res, p["norm_w"], p["scale"], eps=1e-5)
    xz = r["y"] @ p["w_in"]
    xc = ops.m3_causal_conv_step(st["conv"], xz[..., :D], p["conv_w"], p["conv_b"])
    proj = xc @ p["w_x"]
    B, C = (proj[..., R + i * G * N:R + (i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
    y = ops.m3_selective_scan_step(st["h"], xc, proj[..., :R] @ p["w_dt"], p["A"], B, C, p["skip"], None, dt_softplus=True,
                                   dt_bias=p["dt_bias"])
    return r["residual"], ops.m3_gated_norm(y, xz[..., D:], p["gate_w"], groups=G, eps=1e-5) @ p["w_out"]


# Seven stages, each off by at most (its longest sum of 48 + 40) 2^-24 of its terms,
# which cancel by less than ten times in the norm over a tensor.
CHAIN = 7 * 88 * 2.0 ** -24 * 10


def test_block_prompt_and_tokens(ops):
    m = Maker(51)
    p = _params(m)
    Bt, L, T = 3, 40, 6
    x, res = m(Bt, L + T, E), m(Bt, L + T, E)
    p64 = {k: v.double().cpu() for k, v in p.items()}
    h, y, state = _reference(p64, x.double().cpu(), res.double().cpu())
    got_h, got_y, st = _prompt(ops, p, x[:, :L].contiguous(), res[:, :L].contiguous())
    assert rel(got_h, h[:, :L]) <= CHAIN and rel(got_y, y[:, :L]) <= CHAIN
    for t in range(L, L + T):
        th, ty = _token(ops, p, x[:, t].contiguous(), res[:, t].contiguous(), st)
        assert rel(th, h[:, t]) <= CHAIN and rel(ty, y[:, t]) <= CHAIN, t
    assert rel(st["h"], state) <= CHAIN


def test_block_padded_batch_matches_single_items(ops):
    m = Maker(52)
    p = _params(m)
    lengths = [37, 0, 1, 12]
    x, res = m(4, 37, E), m(4, 37, E)
    _, y, st = _prompt(ops, p, x, res, ilen(lengths))
    for b, n in enumerate(lengths):
        if n == 0:
            assert (st["h"][b] == 0).all() and (st["conv"][b] == 0).all()
            continue
        _, y1, s1 = _prompt(ops, p, x[b:b + 1, :n].contiguous(), res[b:b + 1, :n].contiguous())
        assert rel(y[b, :n], y1[0]) <= CHAIN and rel(st["h"][b], s1["h"][0]) <= CHAIN
        assert rel(st["conv"][b] + 1, s1["conv"][0] + 1) <= CHAIN


def _block_gradients(ops, p, x, res, dh, dout):
    """Gradients of sum(h dh) + sum(out dout) through the block, by the operators'
    backward entry points and the products' own."""
    k = {}
    h, _, _ = _prompt(ops, p, x, res, keep=k)
    f = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    g = dict(w_out=f(k["y"]).T @ f(dout))
    n = ops.m3_gated_norm_backward(k["s"], k["xz"][..., D:], p["gate_w"], dy=dout @ p["w_out"].T, groups=G, eps=1e-5)
    s = ops.m3_selective_scan_backward(k["xc"], k["dt"], p["A"], k["B"], k["C"], p["skip"], None, dy=n["dx"], dt_softplus=True,
                                       dt_bias=p["dt_bias"])
    dproj = torch.cat([s["ddt"] @ p["w_dt"].T, s["dB"].flatten(-2), s["dC"].flatten(-2)], -1)
    g.update(gate_w=n["dw"], A=s["dA"], skip=s["dD"], dt_bias=s["ddt_bias"], w_dt=f(k["proj"][..., :R]).T @ f(s["ddt"]),
             w_x=f(k["xc"]).T @ f(dproj))
    c = ops.m3_causal_conv_backward(k["xz"][..., :D], p["conv_w"], p["conv_b"], dy=s["dx"] + dproj @ p["w_x"].T)
    dxz = torch.cat([c["dx"], n["dz"]], -1)
    g.update(conv_w=c["dw"], conv_b=c["dbias"], w_in=f(k["u"]).T @ f(dxz))
    r = ops.m3_residual_norm_backward(h, x, p["norm_w"], p["scale"], dy=dxz @ p["w_in"].T, dresidual=dh, eps=1e-5)
    g.update(norm_w=r["dw"], scale=r["dscale"], x=r["dx"], res=r["dresidual"])
    return g


def test_block_training_step(ops):
    m = Maker(53)
    p = _params(m)
    Bt, L = 2, 70
    x, res, dh, dout = (m(Bt, L, E) for _ in range(4))
    got = _block_gradients(ops, p, x, res, dh, dout)
    leaves = {k: v.double().cpu().requires_grad_() for k, v in dict(p, x=x, res=res).items()}
    h, out, _ = _reference(leaves, leaves["x"], leaves["res"])
    ((h * dh.double().cpu()).sum() + (out * dout.double().cpu()).sum()).backward()
    for k, v in leaves.items():
        # the reverse chain doubles the stages; sums over 140 tokens are its longest
        assert rel(got[k].reshape(v.shape), v.grad) <= 2 * 7 * 180 * 2.0 ** -24 * 10, k
    # against differences of the 64-bit block along one direction
    step = {k: torch.randn(v.shape, generator=m.g, dtype=torch.float64) for k, v in leaves.items()}

    def loss(e):
        q = {k: v.detach() + e * step[k] for k, v in leaves.items()}
        hh, oo, _ = _reference(q, q["x"], q["res"])
        return float((hh * dh.double().cpu()).sum() + (oo * dout.double().cpu()).sum())

    want = sum(float((got[k].double().cpu().reshape(v.shape) * step[k]).sum()) for k, v in leaves.items())
    size = sum(float((got[k].double().cpu().reshape(v.shape) * step[k]).abs().sum()) for k, v in leaves.items())
    # central differences at 1e-5: 1e-10 of third derivatives and 1e-16 / 1e-5 of rounding, both far below
    assert abs((loss(1e-5) - loss(-1e-5)) / 2e-5 - want) <= 2 * 7 * 180 * 2.0 ** -24 * 10 * size


# ---------------------------------------------------------------- every operator as one call
def _calls(ops, dtype, long=False, seed=61):
    """Each entry point on inputs of its own: name -> (inputs, call(inputs, outputs), outputs)."""
    m = Maker(seed)
    Bt, L, Dm, Ns = (1, 700, 64, 16) if long else (3, 50, 96, 16)
    t = dtype
    x, dt, z, dy = (m(Bt, L, Dm, dtype=t) for _ in range(4))
    B, C = (m(Bt, L, 1, Ns, dtype=t) for _ in range(2))
    A, skip, h0, db = -torch.exp(m(Dm, Ns)), m(Dm), m(Bt, Dm, Ns), m(Dm, shift=-3.0)
    w4, bias, st, dhf, gw = m(Dm, 4), m(Dm), m(Bt, 3, Dm, dtype=t), m(Bt, Dm, Ns), m(Dm)
    scan = (x, dt, A, B, C, skip, z, h0)
    tok = (x[:, 0].contiguous(), dt[:, 0].contiguous(), A, B[:, 0].contiguous(), C[:, 0].contiguous(), skip, z[:, 0].contiguous())
    kw = dict(dt_softplus=True, dt_bias=db)
    e = torch.empty_like
    return {
        "conv": lambda **k: ops.m3_causal_conv(x, w4, bias, st, want_state=True, **k),
        "conv_step": lambda **k: dict(y=ops.m3_causal_conv_step(st, x[:, 0], w4, bias, state_out=e(st), **k)),
        "conv_backward": lambda **k: ops.m3_causal_conv_backward(x, w4, bias, st, dy=dy, want_state_grad=True, **k),
        "scan": lambda **k: ops.m3_selective_scan(*scan, **kw, **k),
        "scan_step": lambda **k: dict(y=ops.m3_selective_scan_step(h0, *tok, h_out=e(h0), **kw, **k)),
        "scan_backward": lambda **k: ops.m3_selective_scan_backward(*scan, dy=dy, dh_final=dhf, want_carry_grads=True, **kw, **k),
        "gated": lambda **k: dict(y=ops.m3_gated_norm(x, z, gw, groups=2, **k)),
        "gated_backward": lambda **k: ops.m3_gated_norm_backward(x, z, gw, dy=dy, groups=2, **k),
        "residual": lambda **k: ops.m3_residual_norm(x, z, gw, skip, **k),
        "residual_backward": lambda **k: ops.m3_residual_norm_backward(z, x, gw, skip, dy=dy, dresidual=dt, **k),
    }


def _same(a, b):
    return all(a[k] is None and b[k] is None or torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_again(ops, dtype, long):
    """Nothing depends on what ran before: no atomics, no state between calls."""
    calls = _calls(ops, dtype, long)
    first = {k: f() for k, f in calls.items()}
    for _ in range(2):
        for k, f in calls.items():
            assert _same(first[k], f()), k


@pytest.mark.parametrize("long", [False, True])
def test_other_stream(ops, long):
    calls = _calls(ops, BF, long)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for k, f in calls.items():
        got = f(stream=s)
        # memory freed on the current stream meanwhile is not the call's
        junk = [torch.full((1 << 20,), NAN, device="cuda") for _ in range(4)]
        del junk
        s.synchronize()
        assert _same(want[k], got), k


@pytest.mark.parametrize("long", [False, True])
def test_graph_replays(ops, long):
    calls = _calls(ops, BF, long)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            for k, f in calls.items():
                got[k] = f()
    torch.cuda.synchronize()
    for rep in range(3):
        for o in got.values():
            for t in o.values():
                if t is not None:
                    t.fill_(NAN)
        for k, f in calls.items():  # eager work between the replays
            assert _same(want[k], f()), k
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, o in got.items():
            assert _same(want[k], o), (rep, k)


def test_two_streams_at_once(ops):
    a, b = _calls(ops, BF, True, 61), _calls(ops, BF, True, 62)
    want = [{k: f() for k, f in c.items()} for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [{}, {}]
    for _ in range(3):
        for k in a:
            for i, c in enumerate((a, b)):
                got[i][k] = c[k](stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for k in a:
            assert _same(want[i][k], got[i][k]), (i, k)


# ---------------------------------------------------------------- far offsets
def test_past_32_bit_offsets(ops):
    """Tensors of more than 2^31 elements: the last item's results are those of
    the item alone."""
    Bt, L, Dm, Ns = 3, 400000, 2048, 4
    assert Bt * L * Dm > 1 << 31
    x = torch.randn(Bt, 1, Dm, device="cuda", dtype=BF).expand(Bt, L, Dm).contiguous()
    m = Maker(71)
    x[-1, -300:] = m(300, Dm, dtype=BF)
    w, bias = m(Dm, 4), m(Dm)
    got = ops.m3_causal_conv(x, w, bias)["y"][-1, -200:].clone()
    alone = ops.m3_causal_conv(x[-1:, -300:].contiguous(), w, bias)["y"][0, -200:]
    assert torch.equal(got, alone)
    # rows enough that they are dealt to lanes as in the whole call (2048 or more): a
    # row summed in another order may round to the other neighbour
    last = x[-1, -2500:].contiguous()
    got = ops.m3_gated_norm(x, x, bias, groups=2)[-1, -200:].clone()
    assert torch.equal(got, ops.m3_gated_norm(last, last, bias, groups=2)[-200:])
    got = ops.m3_residual_norm(x, x, bias, want_residual=False)["y"][-1, -200:].clone()
    assert torch.equal(got, ops.m3_residual_norm(last, last, bias)["y"][-200:])
    # decays of 1e-4 and less per token: 100 tokens on, the state is that of the last ones
    A, B = -10.0 - torch.rand(Dm, Ns, generator=m.g).cuda(), m(1, 1, 1, Ns, dtype=BF).expand(Bt, L, 1, Ns).contiguous()
    one = torch.ones(1, 1, Dm, device="cuda", dtype=BF).expand(Bt, L, Dm).contiguous()
    got = ops.m3_selective_scan(x, one, A, B, B, bias)
    alone = ops.m3_selective_scan(x[-1:, -300:].contiguous(), one[:1, :300].contiguous(), A, B[:1, :300].contiguous(),
                                  B[:1, :300].contiguous(), bias)
    # the segments' joins may round the state otherwise: a step of bf16
    assert rel(got["y"][-1, -200:].float(), alone["y"][0, -200:].float()) <= 2.0 ** -8
    assert rel(got["h"][-1], alone["h"][0]) <= 1e-5
    dy = x
    g = ops.m3_selective_scan_backward(x, one, A, B, B, bias, dy=dy)
    ga = ops.m3_selective_scan_backward(x[-1:, -300:].contiguous(), one[:1, :300].contiguous(), A, B[:1, :300].contiguous(),
                                        B[:1, :300].contiguous(), bias, dy=dy[-1:, -300:].contiguous())
    for k in ("dx", "ddt", "dB", "dC"):
        assert rel(g[k][-1, -200:].float(), ga[k][0, -200:].float()) <= 2.0 ** -7, k
    c = ops.m3_causal_conv_backward(x, w, bias, dy=dy)["dx"][-1, -200:].clone()
    assert torch.equal(c, ops.m3_causal_conv_backward(x[-1:, -300:].contiguous(), w, bias, dy=dy[-1:, -300:].contiguous())["dx"][0, -200:])


# ---------------------------------------------------------------- values that stay where they are
def test_not_finite_values_stay_in_their_channels_and_tokens(ops):
    m = Maker(81)
    Bt, L, Dm, Ns = 2, 90, 70, 16
    x, dt, z, B, C = m(Bt, L, Dm), m(Bt, L, Dm), m(Bt, L, Dm), m(Bt, L, 1, Ns), m(Bt, L, 1, Ns)
    A, w, gw = -torch.exp(m(Dm, Ns)), m(Dm, 4), m(Dm)
    t0, d0 = 41, 69
    clean = ops.m3_selective_scan(x, dt, A, B, C, None, z, dt_softplus=True)
    conv = ops.m3_causal_conv(x, w)["y"]
    gated, resid = ops.m3_gated_norm(x, z, gw), ops.m3_residual_norm(x, z, gw)["y"]
    for bad in (NAN, float("inf"), -float("inf"), 3.0e38):
        xb = x.clone()
        xb[1, t0, d0] = bad
        y = ops.m3_selective_scan(xb, dt, A, B, C, None, z, dt_softplus=True)["y"]
        c = ops.m3_causal_conv(xb, w)["y"]
        for got, want in ((y, clean["y"]), (c, conv)):
            keep = torch.ones(Bt, L, Dm, dtype=torch.bool, device="cuda")
            keep[1, t0:, d0] = False
            assert torch.equal(got[keep], want[keep])
        g, r = ops.m3_gated_norm(xb, z, gw), ops.m3_residual_norm(xb, z, gw)["y"]
        keep = torch.ones(Bt, L, dtype=torch.bool, device="cuda")
        keep[1, t0] = False
        assert torch.equal(g[keep], gated[keep]) and torch.equal(r[keep], resid[keep])
        Bb = B.clone()  # a B that is not finite reaches its token and those after it only
        Bb[1, t0, 0, 3] = bad
        y = ops.m3_selective_scan(x, dt, A, Bb, C, None, z, dt_softplus=True)["y"]
        assert torch.equal(y[0], clean["y"][0]) and torch.equal(y[1, :t0], clean["y"][1, :t0])


def test_extreme_steps(ops):
    """delta from the far ends of the softplus: none at all, and one that forgets
    the state at once."""
    m = Maker(82)
    Bt, L, Dm, Ns = 1, 40, 64, 16
    x, B, C, h0 = m(Bt, L, Dm), m(Bt, L, 1, Ns), m(Bt, L, 1, Ns), m(Bt, Dm, Ns)
    A = -torch.exp(m(Dm, Ns))
    still = ops.m3_selective_scan(x, torch.full_like(x, -1000.0), A, B, C, h0=h0, dt_softplus=True)
    assert torch.equal(still["h"], h0)
    far = torch.full_like(x, 1.0e4)
    q = dict(x=x, dt=far, A=A, B=B, C=C, h0=h0)
    got = ops.m3_selective_scan(x, far, A, B, C, h0=h0, dt_softplus=True)
    want = ref.scan(**q, dt_softplus=True)
    # delta itself is exact here, so u, u B and the readout's 17 sums are all that rounds
    assert rel(got["y"], want["y"]) <= 40 * 2.0 ** -24 and rel(got["h"], want["h"]) <= 40 * 2.0 ** -24


@pytest.mark.parametrize("L", [1, 45, 300])
def test_rates_that_forget_at_once(ops, L):
    """A = -inf: every state is its own token's input, and the tokens behind an
    item's length still change nothing."""
    m = Maker(83)
    Bt, Dm, Ns = 2, 24, 16
    x, dt, B, C, dy = m(Bt, L, Dm), m(Bt, L, Dm), m(Bt, L, 1, Ns), m(Bt, L, 1, Ns), m(Bt, L, Dm)
    A = torch.full((Dm, Ns), -float("inf"), device="cuda")
    lengths = ilen([L, (L + 1) // 2])
    got = ops.m3_selective_scan(x, dt, A, B, C, lengths=lengths, dt_softplus=True, y=torch.zeros_like(x))
    u = torch.nn.functional.softplus(dt.double()) * x.double()
    y = u * (B.double() * C.double()).sum(-1)
    last = lengths.long() - 1
    h = torch.stack([u[b, last[b], :, None] * B.double()[b, last[b]] for b in range(Bt)])
    # u: softplus 4 roundings and its product; u B, and 17 sums of the readout
    k = 60 * 2.0 ** -24
    for b, n in enumerate(lengths.tolist()):
        assert rel(got["y"][b, :n], y[b, :n]) <= k
    assert rel(got["h"], h) <= k
    g = ops.m3_selective_scan_backward(x, dt, A, B, C, dy=dy, lengths=lengths, dt_softplus=True, want_carry_grads=True)
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)
    assert (g["dh0"] == 0).all() and (g["dA"] == 0).all()
    step = ops.m3_selective_scan_step(got["h"], x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], dt_softplus=True)
    assert rel(step, y[:, 0]) <= k


def test_binding_refuses_other_places(ops):
    x, w = torch.zeros(2, 5, 16, device="cuda", dtype=BF), torch.zeros(16, 4, device="cuda")
    with pytest.raises(ValueError):
        ops.m3_causal_conv(x, w.cpu())
    with pytest.raises(TypeError):
        ops.m3_causal_conv(x, w.to(BF))
    with pytest.raises(TypeError):
        ops.m3_causal_conv(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ops.m3_causal_conv(x, w, state=torch.zeros(2, 2, 16, device="cuda", dtype=BF))
    with pytest.raises(ops.M3Error):
        ops.m3_causal_conv(x, torch.zeros(16, 6, device="cuda"))
    with pytest.raises(ops.M3Error):
        ops.m3_causal_conv(x, w, y=x)
    with pytest.raises(TypeError):
        ops.m3_gated_norm(x.to(torch.float16))
    with pytest.raises(ValueError):
        ops.m3_gated_norm(wide(x)[:, :4])
    with pytest.raises(ops.M3Error):
        ops.m3_gated_norm(x, groups=3)
    with pytest.raises(ops.M3Error):
        ops.m3_causal_conv_backward(x, w, dy=x.clone(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
