"""Linear attention and the norm and rotation of its queries and keys in use: a whole
retention mixer over prompts, token by token and in a training step; graphs captured and
replayed; other streams; repeated calls; far rows; many tiles; segments of uneven items."""
import pytest

torch = pytest.importorskip("torch")

from tests import mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import BF, F32, NAN, Maker, ilen  # noqa: E402
from tests.test_gpu_mixer import close, k_attention, parts_of, slice_of  # noqa: E402

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


# ---------------------------------------------------------------- a retention mixer
E, H, Hk, K, V, W = 40, 4, 2, 32, 48, 4  # model width, heads, shared heads, head sizes, taps
QK, ALL = (H + Hk) * K, (H + Hk) * K + Hk * V + H * V  # projection: q, k, v, gate


def _params(m):
    return dict(w_in=m(E, ALL, scale=E ** -0.5), w_out=m(H * V, E, scale=(H * V) ** -0.5), conv_w=m(QK, W, scale=0.5), conv_b=m(QK, scale=0.1),
                q_w=m(K, shift=1.0, scale=0.1), k_w=m(K, shift=1.0, scale=0.1), gate_w=m(H * V, shift=1.0, scale=0.1),
                norm_w=m(E, shift=1.0, scale=0.1), freqs=torch.exp(-torch.arange(K // 2, dtype=F32) * 0.5).cuda(),
                g=torch.log1p(-torch.exp2(-torch.arange(3.0, 3.0 + H))).cuda())


def _reference(p, x, res, h0):
    """The block in the inputs' own precision, token by token, by torch operations that
    differentiate: the residual stream, the block's output and the last state."""
    h = res + x
    u = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * p["norm_w"]
    proj = u @ p["w_in"]
    Bt, L = x.shape[:2]
    pad = torch.cat([proj.new_zeros(Bt, W - 1, QK), proj[..., :QK]], 1)
    qk = torch.nn.functional.silu(p["conv_b"] + sum(p["conv_w"][:, k] * pad[:, k:k + L] for k in range(W))).unflatten(-1, (H + Hk, K))
    v = proj[..., QK:QK + Hk * V].unflatten(-1, (Hk, V))
    angle = torch.arange(L, device=x.device, dtype=x.dtype)[:, None] * p["freqs"]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    n = qk * (qk.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    n = torch.cat([n[:, :, :H] * p["q_w"], n[:, :, H:] * p["k_w"]], 2)
    a, b = n[..., :K // 2], n[..., K // 2:]
    n = torch.cat([a * c - b * s, b * c + a * s], -1)
    S, ys, lam = h0, [], torch.exp(p["g"])[:, None, None]
    for t in range(L):
        kt, vt = n[:, t, H:].repeat_interleave(H // Hk, 1), v[:, t].repeat_interleave(H // Hk, 1)
        S = lam * S + kt[..., None] * vt[:, :, None]
        ys.append(K ** -0.5 * (n[:, t, :H, :, None] * S).sum(-2))
    y = torch.stack(ys, 1)
    y = (y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).flatten(-2) * p["gate_w"]
    return h, (y * torch.nn.functional.silu(proj[..., QK + Hk * V:])) @ p["w_out"], S


def _block(ops, p, x, res, h0, lengths=None):
    """The same through the library, over a prompt; what a decoder keeps."""
    r = ops.m3_residual_norm(x, res, p["norm_w"])
    proj = (r["y"].float() @ p["w_in"]).to(x.dtype)
    c = ops.m3_causal_conv(proj[..., :QK], p["conv_w"], p["conv_b"], lengths=lengths, want_state=True)
    qk = c["y"].unflatten(-1, (H + Hk, K))
    q, k = (slice_of(t.contiguous()) for t in (qk[:, :, :H], qk[:, :, H:]))
    n = ops.m3_qk_norm_rope(q, k, p["q_w"], p["k_w"], freqs=p["freqs"], lengths=lengths)
    v = proj[..., QK:QK + Hk * V].unflatten(-1, (Hk, V))
    o = ops.m3_linear_attention(n["q"], n["k"], v, p["g"], h0, lengths=lengths)
    y = ops.m3_gated_norm(o["y"].flatten(-2), proj[..., QK + Hk * V:], p["gate_w"], groups=H, gate_first=False)
    return r["residual"], y.float() @ p["w_out"], dict(conv=c["state"], h=o["h"])


def _step(ops, p, x, res, kept, at):
    """One token of it against the kept state."""
    r = ops.m3_residual_norm(x, res, p["norm_w"])
    proj = (r["y"].float() @ p["w_in"]).to(x.dtype)
    qk = ops.m3_causal_conv_step(kept["conv"], proj[..., :QK], p["conv_w"], p["conv_b"]).unflatten(-1, (H + Hk, K))[:, None]
    pos = torch.full((x.shape[0], 1), at, dtype=torch.int32, device="cuda")
    n = ops.m3_qk_norm_rope(qk[:, :, :H].contiguous(), qk[:, :, H:].contiguous(), p["q_w"], p["k_w"], freqs=p["freqs"], positions=pos)
    y = ops.m3_linear_attention_step(kept["h"], n["q"][:, 0], n["k"][:, 0], proj[..., QK:QK + Hk * V].unflatten(-1, (Hk, V)), p["g"])
    y = ops.m3_gated_norm(y.flatten(-2), proj[..., QK + Hk * V:], p["gate_w"], groups=H, gate_first=False)
    return r["residual"], y.float() @ p["w_out"]


# fp32: a few hundred roundings of 2^-24 on any path, with the norms' division by sums that may
# cancel to a tenth: 1e-4.  bf16: every operator rounds its output to 2^-8, eight of them in a row.
BAR = {F32: 1e-4, BF: 4e-2}


@pytest.mark.parametrize("t", [F32, BF])
def test_mixer_prompt_and_tokens(ops, t):
    m = Maker(81)
    p, Bt, L = _params(m), 3, 150
    x, res, h0 = m(Bt, L, E, dtype=t), m(Bt, L, E), m(Bt, H, K, V, scale=0.1)
    d = {k: v.double() for k, v in p.items()}
    want = _reference(d, x.double(), res.double(), h0.double())
    cut = 131
    head = _block(ops, p, x[:, :cut].contiguous(), res[:, :cut].contiguous(), h0)
    kept, outs = head[2], [head[1]]
    for at in range(cut, L):
        outs.append(_step(ops, p, x[:, at].contiguous(), res[:, at].contiguous(), kept, at)[1][:, None])
    assert rel(torch.cat(outs, 1), want[1]) < BAR[t] and rel(kept["h"], want[2]) < BAR[t] and rel(head[0], want[0][:, :cut]) < BAR[t]
    whole = _block(ops, p, x, res, h0)
    assert rel(whole[1], want[1]) < BAR[t] and rel(whole[2]["h"], want[2]) < BAR[t]


@pytest.mark.parametrize("t", [F32, BF])
def test_mixer_padded_batch_matches_single_items(ops, t):
    """Items of a padded batch, with anything behind their tokens, are those alone."""
    m, lengths = Maker(82), [90, 1, 65, 0]
    p, L = _params(m), 90
    x, res, h0 = m(4, L, E, dtype=t), m(4, L, E), m(4, H, K, V, scale=0.1)
    for b, n in enumerate(lengths):
        x[b, n:] = NAN
    got = _block(ops, p, x, res, h0, ilen(lengths))
    for b, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(got[2]["h"][b], h0[b])
            continue
        one = _block(ops, p, x[b:b + 1, :n].contiguous(), res[b:b + 1, :n].contiguous(), h0[b:b + 1].contiguous())
        assert rel(got[1][b, :n], one[1][0]) < BAR[t] and rel(got[2]["h"][b], one[2]["h"][0]) < BAR[t]


def test_mixer_training_step(ops):
    """Gradients of a block's core (norm and rotation, attention, gated norm) through the
    `_backward` calls against automatic differentiation of the definition."""
    m = Maker(83)
    p, Bt, L = _params(m), 2, 100
    q, k, v, z = m(Bt, L, H, K), m(Bt, L, Hk, K), m(Bt, L, Hk, V), m(Bt, L, H * V)
    h0, dout = m(Bt, H, K, V, scale=0.1), m(Bt, L, H * V)
    n = ops.m3_qk_norm_rope(q, k, p["q_w"], p["k_w"], freqs=p["freqs"])
    o = ops.m3_linear_attention(n["q"], n["k"], v, p["g"], h0)
    gn = ops.m3_gated_norm_backward(o["y"].flatten(-2), z, p["gate_w"], dy=dout, groups=H, gate_first=False)
    at = ops.m3_linear_attention_backward(n["q"], n["k"], v, p["g"], h0, dy=gn["dx"].unflatten(-1, (H, V)), want_carry_grads=True)
    nr = ops.m3_qk_norm_rope_backward(q, k, p["q_w"], p["k_w"], dq_out=at["dq"], dk_out=at["dk"], freqs=p["freqs"])
    leaves = [t.double().requires_grad_() for t in (q, k, v, z, h0, p["q_w"], p["k_w"], p["gate_w"])]
    ql, kl, vl, zl, hl, qw, kw, gw = leaves
    angle = torch.arange(L, device="cuda", dtype=torch.float64)[:, None] * p["freqs"].double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turned(x, w):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = x[..., :K // 2], x[..., K // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    qn, kn = turned(ql, qw), turned(kl, kw)
    S, ys, lam = hl, [], torch.exp(p["g"].double())[:, None, None]
    for t in range(L):
        S = lam * S + kn[:, t].repeat_interleave(H // Hk, 1)[..., None] * vl[:, t].repeat_interleave(H // Hk, 1)[:, :, None]
        ys.append(K ** -0.5 * (qn[:, t, :, :, None] * S).sum(-2))
    y = torch.stack(ys, 1)
    y = (y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).flatten(-2) * gw * torch.nn.functional.silu(zl)
    (y * dout.double()).sum().backward()
    for name, got, leaf in zip(("q", "k", "v", "z", "h0", "q_w", "k_w", "gate_w"),
                               (nr["dq"], nr["dk"], at["dv"], gn["dz"], at["dh0"], nr["dq_w"], nr["dk_w"], gn["dw"]), leaves):
        assert rel(got, leaf.grad) < BAR[F32], name


# ---------------------------------------------------------------- repeated, streamed, captured
def _calls(ops, t, seed=84):
    """Every call at sizes that use its paths: segments, shared heads, column tiles."""
    m = Maker(seed)
    Bt, L, nh, nk, k_, v_ = 2, 1300, 4, 2, 64, 96
    q, k, v = m(Bt, L, nh, k_, dtype=t), m(Bt, L, nk, k_, dtype=t), m(Bt, L, nk, v_, dtype=t)
    g, h0, dy, dh = -torch.tensor([0.03, 0.01, 0.002, 0.3]).cuda(), m(Bt, nh, k_, v_), m(Bt, L, nh, v_, dtype=t), m(Bt, nh, k_, v_)
    n = ilen([1300, 700])
    fr, w = torch.rand(16, generator=m.g).cuda(), m(k_)
    big = [m(1, 200, 2, 256, dtype=t) for _ in range(3)]
    gb = -torch.tensor([0.03, 0.01]).cuda()
    return {
        "attention": lambda **kw: ops.m3_linear_attention(q, k, v, g, h0, lengths=n, **kw),
        "whole": lambda **kw: ops.m3_linear_attention(q, k, v, g, h0, workspace=False, **kw),
        "backward": lambda **kw: ops.m3_linear_attention_backward(q, k, v, g, h0, dy=dy, dh_final=dh, lengths=n, want_carry_grads=True, **kw),
        "large": lambda **kw: ops.m3_linear_attention(*big, gb, **kw),
        "step": lambda **kw: {"y": ops.m3_linear_attention_step(h0, q[:, 5], k[:, 5], v[:, 5], g, h_out=torch.empty_like(h0), **kw)},
        "rope": lambda **kw: ops.m3_qk_norm_rope(q, k, w, w, freqs=fr, **kw),
        "rope_backward": lambda **kw: ops.m3_qk_norm_rope_backward(q, k, w, w, dq_out=q, dk_out=k, freqs=fr, **kw),
    }


def _same(a, b):
    # rows behind the second item's 700 tokens are left as they were in a new output
    return all((x is None and b[k] is None) or torch.equal(x.flatten(0, 1)[:2000] if k == "y" and x.dim() == 4 and x.shape[1] == 1300 else x,
                                                           b[k].flatten(0, 1)[:2000] if k == "y" and x.dim() == 4 and x.shape[1] == 1300 else b[k])
               for k, x in a.items())


@pytest.mark.parametrize("t", [F32, BF])
def test_same_bits_again_and_on_another_stream(ops, t):
    calls = _calls(ops, t)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for k, f in calls.items():
        assert _same(want[k], f()), k
        torch.cuda.synchronize()
        got = f(stream=s)
        s.synchronize()
        assert _same(want[k], got), k


@pytest.mark.parametrize("t", [F32, BF])
def test_graph_replays(ops, t):
    calls = _calls(ops, t)
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
            for x in o.values():
                if x is not None:
                    x.fill_(NAN)
        for k, f in calls.items():  # eager work between the replays
            assert _same(want[k], f()), k
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, o in got.items():
            assert _same(want[k], o), (rep, k)


def test_two_streams_at_once(ops):
    a, b = _calls(ops, BF, 91), _calls(ops, BF, 92)
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


# ---------------------------------------------------------------- far rows, many tiles, odd walks
def test_far_rows(ops):
    """Tokens 2^23 elements apart (offsets past 2^31 elements and 2^32 bytes) and a token's rows
    further apart than a prompt's may be."""
    m, L, ld = Maker(85), 300, (1 << 23) + 64
    big = torch.empty(L * ld, dtype=BF, device="cuda")
    rows = big.view(1, L, ld)
    q, k, v = (rows[..., i * 128:(i + 1) * 128].unflatten(-1, (2, 64)) for i in range(3))
    vals = [m(1, L, 2, 64, dtype=BF) for _ in range(3)]
    for t, x in zip((q, k, v), vals):
        t.copy_(x)
    g = -torch.tensor([0.01, 0.001]).cuda()
    got, want = ops.m3_linear_attention(q, k, v, g), ops.m3_linear_attention(*vals, g)
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["h"], want["h"])
    dy = m(1, L, 2, 64, dtype=BF)
    got, want = (ops.m3_linear_attention_backward(*x, g, dy=dy) for x in ((q, k, v), vals))
    assert all(torch.equal(got[n], want[n]) for n in ("dq", "dk", "dv"))
    got, want = (ops.m3_qk_norm_rope(*x[:2], freqs=torch.ones(32, device="cuda")) for x in ((q, k, v), vals))
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])
    far = big[:3 * (L // 3) * ld].view(3, (L // 3) * ld)  # a batch of three, one position of each
    q, k, v = (far[:, i * 128:(i + 1) * 128].unflatten(-1, (2, 64)) for i in range(3))
    assert q.stride(0) > 1 << 24
    h = m(3, 2, 64, 64)
    h2 = h.clone()
    assert torch.equal(ops.m3_linear_attention_step(h, q, k, v, g),
                       ops.m3_linear_attention_step(h2, q.contiguous(), k.contiguous(), v.contiguous(), g)) and torch.equal(h, h2)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("L", [63, 64, 65, 128, 191, 192, 193, 256, 257, 320, 321, 384, 449, 512, 1000])
def test_every_number_of_chunks(ops, t, L):
    """Walks of every short number of chunks, whole and part, forward and reverse: the first and last
    ones go by other code than those between."""
    m, dt = Maker(86), {"bf16": BF, "f32": F32}[t]
    q, k, v, dy = m(1, L, 2, 64, dtype=dt), m(1, L, 1, 64, dtype=dt), m(1, L, 1, 64, dtype=dt), m(1, L, 2, 64, dtype=dt)
    g, h0, dh = -torch.tensor([0.02, 0.0003]).cuda(), m(1, 2, 64, 64), m(1, 2, 64, 64)
    want, mag = (ref.attention(q, k, v, g, h0, mag=x, dy=dy, dh_final=dh) for x in (False, True))
    kk, parts = k_attention(L, 64, 64, g.cpu(), t) + 2, parts_of(t)
    y = ops.m3_linear_attention(q, k, v, g, h0, workspace=False)
    close("y", y["y"], want["y"], mag["y"], kk, parts)
    close("h", y["h"], want["h"], mag["h"], kk)
    got = ops.m3_linear_attention_backward(q, k, v, g, h0, dy=dy, dh_final=dh, want_carry_grads=True)
    for n in ("dq", "dk", "dv"):
        close(n, got[n], want[n], mag[n], kk, parts)
    close("dh0", got["dh0"], want["dh0"], mag["dh0"], kk)


def test_values_that_are_not_finite(ops):
    """They reach no other item and head, and no token more than a chunk in front of theirs."""
    m, L = Maker(87), 200
    for dt in (BF, F32):
        q, k, v = (m(2, L, 2, 32, dtype=dt) for _ in range(3))
        g = -torch.tensor([0.02, 0.1]).cuda()
        want = ops.m3_linear_attention(q, k, v, g)
        for x, bad in ((q, NAN), (k, float("inf")), (v, float("-inf")), (v, NAN)):
            at = x[1, 150, 1].clone()
            x[1, 150, 1] = bad
            got = ops.m3_linear_attention(q, k, v, g)
            assert torch.equal(got["y"][0], want["y"][0]) and torch.equal(got["y"][:, :, 0], want["y"][:, :, 0])
            assert torch.equal(got["y"][1, :128], want["y"][1, :128]) and not torch.isfinite(got["y"][1, 150, 1]).all()
            if x is q:  # a query is its own token's
                ok = torch.arange(L) != 150
                assert torch.equal(got["y"][1, ok], want["y"][1, ok]) and torch.equal(got["h"], want["h"])
            x[1, 150, 1] = at


def test_rope_far_angles_and_large_rates(ops):
    """Positions at both ends of 32 bits; a rate of zero and one of many turns a token.  Angles are
    products in 64 bits, off by 2^-52 of up to 2^31 x 50 radians: 3e-5 here."""
    m = Maker(88)
    q = m(1, 4, 1, 8)
    pos = torch.tensor([[-(1 << 31), -1, 1, (1 << 31) - 1]], dtype=torch.int32, device="cuda")
    freqs = torch.tensor([0.0, 1e-4, 1.0, 50.0], device="cuda")
    got = ops.m3_qk_norm_rope(q, None, freqs=freqs, positions=pos)["q"]
    want, mag = (ref.rope(q, freqs=freqs, positions=pos, mag=x) for x in (False, True))
    close("q", got, want["y"], mag["y"] + 0.0, 48 + 3e-5 / 2 ** -23)


@pytest.mark.parametrize("D,R,adjacent,t", [(128, 128, False, BF), (80, 40, True, F32), (57, 34, False, BF), (33, 6, True, F32)])
def test_rope_backward_in_place(ops, D, R, adjacent, t):
    """dq and dk where dq_out and dk_out were, uneven numbers of heads over a wave's teams."""
    m = Maker(89)
    q, k, dq, dk, w = m(2, 37, 5, D, dtype=t), m(2, 37, 3, D, dtype=t), m(2, 37, 5, D, dtype=t), m(2, 37, 3, D, dtype=t), m(D, shift=1.0)
    how = dict(freqs=torch.rand(R // 2, generator=m.g).cuda(), adjacent=adjacent, lengths=ilen([37, 11]))
    want = ops.m3_qk_norm_rope_backward(q, k, w, w, dq_out=dq, dk_out=dk, **how)
    got = ops.m3_qk_norm_rope_backward(q, k, w, w, dq_out=dq, dk_out=dk, out=dict(dq=dq, dk=dk), **how)
    assert got["dq"] is dq and all(torch.equal(want[n], got[n]) for n in want)
