"""Layer operators at the edges of what they take."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref as ref  # noqa: E402
from tests import test_gpu_layers as base  # noqa: E402
from tests.test_gpu_layers import DT, BF, NAN, Maker, close, ilen  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


# ---------------------------------------------------------------- tiles side by side
# The reverse walk finishes one tile, walks the next and stages the one after at once:
# each number of state blocks and of states per lane over tiles enough (129 tokens and
# 41) that every slot of LDS is used again, whole and cut into segments.
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,N", [(64, 4), (70, 8), (64, 12), (130, 16), (40, 24), (64, 32), (16, 48), (33, 64)])
def test_scan_backward_over_many_tiles(ops, D, N, dt):
    for Bt, L, lengths in ((2, 129, [129, 41]), (1, 127, None), (1, 290, None)):
        base.test_scan_backward(ops, (Bt, L, D, N, 1, dt, lengths, True, True, True, True, True, False))


@pytest.mark.parametrize("N", [4, 8, 12, 16, 24, 32, 48, 64])
def test_scan_backward_same_bits_beside_other_work(ops, N):
    """dB and dC join what several waves wrote: the same bits whatever shares the card."""
    q, m = base._scan_inputs((3, 200, 96, N, 1, "bf16", None, True, True, True, True, True, False), 91)
    args, kw = base._scan_call(q, True)
    dy = m(3, 200, 96, dtype=BF)
    first = ops.m3_selective_scan_backward(*args, dy=dy, want_carry_grads=True, **kw)
    torch.cuda.synchronize()
    side, a = torch.cuda.Stream(), torch.randn(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            a.mul_(1.0001)
        again = ops.m3_selective_scan_backward(*args, dy=dy, want_carry_grads=True, **kw)
        torch.cuda.synchronize()
        for k, v in first.items():
            assert torch.equal(v, again[k]), k


# ---------------------------------------------------------------- rows that count for nothing
@pytest.mark.parametrize("L", [1, 45, 300])
def test_scan_backward_rates_that_forget_at_once(ops, L):
    """A = -inf in every other state, with a gradient of the last state: the tokens that
    fill an item's last tile have no step, and add nothing to the bias's gradient."""
    q, m = base._scan_inputs((2, L, 70, 16, 1, "f32", [L, (L + 1) // 2], True, True, True, True, True, False), 92)
    lengths = [L, (L + 1) // 2]
    dy, dhf = base.spoil(m(2, L, 70), lengths), m(2, 70, 16, scale=3.0)
    forget = torch.zeros(70, 16, dtype=torch.bool, device="cuda")
    forget[:, ::2] = True
    steepest = float((torch.nn.functional.softplus(torch.nan_to_num(q["dt"]) + q["dt_bias"])[..., None] * q["A"]).abs().max())
    args, kw = base._scan_call(dict(q, A=torch.where(forget, -float("inf"), q["A"])), True)
    got = ops.m3_selective_scan_backward(*args, dy=dy, dh_final=dhf, lengths=ilen(lengths), want_carry_grads=True, **kw)
    # 64 bits: -1e30 times any step here is an exponent whose power is zero too
    q["A"] = torch.where(forget, -1e30, q["A"])
    want, mag = (ref.scan(**q, lengths=lengths, dt_softplus=True, dy=dy, dh_final=dhf, mag=v) for v in (False, True))
    # a decay of exactly zero has no error, so the steepest of the others counts
    k = 2 * base.k_scan(L, 16, steepest, base._zmax(q["z"]))
    for name, extra in (("dz", 0), ("dx", 16), ("ddt", 48), ("dB", 70), ("dC", 70), ("dh0", 0), ("dA", 2 * L), ("dD", 2 * L),
                        ("ddt_bias", 2 * L + 32)):
        close(name, got[name], want[name], mag[name], k + extra)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,W", [(24, 4), (37, 3), (3, 2)])
def test_conv_backward_rows_behind_an_infinite_one(ops, D, W, dt):
    """An item's last input is infinite: the gradients behind its length are zeros, and
    without an activation only the newest tap's gradient sees it."""
    for L, n in ((9, 1), (9, 4), (70, 3), (70, 64), (300, 8), (300, 129), (300, 297)):
        m, t = Maker(93), DT[dt]
        x, dy, w, bias = m(2, L, D, dtype=t), m(2, L, D, dtype=t), m(D, W, scale=0.5), m(D)
        x[1, n - 1, D - 1] = float("inf")
        lengths = [L, n]
        base.spoil(dy, lengths)
        for act in (True, False):
            got = ops.m3_causal_conv_backward(x, w, bias, dy=dy, lengths=ilen(lengths), silu=act, want_state_grad=True)
            assert (got["dx"][1, n:] == 0).all(), (L, n, act)
            z = x.clone()
            z[1, n - 1, D - 1] = 0
            clean = ops.m3_causal_conv_backward(z, w, bias, dy=dy, lengths=ilen(lengths), silu=act, want_state_grad=True)
            for k in ("dx", "dw", "dbias", "dstate"):
                other = (..., slice(0, D - 1)) if k in ("dx", "dstate") else slice(0, D - 1)
                assert torch.equal(got[k][other], clean[k][other]), (k, L, n, act)
            if not act:
                assert torch.equal(got["dw"][-1, :-1], clean["dw"][-1, :-1]) and not got["dw"][-1, -1].isfinite(), (L, n)
                assert torch.equal(got["dx"], clean["dx"]) and torch.equal(got["dbias"], clean["dbias"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", [True, False])
def test_conv_backward_carry_of_an_empty_item(ops, act, dt):
    """An item without tokens: whatever its carry holds, it has no part in any gradient."""
    for L in (1, 6, 200):
        m, t = Maker(94), DT[dt]
        x, dy, w, bias, state = m(3, L, 40, dtype=t), m(3, L, 40, dtype=t), m(40, 4, scale=0.5), m(40), m(3, 3, 40, dtype=t)
        lengths = ilen([L, 0, L])
        want = ops.m3_causal_conv_backward(x, w, bias, state, dy=dy, lengths=lengths, silu=act, want_state_grad=True)
        assert (want["dstate"][1] == 0).all() and (want["dx"][1] == 0).all()
        for bad in (NAN, float("inf")):
            state[1] = bad
            got = ops.m3_causal_conv_backward(x, w, bias, state, dy=dy, lengths=lengths, silu=act, want_state_grad=True)
            for k, v in want.items():
                assert torch.equal(v, got[k]), (k, L, bad)


# ---------------------------------------------------------------- arguments by their names
def test_arguments_by_name(ops):
    m = Maker(95)
    Bt, L, D, N = 2, 20, 24, 8
    x, dt, z, dy, h = (m(Bt, L, D, dtype=BF) for _ in range(5))
    B, C = (m(Bt, L, 1, N, dtype=BF) for _ in range(2))
    w, b, st, A, h0 = m(D, 4), m(D), m(Bt, 3, D, dtype=BF), -torch.exp(m(D, N)), m(Bt, D, N)
    tok = dict(x=x[:, 0], dt=dt[:, 0], A=A, B=B[:, 0], C=C[:, 0], D=b, z=z[:, 0])
    for fn, args in ((ops.m3_causal_conv, dict(x=x, w=w, bias=b, state=st)), (ops.m3_causal_conv_step, dict(state=st.clone(), x=x[:, 0], w=w)),
                     (ops.m3_causal_conv_backward, dict(x=x, w=w, bias=b, state=st, dy=dy)),
                     (ops.m3_selective_scan, dict(x=x, dt=dt, A=A, B=B, C=C, D=b, z=z, h0=h0)),
                     (ops.m3_selective_scan_step, dict(h=h0, **tok, h_out=torch.empty_like(h0))),
                     (ops.m3_selective_scan_backward, dict(x=x, dt=dt, A=A, B=B, C=C, D=b, z=z, h0=h0, dy=dy)),
                     (ops.m3_gated_norm, dict(x=x, z=z, w=b)), (ops.m3_gated_norm_backward, dict(x=x, z=z, w=b, dy=dy)),
                     (ops.m3_residual_norm, dict(x=x, residual=z, w=b, scale=b)),
                     (ops.m3_residual_norm_backward, dict(h=h, x=x, w=b, scale=b, dy=dy))):
        first = next(iter(args))
        rest = {k: v.clone() if k == "state" else v for k, v in args.items() if k != first}
        a, c = fn(args[first].clone(), **rest), fn(**args)
        for p, q in zip(a.values(), c.values()) if isinstance(a, dict) else ((a, c),):
            # steps of either sign overflow here: bits, since no NaN equals itself
            assert p is None and q is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8)), fn.__name__


# ---------------------------------------------------------------- far slices
def test_scan_step_at_one_position_of_long_sequences(ops):
    """Rows 2^24 elements apart: 8192 positions of 2048 channels, 2^20 of 16 states."""
    m = Maker(96)
    Bt, D, N, t = 2, 2048, 16, 17
    x, dt, z = (torch.zeros(Bt, 8192, D, device="cuda", dtype=BF) for _ in range(3))
    B, C = (torch.zeros(Bt, 1 << 20, 1, N, device="cuda", dtype=BF) for _ in range(2))
    for v in (x, dt, z, B, C):
        v[:, t] = m(*v[:, t].shape, dtype=BF)
    A, skip, db, h0 = -torch.exp(m(D, N)), m(D), m(D, shift=-3.0), m(Bt, D, N)
    h, ho = h0.clone(), torch.empty_like(h0)
    kw = dict(dt_softplus=True, dt_bias=db)
    assert x[:, t].stride(0) == B[:, t].stride(0) == 1 << 24
    y = ops.m3_selective_scan_step(h, x[:, t], dt[:, t], A, B[:, t], C[:, t], skip, z[:, t], **kw)
    near = [v[:, t].contiguous() for v in (x, dt, B, C, z)]
    want = ops.m3_selective_scan_step(h0, near[0], near[1], A, near[2], near[3], skip, near[4], h_out=ho, **kw)
    assert torch.equal(y, want) and torch.equal(h, ho)
    st = m(Bt, 3, D, dtype=BF)
    w = m(D, 4)
    assert torch.equal(ops.m3_causal_conv_step(st.clone(), x[:, t], w), ops.m3_causal_conv_step(st.clone(), near[0], w))


# ---------------------------------------------------------------- captured first
def test_first_call_of_a_kernel_is_captured(ops):
    """Kernels that nothing has launched before, captured at once: what a launch sets up
    the first time does not belong to the stream."""
    m = Maker(97)
    Bt, L, D, N = 2, 70, 3, 41
    x, dt, z, dy = (m(Bt, L, D) for _ in range(4))
    B, C = (m(Bt, L, 1, N) for _ in range(2))
    A, skip, db, w, gain = -torch.exp(m(D, N)), m(D), m(D, shift=-3.0), m(D, 3), m(D)

    def calls():
        c = ops.m3_causal_conv(x, w, skip)["y"]
        s = ops.m3_selective_scan(c, dt, A, B, C, skip, z, dt_softplus=True, dt_bias=db)
        g = ops.m3_selective_scan_backward(c, dt, A, B, C, skip, z, dy=dy, dt_softplus=True, dt_bias=db)
        v = ops.m3_causal_conv_backward(x, w, skip, dy=g["dx"])
        n = ops.m3_gated_norm_backward(s["y"], z, gain, dy=dy)
        return [c] + [o for d in (s, g, v, n) for o in d.values() if o is not None]

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = calls()
    for _ in range(3):
        for o in held:
            o.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(calls(), held):
            assert torch.equal(p, q) and p.isfinite().all()
        torch.cuda.synchronize()


@pytest.mark.parametrize("L", [1, 16, 45, 300])
@pytest.mark.parametrize("N", [4, 12, 16, 24, 64])
def test_scan_backward_behind_an_infinite_input(ops, L, N):
    """An item's last input is infinite, and so is its last state.  The gradients of A
    and of the first state, and those of the tokens before, do not depend on it: the
    tokens that fill the last tile bring it nowhere."""
    q, m = base._scan_inputs((2, L, 40, N, 1, "f32", [L, (L + 1) // 2], True, True, True, True, True, False), 98)
    lengths = [L, (L + 1) // 2]
    dy, dhf = base.spoil(m(2, L, 40), lengths), m(2, 40, N)
    for last in (None, dhf):
        got = []
        for value in (0.0, float("inf")):
            for b, n in enumerate(lengths):
                q["x"][b, n - 1, 7] = value
            args, kw = base._scan_call(q, True)
            got.append(ops.m3_selective_scan_backward(*args, dy=dy, dh_final=last, lengths=ilen(lengths), want_carry_grads=True, **kw))
        clean, bad = got
        assert torch.equal(clean["dA"], bad["dA"]) and torch.equal(clean["dh0"], bad["dh0"]), last is None
        for b, n in enumerate(lengths):
            for k in ("dx", "ddt", "dz", "dB", "dC"):
                assert torch.equal(clean[k][b, :n - 1], bad[k][b, :n - 1]) and (bad[k][b, n:] == 0).all(), k
        keep = torch.arange(40, device="cuda") != 7
        for k in ("dD", "ddt_bias"):
            assert torch.equal(clean[k][keep], bad[k][keep]), k


# ---------------------------------------------------------------- several items per lane
@pytest.mark.parametrize("Bt,D,N,dt,strided", [(259, 1030, 13, "bf16", True), (258, 1040, 16, "f32", False), (133, 500, 61, "f32", True)])
def test_scan_step_of_many_items(ops, Bt, D, N, dt, strided):
    """Batches large enough that a lane takes four items, and no multiple of four."""
    base.test_scan_step(ops, Bt, D, N, 1, dt, strided)
