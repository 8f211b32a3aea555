"""Linear attention with a decay per head and the norm and rotation of its queries and
keys on the GPU against their 64-bit reference (tests/mixer_ref.py).

Tolerance of one value: half a step of the output type on the value, plus
(k 2^-24 + parts) times the magnitude (the sum of the absolute values of the terms).  k
bounds the fp32 roundings on any path from an input to the value, each counted twice as the
matrix cores may drop what they round; `parts` is what splitting scores and states into two
bf16 parts leaves, 2^-16 (three parts: 2^-24, in k; fp32 inputs are not split).  Rows behind
an item's length hold NaN on input, outputs are filled with NaN or a marker before each call.
fp32 holds nothing below 2^-126: a power or a term of that size may be lost, times the other
factors of its products, which are below 2^7 here, for each of k roundings: k 2^-119 beside.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref, mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import BF, DT, F32, HALF, NAN, U, Maker, ilen, spoil  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


def slice_of(t, before=8, after=8):
    """The same values [..., H, D] as a slice of wider rows (NaN around them)."""
    *lead, H, D = t.shape
    big = torch.full((*lead, before + H * D + after), NAN, dtype=t.dtype, device=t.device)
    part = big[..., before:before + H * D].unflatten(-1, (H, D))
    part.copy_(t)
    return part


def close(name, got, want, mag, k, parts=0.0):
    got = got.detach().cpu()
    assert torch.isfinite(got.double()).all(), f"{name}: not finite"
    tol = HALF[got.dtype] * want.abs() + (2 * k * U + parts) * mag.abs() + k * 2.0 ** -119
    off = (got.double() - want).abs()
    if off.numel() and float((off - tol).max()) > 0:
        i = int((off - tol).argmax())
        raise AssertionError(f"{name}: off by {float(off.flatten()[i]):.3e} at {i} (value {float(want.flatten()[i]):.3e}, "
                             f"allowed {float(tol.flatten()[i]):.3e})")


# ---------------------------------------------------------------- linear attention
def k_attention(L, K, V, log_decay, dtype):
    """Scores: max(K, V) sums; their part of an output: 64 tokens in two parts; the state's part:
    max(K, V) sums in two parts behind, for each chunk, 64 tokens in three parts and a product.  A
    power exp2(x): two roundings of x make x of its steps, x at most 100 before it is nothing, and
    one of its own; on a path one in the scores or three in the state, and one for each chunk."""
    wide, chunks = max(K, V), -(-L // 64)
    g = log_decay[torch.isfinite(log_decay)].abs()
    x = min(100.0, float(g.max()) * L if g.numel() else 0.0)
    return wide + 2 * 64 + 2 * wide + chunks * (3 * 64 + 4) + 4 * x + 12


def parts_of(dtype):
    return 2.0 ** -16 if dtype == "bf16" else 0.0


ATT = [
    # Bt, L, H, Hk, K, V, dtype, lengths, state, strided, decays
    (1, 1, 1, 1, 1, 1, "f32", None, True, False, [-0.5]),
    (1, 1, 2, 1, 16, 8, "bf16", None, True, False, [-0.5, 0.0]),
    (2, 64, 2, 1, 32, 64, "bf16", None, False, False, [-0.03, -0.001]),
    (2, 65, 4, 2, 64, 64, "bf16", [65, 0], True, True, [-0.03, 0.0, -INF, -4.0]),
    (3, 130, 3, 1, 40, 100, "f32", [130, 1, 63], True, True, [-0.03, -0.4, -0.001]),
    (1, 200, 2, 2, 128, 128, "bf16", None, True, False, [-0.02, -0.0005]),
    (2, 77, 4, 4, 33, 37, "bf16", [77, 128], True, True, [-0.03, -0.1, -30.0, -0.002]),
    (2, 77, 2, 2, 37, 33, "f32", [-3, 64], False, True, [-0.03, -200.0]),
    (1, 300, 2, 1, 256, 256, "bf16", None, True, False, [-0.02, -0.0005]),
    (1, 129, 2, 1, 256, 200, "f32", None, True, False, [-0.02, -0.0005]),
    (1, 70, 1, 1, 20, 256, "f32", None, True, False, [-0.02]),
    (1, 70, 3, 1, 256, 20, "bf16", None, True, False, [-0.02, -0.01, -0.005]),
    (1, 1500, 1, 1, 64, 128, "bf16", None, True, False, [-0.001]),       # the token axis in segments
    (2, 1100, 2, 1, 80, 100, "f32", [1100, 257], True, True, [-0.004, 0.0]),
    (3, 1024, 2, 2, 64, 32, "bf16", [1024, 512, 256], False, False, [-0.01, -INF]),
    (2, 513, 1, 1, 96, 48, "f32", [0, 513], True, False, [-0.0001]),
]


def _attention_inputs(c, seed):
    Bt, L, H, Hk, K, V, dt, lengths, state, strided, decays = c
    m, t = Maker(seed), DT[dt]
    q, k, v = (spoil(m(Bt, L, h, d, dtype=t), lengths) for h, d in ((H, K), (Hk, K), (Hk, V)))
    if strided:
        q, k, v = slice_of(q), slice_of(k, 3, 5), slice_of(v, 16, 0)
    h0 = m(Bt, H, K, V) if state else None
    return q, k, v, torch.tensor(decays, device="cuda"), h0, m


@pytest.mark.parametrize("c", ATT, ids=str)
def test_attention(ops, c):
    Bt, L, H, Hk, K, V, dt, lengths = c[:8]
    q, k, v, g, h0, _ = _attention_inputs(c, 31)
    want, mag = (ref.attention(q, k, v, g, h0, lengths=lengths, mag=x) for x in (False, True))
    kk, parts = k_attention(L, K, V, g.cpu(), dt), parts_of(dt)
    for workspace in (None, False):
        y = torch.full((Bt, L, H, V), 7.0, dtype=q.dtype, device="cuda")
        hf = torch.full((Bt, H, K, V), NAN, device="cuda")
        ops.m3_linear_attention(q, k, v, g, h0, lengths=ilen(lengths), y=y, h_final=hf, workspace=workspace)
        for b, n in enumerate(layer_ref.held(lengths, Bt, L)):
            close("y", y[b, :n], want["y"][b, :n], mag["y"][b, :n], kk, parts)
            assert (y[b, n:] == 7).all()
        close("h", hf, want["h"], mag["h"], kk)
        if h0 is not None:  # the state in place
            s = h0.clone()
            ops.m3_linear_attention(q, k, v, g, s, lengths=ilen(lengths), h_final=s, workspace=workspace)
            assert torch.equal(s, hf)


@pytest.mark.parametrize("c", ATT, ids=str)
def test_attention_backward(ops, c):
    Bt, L, H, Hk, K, V, dt, lengths = c[:8]
    q, k, v, g, h0, m = _attention_inputs(c, 32)
    dy = spoil(m(Bt, L, H, V, dtype=q.dtype), lengths)
    dh = m(Bt, H, K, V) if h0 is not None else None
    shapes = dict(dq=(Bt, L, H, K), dk=(Bt, L, Hk, K), dv=(Bt, L, Hk, V))
    out = {n: torch.full(s, NAN, dtype=q.dtype, device="cuda") for n, s in shapes.items()}
    out["dh0"] = torch.full((Bt, H, K, V), NAN, device="cuda")
    got = ops.m3_linear_attention_backward(q, k, v, g, h0, dy=dy, dh_final=dh, lengths=ilen(lengths), scale=0.3, out=out)
    want, mag = (ref.attention(q, k, v, g, h0, scale=0.3, lengths=lengths, mag=x, dy=dy, dh_final=dh) for x in (False, True))
    kk, parts = k_attention(L, K, V, g.cpu(), dt) + H // Hk, parts_of(dt)
    for n in ("dq", "dk", "dv"):
        close(n, got[n], want[n], mag[n], kk, parts)
    close("dh0", got["dh0"], want["dh0"], mag["dh0"], kk)


STEP = [
    # Bt, H, Hk, K, V, dtype, strided
    (1, 1, 1, 1, 1, "f32", False), (3, 4, 2, 64, 64, "bf16", True), (2, 3, 1, 33, 37, "bf16", False),
    (2, 2, 2, 128, 128, "f32", True), (5, 2, 1, 256, 256, "bf16", False), (2, 6, 3, 80, 100, "f32", False),
]


@pytest.mark.parametrize("c", STEP, ids=str)
def test_attention_step(ops, c):
    Bt, H, Hk, K, V, dt, strided = c
    m, t = Maker(33), DT[dt]
    q, k, v = (m(Bt, h, d, dtype=t) for h, d in ((H, K), (Hk, K), (Hk, V)))
    if strided:
        q, k, v = slice_of(q), slice_of(k, 1, 0), slice_of(v)
    g, h = -torch.rand(H, device="cuda"), m(Bt, H, K, V)
    h_out, y = torch.full_like(h, NAN), torch.full((Bt, H, V), NAN, dtype=t, device="cuda")
    before = h.clone()
    ops.m3_linear_attention_step(h, q, k, v, g, y=y, h_out=h_out)
    assert torch.equal(h, before)
    want, mag = (ref.attention(q[:, None], k[:, None], v[:, None], g, h, mag=x) for x in (False, True))
    close("y", y, want["y"][:, 0], mag["y"][:, 0], K + 12)
    close("h", h_out, want["h"], mag["h"], 8)
    y2 = ops.m3_linear_attention_step(h, q, k, v, g)  # in place
    assert torch.equal(h, h_out) and torch.equal(y, y2)


# ---------------------------------------------------------------- norm and rotation
# Sum of squares: at most 16 values a lane (8 of single elements) and 6 joins, halved by the root;
# root, gain and products 4; sine and cosine 3 (argument, series, and 2e-9 of it); the turn 3; the
# gradient's second sum as the first.
K_ROPE = 48

ROPE = [
    # Bt, L, H, Hk, D, R, adjacent, dtype, lengths, norm, gains, positions, strided
    (1, 1, 1, 0, 1, 0, False, "f32", None, True, True, None, False),
    (1, 1, 1, 1, 2, 2, True, "bf16", None, True, True, None, False),
    (2, 5, 4, 2, 128, 128, False, "bf16", None, True, True, None, True),
    (2, 33, 3, 1, 80, 40, True, "f32", [33, 7], True, True, "far", False),
    (2, 33, 3, 1, 80, 40, False, "bf16", [0, 33], True, True, "far", True),
    (1, 40, 2, 2, 64, 64, True, "bf16", None, False, False, None, True),
    (1, 17, 5, 3, 57, 34, False, "bf16", None, True, True, None, False),
    (1, 17, 5, 3, 57, 34, True, "f32", [11], True, False, None, True),
    (3, 9, 2, 2, 33, 32, False, "f32", [9, 1, 0], True, True, "far", False),
    (1, 6, 2, 1, 256, 128, False, "f32", None, True, True, None, False),
    (1, 3, 2, 1, 1024, 1024, False, "f32", None, True, True, "far", False),
    (1, 3, 2, 1, 1024, 512, True, "bf16", None, True, True, None, False),
    (1, 3, 1, 1, 1021, 6, False, "f32", None, True, True, None, False),
    (2, 4, 3, 2, 1023, 1022, True, "bf16", [4, 2], True, True, None, False),
    (1, 5, 70, 9, 16, 16, False, "bf16", None, True, True, None, False),
    (2, 4500, 2, 1, 32, 32, False, "bf16", [4500, 300], True, True, None, False),
    (1, 50, 4, 4, 72, 0, False, "bf16", None, True, True, None, False),
]


def _rope_inputs(c, seed):
    Bt, L, H, Hk, D, R, adjacent, dt, lengths, norm, gains, far, strided = c
    m, t = Maker(seed), DT[dt]
    x = {"q": spoil(m(Bt, L, H, D, dtype=t), lengths), "k": spoil(m(Bt, L, Hk, D, dtype=t), lengths) if Hk else None}
    d = {n: None if x[n] is None else spoil(m(*x[n].shape, dtype=t), lengths) for n in x}
    w = {n: m(D, shift=1.0, scale=0.2) if gains and x[n] is not None else None for n in x}
    if strided:
        x = {n: None if v is None else slice_of(v, 24, 8) for n, v in x.items()}
    freqs = None if R == 0 else torch.exp(-torch.arange(R // 2, dtype=F32) * (9.2 / max(1, R // 2))).cuda()
    pos = None if far is None else torch.randint(-(1 << 20), 1 << 30, (Bt, L), generator=m.g).to(torch.int32).cuda()
    how = dict(freqs=freqs, positions=pos, start=0 if pos is not None else 5, eps=1e-6, norm=norm, adjacent=adjacent)
    return x, d, w, how, lengths


@pytest.mark.parametrize("c", ROPE, ids=str)
def test_rope(ops, c):
    x, _, w, how, lengths = _rope_inputs(c, 34)
    outs = {n: None if v is None else torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda") for n, v in x.items()}
    got = ops.m3_qk_norm_rope(x["q"], x["k"], w["q"], w["k"], lengths=ilen(lengths), q_out=outs["q"], k_out=outs["k"], **how)
    for n in "qk":
        if x[n] is None:
            assert got[n] is None
            continue
        want, mag = (ref.rope(x[n], w[n], lengths=lengths, mag=s, **how) for s in (False, True))
        for b, held in enumerate(layer_ref.held(lengths, *x[n].shape[:2])):
            close(n, got[n][b, :held], want["y"][b, :held], mag["y"][b, :held], K_ROPE)
            assert (got[n][b, held:] == 7).all()
        if x[n].is_contiguous():
            x[n] = x[n].clone()
    q, k = x["q"], x["k"]
    if q.is_contiguous():  # in place
        ops.m3_qk_norm_rope(q, k, w["q"], w["k"], lengths=ilen(lengths), q_out=q, k_out=k, **how)
        for n in "qk":
            for b, held in enumerate(layer_ref.held(lengths, *q.shape[:2])):
                assert x[n] is None or torch.equal(x[n][b, :held], got[n][b, :held])


@pytest.mark.parametrize("c", ROPE, ids=str)
def test_rope_backward(ops, c):
    x, d, w, how, lengths = _rope_inputs(c, 35)
    rows = x["q"].shape[0] * x["q"].shape[1]
    out = {"d" + n: torch.full(v.shape, NAN, dtype=v.dtype, device="cuda") for n, v in x.items() if v is not None}
    out.update({"d" + n + "_w": torch.full(v.shape, NAN, device="cuda") for n, v in w.items() if v is not None})
    got = ops.m3_qk_norm_rope_backward(x["q"], x["k"], w["q"], w["k"], dq_out=d["q"], dk_out=d["k"], lengths=ilen(lengths), out=out, **how)
    for n in "qk":
        if x[n] is None:
            assert got["d" + n] is None
            continue
        want, mag = (ref.rope(x[n], w[n], lengths=lengths, mag=s, dy=d[n], **how) for s in (False, True))
        close("d" + n, got["d" + n], want["dx"], mag["dx"], 2 * K_ROPE)
        if w[n] is None:
            assert got["d" + n + "_w"] is None
        else:
            close("d" + n + "_w", got["d" + n + "_w"], want["dw"], mag["dw"], K_ROPE + rows * x[n].shape[2])
    again = ops.m3_qk_norm_rope_backward(x["q"], x["k"], w["q"], w["k"], dq_out=d["q"].clone(), dk_out=None if d["k"] is None else d["k"].clone(),
                                         lengths=ilen(lengths), **how)
    for n, v in got.items():
        assert v is None or torch.equal(v, again[n]), n
