"""Layer operators on the GPU against their 64-bit reference (tests/layer_ref.py).

Tolerance of one value: half a step of the output type on the value, plus
k 2^-24 times the magnitude (the sum of the absolute values of the terms), where
k bounds the fp32 roundings on any path from an input to the value; a hardware
exponential, reciprocal or logarithm counts as the few steps its argument's
rounding makes of it.  Rows behind an item's length hold NaN on input, outputs
are filled with NaN (or a marker) before each call.
"""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F32}
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


class Maker:
    """Seeded inputs made on the CPU."""

    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=F32, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=self.g) * scale + shift).to(dtype).cuda()


def wide(t, pad_left=8, pad_right=8):
    """The same values as a slice of wider rows (NaN around them)."""
    lead, width = t.shape[:-1], t.shape[-1]
    big = torch.full((*lead, pad_left + width + pad_right), NAN, dtype=t.dtype, device=t.device)
    big[..., pad_left:pad_left + width] = t
    return big[..., pad_left:pad_left + width]


def spoil(t, lengths):
    """NaN behind the lengths of a [Bt, L, ...] tensor."""
    if lengths is not None:
        for b, n in enumerate(ref.held(lengths, t.shape[0], t.shape[1])):
            t[b, n:] = NAN
    return t


def close(name, got, want, mag, k):
    got = got.detach().cpu()
    assert torch.isfinite(got.double()).all(), f"{name}: not finite"
    tol = HALF[got.dtype] * want.abs() + k * U * mag.abs()
    over = (got.double() - want).abs() - tol
    worst = float(over.max())
    if worst > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}: off by {float((got.double() - want).abs().flatten()[i]):.3e} at {i} (value "
                             f"{float(want.flatten()[i]):.3e}, allowed {float(tol.flatten()[i]):.3e})")


def ilen(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- convolution
# pre: W products and sums; SiLU: the exponential's argument is rounded once (an
# error of |pre| 2^-24 of it), plus exponential, sum, reciprocal and product.
def k_conv(W, pre):
    return 2 * W + 12 + 2 * float(pre.abs().max())


CONV = [
    # Bt, L, D, W, dtype, lengths, state, bias, act, strided
    (1, 1, 8, 4, "bf16", None, True, True, True, False),
    (2, 2, 16, 4, "f32", None, True, True, True, False),
    (3, 77, 64, 4, "bf16", [77, 0, 1], True, True, True, True),
    (2, 300, 24, 3, "f32", [300, 123], False, False, True, False),
    (2, 65, 37, 4, "bf16", [64, 65], True, True, False, True),
    (1, 131, 13, 2, "f32", None, True, True, True, True),
    (4, 33, 520, 4, "bf16", [2, 3, 33, 32], True, True, True, False),
    (2, 64, 1000, 2, "bf16", [-3, 99], True, True, True, False),
]


def _conv_inputs(c, seed):
    Bt, L, D, W, dt, lengths, has_state, has_bias, act, strided = c
    m, t = Maker(seed), DT[dt]
    x = spoil(m(Bt, L, D, dtype=t), lengths)
    w, bias, state = m(D, W, scale=0.5), m(D) if has_bias else None, m(Bt, W - 1, D, dtype=t) if has_state else None
    return (wide(x, *(strided if isinstance(strided, tuple) else ())) if strided else x), w, bias, state, m(Bt, L, D, dtype=t)


@pytest.mark.parametrize("c", CONV, ids=str)
def test_conv(ops, c):
    Bt, L, D, W, dt, lengths, has_state, _, act, _ = c
    x, w, bias, state, _ = _conv_inputs(c, 11)
    y = torch.full((Bt, L, D), 7.0, dtype=x.dtype, device="cuda")
    so = torch.full((Bt, W - 1, D), NAN, dtype=x.dtype, device="cuda")
    ops.m3_causal_conv(x, w, bias, state, lengths=ilen(lengths), silu=act, y=y, state_out=so)
    want = ref.conv(x, w, bias, state, lengths, act)
    mag = ref.conv(x, w, bias, state, lengths, act, mag=True)
    assert torch.equal(so.cpu().double(), want["state"])
    k = k_conv(W, mag["y"])
    for b, n in enumerate(ref.held(lengths, Bt, L)):
        close("y", y[b, :n], want["y"][b, :n], mag["y"][b, :n], k) if n else None
        assert (y[b, n:] == 7).all()
    if state is not None:  # the carry updated in place
        s2 = state.clone()
        ops.m3_causal_conv(x, w, bias, s2, lengths=ilen(lengths), silu=act, state_out=s2)
        assert torch.equal(s2, so)


@pytest.mark.parametrize("c", CONV, ids=str)
def test_conv_backward(ops, c):
    Bt, L, D, W, dt, lengths, has_state, has_bias, act, _ = c
    x, w, bias, state, dy = _conv_inputs(c, 12)
    spoil(dy, lengths)
    t = x.dtype
    out = dict(dx=torch.full((Bt, L, D), NAN, dtype=t, device="cuda"), dw=torch.full((D, W), NAN, device="cuda"),
               dbias=torch.full((D,), NAN, device="cuda"), dstate=torch.full((Bt, W - 1, D), NAN, dtype=t, device="cuda"))
    got = ops.m3_causal_conv_backward(x, w, bias, state, dy=dy, lengths=ilen(lengths), silu=act, out=out)
    want = ref.conv(x, w, bias, state, lengths, act, dy=dy)
    mag = ref.conv(x, w, bias, state, lengths, act, mag=True, dy=dy)
    k = k_conv(W, mag["y"])
    close("dx", got["dx"], want["dx"], mag["dx"], k + W)
    close("dstate", got["dstate"], want["dstate"], mag["dstate"], k + W)
    close("dw", got["dw"], want["dw"], mag["dw"], k + Bt * L)
    if has_bias:
        close("dbias", got["dbias"], want["dbias"], mag["dbias"], k + Bt * L)
    else:
        assert got["dbias"] is None


@pytest.mark.parametrize("Bt,D,W,dt,strided", [(1, 8, 4, "bf16", False), (5, 64, 4, "f32", True), (3, 37, 3, "bf16", True),
                                               (300, 40, 2, "bf16", False)])
def test_conv_step(ops, Bt, D, W, dt, strided):
    m, t = Maker(13), DT[dt]
    state, w, bias = m(Bt, W - 1, D, dtype=t), m(D, W, scale=0.5), m(D)
    xs = m(Bt, 6, D, dtype=t)
    whole = ops.m3_causal_conv(xs, w, bias, state, want_state=True)
    s = state.clone()
    for i in range(6):
        x = wide(xs[:, i]) if strided else xs[:, i].contiguous()
        so = torch.full_like(s, NAN)
        kept = s.clone()
        y2 = ops.m3_causal_conv_step(s, x, w, bias, state_out=so)
        assert torch.equal(s, kept)
        y = ops.m3_causal_conv_step(s, x, w, bias, y=torch.full_like(y2, NAN))
        assert torch.equal(y, y2) and torch.equal(s, so)
        assert torch.equal(y, whole["y"][:, i])  # the same sums in the same order
    assert torch.equal(s, whole["state"])


# ---------------------------------------------------------------- selective scan
# One token multiplies the state by a decay (relative error: that of its argument,
# at most |delta A| (softplus ~4, bias sum, A log2 e, product: 8 in all), plus the
# exponential's and the product's), adds u B (u: softplus, product; 8) and rounds
# the sum; so a path through L tokens has at most L (8 steepest + 4) + 8 roundings,
# the readout N + 3 more, the gate about 12 + 2 |z|.
def k_scan(L, N, steepest, zmax):
    return L * (8 * steepest + 4) + N + 40 + 2 * zmax


SCAN = [
    # Bt, L, D, N, G, dtype, lengths, z, D_skip, h0, softplus, bias, strided
    (1, 1, 8, 16, 1, "bf16", None, True, True, True, True, True, False),
    (2, 37, 64, 16, 1, "bf16", None, True, True, True, True, True, True),
    (3, 70, 48, 4, 1, "f32", [70, 0, 1], True, True, True, True, True, False),
    (2, 33, 40, 8, 2, "bf16", [33, 32], True, False, False, True, False, True),
    (2, 50, 130, 16, 2, "f32", None, False, True, True, False, False, False),
    (1, 100, 37, 24, 1, "bf16", None, True, True, True, True, True, True),
    (2, 45, 36, 32, 3, "f32", [45, 17], True, True, False, True, True, False),
    (1, 64, 20, 64, 1, "bf16", None, True, True, True, True, True, False),
    (2, 31, 6, 13, 2, "f32", [-1, 99], True, True, True, True, True, True),
    (1, 20, 5, 1, 5, "bf16", None, False, False, False, False, False, False),
    (2, 300, 32, 16, 1, "f32", [300, 150], True, True, True, True, True, False),   # two segments of the token axis
    (2, 700, 24, 16, 1, "bf16", [700, 200], True, True, True, True, True, True),   # several, some empty
    (1, 520, 70, 30, 1, "f32", None, True, True, True, True, True, True),
]


def _scan_inputs(c, seed):
    Bt, L, D, N, G, dt, lengths, hz, hd, hh, sp, hb, strided = c
    m, t = Maker(seed), DT[dt]
    q = dict(x=m(Bt, L, D, dtype=t), dt=m(Bt, L, D, dtype=t) if sp else m(Bt, L, D, scale=0.2, shift=0.3, dtype=t).abs(),
             B=m(Bt, L, G * N, dtype=t), C=m(Bt, L, G * N, dtype=t), z=m(Bt, L, D, dtype=t) if hz else None)
    A = -torch.exp(torch.rand(D, N, generator=m.g) * 2.77).cuda()
    q = {k: None if v is None else spoil(v, lengths) for k, v in q.items()}
    if strided:
        q = {k: None if v is None else wide(v, *(strided if isinstance(strided, tuple) else ())) for k, v in q.items()}
    q["B"], q["C"] = q["B"].unflatten(-1, (G, N)), q["C"].unflatten(-1, (G, N))
    q.update(A=A, D=m(D) if hd else None, h0=m(Bt, D, N, scale=0.5) if hh else None, dt_bias=m(D, shift=-3.0) if hb else None)
    return q, m


def _scan_call(q, sp):
    return (q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["z"], q["h0"]), dict(dt_softplus=sp, dt_bias=q["dt_bias"])


def _zmax(z):
    return 0.0 if z is None else float(torch.nan_to_num(z.float()).abs().max())


@pytest.mark.parametrize("c", SCAN, ids=str)
def test_scan(ops, c):
    Bt, L, D, N, G, dt, lengths, *_, sp, _, _ = c
    q, m = _scan_inputs(c, 21)
    args, kw = _scan_call(q, sp)
    y = torch.full((Bt, L, D), 7.0, dtype=q["x"].dtype, device="cuda")
    h = torch.full((Bt, D, N), NAN, device="cuda")
    ops.m3_selective_scan(*args, lengths=ilen(lengths), y=y, h_final=h, **kw)
    want = ref.scan(**q, lengths=lengths, dt_softplus=sp)
    mag = ref.scan(**q, lengths=lengths, dt_softplus=sp, mag=True, dy=torch.zeros(Bt, L, D))
    k = k_scan(L, N, mag["steepest"], _zmax(q["z"]))
    close("h", h, want["h"], mag["h"], k)
    for b, n in enumerate(ref.held(lengths, Bt, L)):
        close("y", y[b, :n], want["y"][b, :n], mag["y"][b, :n], k) if n else None
        assert (y[b, n:] == 7).all()
    # without a workspace the token axis is not cut; the same to rounding
    r = ops.m3_selective_scan(*args, lengths=ilen(lengths), workspace=False, **kw)
    close("h, uncut", r["h"], want["h"], mag["h"], k)


@pytest.mark.parametrize("c", SCAN, ids=str)
def test_scan_backward(ops, c):
    Bt, L, D, N, G, dt, lengths, *_, sp, _, _ = c
    q, m = _scan_inputs(c, 22)
    t = q["x"].dtype
    dy, dhf = spoil(m(Bt, L, D, dtype=t), lengths), m(Bt, D, N) if L % 2 == 0 else None
    args, kw = _scan_call(q, sp)
    full = lambda *s, dtype=F32: torch.full(s, NAN, dtype=dtype, device="cuda")  # noqa: E731
    out = dict(dx=full(Bt, L, D, dtype=t), ddt=full(Bt, L, D, dtype=t), dA=full(D, N), dB=full(Bt, L, G, N, dtype=t),
               dC=full(Bt, L, G, N, dtype=t), dD=full(D), dz=full(Bt, L, D, dtype=t), ddt_bias=full(D), dh0=full(Bt, D, N))
    got = ops.m3_selective_scan_backward(*args, dy=dy, dh_final=dhf, lengths=ilen(lengths), out=out, **kw)
    want = ref.scan(**q, lengths=lengths, dt_softplus=sp, dy=dy, dh_final=dhf)
    mag = ref.scan(**q, lengths=lengths, dt_softplus=sp, dy=dy, dh_final=dhf, mag=True)
    # forward and reverse paths, then the sums over channels or over items and tokens
    k = 2 * k_scan(L, N, mag["steepest"], _zmax(q["z"]))
    for name, extra in (("dz", 0), ("dx", N), ("ddt", 2 * N + 16), ("dB", D), ("dC", D), ("dh0", 0), ("dA", Bt * L), ("dD", Bt * L),
                        ("ddt_bias", Bt * L + 2 * N)):
        if want[name] is None:
            assert got[name] is None, name
        else:
            close(name, got[name], want[name], mag[name], k + extra)


@pytest.mark.parametrize("Bt,D,N,G,dt,strided", [(1, 8, 16, 1, "bf16", False), (5, 64, 16, 2, "f32", True), (3, 37, 4, 1, "bf16", True),
                                                 (2, 30, 24, 1, "bf16", False), (7, 12, 64, 3, "f32", False), (2, 9, 13, 1, "bf16", True),
                                                 (300, 33, 8, 1, "bf16", False), (2, 6, 1, 2, "f32", False)])
def test_scan_step(ops, Bt, D, N, G, dt, strided):
    m, t, T = Maker(23), DT[dt], 5
    q, m = _scan_inputs((Bt, T, D, N, G, dt, None, True, True, True, True, True, False), 23)
    args, kw = _scan_call(q, True)
    whole = ref.scan(**q, dt_softplus=True)
    mag = ref.scan(**q, dt_softplus=True, mag=True, dy=torch.zeros(Bt, T, D))
    k = k_scan(T, N, mag["steepest"], _zmax(q["z"]))
    h = q["h0"].clone()
    for i in range(T):
        tok = {n: q[n][:, i] for n in ("x", "dt", "B", "C", "z")}
        if strided:
            tok = {n: (wide(v) if v.dim() == 2 else wide(v.flatten(1)).unflatten(-1, (G, N))) for n, v in tok.items()}
        else:
            tok = {n: v.contiguous() for n, v in tok.items()}
        call = (tok["x"], tok["dt"], q["A"], tok["B"], tok["C"], q["D"], tok["z"])
        kept, ho = h.clone(), torch.full_like(h, NAN)
        y2 = ops.m3_selective_scan_step(h, *call, h_out=ho, **kw)
        assert torch.equal(h, kept)
        y = ops.m3_selective_scan_step(h, *call, y=torch.full_like(y2, NAN), **kw)
        assert torch.equal(y, y2) and torch.equal(h, ho)
        close(f"y[{i}]", y, whole["y"][:, i], mag["y"][:, i], k)
    close("h", h, whole["h"], mag["h"], k)


# ---------------------------------------------------------------- norms
# The mean of squares: width roundings of one sign, so width / 2 on the root; the
# gate 12 + 2 |z|; a handful for the rest.
GATED = [
    # shape, groups, dtype, gate_first, z, w, strided
    ((1, 8), 1, "bf16", True, True, True, False),
    ((3, 5, 64), 4, "bf16", True, True, True, True),
    ((7, 37), 1, "f32", False, True, True, False),
    ((2500, 96), 3, "bf16", False, True, True, True),
    ((5, 1000), 1, "f32", True, True, False, False),
    ((9, 2048), 8, "bf16", True, False, True, True),
    ((3000, 1024), 1, "bf16", False, True, True, False),
    ((2200, 1040), 1, "bf16", True, True, True, False),
    ((4, 5000), 1, "bf16", True, True, True, False),
    ((3, 20008), 1, "f32", False, True, True, False),
    ((2, 40001), 1, "bf16", True, True, True, False),
    ((2, 36002), 1, "f32", False, True, True, True),
    ((5, 8192), 1, "f32", True, True, True, False),
    ((270, 6000), 1, "f32", False, False, True, True),
    ((300, 8448), 1, "bf16", False, True, True, False),
    ((5, 16384), 1, "bf16", True, True, False, True),
]


@pytest.mark.parametrize("c", GATED, ids=str)
def test_gated_norm(ops, c):
    shape, groups, dt, first, hz, hw, strided = c
    m, t = Maker(31), DT[dt]
    x, z, w, dy = m(*shape, dtype=t), m(*shape, dtype=t) if hz else None, m(shape[-1]) if hw else None, m(*shape, dtype=t)
    if strided:
        x, z = wide(x), wide(z) if hz else None
    kw = dict(groups=groups, eps=1e-5, gate_first=first)
    want = ref.gated_norm(x, z, w, dy=dy, **kw)
    mag = ref.gated_norm(x, z, w, dy=dy, mag=True, **kw)
    k = shape[-1] // groups + 40 + 4 * _zmax(z)
    y = ops.m3_gated_norm(x, z, w, y=torch.full(shape, NAN, dtype=t, device="cuda"), **kw)
    close("y", y, want["y"], mag["y"], k)
    out = dict(dx=torch.full(shape, NAN, dtype=t, device="cuda"), dz=torch.full(shape, NAN, dtype=t, device="cuda"),
               dw=torch.full((shape[-1],), NAN, device="cuda"))
    got = ops.m3_gated_norm_backward(x, z, w, dy=dy, out=out, **kw)
    rows = x.numel() // shape[-1]
    close("dx", got["dx"], want["dx"], mag["dx"], 2 * k)
    if hz:
        close("dz", got["dz"], want["dz"], mag["dz"], 2 * k)
    if hw:
        close("dw", got["dw"], want["dw"], mag["dw"], k + rows)
    if not strided:  # in place
        for which in (0, 1) if hz else (0,):
            q = [x.clone(), z.clone() if hz else None]
            assert torch.equal(ops.m3_gated_norm(q[0], q[1], w, y=q[which], **kw), y)


RESIDUAL = [
    # shape, dtype, residual type (None: no residual), scale, w, strided
    ((1, 8), "bf16", "f32", True, True, False),
    ((3, 5, 64), "bf16", "bf16", False, True, True),
    ((7, 37), "f32", "f32", True, True, False),
    ((2500, 96), "bf16", "f32", True, False, True),
    ((5, 1000), "bf16", "bf16", True, True, False),
    ((3000, 2048), "bf16", "f32", False, True, False),
    ((9, 2048), "bf16", None, True, True, False),
    ((2100, 1000), "f32", "f32", True, True, True),
    ((4, 8200), "bf16", "bf16", True, True, False),
    ((3, 40001), "bf16", "f32", True, True, True),
    ((270, 8192), "f32", "f32", True, True, False),
    ((300, 8448), "bf16", "bf16", False, True, True),
    ((5, 16384), "bf16", "f32", True, True, False),
]


@pytest.mark.parametrize("c", RESIDUAL, ids=str)
def test_residual_norm(ops, c):
    shape, dt, rdt, hs, hw, strided = c
    m, t = Maker(41), DT[dt]
    rt = DT[rdt] if rdt else t
    x, res = m(*shape, dtype=t), m(*shape, dtype=rt) if rdt else None
    w, scale = m(shape[-1]) if hw else None, m(shape[-1]) if hs else None
    dy, dr = m(*shape, dtype=t), m(*shape, dtype=rt) if rdt else None
    if strided:
        x = wide(x)
    kw = dict(eps=1e-5)
    want = ref.residual_norm(x, res, w, scale, **kw)
    mag = ref.residual_norm(x, res, w, scale, mag=True, **kw)
    k = shape[-1] + 20
    got = ops.m3_residual_norm(x, res, w, scale, y=torch.full(shape, NAN, dtype=t, device="cuda"),
                               residual_out=torch.full(shape, NAN, dtype=rt, device="cuda"), **kw)
    close("residual", got["residual"], want["residual"], mag["residual"], 2)
    close("y", got["y"], want["y"], mag["y"], k)
    if res is not None:  # the residual stream updated in place
        r2 = res.clone()
        g2 = ops.m3_residual_norm(x, r2, w, scale, residual_out=r2, **kw)
        assert torch.equal(r2, got["residual"]) and torch.equal(g2["y"], got["y"])
    h = got["residual"]
    want = ref.residual_norm_backward(h, x, w, scale, dy, dr, **kw)
    mag = ref.residual_norm_backward(h, x, w, scale, dy, dr, mag=True, **kw)
    out = dict(dresidual=torch.full(shape, NAN, dtype=rt, device="cuda"), dx=torch.full(shape, NAN, dtype=t, device="cuda"))
    bw = ops.m3_residual_norm_backward(h, x, w, scale, dy=dy, dresidual=dr, out=out, **kw)
    rows = x.numel() // shape[-1]
    for name, extra in (("dresidual", 0), ("dx", 0), ("dw", rows), ("dscale", rows)):
        if want[name] is None:
            assert bw[name] is None
        else:
            close(name, bw[name], want[name], mag[name], 2 * k + extra)
    if dr is not None:  # the gradient of the residual stream updated in place
        d2 = dr.clone()
        b2 = ops.m3_residual_norm_backward(h, x, w, scale, dy=dy, dresidual=d2, out=dict(dresidual=d2), **kw)
        assert torch.equal(d2, bw["dresidual"]) and torch.equal(b2["dx"], bw["dx"])


# Widths that end inside a 16-byte word and rows off its alignment, at each way that
# units are dealt to lanes.
UNALIGNED = [(2100, 9, 1), (2500, 49, 1), (2100, 515, 1), (2100, 1030, 1), (30, 1041, 3), (5, 2051, 1), (5, 4099, 1),
             (5, 6001, 1), (4, 8209, 1), (70, 1024, 2)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,groups", UNALIGNED)
def test_norms_off_alignment(ops, M, D, groups, dt):
    for first in (True, False):
        test_gated_norm(ops, ((M, D), groups, dt, first, True, True, False))
    test_residual_norm(ops, ((M, D), dt, "f32", True, True, False))
    test_residual_norm(ops, ((M, D), dt, dt, False, True, False))
    # one element off: rows, residual, gate, gain and outputs at odd addresses
    m, t = Maker(43), DT[dt]
    x, z, res, w, scale, dy = m(M, D, dtype=t), m(M, D, dtype=t), m(M, D, dtype=t), m(D), m(D), m(M, D, dtype=t)

    def off(v):
        o = torch.full((v.numel() + 1,), NAN, dtype=v.dtype, device="cuda")[1:].view(v.shape)
        return o.copy_(v)

    kw, k = dict(groups=groups, eps=1e-5), D // groups + 40 + 4 * _zmax(z)
    want, mag = ref.gated_norm(x, z, w, dy=dy, **kw), ref.gated_norm(x, z, w, dy=dy, mag=True, **kw)
    xs, zs = wide(x, 1, 2), wide(z, 3, 2)
    close("y", ops.m3_gated_norm(xs, zs, off(w), y=off(x), **kw), want["y"], mag["y"], k)
    got = ops.m3_gated_norm_backward(xs, zs, off(w), dy=off(dy), out=dict(dx=off(x), dz=off(x), dw=off(w)), **kw)
    for name, extra in (("dx", k), ("dz", k), ("dw", M)):
        close(name, got[name], want[name], mag[name], k + extra)
    want, mag = ref.residual_norm(x, res, w, scale, eps=1e-5), ref.residual_norm(x, res, w, scale, eps=1e-5, mag=True)
    got = ops.m3_residual_norm(xs, off(res), off(w), off(scale), y=off(x), residual_out=off(x), eps=1e-5)
    close("residual", got["residual"], want["residual"], mag["residual"], 2)
    close("y", got["y"], want["y"], mag["y"], D + 20)
    h, dr = off(got["residual"]), off(m(M, D, dtype=t))
    want, mag = (ref.residual_norm_backward(h, x, w, scale, dy, dr, eps=1e-5, mag=q) for q in (False, True))
    bw = ops.m3_residual_norm_backward(h, xs, off(w), off(scale), dy=off(dy), dresidual=dr, eps=1e-5,
                                       out=dict(dx=off(x), dresidual=off(x), dw=off(w), dscale=off(w)))
    for name, extra in (("dresidual", 0), ("dx", 0), ("dw", M), ("dscale", M)):
        close(name, bw[name], want[name], mag[name], 2 * (D + 20) + extra)


@pytest.mark.parametrize("at", [0, 1021, 1022, 1023, 1029])
def test_infinity_in_a_shared_word(ops, at):
    """A row of 1030 ends in a word that shares two elements with the one before: an
    infinity there counts once, so the row's other outputs are zeros, not NaN."""
    x = Maker(44)(3, 1030, dtype=torch.bfloat16)
    x[1, at] = float("inf")
    y = ops.m3_gated_norm(x)
    r = ops.m3_residual_norm(x)["y"]
    for o in (y, r):
        keep = torch.arange(1030, device="cuda") != at
        assert (o[1, keep] == 0).all() and o[1, at].isnan()
        assert o[0].isfinite().all() and o[2].isfinite().all() and (o[0] != 0).any()


# Widths that leave one, two or three channels of a word, and fewer than one, in every
# block of channels (64, 32 and 16 of them); state sizes that end inside a word; rows
# an element or two off a word.
SCAN_OFF = [(D, N, G, dt, off) for D, N, G, dt, off in [
    (65, 16, 1, "bf16", (1, 2)), (66, 15, 1, "f32", (2, 1)), (67, 14, 1, "bf16", False), (71, 13, 1, "f32", False), (5, 4, 1, "bf16", (3, 0)),
    (4, 5, 1, "f32", (1, 0)), (33, 17, 1, "bf16", (1, 2)), (35, 31, 1, "f32", False), (38, 30, 2, "bf16", (1, 1)), (17, 33, 1, "f32", (1, 0)),
    (18, 62, 1, "bf16", False), (19, 63, 1, "f32", (1, 1)), (21, 61, 3, "bf16", (5, 2)), (64, 16, 1, "bf16", (1, 0)), (64, 16, 2, "f32", (1, 3)),
    (72, 12, 1, "bf16", False), (65, 9, 1, "f32", (1, 0)), (40, 24, 2, "bf16", False), (33, 20, 1, "f32", (1, 1)),
    (36, 48, 1, "f32", False), (18, 40, 2, "bf16", (2, 1)), (48, 8, 1, "bf16", False), (40, 7, 1, "f32", (1, 0)), (130, 6, 2, "bf16", (1, 1)), (3, 16, 1, "bf16", (1, 0)), (64, 3, 1, "f32", (1, 0)), (1, 1, 1, "bf16", False), (2, 2, 1, "f32", (1, 0))]]


@pytest.mark.parametrize("D,N,G,dt,off", SCAN_OFF)
def test_scans_off_alignment(ops, D, N, G, dt, off):
    for Bt, L, lengths in ((1, 1, None), (2, 65, [65, 34]), (1, 290, None)):
        c = (Bt, L, D, N, G, dt, lengths, True, True, True, True, True, off)
        test_scan(ops, c)
        test_scan_backward(ops, c)


# Widths around one word, that end inside one, and in the second block of columns; rows
# an element or more off a word.
CONV_OFF = [(D, W, dt, off) for D, W, dt, off in [
    (3, 4, "bf16", (1, 0)), (4, 2, "f32", (1, 0)), (5, 3, "f32", False), (7, 4, "bf16", False), (8, 4, "bf16", (1, 1)), (9, 4, "bf16", False),
    (15, 3, "bf16", (3, 2)), (39, 2, "bf16", False), (66, 4, "f32", (1, 0)), (257, 4, "f32", False), (513, 4, "bf16", (2, 1)), (1030, 3, "bf16", False)]]


@pytest.mark.parametrize("D,W,dt,off", CONV_OFF)
def test_conv_off_alignment(ops, D, W, dt, off):
    for Bt, L, lengths in ((1, 1, None), (2, 2, None), (3, 67, [67, 0, 2]), (1, 300, None)):
        c = (Bt, L, D, W, dt, lengths, True, True, True, off)
        test_conv(ops, c)
        test_conv_backward(ops, c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shared_words_repeat(ops, dt):
    """Channels that two words share are written twice with the same value: every call
    gives the same bits, eager and replayed from a graph."""
    m, t = Maker(45), DT[dt]
    Bt, L, D, N = 3, 70, 1031, 11
    x, z, dy, dl, C, B = (m(Bt, L, n, dtype=t) for n in (D, D, D, D, N, N))
    B, C = B.unflatten(-1, (1, N)), C.unflatten(-1, (1, N))
    w, b, gain, A = m(D, 4, scale=0.5), m(D), m(D), -torch.exp(m(D, N))

    def calls():
        y = ops.m3_causal_conv(x, w, b)["y"]
        s = ops.m3_selective_scan(y, dl, A, B, C, gain, z, dt_softplus=True, dt_bias=b)
        n = ops.m3_gated_norm(s["y"], z, gain)
        r = ops.m3_residual_norm(n, x, gain)
        g = ops.m3_residual_norm_backward(r["residual"], w=gain, dy=dy)
        q = ops.m3_gated_norm_backward(s["y"], z, gain, dy=g["dx"])
        u = ops.m3_selective_scan_backward(y, dl, A, B, C, gain, z, dy=q["dx"], dt_softplus=True, dt_bias=b)
        v = ops.m3_causal_conv_backward(x, w, b, dy=u["dx"])
        return [y, n] + [o for d in (s, r, g, q, u, v) for o in d.values() if o is not None]

    first = calls()
    assert all(torch.equal(p, q) for _ in range(3) for p, q in zip(first, calls()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = calls()
    for _ in range(3):
        for o in held:
            o.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, held))
        assert all(torch.equal(p, q) for p, q in zip(first, calls()))
