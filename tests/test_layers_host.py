"""Layer operators without a GPU: the 64-bit reference's gradients against
automatic differentiation and differences, and the refusals of the C ABI and of
the torch binding."""
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from state_space_sequence_ssm_amd import _lib  # noqa: E402
from tests import layer_ref as ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_SAN_LIB = os.environ.get("M3SSM_HOSTSAN_LIB")
if _SAN_LIB:
    _lib.load(_SAN_LIB)

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libm3ssm.so not built (run __graft_entry__.build())")
F64 = torch.float64
INV, UNS = _lib.M3_ERR_INVALID_ARG, _lib.M3_ERR_UNSUPPORTED


def _rand(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=F64) * scale


# ---------------------------------------------------------------- the reference itself
@pytest.mark.parametrize("lengths", [None, [5, 0, 1]])
def test_reference_conv_gradients(lengths):
    Bt, L, D, W = 3, 7, 4, 4
    ins = [_rand(Bt, L, D, seed=1), _rand(D, W, seed=2), _rand(D, seed=3), _rand(Bt, W - 1, D, seed=4)]
    dy = _rand(Bt, L, D, seed=5)
    leaves = [t.clone().requires_grad_() for t in ins]
    x, w, bias, state = leaves
    ys = []
    for b, n in enumerate(ref.held(lengths, Bt, L)):
        xs = torch.cat([state[b], x[b, :n]])
        pre = bias + sum(w[:, k] * xs[k:k + n] for k in range(W))
        ys.append((dy[b, :n] * torch.nn.functional.silu(pre)).sum())
    sum(ys).backward()
    got = ref.conv(*ins, lengths=lengths, dy=dy)
    for k, leaf in zip(("dx", "dw", "dbias", "dstate"), leaves):
        assert torch.allclose(got[k], leaf.grad, rtol=1e-12, atol=1e-13), k


def _scan_case(Bt=2, L=6, D=6, N=3, G=2):
    return dict(x=_rand(Bt, L, D, seed=1), dt=_rand(Bt, L, D, seed=2), A=-_rand(D, N, seed=3).abs(), B=_rand(Bt, L, G, N, seed=4),
                C=_rand(Bt, L, G, N, seed=5), D=_rand(D, seed=6), z=_rand(Bt, L, D, seed=7), h0=_rand(Bt, D, N, seed=8),
                dt_bias=_rand(D, seed=9))


@pytest.mark.parametrize("lengths", [None, [6, 1], [0, 4]])
def test_reference_scan_gradients(lengths):
    c = _scan_case()
    dy, dhf = _rand(2, 6, 6, seed=10), _rand(2, 6, 3, seed=11)
    lv = {k: v.clone().requires_grad_() for k, v in c.items()}
    per = 3
    delta = torch.nn.functional.softplus(lv["dt"] + lv["dt_bias"])
    loss = 0.0
    for b, n in enumerate(ref.held(lengths, 2, 6)):
        h = lv["h0"][b]
        for t in range(n):
            Bw, Cw = lv["B"][b, t].repeat_interleave(per, 0), lv["C"][b, t].repeat_interleave(per, 0)
            h = torch.exp(delta[b, t][:, None] * lv["A"]) * h + (delta[b, t] * lv["x"][b, t])[:, None] * Bw
            y = ((h * Cw).sum(-1) + lv["D"] * lv["x"][b, t]) * torch.nn.functional.silu(lv["z"][b, t])
            loss = loss + (dy[b, t] * y).sum()
        loss = loss + (dhf[b] * h).sum()
    loss.backward()
    got = ref.scan(**c, lengths=lengths, dt_softplus=True, dy=dy, dh_final=dhf)
    for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"):
        assert torch.allclose(got["d" + k], lv[k].grad, rtol=1e-11, atol=1e-12), k


def test_reference_scan_against_differences():
    c = _scan_case()
    dy, dhf = _rand(2, 6, 6, seed=10), _rand(2, 6, 3, seed=11)
    got = ref.scan(**c, dt_softplus=True, dy=dy, dh_final=dhf)

    def loss(q):
        o = ref.scan(**q, dt_softplus=True)
        return float((o["y"] * dy).sum() + (o["h"] * dhf).sum())

    for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"):
        step = _rand(*c[k].shape, seed=20)
        e = 1e-5
        up, down = (loss({**c, k: c[k] + s * e * step}) for s in (1, -1))
        want = float((got["d" + k] * step).sum())
        assert abs((up - down) / (2 * e) - want) <= 1e-6 * (1 + abs(want)), k


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("groups", [1, 3])
def test_reference_gated_norm_gradients(gate_first, groups):
    x, z, w, dy = _rand(5, 12, seed=1), _rand(5, 12, seed=2), _rand(12, seed=3), _rand(5, 12, seed=4)
    lv = [t.clone().requires_grad_() for t in (x, z, w)]
    gate = torch.nn.functional.silu(lv[1])
    v = (lv[0] * gate if gate_first else lv[0]).view(5, groups, -1)
    n = (v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()).reshape(5, 12) * lv[2]
    ((n if gate_first else n * gate) * dy).sum().backward()
    got = ref.gated_norm(x, z, w, groups, 1e-6, gate_first, dy=dy)
    for k, leaf in zip(("dx", "dz", "dw"), lv):
        assert torch.allclose(got[k], leaf.grad, rtol=1e-11, atol=1e-12), k


def test_reference_residual_norm_gradients():
    x, res, w, s = _rand(5, 12, seed=1), _rand(5, 12, seed=2), _rand(12, seed=3), _rand(12, seed=4)
    dy, dr = _rand(5, 12, seed=5), _rand(5, 12, seed=6)
    lv = [t.clone().requires_grad_() for t in (x, res, w, s)]
    h = lv[1] + lv[3] * lv[0]
    n = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * lv[2]
    ((n * dy).sum() + (h * dr).sum()).backward()
    got = ref.residual_norm_backward(res + s * x, x, w, s, dy, dr)
    for k, leaf in zip(("dx", "dresidual", "dw", "dscale"), lv):
        assert torch.allclose(got[k], leaf.grad, rtol=1e-11, atol=1e-12), k


# ---------------------------------------------------------------- refusals of the C ABI
BASE = 0x10000000


def _fill(a, names, start=0):
    for i, f in enumerate(names):
        setattr(a, f, BASE + 0x100000 * (i + start))
    return a


def _conv():
    a = _fill(_lib.ConvArgs(), ("x", "w", "bias", "lengths", "state", "y", "state_out"))
    a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu = 2, 9, 16, 4, _lib.M3_BF16, 1
    return a


def _conv_step():
    a = _fill(_lib.ConvStepArgs(), ("x", "w", "bias", "state", "state_out", "y"))
    a.Bt, a.D, a.W, a.in_dtype, a.silu = 2, 16, 4, _lib.M3_BF16, 1
    return a


def _conv_bw():
    a = _fill(_lib.ConvBackwardArgs(), ("x", "w", "bias", "lengths", "state", "dy", "dx", "dw", "dbias", "dstate", "workspace"))
    a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu = 2, 9, 16, 4, _lib.M3_BF16, 1
    a.workspace_bytes = 1 << 30
    return a


def _scan_fields(a, extra):
    _fill(a, ("x", "dt", "A", "B", "C", "D_skip", "z", "dt_bias", *extra))
    a.Bt, a.D, a.N, a.G, a.in_dtype, a.dt_softplus = 2, 16, 16, 2, _lib.M3_BF16, 1
    return a


def _scan():
    a = _scan_fields(_lib.ScanArgs(), ("h0", "lengths", "y", "h_final", "workspace"))
    a.L, a.workspace_bytes = 9, 1 << 30
    return a


def _scan_step():
    return _scan_fields(_lib.ScanStepArgs(), ("h", "h_out", "y"))


def _scan_bw():
    a = _lib.ScanBackwardArgs()
    f = _scan_fields(a.fwd, ("h0", "lengths"))
    f.L = 9
    _fill(a, ("dy", "dh_final", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0", "workspace"), 20)
    a.workspace_bytes = 1 << 30
    return a


def _gated():
    a = _fill(_lib.GatedNormArgs(), ("x", "z", "w", "y"))
    a.M, a.D, a.G, a.in_dtype, a.gate_first, a.eps = 5, 16, 2, _lib.M3_BF16, 1, 1e-6
    return a


def _gated_bw():
    a = _lib.GatedNormBackwardArgs()
    f = _fill(a.fwd, ("x", "z", "w"))
    f.M, f.D, f.G, f.in_dtype, f.gate_first, f.eps = 5, 16, 2, _lib.M3_BF16, 1, 1e-6
    _fill(a, ("dy", "dx", "dz", "dw", "workspace"), 20)
    a.workspace_bytes = 1 << 30
    return a


def _residual():
    a = _fill(_lib.ResidualNormArgs(), ("x", "residual", "scale", "w", "y", "residual_out"))
    a.M, a.D, a.in_dtype, a.res_dtype, a.eps = 5, 16, _lib.M3_BF16, _lib.M3_F32, 1e-6
    return a


def _residual_bw():
    a = _fill(_lib.ResidualNormBackwardArgs(), ("h", "x", "scale", "w", "dy", "dresidual_out", "dx", "dresidual", "dw", "dscale",
                                                "workspace"))
    a.M, a.D, a.in_dtype, a.res_dtype, a.eps, a.workspace_bytes = 5, 16, _lib.M3_BF16, _lib.M3_F32, 1e-6, 1 << 30
    return a


MAKE = {"m3_causal_conv": _conv, "m3_causal_conv_step": _conv_step, "m3_causal_conv_backward": _conv_bw,
        "m3_selective_scan": _scan, "m3_selective_scan_step": _scan_step, "m3_selective_scan_backward": _scan_bw,
        "m3_gated_norm": _gated, "m3_gated_norm_backward": _gated_bw, "m3_residual_norm": _residual,
        "m3_residual_norm_backward": _residual_bw}


def _set(path, value):
    def change(a):
        *front, last = path.split(".")
        for f in front:
            a = getattr(a, f)
        setattr(a, last, getattr(a, value[1:]) if isinstance(value, str) else value)
    change.__name__ = f"{path}={value}"
    return change


def _bad(name):
    """(field, value, code): one refused argument each; "=f" takes field f's value."""
    f = "fwd." if name in ("m3_selective_scan_backward", "m3_gated_norm_backward") else ""
    out = [(f + "in_dtype", 7, UNS), (f + "D", 0, INV), (f + "x", None, INV) if name != "m3_residual_norm_backward" else ("h", None, INV),
           (f + "x", BASE + 1, INV), (f + "x_ld", 8, INV), (f + "x_ld", -16, INV)]
    if "norm" in name:
        out += [(f + "M", 0, INV), (f + "eps", -1.0, INV), (f + "eps", float("nan"), INV), (f + "M", 1 << 40, UNS)]
    else:
        out += [(f + "Bt", 0, INV), (f + "Bt", 1 << 30, UNS)]
        if "step" not in name:
            out += [(f + "L", 0, INV), (f + "lengths", BASE + 2, INV)]
    if "conv" in name:
        out += [("W", 1, UNS), ("W", 5, UNS), ("silu", 2, INV), ("w", None, INV), ("w", BASE + 2, INV)]
    if "scan" in name:
        out += [(f + "N", 0, INV), (f + "N", 65, UNS), (f + "G", 3, INV), (f + "G", 0, INV), (f + "dt_softplus", 3, INV),
                (f + "dt_softplus", 0, INV), (f + "A", None, INV), (f + "B", None, INV), (f + "B_ld", 31, INV), (f + "C", BASE + 1, INV)]
    if "gated" in name:
        out += [(f + "G", 3, INV), (f + "gate_first", 2, INV)]
    if "scan" in name:
        out += [(f + "x_ld", 1 << 24, INV), (f + "C_ld", 1 << 24, INV)]
    if "residual" in name:
        out += [("res_dtype", 5, UNS)]
    if name.endswith("backward"):
        out += [("dy", None, INV), ("workspace", None, INV), ("workspace", BASE + 0x100000 * 40 + 64, INV), ("workspace_bytes", 16, INV)]
        out += [("dx", "=dy", INV)]
        out += [("dw" if "scan" not in name else "dA", None, INV)]
    elif "step" not in name:
        out += [("y", None, INV), ("y", "=w" if "scan" not in name else "=A", INV)]
    if name == "m3_selective_scan":
        out += [("workspace_bytes", -1, None), ("h_final", "=h0", INV), ("y", "=x", INV), ("workspace", BASE + 8, INV)]
    if name == "m3_selective_scan_backward":
        out += [("dD", None, INV), ("dz", None, INV), ("ddt_bias", None, INV), ("fwd.z", None, INV), ("dB", "=dC", INV)]
    if name == "m3_selective_scan_step":
        out += [("h", None, INV), ("y", "=h", INV), ("h_out", "=A", INV)]
    if name == "m3_causal_conv_step":
        out += [("state", None, INV), ("y", "=state", INV), ("state_out", "=x", INV)]
    if name == "m3_causal_conv":
        out += [("y", "=state", INV), ("y", "=x", INV), ("state_out", "=y", INV)]
    if name == "m3_gated_norm_backward":
        out += [("dz", None, INV), ("fwd.z", None, INV), ("fwd.w", None, INV)]
    if name == "m3_gated_norm":
        out += [("y", "=w", INV)]
    if name == "m3_residual_norm_backward":
        out += [("x", None, INV), ("dscale", None, INV), ("dx", "=dresidual_out", INV), ("dresidual", "=h", INV)]
    if name == "m3_residual_norm":
        out += [("y", "=residual", INV), ("residual_out", "=x", INV)]
    return [c for c in out if c[2] is not None]


@built
@pytest.mark.parametrize("name", list(MAKE))
def test_layer_refusals(name):
    fn = getattr(_lib.load(), name)
    assert fn(None, None) == INV
    for path, value, code in _bad(name):
        a = MAKE[name]()
        _set(path, value)(a)
        assert fn(ctypes.byref(a), None) == code, (path, value)


@built
def test_gated_norm_in_place_needs_dense_rows():
    for src in ("x", "z"):
        a = _gated()
        a.y = getattr(a, src)
        setattr(a, src + "_ld", 32)
        assert _lib.load().m3_gated_norm(ctypes.byref(a), None) == INV


@built
def test_gated_norm_group_limit():
    a = _gated()
    a.D = a.G = 1 << 21
    a.M = 1
    assert _lib.load().m3_gated_norm(ctypes.byref(a), None) == UNS


@built
def test_layer_workspace_sizes():
    lib = _lib.load()
    for name in _lib.LAYER_SIZES:
        assert getattr(lib, name)(None) == 0
    a = _scan()
    assert lib.m3_selective_scan_workspace_size(ctypes.byref(a)) == 0  # 9 tokens: not cut
    a.L = 4096
    need = lib.m3_selective_scan_workspace_size(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    a.N = 65
    assert lib.m3_selective_scan_workspace_size(ctypes.byref(a)) == 0
    for name, make in (("m3_causal_conv_backward", _conv_bw), ("m3_selective_scan_backward", _scan_bw),
                       ("m3_gated_norm_backward", _gated_bw), ("m3_residual_norm_backward", _residual_bw)):
        a = make()
        need = getattr(lib, name + "_workspace_size")(ctypes.byref(a))
        assert need > 0 and need % 256 == 0
        a.workspace_bytes = need - 1
        assert getattr(lib, name)(ctypes.byref(a), None) == INV, name


@pytest.mark.skipif(bool(_SAN_LIB), reason="already the sanitized run")
@built
def test_layer_validation_under_host_sanitizers():
    from state_space_sequence_ssm_amd import build as b
    try:
        lib, rt = b.build_hostsan(), b.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    env = dict(os.environ, LD_PRELOAD=rt, M3SSM_HOSTSAN_LIB=lib, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__), "-k",
                        "refusals or dense_rows or workspace_sizes or group_limit"], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


# ---------------------------------------------------------------- refusals of the torch binding
@built
def test_binding_refuses_host_tensors():
    from state_space_sequence_ssm_amd import ops
    x = torch.zeros(1, 4, 8)
    for call in (lambda: ops.m3_causal_conv(x, torch.zeros(8, 4)), lambda: ops.m3_gated_norm(x),
                 lambda: ops.m3_residual_norm(x), lambda: ops.m3_selective_scan(x, x, torch.zeros(8, 4), x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ops.m3_gated_norm(None)


@built
def test_row_distances():
    from state_space_sequence_ssm_amd import ops
    cpu, f = -1, torch.float32  # the device index of a host tensor
    rows = lambda t, lead, inner: ops._rows(t, f, (*lead, *inner), len(lead), "t", cpu)[1]  # noqa: E731
    wide = torch.zeros(2, 5, 24)
    assert rows(torch.zeros(2, 5, 8), (2, 5), (8,)) == 0
    assert rows(wide[..., 8:16], (2, 5), (8,)) == 24
    assert rows(wide[:1, :, :8], (1, 5), (8,)) == 24
    assert rows(wide[:, :1, :8], (2, 1), (8,)) == 120
    assert rows(wide[..., :12].unflatten(-1, (3, 4)), (2, 5), (3, 4)) == 24
    for bad, lead, inner in ((wide[:, :4, :8], (2, 4), (8,)), (wide[..., ::3], (2, 5), (8,)),
                             (torch.zeros(8).expand(2, 5, 8), (2, 5), (8,)), (torch.zeros(2, 8, 5).transpose(1, 2), (2, 5), (8,))):
        with pytest.raises(ValueError):
            rows(bad, lead, inner)
