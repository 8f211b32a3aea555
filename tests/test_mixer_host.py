"""Linear attention and the norm and rotation of its queries and keys without a GPU: the
64-bit reference's gradients against automatic differentiation and differences, and the
refusals of the C ABI and of the torch binding."""
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from state_space_sequence_ssm_amd import _lib  # noqa: E402
from tests import layer_ref, mixer_ref as ref  # noqa: E402

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
def _recurrence(q, k, v, g, h0, scale, lengths):
    """The definition, token by token."""
    Bt, L, H, K = q.shape
    per = H // k.shape[2]
    ys, hs = [], []
    for b, n in enumerate(layer_ref.held(lengths, Bt, L)):
        S, rows = h0[b], []
        for t in range(n):
            kt, vt = k[b, t].repeat_interleave(per, 0), v[b, t].repeat_interleave(per, 0)
            S = torch.exp(g)[:, None, None] * S + kt[..., None] * vt[:, None]
            rows.append(scale * (q[b, t][..., None] * S).sum(1))
        rows += [torch.zeros(H, v.shape[3], dtype=F64)] * (L - n)
        ys.append(torch.stack(rows))
        hs.append(S)
    return torch.stack(ys), torch.stack(hs)


@pytest.mark.parametrize("lengths", [None, [5, 0], [1, 9]])
def test_reference_attention(lengths):
    Bt, L, H, Hk, K, V = 2, 6, 4, 2, 3, 5
    q, k, v, h0 = _rand(Bt, L, H, K, seed=1), _rand(Bt, L, Hk, K, seed=2), _rand(Bt, L, Hk, V, seed=3), _rand(Bt, H, K, V, seed=4)
    g = -_rand(H, seed=5).abs()
    dy, dh = _rand(Bt, L, H, V, seed=6), _rand(Bt, H, K, V, seed=7)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, h0)]

    def loss(q, k, v, h0):
        y, h = _recurrence(q, k, v, g, h0, 0.7, lengths)
        return (y * dy).sum() + (h * dh).sum()

    got = ref.attention(q, k, v, g, h0, 0.7, lengths, dy=dy, dh_final=dh)
    y, h = _recurrence(q, k, v, g, h0, 0.7, lengths)
    assert torch.allclose(got["y"], y, rtol=1e-12, atol=1e-13) and torch.allclose(got["h"], h, rtol=1e-12, atol=1e-13)
    loss(*leaves).backward()
    for name, leaf in zip(("dq", "dk", "dv", "dh0"), leaves):
        assert torch.allclose(got[name], leaf.grad, rtol=1e-11, atol=1e-12), name
        # and against central differences along a direction
        args = {"dq": 0, "dk": 1, "dv": 2, "dh0": 3}[name]
        way, at = _rand(*leaf.shape, seed=8), [q, k, v, h0]
        up, down = list(at), list(at)
        up[args], down[args] = at[args] + 1e-5 * way, at[args] - 1e-5 * way
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs(float(slope - (got[name] * way).sum())) < 1e-6 * (1 + abs(float(slope)))


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_reference_rope(adjacent, norm):
    Bt, L, H, D, R = 2, 3, 2, 9, 6
    x, dy = _rand(Bt, L, H, D, seed=1), _rand(Bt, L, H, D, seed=2)
    w = _rand(D, seed=3) if norm else None
    freqs, lengths = torch.tensor([1.0, 0.3, 0.01], dtype=F64), [3, 1]
    how = dict(freqs=freqs, start=11, lengths=lengths, norm=norm, adjacent=adjacent)
    xl, wl = x.clone().requires_grad_(), None if w is None else w.clone().requires_grad_()
    ys = []
    for b in range(Bt):  # element by element
        for t in range(lengths[b]):
            for h in range(H):
                v = xl[b, t, h]
                n = v / torch.sqrt((v * v).sum() / D + 1e-6) * wl if norm else v
                y = list(n)
                for i in range(R // 2):
                    lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)
                    c, s = torch.cos((11 + t) * freqs[i]), torch.sin((11 + t) * freqs[i])
                    y[lo], y[hi] = n[lo] * c - n[hi] * s, n[hi] * c + n[lo] * s
                ys.append(((b, t, h), torch.stack(y)))
    got = ref.rope(x, w, dy=dy, **how)
    sum((y * dy[at]).sum() for at, y in ys).backward()
    for at, y in ys:
        assert torch.allclose(got["y"][at], y, rtol=1e-12, atol=1e-13)
    assert torch.allclose(got["dx"], xl.grad, rtol=1e-11, atol=1e-12)
    assert w is None or torch.allclose(got["dw"], wl.grad, rtol=1e-11, atol=1e-12)


# ---------------------------------------------------------------- refusals of the C ABI
BASE = 0x10000000


def _fill(a, fields, at=0):
    for i, f in enumerate(fields.split()):
        setattr(a, f, BASE + 0x100000 * (at + i))
    return a


def _attention():
    a = _lib.LinearAttentionArgs(Bt=2, L=9, H=4, Hk=2, K=16, V=24, in_dtype=_lib.M3_BF16, scale=0.25)
    return _fill(a, "q k v log_decay h0 lengths y h_final")


def _step():
    a = _lib.LinearAttentionStepArgs(Bt=2, H=4, Hk=2, K=16, V=24, in_dtype=_lib.M3_BF16, scale=0.25)
    return _fill(a, "q k v log_decay h h_out y")


def _backward():
    a = _lib.LinearAttentionBackwardArgs(fwd=_attention())
    _fill(a, "dy dh_final dq dk dv dh0 workspace", 10)
    a.workspace_bytes = 1 << 30
    return a


def _rope():
    a = _lib.QkNormRopeArgs(Bt=2, L=9, H=4, Hk=2, D=16, R=8, in_dtype=_lib.M3_BF16, norm=1, adjacent=0, start=0, eps=1e-6)
    return _fill(a, "q k q_w k_w freqs positions lengths q_out k_out")


def _rope_backward():
    a = _lib.QkNormRopeBackwardArgs(fwd=_rope())
    _fill(a, "dq_out dk_out dq dk dq_w dk_w workspace", 10)
    a.workspace_bytes = 1 << 30
    return a


MAKE = {"m3_linear_attention": _attention, "m3_linear_attention_step": _step, "m3_linear_attention_backward": _backward,
        "m3_qk_norm_rope": _rope, "m3_qk_norm_rope_backward": _rope_backward}


def _bad(name):
    """(field, value, code): one refused argument each; "=f" takes field f's value."""
    f = "fwd." if name.endswith("backward") else ""
    out = [(f + "in_dtype", 7, UNS), (f + "Bt", 0, INV), (f + "Bt", 1 << 30, UNS), (f + "H", 0, INV), (f + "q", None, INV),
           (f + "q", BASE + 1, INV), (f + "q_ld", 8, INV), (f + "q_ld", -64, INV), (f + "k_ld", 8, INV), (f + "k", BASE + 1, INV),
           (f + "k", None, INV)]
    if "step" not in name:
        out += [(f + "L", 0, INV), (f + "L", (1 << 28) + 1, UNS), (f + "lengths", BASE + 2, INV), (f + "q_ld", 1 << 24, INV)]
    if "attention" in name:
        out += [(f + "K", 0, INV), (f + "K", 257, UNS), (f + "V", 257, UNS), (f + "V", -1, INV), (f + "Hk", 3, INV), (f + "Hk", 0, INV),
                (f + "v", None, INV), (f + "v_ld", 47, INV), (f + "log_decay", None, INV), (f + "log_decay", BASE + 2, INV)]
    else:
        out += [(f + "D", 0, INV), (f + "D", 1025, UNS), (f + "R", 7, INV), (f + "R", 18, INV), (f + "R", 0, INV), (f + "norm", 2, INV),
                (f + "norm", 0, INV), (f + "adjacent", -1, INV), (f + "eps", -1.0, INV), (f + "eps", float("nan"), INV),
                (f + "freqs", None, INV), (f + "Hk", 0, INV), (f + "Hk", -1, INV), (f + "positions", BASE + 1, INV)]
    out += {"m3_linear_attention": [("y", None, INV), ("y", "=q", INV), ("y", "=h0", INV), ("y", "=h_final", INV), ("h_final", "=k", INV),
                                    ("y", BASE + 1, INV), ("workspace", BASE + 8, INV), ("workspace", "=h0", INV)],
            "m3_linear_attention_step": [("y", None, INV), ("y", "=h", INV), ("h", None, INV), ("h_out", "=q", INV), ("q_ld", 1 << 40, INV),
                                         ("h", BASE + 2, INV)],
            "m3_linear_attention_backward": [("dy", None, INV), ("dq", None, INV), ("dk", "=dv", INV), ("dv", "=dy", INV), ("dh0", "=dh_final", INV),
                                             ("workspace", None, INV), ("workspace_bytes", 16, INV), ("workspace", BASE + 64, INV),
                                             ("workspace", "=dq", INV)],
            "m3_qk_norm_rope": [("q_out", None, INV), ("k_out", None, INV), ("q_out", "=k", INV), ("k_out", "=q", INV), ("q_out", "=k_out", INV),
                                ("q_out", "=q_w", INV)],
            "m3_qk_norm_rope_backward": [("dq_out", None, INV), ("dk_out", None, INV), ("dq", None, INV), ("dk", None, INV), ("dq_w", None, INV),
                                         ("fwd.q_w", None, INV), ("dq", "=dk_out", INV), ("dq_w", "=dk_w", INV), ("dq", "=dk", INV),
                                         ("workspace", None, INV), ("workspace_bytes", 16, INV), ("workspace", "=dq_out", INV)]}[name]
    return out


def _set(a, path, value):
    *front, last = path.split(".")
    for f in front:
        a = getattr(a, f)
    setattr(a, last, value)


@built
@pytest.mark.parametrize("name", list(MAKE))
def test_mixer_refusals(name):
    fn = getattr(_lib.load(), name)
    assert fn(None, None) == INV
    for path, value, code in _bad(name):
        a = MAKE[name]()
        _set(a, path, getattr(a, value[1:]) if isinstance(value, str) else value)
        assert fn(ctypes.byref(a), None) == code, (path, value)


@built
def test_rows_past_32_bits_are_refused():
    """64 rows of an output are addressed in 32 bits: of many heads over few shared ones too."""
    lib = _lib.load()
    for name, make in (("m3_linear_attention", _attention), ("m3_linear_attention_backward", _backward)):
        a = make()
        f = a.fwd if hasattr(a, "fwd") else a
        f.Bt, f.L, f.H, f.Hk, f.K, f.V = 1, 64, 1 << 17, 1, 1, 128
        if hasattr(a, "fwd"):
            a.workspace_bytes = (1 << 64) - 1
        assert getattr(lib, name)(ctypes.byref(a), None) == UNS, name


@built
def test_calls_past_32_bits_of_work_items_are_refused():
    a = _attention()
    a.Bt, a.L, a.H, a.Hk, a.K, a.V = 1 << 19, 1, 32, 32, 8, 8
    assert _lib.load().m3_linear_attention(ctypes.byref(a), None) == UNS
    b = _step()
    b.Bt, b.H, b.Hk, b.K, b.V = 1 << 19, 64, 64, 1, 1
    assert _lib.load().m3_linear_attention_step(ctypes.byref(b), None) == UNS


@built
def test_rope_in_place_needs_dense_rows():
    for x, width in (("q", 64), ("k", 32)):
        a = _rope()
        setattr(a, x + "_out", getattr(a, x))
        setattr(a, x + "_ld", width + 8)
        assert _lib.load().m3_qk_norm_rope(ctypes.byref(a), None) == INV


@built
def test_mixer_workspace_sizes():
    lib = _lib.load()
    for name in _lib.MIXER_SIZES:
        assert getattr(lib, name)(None) == 0
    a = _attention()
    assert lib.m3_linear_attention_workspace_size(ctypes.byref(a)) == 0  # 9 tokens: not cut
    a.L = 4096
    need = lib.m3_linear_attention_workspace_size(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    a.workspace, a.workspace_bytes = BASE + 0x100000 * 30, need - 1
    assert lib.m3_linear_attention(ctypes.byref(a), None) == INV
    a.K = 257
    assert lib.m3_linear_attention_workspace_size(ctypes.byref(a)) == 0
    for name, make in (("m3_linear_attention_backward", _backward), ("m3_qk_norm_rope_backward", _rope_backward)):
        a = make()
        need = getattr(lib, name + "_workspace_size")(ctypes.byref(a))
        assert need > 0 and need % 256 == 0
        a.workspace_bytes = need - 1
        assert getattr(lib, name)(ctypes.byref(a), None) == INV, name


@pytest.mark.skipif(bool(_SAN_LIB), reason="already the sanitized run")
@built
def test_mixer_validation_under_host_sanitizers():
    from state_space_sequence_ssm_amd import build as b
    try:
        lib, rt = b.build_hostsan(), b.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    env = dict(os.environ, LD_PRELOAD=rt, M3SSM_HOSTSAN_LIB=lib, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__), "-k",
                        "refusals or dense_rows or workspace_sizes"], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


# ---------------------------------------------------------------- the torch binding
NAMES = {"m3_linear_attention": ("q", "k", "v", "log_decay"), "m3_linear_attention_step": ("h", "q", "k", "v", "log_decay"),
         "m3_linear_attention_backward": ("q", "k", "v", "log_decay", "dy"), "m3_qk_norm_rope": ("q",),
         "m3_qk_norm_rope_backward": ("q", "dq_out")}


def test_every_mixer_call_is_named():
    assert set(NAMES) == set(_lib.MIXER_CALLS) and set(MAKE) == set(NAMES)


@pytest.mark.parametrize("name", list(NAMES))
def test_first_argument_by_name(name):
    import state_space_sequence_ssm_amd as pkg
    fn, t = getattr(pkg, name), torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match=f"^{NAMES[name][0]} must be a device tensor"):
        fn(**{k: t for k in NAMES[name]})
    with pytest.raises(TypeError, match=f"^{NAMES[name][0]} must be a torch.Tensor"):
        fn(**{k: t for k in NAMES[name][1:]})


def _ran(monkeypatch):
    """The binding on host tensors, with nothing launched."""
    from state_space_sequence_ssm_amd import ops
    ran = []
    monkeypatch.setattr(ops, "_run_layer", lambda *a: ran.append(a))
    monkeypatch.setattr(ops, "_take_workspace", lambda name, args, given, dev: given)
    return ops, ran


def test_attention_binding_refusals(monkeypatch):
    ops, ran = _ran(monkeypatch)
    call = ops.m3_linear_attention.__wrapped__
    q, k, v, g = torch.zeros(2, 5, 4, 8), torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 2, 6), torch.zeros(4)
    bad = [
        (dict(q=q.half()), TypeError, "unsupported"), (dict(k=k.bfloat16()), TypeError, "k must be"), (dict(k=k[:, :4]), ValueError, "k has shape"),
        (dict(v=v[:1]), ValueError, "v has shape"), (dict(g=g[:3]), ValueError, "log_decay has shape"),
        (dict(g=g.double()), TypeError, "log_decay must be"), (dict(h0=torch.zeros(2, 4, 8, 5)), ValueError, "h0 has shape"),
        (dict(lengths=torch.zeros(2, dtype=torch.int64)), TypeError, "lengths must be"), (dict(y=torch.zeros(2, 5, 4, 8)), ValueError, "y has shape"),
        (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "dense"), (dict(k=torch.zeros(2, 5, 2, 16)[..., ::2]), ValueError, "dense"),
    ]
    for change, error, text in bad:
        kw = dict(q=q, k=k, v=v, g=g, h0=None) | change
        with pytest.raises(error, match=text):
            call(kw.pop("q"), kw.pop("k"), kw.pop("v"), kw.pop("g"), kw.pop("h0"), **kw)
    assert not ran
    out = call(q, k, v, g)
    assert out["y"].shape == (2, 5, 4, 6) and out["h"].shape == (2, 4, 8, 6) and abs(ran[0][1].scale - 8 ** -0.5) < 1e-7
    assert call(q, k, v, g, want_state=False)["h"] is None


def test_rope_binding_refusals(monkeypatch):
    ops, ran = _ran(monkeypatch)
    call = ops.m3_qk_norm_rope.__wrapped__
    q, k, w, f = torch.zeros(2, 5, 4, 8), torch.zeros(2, 5, 2, 8), torch.zeros(8), torch.zeros(4)
    for args, kw, error, text in [
            ((q, k[..., :6]), {}, ValueError, "k has shape"), ((q, k, w[:4]), {}, ValueError, "q_w has shape"),
            ((q, None, None, w), {}, ValueError, "k_w without k"), ((q,), dict(k_out=k), ValueError, "k_out without k"),
            ((q, k), dict(positions=torch.zeros(2, 5, dtype=torch.int64)), TypeError, "positions must be"),
            ((q, k), dict(positions=torch.zeros(2, 4, dtype=torch.int32)), ValueError, "positions has shape"),
            ((q, k), dict(freqs=f.double()), TypeError, "freqs must be"), ((q, k), dict(start=1 << 31), ValueError, "sizes up to"),
            ((q, k), dict(q_out=q[..., :4]), ValueError, "q_out has shape")]:
        with pytest.raises(error, match=text):
            call(*args, **kw)
    with pytest.raises(ValueError, match="goes with k"):
        ops.m3_qk_norm_rope_backward.__wrapped__(q, k, dq_out=q)
    assert not ran
    out = call(q, None, freqs=f)
    assert out["k"] is None and ran[0][1].R == 8 and ran[0][1].Hk == 0
