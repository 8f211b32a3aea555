"""Layer operators at the edges of what they take, without a GPU."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

from state_space_sequence_ssm_amd import _lib  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "state_space_sequence_ssm_amd", "csrc")


# ---------------------------------------------------------------- the staging waves' order
def _body(text, name):
    """The body of the lambda `name` of a kernel."""
    i = text.index(f"auto {name} = [&](")
    i = text.index("{", i)
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


@pytest.mark.parametrize("source,kernel", [("scan.hip", "scan_kernel"), ("scan_backward.hip", "reverse_kernel")])
def test_what_a_step_finishes_is_not_what_it_stages(source, kernel):
    """Between two barriers a staging wave finishes one tile and then stages another in
    the same half of LDS, while the other waves may still be finishing: no array is
    both read by the one and written by the other."""
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text[text.index(f"void {kernel}("):])
    names = "dl|us|ds|bc|ys|o|gB|gA|wp|sdu"
    used = {k: set(re.findall(rf"&?(?:\bsh\.)?\b({names})\[", _body(text, k))) for k in ("finish", "stage")}
    assert used["stage"] >= {"dl", "us", "bc"} and used["finish"]
    assert not used["finish"] & used["stage"]


# ---------------------------------------------------------------- the binding's arguments
# each operator's tensors by their names, the first of them the one whose device it takes
NAMES = {"m3_causal_conv": ("x", "w"), "m3_causal_conv_step": ("state", "x", "w"), "m3_causal_conv_backward": ("x", "w", "dy"),
         "m3_selective_scan": ("x", "dt", "A", "B", "C"), "m3_selective_scan_step": ("h", "x", "dt", "A", "B", "C"),
         "m3_selective_scan_backward": ("x", "dt", "A", "B", "C", "dy"), "m3_gated_norm": ("x",),
         "m3_gated_norm_backward": ("x", "dy"), "m3_residual_norm": ("x",), "m3_residual_norm_backward": ("h", "dy")}


def test_every_operator_is_named():
    assert set(NAMES) == set(_lib.LAYER_CALLS)


@pytest.mark.parametrize("name", list(NAMES))
def test_first_argument_by_name(name):
    from state_space_sequence_ssm_amd import ops
    fn, t = getattr(ops, name), torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match=f"^{NAMES[name][0]} must be a device tensor"):  # found, and on the host
        fn(**{k: t for k in NAMES[name]})
    with pytest.raises(TypeError, match=f"^{NAMES[name][0]} must be a torch.Tensor"):
        fn(**{k: t for k in NAMES[name][1:]})


@pytest.mark.parametrize("bad", [torch.float16, torch.float64, torch.int16])
def test_residual_of_another_type(monkeypatch, bad):
    """A residual stream is bfloat16 or float32: nothing else is read as one of them."""
    from state_space_sequence_ssm_amd import ops
    ran = []
    monkeypatch.setattr(ops, "_run_layer", lambda *a: ran.append(a))  # nothing is launched on these host tensors
    call = ops.m3_residual_norm.__wrapped__
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for kw in (dict(residual=x.to(bad)), dict(residual_out=x.to(bad))):
        with pytest.raises(TypeError, match="unsupported"):
            call(x, **kw)
    assert not ran
    for t in (torch.bfloat16, torch.float32):
        call(x, x.to(t), residual_out=x.to(t))
    assert [a[1].res_dtype for a in ran] == [_lib.M3_BF16, _lib.M3_F32]


# ---------------------------------------------------------------- sizes
BASE = 0x10000000
UNS = _lib.M3_ERR_UNSUPPORTED
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libm3ssm.so not built (run __graft_entry__.build())")
POINTERS = {_lib.ConvBackwardArgs: "x w bias dy dx dw dbias workspace", _lib.ScanArgs: "x dt A B C y workspace",
            _lib.ScanStepArgs: "x dt A B C h h_out y", _lib.ScanBackwardArgs: "fwd.x fwd.dt fwd.A fwd.B fwd.C dy dx ddt dA dB dC workspace",
            _lib.GatedNormArgs: "x w y", _lib.GatedNormBackwardArgs: "fwd.x fwd.w dy dx dw workspace",
            _lib.ResidualNormArgs: "x w y", _lib.ResidualNormBackwardArgs: "h x w scale dy dx dw dscale workspace"}


def _put(a, path, value):
    *front, last = path.split(".")
    for f in front:
        a = getattr(a, f)
    setattr(a, last, value)


def _refused(name, **sizes):
    """The codes of a call of these sizes on addresses that nothing may touch, and the
    workspace that it asks for."""
    lib, args = _lib.load(), _lib.LAYER_CALLS[name]()
    for i, f in enumerate(POINTERS[type(args)].split()):
        _put(args, f, BASE + 0x100000 * i)
    if hasattr(args, "workspace_bytes"):
        args.workspace_bytes = (1 << 64) - 1
    inner = args.fwd if hasattr(args, "fwd") else args
    inner.in_dtype = _lib.M3_BF16
    for k, v in sizes.items():
        setattr(inner, k, v)
    size = getattr(lib, name + "_workspace_size", None)
    return getattr(lib, name)(ctypes.byref(args), None), None if size is None else size(ctypes.byref(args))


@built
@pytest.mark.parametrize("D", [(1 << 28) + 4, (1 << 31) - 1])
def test_rows_past_the_widest_are_refused(D):
    assert _refused("m3_gated_norm", M=1, D=D, G=1, eps=1e-6) == (UNS, None)
    assert _refused("m3_gated_norm_backward", M=1, D=D, G=1, eps=1e-6) == (UNS, 0)
    assert _refused("m3_residual_norm", M=1, D=D, res_dtype=_lib.M3_F32, eps=1e-6) == (UNS, None)
    assert _refused("m3_residual_norm_backward", M=1, D=D, res_dtype=_lib.M3_F32, eps=1e-6) == (UNS, 0)


# one launch of the call just past 2^32 work items, and what it is
LAUNCHES = [
    ("m3_causal_conv_backward", dict(Bt=1 << 24, L=1, D=4, W=4)),           # 256 per item
    ("m3_causal_conv_backward", dict(Bt=64, L=1, D=1 << 24, W=4)),          # 64 per sum: 5 D of them
    ("m3_selective_scan", dict(Bt=32768, L=1, D=4096, N=64, G=1)),          # 512 per item and 16 channels
    ("m3_selective_scan", dict(Bt=1 << 23, L=1, D=64, N=4, G=1)),           # 512 per item
    ("m3_selective_scan_step", dict(Bt=1 << 12, D=1 << 18, N=64, G=1)),     # 16 / 4 per item and channel
    ("m3_selective_scan_backward", dict(Bt=1 << 23, L=1, D=64, N=4, G=1)),  # 512 per item
    ("m3_selective_scan_backward", dict(Bt=8, L=1 << 24, D=4, N=16, G=1)),  # 32 per token
    ("m3_selective_scan_backward", dict(Bt=64, L=1, D=1 << 20, N=64, G=1)),  # 64 per sum: 66 D of them
    ("m3_gated_norm_backward", dict(M=64, D=1 << 26, G=1, eps=1e-6)),       # 64 per sum
    ("m3_residual_norm_backward", dict(M=64, D=1 << 25, res_dtype=_lib.M3_BF16, eps=1e-6)),
]


@built
@pytest.mark.parametrize("name,sizes", LAUNCHES, ids=lambda v: v if isinstance(v, str) else "-".join(map(str, v.values())))
def test_launches_of_more_work_items_than_are_counted_are_refused(name, sizes):
    """Before the first launch, and no workspace is asked for."""
    code, size = _refused(name, **sizes)
    assert code == UNS and not size


FAR = (1 << 32) + 5  # 5 in the structures' 32 bits


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The argument structures hold sizes in 32 bits, and would keep the rest of a larger one."""
    from state_space_sequence_ssm_amd import ops
    ran = []
    monkeypatch.setattr(ops, "_run_layer", lambda name, a, dev: ran.append(name))
    monkeypatch.setattr(ops, "_take_workspace", lambda *a: None)
    monkeypatch.setattr(ops, "_dense", lambda *a: None)
    monkeypatch.setattr(ops, "_rows", lambda *a: (None, 0))

    def calls(b, l, d, n, w, g, groups):
        t = lambda *shape: torch.zeros(()).expand(shape)  # noqa: E731
        x, x1, A, B, out = t(b, l, d), t(b, d), t(d, n), t(b, l, g, n), dict(y=t(1))
        grads = {k: t(1) for k in ("dx", "dw", "ddt", "dA", "dB", "dC", "dresidual")}
        return [lambda: ops.m3_causal_conv.__wrapped__(x, t(d, w), **out),
                lambda: ops.m3_causal_conv_step.__wrapped__(t(b, w - 1, d), x1, t(d, w), **out),
                lambda: ops.m3_causal_conv_backward.__wrapped__(x, t(d, w), dy=x, out=grads),
                lambda: ops.m3_selective_scan.__wrapped__(x, x, A, B, B, want_state=False, **out),
                lambda: ops.m3_selective_scan_step.__wrapped__(t(b, d, n), x1, x1, A, B[:, 0], B[:, 0], **out),
                lambda: ops.m3_selective_scan_backward.__wrapped__(x, x, A, B, B, dy=x, out=grads),
                lambda: ops.m3_gated_norm.__wrapped__(x, groups=groups, **out),
                lambda: ops.m3_gated_norm_backward.__wrapped__(x, dy=x, groups=groups, out=grads),
                lambda: ops.m3_residual_norm.__wrapped__(x, want_residual=False, **out),
                lambda: ops.m3_residual_norm_backward.__wrapped__(x, dy=x, out=grads)]

    small = dict(b=1, l=1, d=1, n=1, w=4, g=1, groups=1)
    for call in calls(**small):
        call()
    assert sorted(ran) == sorted(_lib.LAYER_CALLS)
    conv, scan, gated, residual = (0, 1, 2), (3, 4, 5), (6, 7), (8, 9)
    for field, wide in dict(b=conv + scan, l=(0, 2, 3, 5), d=range(10), n=scan, w=conv, g=scan, groups=gated).items():
        for far in (FAR, 1 - (1 << 32)) if field == "groups" else (FAR,):
            del ran[:]
            todo = calls(**dict(small, **{field: far}))
            for i in wide:
                with pytest.raises(ValueError, match="2147483647"):
                    todo[i]()
            assert not ran
