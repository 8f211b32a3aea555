"""Linear attention at its edges: many items and heads (blocks of 128 columns), what the parts
of bf16 products leave, a token's decay over thousands of steps, the largest calls, gradients
of values that are not finite.  References and tolerances as in tests/test_gpu_mixer.py."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref, mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import BF, DT, NAN, Maker, ilen, spoil  # noqa: E402
from tests.test_gpu_mixer import close, k_attention, parts_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


# From 256 items' heads on a block of fp32 takes 128 columns: whole, part and second tiles of
# them, both walks of the backward by the same kernel and by two, few and many chunks.
MANY = [
    # Bt, L, H, Hk, K, V, dtype, lengths every 4 items
    (64, 70, 4, 2, 128, 128, "f32", None),
    (32, 100, 8, 8, 64, 100, "f32", [100, 0, 1, 65]),
    (16, 65, 16, 4, 32, 128, "f32", [65, 64, 63, 3]),
    (44, 30, 6, 3, 80, 200, "f32", [30, 1, 0, 29]),
    (64, 200, 4, 4, 64, 96, "f32", [200, 129, 128, 5]),
    (32, 20, 8, 2, 100, 40, "f32", None),
    (64, 70, 4, 2, 64, 128, "bf16", [70, 0, 64, 1]),
]


@pytest.mark.parametrize("c", MANY, ids=str)
def test_many_items_and_heads(ops, c):
    Bt, L, H, Hk, K, V, dt, some = c
    lengths = None if some is None else [some[b % 4] for b in range(Bt)]
    m, t = Maker(51), DT[dt]
    q, k, v, dy = (spoil(m(Bt, L, h, d, dtype=t), lengths) for h, d in ((H, K), (Hk, K), (Hk, V), (H, V)))
    h0, dh = m(Bt, H, K, V), m(Bt, H, K, V)
    g = -torch.linspace(0.0, 0.4, H, device="cuda") ** 2
    want, mag = (ref.attention(q, k, v, g, h0, lengths=lengths, mag=x, dy=dy, dh_final=dh) for x in (False, True))
    kk, parts = k_attention(L, K, V, g.cpu(), dt), parts_of(dt)
    y = torch.full((Bt, L, H, V), 7.0, dtype=t, device="cuda")
    hf = torch.full((Bt, H, K, V), NAN, device="cuda")
    ops.m3_linear_attention(q, k, v, g, h0, lengths=ilen(lengths), y=y, h_final=hf)
    for b, n in enumerate(layer_ref.held(lengths, Bt, L)):
        close("y", y[b, :n], want["y"][b, :n], mag["y"][b, :n], kk, parts)
        assert (y[b, n:] == 7).all()
    close("h", hf, want["h"], mag["h"], kk)
    shapes = dict(dq=(Bt, L, H, K), dk=(Bt, L, Hk, K), dv=(Bt, L, Hk, V))
    out = {n: torch.full(s, NAN, dtype=t, device="cuda") for n, s in shapes.items()}
    out["dh0"] = torch.full((Bt, H, K, V), NAN, device="cuda")
    got = ops.m3_linear_attention_backward(q, k, v, g, h0, dy=dy, dh_final=dh, lengths=ilen(lengths), out=out)
    for n in ("dq", "dk", "dv"):
        close(n, got[n], want[n], mag[n], kk + H // Hk, parts)
    close("dh0", got["dh0"], want["dh0"], mag["dh0"], kk)


# What parts leave.  One token of an item holds values, so that nothing hides it behind sums.
# With U = 2^-24: its state is w k v^T; the power w = exp2(x), x = d log2(e) log_decay below 1 here,
# is off by x's two roundings and its own step (4 U), w v rounds once, three parts leave 2^-24, and
# three sums of them, counted twice as the matrix cores may drop what they round, are 6 U: 12 U;
# every further chunk multiplies by another power, 5 U.  Two parts would leave up to 2^-16 = 256 U.
@pytest.mark.parametrize("L,at,chunks", [(64, 20, 1), (64, 63, 1), (40, 7, 1), (200, 130, 2), (1500, 1400, 3)])
@pytest.mark.parametrize("K,V", [(32, 32), (64, 64), (128, 96), (256, 64)])
def test_states_keep_what_three_parts_hold(ops, K, V, L, at, chunks):
    m = Maker(52)
    q, k, v = (torch.zeros(1, L, 2, d, dtype=BF, device="cuda") for d in (K, K, V))
    k[:, at], v[:, at] = m(1, 2, K, dtype=BF), m(1, 2, V, dtype=BF)
    g = -torch.tensor([0.0061, 0.0003], device="cuda")
    want = ref.attention(q, k, v, g)["h"]
    bound = (12 + 5 * (chunks - 1)) * 2.0 ** -24 * want.abs()
    for workspace in (None, False):
        h = ops.m3_linear_attention(q, k, v, g, workspace=workspace)["h"].cpu().double()
        assert ((h - want).abs() <= bound).all(), float(((h - want).abs() / want.abs().clamp(min=1e-30)).max() * 2 ** 24)
    two = (w2 := (want / k[0, at].cpu().double()[..., None]).float()).bfloat16().float()
    two = two + (w2 - two).bfloat16().float()
    # (the last token's weight is 1 and leaves v, which one part holds)
    assert at == L - 1 or ((two.double() * k[0, at].cpu().double()[..., None] - want).abs() > bound).any(), "two parts would pass"


# Scores and the state read are in two parts, 2^-16 of a term.  Two terms that nearly cancel
# show it through the rounding of the output, 2^-8 of what is left of them: s - s' is a 64th of
# either.  One part would be off by up to 2^-8 of the terms.  Powers are 1 (no decay) and few
# elements are not zero, so that a handful of roundings is all there is beside.
@pytest.mark.parametrize("where", ["scores", "state"])
@pytest.mark.parametrize("K,V", [(32, 32), (64, 64), (128, 96), (256, 64)])
def test_outputs_keep_what_two_parts_hold(ops, K, V, where):
    m, L = Maker(53), 64
    q, k, v = (torch.zeros(1, L, 1, d, dtype=BF, device="cuda") for d in (K, K, V))
    g, h0 = torch.zeros(1, device="cuda"), None
    a = m(V)
    q[..., 0] = m(1, L, 1, shift=2.0, scale=0.3, dtype=BF)
    if where == "scores":  # keys equal but for a small element, values opposite
        q[..., 5] = q[..., 0]
        k[0, 3, 0, 0], k[0, 9, 0, 0], k[0, 9, 0, 5] = 1.3, 1.3, 1.3 / 64
        v[0, 3, 0], v[0, 9, 0] = a.bfloat16(), -a.bfloat16()
    else:  # two rows of the state met by queries of opposite sign
        q[..., 1] = -q[..., 0]
        h0 = torch.zeros(1, 1, K, V, device="cuda")
        h0[0, 0, 0], h0[0, 0, 1] = a, a * (1 + 1 / 64)
    want, mag = (ref.attention(q, k, v, g, h0, mag=x) for x in (False, True))
    y = ops.m3_linear_attention(q, k, v, g, h0)["y"]
    close("y", y, want["y"], mag["y"], 8, 2.0 ** -16)


def test_a_tokens_decay_over_thousands_of_steps(ops):
    """States of k = 0 after n steps are exp(n log_decay) of what they were.  Every step rounds
    the state, by up to 2^-24 either way: over 4096 steps and the mean of 4096 elements six times
    2^-24 / sqrt(3) stay below 2.1e-7.  The decay itself, 1 - l to a few 2^-24 of it, adds
    n |log_decay| 2^-22 = 6e-7 at most here; l rounded to 2^-24 would add up to n 2^-25 = 1.2e-4."""
    n, K = 4096, 64
    m = Maker(54)
    g = -torch.tensor([0.00061, 0.00027, 0.000071, 0.0005], device="cuda")
    h = m(1, 4, K, K, shift=3.0)
    want = h.cpu().double() * torch.exp(g.cpu().double() * n)[:, None, None]
    z, q = torch.zeros(1, 4, K, device="cuda"), m(1, 4, K)
    for _ in range(n):
        ops.m3_linear_attention_step(h, q, z, z, g)
    off = (h.cpu().double() / want - 1).mean((0, 2, 3))
    assert (off.abs() < 1e-6).all(), off


def test_a_tokens_decay_of_any_size(ops):
    """l s + k v from no decay through l of one half, where its form changes, to l = 0 and growth."""
    K, V = 24, 40
    g = torch.tensor([0.0, -1e-9, -1e-4, -0.3, -0.4999, -0.5, -0.5001, -0.7, -3.0, -20.0, -80.0, -float("inf"), 0.2, 0.4999, 0.6, 5.0], device="cuda")
    H, m = len(g), Maker(55)
    for size in (1.0, 1e-6, 1e6):
        h, q, k, v = m(2, H, K, V, scale=size), m(2, H, K), m(2, H, K), m(2, H, V)
        want, mag = (ref.attention(q[:, None], k[:, None], v[:, None], g, h, mag=x) for x in (False, True))
        y = ops.m3_linear_attention_step(h, q, k, v, g)
        close("h", h, want["h"], mag["h"], 8)
        close("y", y, want["y"][:, 0], mag["y"][:, 0], K + 12)
    h = torch.full((2, H, K, V), float("inf"), device="cuda")
    ops.m3_linear_attention_step(h, q, k, v, g)
    held = torch.exp(g) > 0
    assert (h[:, held] == float("inf")).all()


def test_many_large_states(ops):
    """65,536 items and heads of 256 x 256: within the documented limits, states apart."""
    n, D = 65536, 256
    gen = torch.Generator(device="cuda").manual_seed(56)
    q, k, v, dy = (torch.randn(n, 1, 1, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
    g = torch.zeros(1, device="cuda")
    y = ops.m3_linear_attention(q, k, v, g, want_state=False)["y"]
    out = ops.m3_linear_attention_backward(q, k, v, g, dy=dy)
    s = D ** -0.5
    q, k, v, dy = (t.double() for t in (q, k, v, dy))
    kk = k_attention(1, D, D, g.cpu(), "bf16")
    qk, dv = (q * k).sum(-1, keepdim=True), (dy * v).sum(-1, keepdim=True)
    mqk, mdv = (q * k).abs().sum(-1, keepdim=True), (dy * v).abs().sum(-1, keepdim=True)
    for name, got, want, mag in (("y", y, s * qk * v, s * mqk * v.abs()), ("dq", out["dq"], s * dv * k, s * mdv * k.abs()),
                                 ("dk", out["dk"], s * dv * q, s * mdv * q.abs()), ("dv", out["dv"], s * qk * dy, s * mqk * dy.abs())):
        close(name, got, want.cpu(), mag.cpu(), kk, parts_of("bf16"))


def test_gradients_of_many_shared_heads(ops):
    """2^24 and more elements of dk and dv: the sums over the heads that share one are those of the
    heads alone, in order."""
    m, Bt, L, H, Hk, K, V = Maker(57), 33, 1024, 8, 4, 128, 8
    q, k, v, dy = m(Bt, L, H, K), m(Bt, L, Hk, K), m(Bt, L, Hk, V), m(Bt, L, H, V)
    g = -torch.linspace(0.001, 0.1, H, device="cuda")
    n = ilen([L - 31 * b for b in range(Bt)])
    got = ops.m3_linear_attention_backward(q, k, v, g, dy=dy, lengths=n)
    each = ops.m3_linear_attention_backward(q, *(x.repeat_interleave(H // Hk, 2) for x in (k, v)), g, dy=dy, lengths=n)
    assert Bt * L * Hk * K > 1 << 24 and torch.equal(got["dq"], each["dq"])
    for x in ("dk", "dv"):
        a, b = each[x].unflatten(2, (Hk, 2)).unbind(3)
        assert torch.equal(got[x], a + b), x


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_values_that_are_not_finite(ops, dt):
    """They reach no other item and head, dq no more than 63 tokens in front of a k or v, dk and dv
    no more than 63 behind a q or dy; of a token's own row only, where it is the row's factor."""
    m, L, at = Maker(58), 200, 100
    q, k, v, dy = (m(2, L, 2, 32, dtype=DT[dt]) for _ in range(4))
    g = -torch.tensor([0.02, 0.1]).cuda()
    want = ops.m3_linear_attention_backward(q, k, v, g, dy=dy, want_carry_grads=True)
    own = {"q": "", "k": "dv", "v": "dk", "dy": "dq"}  # outputs whose row is a sum times this row
    for name, x in (("q", q), ("k", k), ("v", v), ("dy", dy)):
        for bad in (NAN, float("inf")):
            kept = x[1, at, 1].clone()
            x[1, at, 1] = bad
            got = ops.m3_linear_attention_backward(q, k, v, g, dy=dy, want_carry_grads=True)
            x[1, at, 1] = kept
            for o in ("dq", "dk", "dv"):
                assert torch.equal(got[o][0], want[o][0]) and torch.equal(got[o][1, :, 0], want[o][1, :, 0])
                row, was = got[o][1, :, 1], want[o][1, :, 1]
                if o == own[name]:
                    same = torch.arange(L, device="cuda") != at
                elif name in ("k", "v"):  # dq of its token and those behind; dk and dv of none
                    same = torch.arange(L, device="cuda") < at - 63 if o == "dq" else torch.ones(L, dtype=torch.bool, device="cuda")
                else:  # dk and dv of its token and those in front; dq of none
                    same = torch.arange(L, device="cuda") > at + 63 if o != "dq" else torch.ones(L, dtype=torch.bool, device="cuda")
                assert torch.equal(row[same], was[same]), (name, bad, o)
                if not same.all():
                    assert not torch.isfinite(row[at]).all(), (name, bad, o)
            if name in ("k", "v"):
                assert torch.equal(got["dh0"], want["dh0"])
            else:
                assert torch.equal(got["dh0"][0], want["dh0"][0]) and torch.equal(got["dh0"][1, 0], want["dh0"][1, 0])
