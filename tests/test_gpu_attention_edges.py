"""Linear attention at its edges: a token's decay over thousands of steps, the largest calls.
References and tolerances as in tests/test_gpu_mixer.py."""
import pytest

torch = pytest.importorskip("torch")

from tests import mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import Maker, ilen  # noqa: E402
from tests.test_gpu_mixer import close, k_attention, parts_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


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
