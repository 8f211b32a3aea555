"""Linear attention at its edges: a token's decay over thousands of steps.
References and tolerances as in tests/test_gpu_mixer.py."""
import pytest

torch = pytest.importorskip("torch")

from tests import mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import Maker  # noqa: E402
from tests.test_gpu_mixer import close  # noqa: E402

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
