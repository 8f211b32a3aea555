"""The norm and rotation of queries and keys at its edges: the largest heads, values that
are not finite in elements that are not rotated, positions past 32 bits, far rows.
References and tolerances as in tests/test_gpu_mixer.py."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_ref, mixer_ref as ref  # noqa: E402
from tests.test_gpu_layers import BF, F32, NAN, Maker, ilen  # noqa: E402
from tests.test_gpu_mixer import K_ROPE, _rope_inputs, close  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops as o
    return o


# Heads of which a wave's lanes hold more than their usual number of words: both ranges of the
# head end inside a word of 16 bytes (65 words in bf16, 129 in fp32), and their neighbours.
LARGE = [(D, R, adjacent, dt)
         for dt, sizes in (("bf16", [(1024, 20), (1024, 1000), (1011, 18), (1023, 514), (1010, 18), (1024, 1008)]),
                           ("f32", [(1024, 10), (1024, 510), (1019, 10), (1023, 1014), (1018, 10), (520, 10)]))
         for D, R in sizes for adjacent in (False, True)]


@pytest.mark.parametrize("D,R,adjacent,dt", LARGE)
def test_rope_of_the_largest_heads(ops, D, R, adjacent, dt):
    c = (2, 3, 3, 2, D, R, adjacent, dt, [3, 2], True, True, None, False)
    x, d, w, how, lengths = _rope_inputs(c, 41)
    outs = {n: torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda") for n, v in x.items()}
    got = ops.m3_qk_norm_rope(x["q"], x["k"], w["q"], w["k"], lengths=ilen(lengths), q_out=outs["q"], k_out=outs["k"], **how)
    out = {"d" + n: torch.full(v.shape, NAN, dtype=v.dtype, device="cuda") for n, v in x.items()}
    out.update({"d" + n + "_w": torch.full(v.shape, NAN, device="cuda") for n, v in w.items()})
    grad = ops.m3_qk_norm_rope_backward(x["q"], x["k"], w["q"], w["k"], dq_out=d["q"], dk_out=d["k"], lengths=ilen(lengths), out=out, **how)
    for n in "qk":
        want, mag = (ref.rope(x[n], w[n], lengths=lengths, mag=s, dy=d[n], **how) for s in (False, True))
        for b, held in enumerate(layer_ref.held(lengths, 2, 3)):
            close(n, got[n][b, :held], want["y"][b, :held], mag["y"][b, :held], K_ROPE)
            assert (got[n][b, held:] == 7).all()
        close("d" + n, grad["d" + n], want["dx"], mag["dx"], 2 * K_ROPE)
        close("d" + n + "_w", grad["d" + n + "_w"], want["dw"], mag["dw"], K_ROPE + 6 * x[n].shape[2])


# Elements behind R, and with norm = 0 all of them, take no part in others: words in pairs of 16
# bytes, moved back to end with the head, and single elements.
PASSED = [(128, 64, BF), (80, 40, BF), (57, 34, BF), (72, 64, BF), (40, 0, BF), (33, 6, F32), (128, 32, F32), (60, 26, F32), (13, 4, F32)]


def _spread(D, R, t):
    """[1, 7, 2, D] with a value that is not finite in single elements, each in its own head, and where."""
    bad = torch.zeros(1, 7, 2, D, dtype=torch.bool)
    for i in range(14):
        bad[0, i // 2, i % 2, (i * 5 + 3 * (i // 3)) % D] = i % 7 != 6
    values = torch.tensor([INF, -INF, NAN])[torch.arange(14).view(1, 7, 2, 1) % 3]
    return bad.cuda(), values.to(t).cuda()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D,R,t", PASSED)
def test_values_that_are_not_finite_stay_where_they_are(ops, D, R, t, adjacent):
    m = Maker(42)
    x = m(1, 7, 2, D, dtype=t)
    bad, values = _spread(D, R, t)
    dirty = torch.where(bad, values, x)
    freqs = torch.rand(R // 2, generator=m.g).cuda() if R else None
    # a rotated element's value reaches its partner too
    reach = bad.clone()
    if R:
        lo, hi = (slice(0, R, 2), slice(1, R, 2)) if adjacent else (slice(0, R // 2), slice(R // 2, R))
        both = bad[..., lo] | bad[..., hi]
        reach[..., lo], reach[..., hi] = both, both
    how = dict(freqs=freqs, norm=False, adjacent=adjacent, start=3)
    runs = [lambda v: ops.m3_qk_norm_rope(v, None, **how)["q"], lambda v: ops.m3_qk_norm_rope_backward(x, dq_out=v, **how)["dq"]]
    for run in runs:
        clean, got = run(x), run(dirty)
        assert torch.equal(got[~reach], clean[~reach])
        assert torch.equal(got[..., R:].nan_to_num(9e9), dirty[..., R:].nan_to_num(9e9))
        assert not torch.isfinite(got[..., :R][bad[..., :R]]).any()


@pytest.mark.parametrize("start", [(1 << 31) - 3, (1 << 31) - 1, -(1 << 31) + 1])
def test_rope_positions_past_32_bits(ops, start):
    """Token t is at start + t, also where that is 2^31 and more.  Rates are whole multiples of
    2^-12 and 2^-24, so that the reference's angles are exact."""
    m = Maker(43)
    q, dy = m(2, 6, 1, 8), m(2, 6, 1, 8)
    freqs = torch.tensor([1.0, 3 * 2.0 ** -12, 2.0 ** -24, 0.0], device="cuda")
    got = ops.m3_qk_norm_rope(q, None, freqs=freqs, start=start)["q"]
    grad = ops.m3_qk_norm_rope_backward(q, dq_out=dy, freqs=freqs, start=start)["dq"]
    want, mag = (ref.rope(q, freqs=freqs, start=start, mag=x, dy=dy) for x in (False, True))
    close("q", got, want["y"], mag["y"], K_ROPE)
    close("dq", grad, want["dx"], mag["dx"], 2 * K_ROPE)


def test_single_tokens_rows_further_apart_than_a_prompts(ops):
    """One position of each sequence of a long batch: rows 2^24 elements apart and more."""
    m, Bt, H, Hk, D, ld = Maker(44), 3, 4, 2, 64, (1 << 24) + 64
    big = torch.empty(Bt * ld, dtype=BF, device="cuda").view(Bt, 1, ld)
    q, k = (big[..., a * D:b * D].unflatten(-1, (b - a, D)) for a, b in ((0, H), (H, H + Hk)))
    x, y = m(Bt, 1, H, D, dtype=BF), m(Bt, 1, Hk, D, dtype=BF)
    q.copy_(x)
    k.copy_(y)
    w, freqs, pos = m(D), torch.rand(D // 2, generator=m.g).cuda(), torch.tensor([[5], [70000], [0]], dtype=torch.int32, device="cuda")
    calls = (lambda q, k: ops.m3_qk_norm_rope(q, k, w, w, freqs=freqs, positions=pos),
             lambda q, k: ops.m3_qk_norm_rope_backward(q, k, w, w, dq_out=x, dk_out=y, freqs=freqs, positions=pos))
    for call in calls:
        got, want = call(q, k), call(x, y)
        assert all(torch.equal(got[n], want[n]) for n in want)
    two = torch.empty(2 * ld, dtype=BF, device="cuda").view(1, 2, ld)[..., :H * D].unflatten(-1, (H, D))  # two tokens of one
    with pytest.raises(ops.M3Error, match="invalid argument"):
        ops.m3_qk_norm_rope(two, freqs=freqs)
