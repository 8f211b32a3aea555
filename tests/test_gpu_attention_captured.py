"""Linear attention and rotation captured before anything has launched them: what a launch
sets up the first time (leave for much LDS) does not belong to the stream.  The name of this
file puts it in front of those that use the kernels otherwise."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_layers import BF, F32, NAN, Maker  # noqa: E402

pytestmark = pytest.mark.gpu


def test_first_calls_are_captured():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    from state_space_sequence_ssm_amd import ops
    m = Maker(71)
    sizes = [(BF, 32, 48), (BF, 64, 64), (BF, 128, 128), (BF, 256, 40), (F32, 32, 100), (F32, 64, 64), (F32, 128, 64), (F32, 256, 256)]
    ins = [(m(1, 600, 2, K, dtype=t), m(1, 600, 1, K, dtype=t), m(1, 600, 1, V, dtype=t), m(1, 600, 2, V, dtype=t), m(1, 2, K, V))
           for t, K, V in sizes]
    g, freqs = -torch.tensor([0.02, 0.002]).cuda(), torch.rand(16, generator=m.g).cuda()

    def calls():
        out = []
        for q, k, v, dy, h in ins:
            r = ops.m3_qk_norm_rope(q, k, freqs=freqs)
            o = ops.m3_linear_attention(r["q"], r["k"], v, g)
            b = ops.m3_linear_attention_backward(r["q"], r["k"], v, g, dy=dy, want_carry_grads=True)
            n = ops.m3_qk_norm_rope_backward(q, k, dq_out=b["dq"], dk_out=b["dk"], freqs=freqs)
            s = dict(y=ops.m3_linear_attention_step(h, q[:, 3], k[:, 3], v[:, 3], g, h_out=torch.empty_like(h)))
            out += [x for d in (r, o, b, n, s) for x in d.values() if x is not None]
        return out

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
