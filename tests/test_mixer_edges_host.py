"""Linear attention and rotation at the edges of what they take, without a GPU."""
import ctypes
import os

import pytest

from state_space_sequence_ssm_amd import _lib

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libm3ssm.so not built (run __graft_entry__.build())")


@built
def test_large_calls_have_a_workspace():
    """A backward that is taken and shares heads needs a workspace; a size of 0 is a refusal."""
    need = _lib.load().m3_linear_attention_backward_workspace_size
    for Bt, L, H, Hk, K, V in ((8, 1 << 17, 64, 32, 128, 128), (1 << 15, 1, 2, 1, 256, 256), (1 << 17, 1, 2, 1, 128, 128)):
        a = _lib.LinearAttentionBackwardArgs(fwd=_lib.LinearAttentionArgs(Bt=Bt, L=L, H=H, Hk=Hk, K=K, V=V, in_dtype=_lib.M3_BF16))
        assert need(ctypes.byref(a)) == Bt * L * H * (K + V) * 4, (Bt, L, H)
    a.fwd.Bt, a.fwd.H, a.fwd.V = 1 << 20, 16, 64  # 2^24 items' heads: past what a launch counts
    assert need(ctypes.byref(a)) == 0


@built
def test_rows_too_far_apart_are_refused():
    """Below 2^24 elements for prompts, 2^40 for single tokens."""
    lib, base = _lib.load(), 0x10000000
    for L, ld in ((2, 1 << 24), (1, 1 << 40)):
        for x in ("q_ld", "k_ld"):
            f = _lib.QkNormRopeArgs(Bt=3, L=L, H=4, Hk=2, D=16, R=8, in_dtype=_lib.M3_BF16, norm=1, eps=1e-6, q=base, k=base * 2,
                                    freqs=base * 3, q_out=base * 4, k_out=base * 5)
            setattr(f, x, ld)
            assert lib.m3_qk_norm_rope(ctypes.byref(f), None) == _lib.M3_ERR_INVALID_ARG, (L, x)
