"""Linear attention at the edges of what it takes, without a GPU."""
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
