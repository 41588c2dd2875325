"""One tensor where two are written: refused on the host, no device is needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def T():
    from tensor_transformer_mlp_rmsnorm_gb300 import build
    build.build()
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


def test_one_gradient_tensor_for_both_weights(T):
    L = T.lib()
    desc = T.tpmlp.QkDesc(4, 2, 1, 64, T.BF16, None, 0, 64, 64, 1e-6, 0)  # one weight for both is fine: it is read
    need = L.tpattn_qk_rope_workspace_bytes(64)

    def bwd(dq, dk):
        return L.tpattn_qk_rope_backward(ctypes.byref(desc), None, 1024, 192, 2048, 192, 4096, 192, dq, dk, 256,
                                         need - 1, None)  # (refused in any case: the workspace is too small)

    assert bwd(128, 128) == T.ERR_ARG and b"same tensor" in L.tpmlp_last_error(None)
    assert bwd(128, 512) == T.ERR_ARG and b"workspace" in L.tpmlp_last_error(None)
