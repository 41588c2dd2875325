"""Norm and rotation of query and key heads: an eps of 0, head counts that leave part of a warp idle."""
import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("rows,nq,nkv,d,kind", [(3, 5, 1, 128, "bf16"), (700, 1, 3, 64, "f32"), (40, 3, 1, 192, "bf16"),
                                                (9, 1, 1, 256, "f32")])
def test_an_eps_of_zero(rows, nq, nkv, d, kind):
    """eps = 0 is allowed where no head is 0; lanes without a head add nothing to the weight gradients."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = torch.Generator().manual_seed(d + rows)
    x = torch.randn((rows, (nq + nkv) * d), generator=g).to(DT[kind])
    dout = (torch.randn((rows, (nq + nkv) * d), generator=g) * 0.05).to(DT[kind])
    qw, kw = ((torch.randn(d, generator=g) * 0.1 + 1).to(DT[kind]) for _ in "qk")
    r, pos = T.Rotary(d), np.arange(rows)
    out = T.qk_norm_rope(x.cuda(), nq, nkv, d, r, q_norm_w=qw.cuda(), k_norm_w=kw.cuda(), eps=0.0)
    R.within("out", to_np(out), *R.rope(to_np(x), nq, nkv, d, pos, d, False, to_np(qw), to_np(kw), 0.0, kind))
    got = T.qk_norm_rope_backward(dout.cuda(), x.cuda(), nq, nkv, d, r, q_norm_w=qw.cuda(), k_norm_w=kw.cuda(), eps=0.0)
    want = R.rope_bwd(to_np(x), to_np(dout), nq, nkv, d, pos, d, False, to_np(qw), to_np(kw), 0.0, kind)
    for name, a, b in zip(("dx", "dq_norm_w", "dk_norm_w"), got, want):
        R.within(name, to_np(a), *b)
