"""Every variant of the norm and rotation kernels, forward and backward, and rows beyond 2^31 elements."""
import itertools

import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.mark.parametrize("d,kind,il,rot", [(d, k, il, r) for d, k, il in itertools.product((64, 128, 192, 256), DT, (False, True))
                                           for r in (0, 16, d // 2, d - 16, d)])
def test_rows(d, kind, il, rot):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    rows, (nq, nkv) = 37, ((7, 2), (1, 1), (0, 3), (9, 0))[(d // 64 + rot // 16) % 4]
    g = torch.Generator().manual_seed(d + rot)
    x = (torch.randn((rows, (nq + nkv) * d + 8), generator=g) * 1.5).to(DT[kind])
    dout = (torch.randn((rows, (nq + nkv) * d), generator=g) * 0.05).to(DT[kind])
    w = (torch.randn(d, generator=g) * 0.1 + 1).to(DT[kind])
    qw, kw = w if nq and rot != 16 else None, w if nkv and rot != d // 2 else None
    pos = torch.randint(-5000, 1 << 20, (rows,), generator=g).to(torch.int32)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = lambda t: None if t is None else to_np(t)  # noqa: E731
    args = (nq, nkv, d, T.Rotary(rot, interleaved=il) if rot else None, pos.cuda(), 0, c(qw), c(kw), EPS)
    ref = (nq, nkv, d, pos.numpy(), rot, il, n(qw), n(kw), EPS, kind)
    R.within("out", to_np(T.qk_norm_rope(x.cuda(), *args)), *R.rope(to_np(x), *ref))
    got = T.qk_norm_rope_backward(dout.cuda(), x.cuda(), *args)
    for name, a, b in zip(("dx", "dq_norm_w", "dk_norm_w"), got, R.rope_bwd(to_np(x), to_np(dout), *ref)):
        assert (a is None) == (b is None), name
        if b is not None:
            R.within(name, to_np(a), *b)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_beyond_2_31_elements(kind):
    """The last rows have the bits that they get alone, and the weight gradients theirs, as the others are 0."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    nq, nkv, d, last = 3, 1, 256, 500
    W = (nq + nkv) * d
    rows = (1 << 31) // W + 77
    g = torch.Generator().manual_seed(3)
    x = torch.ones((rows, W), dtype=DT[kind], device="cuda")
    dout = torch.zeros((rows, W), dtype=DT[kind], device="cuda")
    xt, dt = (torch.randn((last, W), generator=g).to(DT[kind]).cuda() for _ in range(2))
    x[-last:], dout[-last:] = xt, dt
    w = (torch.randn(d, generator=g) * 0.1 + 1).to(DT[kind]).cuda()
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pt = torch.randint(0, 9000, (last,), generator=g).to(torch.int32).cuda()
    pos[-last:] = pt
    r = T.Rotary(d)
    dx, dq, dk = T.qk_norm_rope_backward(dout, x, nq, nkv, d, r, pos, 0, w, w, EPS, dx=dout)
    a, b, c = T.qk_norm_rope_backward(dt, xt, nq, nkv, d, r, pt, 0, w, w, EPS)
    assert torch.equal(dx[-last:], a) and not dx[:-last].any()
    # the same terms, added in another order: n of them, each at most max|dout| sqrt(d), 2^-24 a sum and 24 levels
    bound = 24 * 2.0 ** -24 * float((dt.double().abs().max() * d ** 0.5) * last * nq)
    assert float((dq - b).abs().max()) <= bound and float((dk - c).abs().max()) <= bound
    T.qk_norm_rope(x, nq, nkv, d, r, pos, 0, w, w, EPS, out=x)
    assert torch.equal(x[-last:], T.qk_norm_rope(xt, nq, nkv, d, r, pt, 0, w, w, EPS))
    assert np.isfinite(float(x[0].float().sum()))
    del x, dout, dx
    torch.cuda.empty_cache()
