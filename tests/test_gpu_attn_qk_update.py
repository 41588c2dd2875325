"""Updates of the attention sublayer's query and key norm weights: inside backward, and after a decode.

Each new fp32 master equals fmaf(-lr, g, w) of the gradient that the same backward wrote, bit for bit, and its bf16
copy is that rounded; on the unfused path, which has no atomics, the whole step has the bits of backward followed by
``sgd_step``.
"""
import numpy as np
import pytest
import torch

from tests._util import fma_f32, to_np

pytestmark = pytest.mark.gpu

EPS, LR = 1e-6, 0.1
MAIN, QK = ("norm_w", "w_qkv", "w_o", "b_o"), ("q_norm_w", "k_norm_w")


def _inputs(N, H, nq, nkv, d):
    g = torch.Generator().manual_seed(N + H + d)
    r = lambda *shape, std=1.0, mean=0.0: (torch.randn(*shape, generator=g) * std + mean).to(torch.bfloat16)  # noqa: E731
    p = {"norm_w": r(H, std=0.1, mean=1.0), "w_qkv": r((nq + 2 * nkv) * d, H, std=0.05), "w_o": r(H, nq * d, std=0.05),
         "b_o": r(H, std=0.01), "q_norm_w": r(d, std=0.1, mean=1.2), "k_norm_w": r(d, std=0.1, mean=1.2)}
    return r(N, H), r(N, H, std=0.01), p


def _step(B, S, H, nq, nkv, d, in_backward):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x, dy, p = _inputs(B * S, H, nq, nkv, d)
    dev = {k: v.cuda() for k, v in p.items()}
    ms = {k: v.float() for k, v in dev.items()}
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1)
    m.bind_master({k: ms[k] for k in MAIN})
    qk = m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS, (ms["q_norm_w"], ms["k_norm_w"]))
    if in_backward:
        m.set_update_in_backward(True, LR)
    y = m.forward(x.cuda(), dev["norm_w"], dev["w_qkv"], dev["w_o"], dev["b_o"], EPS, 1, B, S)
    dx, g = m.backward(dy.cuda())
    if in_backward:
        with pytest.raises(T.TPMLPError) as e:
            m.sgd_step(LR)
        assert e.value.status == T.ERR_ORDER
    else:
        m.sgd_step(LR)
    m.sync()
    assert m.update_in_epilogue() == (in_backward and B * S >= 8192)
    return p, {**g, **qk}, ms, dev, y, dx, m.fused_active()


@pytest.mark.parametrize("B,S,H,nq,nkv,d", [
    (2, 128, 256, 4, 2, 64),    # unfused, the update kernel
    (2, 256, 512, 4, 1, 128),   # fused, the update kernel
    (9, 960, 328, 4, 2, 64),    # unfused, matrices updated in their epilogues
    (4, 2048, 512, 4, 2, 128),  # fused, the same
])
def test_update_in_backward(B, S, H, nq, nkv, d):
    runs = {b: _step(B, S, H, nq, nkv, d, b) for b in (False, True)}
    for p, g, ms, dev, *_ in runs.values():
        for k in MAIN + QK:
            want = fma_f32(np.float32(-LR), g[k].cpu().numpy(), p[k].float().numpy())
            np.testing.assert_array_equal(ms[k].cpu().numpy(), want, err_msg=k)
            assert torch.equal(dev[k], ms[k].to(torch.bfloat16)), k
    (_, g0, m0, d0, y0, dx0, fused), (_, g1, m1, d1, y1, dx1, _) = runs[False], runs[True]
    assert torch.equal(y0, y1)
    if not fused:
        assert torch.equal(dx0, dx1)
        for a, b in ((g0, g1), (m0, m1), (d0, d1)):
            assert all(torch.equal(a[k], b[k]) for k in MAIN + QK)


def test_update_in_backward_needs_every_master():
    """Without masters of the norm weights the update would be lost in bf16 roundings: refused, nothing written."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 1, 64, 128, 2, 1, 64
    x, dy, p = _inputs(B * S, H, nq, nkv, d)
    dev = {k: v.cuda() for k, v in p.items()}
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1)
    m.bind_master({k: dev[k].float() for k in MAIN})
    m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
    m.set_update_in_backward(True, LR)
    m.forward(x.cuda(), dev["norm_w"], dev["w_qkv"], dev["w_o"], dev["b_o"], EPS, 1, B, S)
    with pytest.raises(T.TPMLPError) as e:
        m.backward(dy.cuda())
    assert e.value.status == T.ERR_ORDER
    m.sync()
    assert all(torch.equal(dev[k].cpu(), p[k]) for k in p)
    m.set_update_in_backward(False)
    m.backward(dy.cuda())
    m.sgd_step(LR)  # in bf16, as asked for
    m.sync()
    assert not torch.equal(dev["q_norm_w"].cpu(), p["q_norm_w"])


def test_update_after_a_decode():
    """A decode between backward and the update takes the forward's workspace, not the gradients."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 1, 64, 128, 2, 1, 64
    x, dy, p = _inputs(B * S, H, nq, nkv, d)
    got = []
    for decode in (False, True):
        dev = {k: v.cuda() for k, v in p.items()}
        m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1)
        m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
        w = [dev[k] for k in MAIN]
        m.forward(x.cuda(), *w, EPS, 1, B, S)
        m.backward(dy.cuda())
        if decode:
            k = torch.zeros(1, nkv, 16, d, dtype=torch.bfloat16, device="cuda")
            kv = T.TPKV(k, k.clone(), nq, max_batch=1)
            z = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
            m.decode(kv, x[:1].cuda(), *w, EPS, 1, z[0], z)
            with pytest.raises(T.TPMLPError) as e:
                m.backward(dy.cuda())
            assert e.value.status == T.ERR_ORDER
        m.sgd_step(LR)
        m.sync()
        got.append({k: to_np(v) for k, v in dev.items()})
    for k in p:
        np.testing.assert_array_equal(got[0][k], got[1][k], err_msg=k)
