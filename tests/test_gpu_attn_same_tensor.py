"""One tensor given where a call writes two: refused, and where it only reads them: allowed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _refused(T, status, f):
    with pytest.raises(T.TPMLPError) as e:
        f()
    assert e.value.status == status and "same tensor" in str(e.value)


def test_norm_weights_of_queries_and_keys():
    """A weight shared by queries and keys answers, and trains no further than its gradients: an update would write it
    twice at once."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 1, 64, 128, 2, 1, 64
    g = torch.Generator().manual_seed(1)
    r = lambda *s: (torch.randn(*s, generator=g) * 0.05).to(torch.bfloat16).cuda()  # noqa: E731
    w = (1 + r(H), r((nq + 2 * nkv) * d, H), r(H, nq * d), r(H))
    x, one = r(B * S, H), 1 + r(d)
    f32 = [torch.ones(d, device="cuda") for _ in range(4)]
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1)
    m.set_qk(T.Rotary(d), one, one.clone(), EPS)
    want = m.forward(x, *w, EPS, 1, B, S)
    m.set_qk(T.Rotary(d), one, one, EPS)
    assert torch.equal(m.forward(x, *w, EPS, 1, B, S), want)
    m.backward(x)
    before = one.clone()
    _refused(T, T.ERR_ARG, lambda: m.sgd_step(0.1))
    m.new_adam_state()
    m.set_qk(T.Rotary(d), one, one, EPS, None, f32)
    m.forward(x, *w, EPS, 1, B, S)
    m.backward(x)
    _refused(T, T.ERR_ARG, lambda: m.adamw_step(1e-3, 1))
    m.sync()
    assert torch.equal(one, before)
    two = one.clone()
    _refused(T, T.ERR_ARG, lambda: m.set_qk(T.Rotary(d), one, two, EPS, (f32[0], f32[0])))
    _refused(T, T.ERR_ARG, lambda: m.set_qk(T.Rotary(d), one, two, EPS, None, (f32[0], f32[1], f32[2], f32[1])))
    m.set_qk(T.Rotary(d), one, one, EPS, f32[:2])
    m.bind_master({k: t.float() for k, t in zip(("norm_w", "w_qkv", "w_o", "b_o"), w)})
    m.set_update_in_backward(True, 0.1)
    m.forward(x, *w, EPS, 1, B, S)
    _refused(T, T.ERR_ARG, lambda: m.backward(x))


def test_keys_and_values():
    """A cache whose values are its keys can be read; an append would write each slot twice."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k = torch.randn(2, 1, 16, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv, apart = T.TPKV(k, k, 1, max_batch=1), T.TPKV(k, k.clone(), 1, max_batch=1)
    q, lens, table = k[0, 0, :1].contiguous(), torch.tensor([20], **i32), torch.tensor([[1, 0]], **i32)
    assert torch.equal(kv.decode(q, lens, table), apart.decode(q, lens, table))
    before = k.clone()
    _refused(T, T.ERR_ARG, lambda: kv.append(torch.ones(1, 192, dtype=torch.bfloat16, device="cuda"), lens, table))
    kv.sync()
    assert torch.equal(k, before)
