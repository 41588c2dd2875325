"""The attention sublayer with rotation, per-head norms and a cache: a training step against float64 autograd of the
formulas, and prompts plus single tokens through the cache against the float64 forward of the whole sequences.

Tolerances are the bf16 ones of tests/_util.py.
"""
import numpy as np
import pytest
import torch

from tests._util import compare, fma_f32, to_np

pytestmark = pytest.mark.gpu

EPS = 1e-6
LR = 0.1


def _inputs(B, S, H, nq, nkv, d, norm, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *shape, std=1.0, mean=0.0: (torch.randn(*shape, generator=g) * std + mean).to(torch.bfloat16)  # noqa: E731
    p = {"norm_w": r(H, std=0.1, mean=1.0), "w_qkv": r((nq + 2 * nkv) * d, H, std=0.05), "w_o": r(H, nq * d, std=0.05),
         "b_o": r(H, std=0.01)}
    if norm:
        p["q_norm_w"], p["k_norm_w"] = r(d, std=0.1, mean=1.2), r(d, std=0.1, mean=1.2)
    return r(B * S, H), p


def _rms(h, w):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w


def _rotate(h, rot, il):
    """h [B, S, heads, d] float64 at positions 0 .. S-1."""
    S = h.shape[1]
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    a = torch.arange(S, dtype=torch.float64)[:, None] * f
    c, s = a.cos()[None, :, None, :], a.sin()[None, :, None, :]
    x, y = (h[..., 0:rot:2], h[..., 1:rot:2]) if il else (h[..., : rot // 2], h[..., rot // 2: rot])
    u, v = x * c - y * s, y * c + x * s
    z = torch.stack([u, v], -1).flatten(-2) if il else torch.cat([u, v], -1)
    return torch.cat([z, h[..., rot:]], -1)


def _reference(x, p, B, S, nq, nkv, d, rot, il, window=0, sinks=0):
    """y [B S, H] in float64 (autograd follows)."""
    n = _rms(x, p["norm_w"])
    qkv = (n @ p["w_qkv"].T).reshape(B, S, nq + 2 * nkv, d)
    q, k, v = qkv[:, :, :nq], qkv[:, :, nq: nq + nkv], qkv[:, :, nq + nkv:]
    if "q_norm_w" in p:
        q, k = _rms(q, p["q_norm_w"]), _rms(k, p["k_norm_w"])
    if rot:
        q, k = _rotate(q, rot, il), _rotate(k, rot, il)
    k, v = (t.repeat_interleave(nq // nkv, 2) for t in (k, v))
    sc = torch.einsum("bihd,bjhd->bhij", q, k) / d ** 0.5
    i, j = torch.arange(S)[:, None], torch.arange(S)[None, :]
    seen = j <= i
    if window:
        seen = seen & ((j > i - window) | (j < sinks))
    z = torch.einsum("bhij,bjhd->bihd", sc.masked_fill(~seen, float("-inf")).softmax(-1), v)
    return x + z.reshape(B * S, nq * d) @ p["w_o"].T + p["b_o"]


TRAIN = [  # B, S, H, nq, nkv, d, rot, il, norm
    (2, 128, 256, 4, 2, 64, 64, False, True),     # unfused path
    (2, 256, 512, 4, 1, 128, 128, False, True),   # fused
    (1, 384, 256, 3, 3, 128, 64, True, False),    # fused, rotation only
    (3, 64, 128, 2, 1, 192, 96, True, True),
    (2, 128, 256, 2, 2, 128, 0, False, True),     # norms only
]


@pytest.mark.parametrize("B,S,H,nq,nkv,d,rot,il,norm", TRAIN)
def test_training_step(B, S, H, nq, nkv, d, rot, il, norm):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x, p = _inputs(B, S, H, nq, nkv, d, norm, B * 100 + S + d)
    g = torch.Generator().manual_seed(9)
    dy = (torch.randn(B * S, H, generator=g) * 0.01).to(torch.bfloat16)
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1)
    dev = {k: v.cuda() for k, v in p.items()}
    masters = {k: v.float() for k, v in dev.items()}
    main = ("norm_w", "w_qkv", "w_o", "b_o")
    m.bind_master({k: masters[k] for k in main})
    qk = {}
    if norm:
        mom = [torch.zeros(d, device="cuda") for _ in range(4)]
        qk = m.set_qk(T.Rotary(rot, interleaved=il) if rot else None, dev["q_norm_w"], dev["k_norm_w"], EPS,
                      (masters["q_norm_w"], masters["k_norm_w"]), mom)
    else:
        m.set_qk(T.Rotary(rot, interleaved=il))
    fwd = lambda: m.forward(x.cuda(), dev["norm_w"], dev["w_qkv"], dev["w_o"], dev["b_o"], EPS, 1, B, S)  # noqa: E731
    y = fwd()
    dx, gr = m.backward(dy.cuda())
    m.sync()
    assert m.fused_active() == (d == 128 and S % 128 == 0)
    gr = {**{k: v.clone() for k, v in gr.items()}, **{k: v.clone() for k, v in qk.items()}}
    X = x.double().requires_grad_()
    P = {k: v.double().requires_grad_() for k, v in p.items()}
    Y = _reference(X, P, B, S, nq, nkv, d, rot, il)
    Y.backward(dy.double())
    compare("y", to_np(y), to_np(Y), "bf16")
    compare("dx", to_np(dx), to_np(X.grad), "bf16")
    for k in P:
        compare("d" + k, to_np(gr[k]), to_np(P[k].grad), "bf16")
    # the update reaches the norm weights with the others: w - lr g of the gradient that backward wrote, one rounding
    before = {k: v.clone() for k, v in masters.items()}
    m.sgd_step(LR)
    m.sync()
    for k in qk:
        want = fma_f32(np.float32(-LR), gr[k].cpu().numpy(), before[k].cpu().numpy())
        assert np.array_equal(masters[k].cpu().numpy(), want), k
        assert torch.equal(dev[k], masters[k].to(torch.bfloat16))
    if norm:
        m.new_adam_state()
        fwd()
        m.backward(dy.cuda())
        before = {k: masters[k].clone() for k in qk}
        gn = m.adamw_step(1e-3, 1, weight_decay=0.0)
        m.sync()
        total = sum(float(t.double().square().sum()) for t in {**m._grads, **qk}.values()) ** 0.5
        assert abs(float(gn) - total) <= 1e-5 * total
        for k in qk:  # a first step moves each weight by lr against its gradient's sign (g >> eps here)
            move, clip = masters[k] - before[k], min(1.0, 1.0 / (total + 1e-6))
            gk = qk[k] * clip
            want = -1e-3 * gk / (gk.abs() + 1e-8)
            # lr, the moments and the division round a few times each, the sum once more
            assert (move - want).abs().max() <= 1e-3 * 2.0 ** -18 + 2.0 ** -23 * 2


SERVE = [  # B, H, nq, nkv, d, cache, page, window, sinks
    (3, 256, 4, 2, 64, torch.bfloat16, 16, 0, 0),
    (2, 512, 8, 1, 128, torch.bfloat16, 48, 50, 4),
    (3, 256, 6, 3, 128, torch.float8_e4m3fn, 32, 0, 0),
]


@pytest.mark.parametrize("B,H,nq,nkv,d,cache,page,window,sinks", SERVE)
def test_prompt_then_decode(B, H, nq, nkv, d, cache, page, window, sinks):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    S, steps = 128, 20
    lens = [64, 37, 1][:B]
    x, p = _inputs(B, S, H, nq, nkv, d, True, 77 + d)
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=nkv)
    dev = {k: v.cuda() for k, v in p.items()}
    m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
    w = (dev["norm_w"], dev["w_qkv"], dev["w_o"], dev["b_o"], EPS)
    pages = 2 + B * ((S + page - 1) // page)
    kc = torch.full((pages, nkv, page, d), float("nan"), device="cuda").to(cache)
    sc = torch.full((nkv,), 0.02, device="cuda") if cache != torch.bfloat16 else None
    kv = T.TPKV(kc, kc.clone(), nq, max_batch=B, k_inv_scale=sc, v_inv_scale=sc)
    width = (S + page - 1) // page
    table = torch.randperm(pages)[: B * width].reshape(B, width).to(torch.int32).cuda()
    X = x.reshape(B, S, H)
    xp = X[:, :64].reshape(B * 64, H).contiguous().cuda()  # prompts padded to 64 rows
    m.forward(xp, *w, 1, B, 64)
    m.append_kv(kv, table, torch.tensor(lens, dtype=torch.int32).cuda())
    past = torch.tensor(lens, dtype=torch.int32).cuda()
    xt, y = torch.empty(B, H, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
    got = []
    for i in range(steps):
        xt.copy_(torch.stack([X[b, lens[b] + i] for b in range(B)]))
        m.decode(kv, xt, *w, nkv, past, table, window, sinks, y=y)
        past.add_(1)
        got.append(to_np(y))
    m.sync()
    kv.sync()
    P = {k: v.double() for k, v in p.items()}
    Y = to_np(_reference(x.double(), P, B, S, nq, nkv, d, d, False, window, sinks)).reshape(B, S, H)
    want = np.stack([np.stack([Y[b, lens[b] + i] for b in range(B)]) for i in range(steps)])
    # a bf16 cache rounds keys and values as the training forward's tensors are; E4M3 codes are off by up to 2^-4
    compare("y", np.stack(got), want, "bf16" if cache == torch.bfloat16 else "fp8")
    with pytest.raises(T.TPMLPError) as e:
        m.backward(xp)  # the decode has taken the forward's workspace
    assert e.value.status == T.ERR_ORDER


def test_refusals():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    m = T.TPAttn(128, 128, 2, 1, 64, 64, max_t=1)
    k = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    kv, other = T.TPKV(k, k.clone(), 2, max_batch=2), T.TPKV(k, k.clone(), 4, max_batch=2)
    tb = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for cache, status in ((kv, T.ERR_ORDER), (other, T.ERR_SHAPE)):
        with pytest.raises(T.TPMLPError) as e:
            m.append_kv(cache, tb)
        assert e.value.status == status
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(T.TPMLPError) as e:
        m.set_qk(None, one, None)
    assert e.value.status == T.ERR_ARG
    with pytest.raises(T.TPMLPError) as e:
        m.set_qk(T.Rotary(128))  # wider than the head
    assert e.value.status == T.ERR_SHAPE
    with pytest.raises(T.TPMLPError) as e:  # three sequences for a cache context of two
        z = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
        h = torch.ones(128, dtype=torch.bfloat16, device="cuda")
        m.decode(kv, z, h, torch.zeros(256, 128, dtype=torch.bfloat16, device="cuda"),
                 torch.zeros(128, 128, dtype=torch.bfloat16, device="cuda"), h, EPS, 1,
                 torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    assert e.value.status == T.ERR_SHAPE
