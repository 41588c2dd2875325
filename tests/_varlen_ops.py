"""Plain float64 forms of the attention operators over sequences of different lengths, with bounds on what a kernel
with f32 sums, one bf16 rounding of the probabilities and of the scores' gradients, and a bf16 result may be off."""
import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # 2^-8, half a step relative to the value
HALF_F32 = torch.finfo(torch.float32).eps / 2


def seen(new, past, window, sinks, device="cuda"):
    """[new, past + new]: which tokens the new ones see."""
    p = torch.arange(past, past + new, device=device)[:, None]
    t = torch.arange(past + new, device=device)[None, :]
    m = t <= p
    if window:
        m = m & ((t > p - window) | (t < sinks))
    return m


def forward(q, k, v, mask, scale):
    """q [n, nq, d], k and v [t, nkv, d] float64, mask [n, t] -> out [n, nq, d], lse [n, nq] and their bounds."""
    n, nq, d = q.shape
    hpg = nq // k.shape[1]
    K, V = (x.repeat_interleave(hpg, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, K) * scale
    # Every product is exact in f32; d additions, the scaling and the exponential's argument each round once.  The
    # exponential is off by 2^-22 and the sum of t terms by t 2^-24 at worst.
    es = torch.einsum("ihd,jhd->hij", q.abs(), K.abs()) * abs(scale) * ((d + 8) * HALF_F32)
    es = es.masked_fill(~mask, 0.0).amax(-1) + (8 + K.shape[0]) * HALF_F32 if K.shape[0] else es.sum(-1)
    s = s.masked_fill(~mask, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None]).masked_fill(~mask, 0.0)
    out = torch.einsum("hij,jhd->ihd", p, V)
    weight = torch.einsum("hij,jhd->ihd", p, V.abs())
    # probabilities rounded to bf16, the result rounded to bf16, and twice the scores' error in every probability
    tol = HALF_BF16 * (out.abs() + weight) * (1 + HALF_BF16) + 2 * es.T[..., None] * weight + 1e-30
    ltol = es.T + lse.T.abs() * 4 * HALF_F32 + 1e-6
    return out, lse.T, tol, ltol


def backward(q, k, v, dout, mask, scale):
    """Gradients of q, k, v with their bounds (shapes as in forward)."""
    nq, d = q.shape[1:]
    nkv = k.shape[1]
    hpg = nq // nkv
    K, V = (x.repeat_interleave(hpg, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, K) * scale
    es = torch.einsum("ihd,jhd->hij", q.abs(), K.abs()) * abs(scale) * ((d + 8) * HALF_F32)
    es = 2 * es.masked_fill(~mask, 0.0).amax(-1) + (16 + K.shape[0]) * HALF_F32
    p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
    out = torch.einsum("hij,jhd->ihd", p, V)
    dp = torch.einsum("ihd,jhd->hij", dout, V)
    D = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - D) * scale
    # D = sum dout . out takes the output as it was rounded (and as its probabilities were): what that may be off,
    # with the f32 sums of dP and D; P itself is off by the scores' error
    ap = torch.einsum("hij,jhd->ihd", p, V.abs())
    eD = torch.einsum("ihd,ihd->hi", dout.abs(), HALF_BF16 * (out.abs() + ap)) * (1 + HALF_BF16)
    edp = torch.einsum("ihd,jhd->hij", dout.abs(), V.abs()) * ((d + 8) * HALF_F32)
    eds = HALF_BF16 * ds.abs() * (1 + HALF_BF16) + p * (eD[..., None] + edp + edp.amax(-1, keepdim=True)) * abs(scale)
    eds = eds + es[..., None] * ds.abs()
    ep = (HALF_BF16 + es[..., None]) * p

    def group(x):  # sum over the query heads of a key head
        return x.unflatten(1, (nkv, hpg)).sum(2)

    dq = torch.einsum("hij,jhd->ihd", ds, K)
    dk = group(torch.einsum("hij,ihd->jhd", ds, q))
    dv = group(torch.einsum("hij,ihd->jhd", p, dout))
    tq = HALF_BF16 * dq.abs() + torch.einsum("hij,jhd->ihd", eds, K.abs()) * 1.01
    tk = HALF_BF16 * dk.abs() + group(torch.einsum("hij,ihd->jhd", eds, q.abs())) * 1.01
    tv = HALF_BF16 * dv.abs() + group(torch.einsum("hij,ihd->jhd", ep, dout.abs())) * 1.01
    # f32 sums of the products over tokens
    n = K.shape[0]
    tq = tq + torch.einsum("hij,jhd->ihd", ds.abs(), K.abs()) * (n * HALF_F32) + 1e-30
    tk = tk + group(torch.einsum("hij,ihd->jhd", ds.abs(), q.abs())) * (n * hpg * HALF_F32) + 1e-30
    tv = tv + group(torch.einsum("hij,ihd->jhd", p, dout.abs())) * (n * hpg * HALF_F32) + 1e-30
    return (dq, dk, dv), (tq, tk, tv)


def close(got, want, tol, what):
    """Element by element; infinities and NaN must be the same."""
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first {i}: {got[i].item()} for "
                             f"{want[i].item()} +- {tol[i].item()}")
