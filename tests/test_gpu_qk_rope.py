"""Norm and rotation of query and key heads, forward and backward, against the formulas in float64."""
import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np

pytestmark = pytest.mark.gpu

EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _randn(g, shape, dt, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dt)


def _case(rows, nq, nkv, d, rot, kind, norm, interleaved, pos, seed=0, extra=16):
    g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + d + nq)
    dt = DT[kind]
    x = _randn(g, (rows, (nq + nkv) * d + extra), dt, 1.5)
    qw = _randn(g, (d,), dt, 0.1, 1.0) if norm in ("both", "q") else None
    kw = _randn(g, (d,), dt, 0.1, 1.0) if norm in ("both", "k") else None
    dout = _randn(g, (rows, (nq + nkv) * d), dt, 0.05)
    if pos == "far":
        p = torch.randint(-(1 << 31), (1 << 31) - 1, (rows,), generator=g).to(torch.int32)
        seq = 0
    elif pos == "given":
        p, seq = torch.randint(0, 9000, (rows,), generator=g).to(torch.int32), 0
    else:
        p, seq = None, int(pos)
    posn = p.numpy() if p is not None else (np.arange(rows) % seq if seq else np.arange(rows))
    return x, dout, qw, kw, p, seq, posn


def _cu(t):
    return None if t is None else t.cuda()


def _np(t):
    return None if t is None else to_np(t)


CASES = [  # rows, nq, nkv, d, rot, kind, norm, interleaved, positions
    (1, 32, 8, 128, 128, "bf16", "both", False, "0"),
    (1, 1, 0, 64, 64, "f32", "q", False, "0"),
    (7, 3, 1, 192, 192, "bf16", "both", True, "given"),
    (33, 4, 4, 64, 32, "f32", "both", True, "far"),
    (129, 6, 2, 256, 256, "bf16", "k", False, "far"),
    (130, 0, 5, 128, 64, "bf16", "both", False, "64"),
    (257, 5, 1, 192, 16, "f32", "none", False, "given"),
    (64, 2, 2, 128, 0, "bf16", "both", False, "0"),
    (1000, 16, 2, 128, 128, "bf16", "none", False, "100"),
    (5003, 7, 1, 128, 128, "bf16", "both", False, "given"),
    (6000, 1, 1, 64, 48, "f32", "both", True, "2000"),
    (3, 70, 1, 256, 128, "f32", "q", False, "far"),
]


@pytest.mark.parametrize("rows,nq,nkv,d,rot,kind,norm,il,pos", CASES)
def test_forward(rows, nq, nkv, d, rot, kind, norm, il, pos):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x, _, qw, kw, p, seq, posn = _case(rows, nq, nkv, d, rot, kind, norm, il, pos)
    r = T.Rotary(rot, interleaved=il) if rot else None
    xd = x.cuda()
    out = T.qk_norm_rope(xd, nq, nkv, d, r, _cu(p), seq, _cu(qw), _cu(kw), EPS)
    want, tol = R.rope(to_np(x), nq, nkv, d, posn, rot, il, _np(qw), _np(kw), EPS, kind)
    R.within("out", to_np(out), want, tol)
    # in place: the same bits, and the columns behind the heads untouched
    T.qk_norm_rope(xd, nq, nkv, d, r, _cu(p), seq, _cu(qw), _cu(kw), EPS, out=xd)
    w = (nq + nkv) * d
    assert torch.equal(xd[:, :w], out)
    assert torch.equal(xd[:, w:].cpu(), x[:, w:])


@pytest.mark.parametrize("rows,nq,nkv,d,rot,kind,norm,il,pos", CASES)
def test_backward(rows, nq, nkv, d, rot, kind, norm, il, pos):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x, dout, qw, kw, p, seq, posn = _case(rows, nq, nkv, d, rot, kind, norm, il, pos, seed=1)
    r = T.Rotary(rot, interleaved=il) if rot else None
    args = (nq, nkv, d, r, _cu(p), seq, _cu(qw), _cu(kw), EPS)
    dd, xd = dout.cuda(), x.cuda()
    dx, dqw, dkw = T.qk_norm_rope_backward(dd, xd, *args)
    (wx, tx), wq, wk = R.rope_bwd(to_np(x), to_np(dout), nq, nkv, d, posn, rot, il, _np(qw), _np(kw), EPS, kind)
    R.within("dx", to_np(dx), wx, tx)
    for name, got, want in (("dq_norm_w", dqw, wq), ("dk_norm_w", dkw, wk)):
        assert (got is None) == (want is None)
        if want is not None:
            R.within(name, to_np(got), *want)
    # in place, and again: the same bits (partial sums are added in a fixed order)
    dx2, dqw2, dkw2 = T.qk_norm_rope_backward(dd, xd, *args, dx=dd)
    assert torch.equal(dx2, dx)
    for a, b in ((dqw, dqw2), (dkw, dkw2)):
        assert a is None or torch.equal(a, b)


def test_backward_against_differences():
    """The gradient of sum(out * dout) by central differences of the float64 formula."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    rows, nq, nkv, d, rot = 3, 2, 1, 64, 32
    x, dout, qw, kw, p, seq, posn = _case(rows, nq, nkv, d, rot, "f32", "both", False, "given", extra=0)
    dx, dqw, dkw = T.qk_norm_rope_backward(dout.cuda(), x.cuda(), nq, nkv, d, T.Rotary(rot), p.cuda(), 0, qw.cuda(),
                                           kw.cuda(), EPS)
    X, Q, K, G = to_np(x), to_np(qw), to_np(kw), to_np(dout)

    def f(X, Q, K):
        return float((R.rope(X, nq, nkv, d, posn, rot, False, Q, K, EPS, "f32")[0] * G).sum())

    e = 1e-4  # truncation e^2 f''' ~ 1e-8 of the gradient's scale, cancellation 1e-16 / 1e-4
    rng = np.random.default_rng(0)
    for i, j in zip(rng.integers(0, rows, 12), rng.integers(0, X.shape[1], 12)):
        a, b = X.copy(), X.copy()
        a[i, j] += e
        b[i, j] -= e
        assert abs((f(a, Q, K) - f(b, Q, K)) / (2 * e) - float(dx[i, j])) < 2e-6
    for j in range(0, d, 7):
        a, b = Q.copy(), Q.copy()
        a[j] += e
        b[j] -= e
        assert abs((f(X, a, K) - f(X, b, K)) / (2 * e) - float(dqw[j])) < 2e-6
        a, b = K.copy(), K.copy()
        a[j] += e
        b[j] -= e
        assert abs((f(X, Q, a) - f(X, Q, b)) / (2 * e) - float(dkw[j])) < 2e-6


def test_strided_rows_and_guards():
    """Rows inside wider ones on both sides: nothing outside the heads' columns or rows is written."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    rows, nq, nkv, d = 19, 2, 1, 64
    w = (nq + nkv) * d
    base = torch.randn(rows + 2, w + 40).to(torch.bfloat16).cuda()
    x = base[1:-1, 8: 8 + w]
    dst = torch.full((rows + 2, w + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = dst[1:-1, 16: 16 + w]
    T.qk_norm_rope(x, nq, nkv, d, T.Rotary(d), seq=5, out=out)
    want, tol = R.rope(to_np(x), nq, nkv, d, np.arange(rows) % 5, d, False, None, None, EPS, "bf16")
    R.within("out", to_np(out), want, tol)
    mask = torch.ones_like(dst, dtype=torch.bool)
    mask[1:-1, 16: 16 + w] = False
    assert (dst[mask] == 7.0).all()


def test_empty_rows_zero_gradients():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x = torch.empty(0, 192, device="cuda")
    w = torch.ones(64, device="cuda")
    assert T.qk_norm_rope(x, 2, 1, 64, T.Rotary(64), q_norm_w=w).shape == (0, 192)
    dx, dqw, dkw = T.qk_norm_rope_backward(x, x, 2, 1, 64, T.Rotary(64), q_norm_w=w, k_norm_w=w)
    torch.cuda.synchronize()
    assert dx.shape == (0, 192) and not dqw.any() and not dkw.any()


def test_graph_replay_and_side_stream():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x = torch.randn(300, 3 * 128, device="cuda").to(torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    r = T.Rotary(128)
    ws = torch.empty(T.lib().tpattn_qk_rope_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    out, dx, dq, dk = torch.empty_like(x), torch.empty_like(x), torch.empty(128, **f32), torch.empty(128, **f32)

    def step():
        T.qk_norm_rope(x, 2, 1, 128, r, q_norm_w=w, k_norm_w=w, out=out)
        T.qk_norm_rope_backward(out, x, 2, 1, 128, r, q_norm_w=w, k_norm_w=w, dx=dx, dq_norm_w=dq, dk_norm_w=dk,
                                workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (out, dx, dq, dk)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    # every output is odd in x but the weight gradients, which are even
    assert torch.equal(out, -ref[0]) and torch.equal(dx, -ref[1])
    assert torch.equal(dq, ref[2]) and torch.equal(dk, ref[3])


@pytest.mark.parametrize("il", [False, True])
def test_infinity_behind_the_rotated_part_stays_there(il):
    """Values that pass take nothing from, and give nothing to, what lies beside them."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    x = torch.randn(5, 192).cuda()
    x[2, 64 + 40] = float("inf")
    x[3, 64 + 63] = float("nan")
    r = T.Rotary(32, interleaved=il)
    out = T.qk_norm_rope(x, 2, 1, 64, r)
    bad = ~out.isfinite()
    want = torch.zeros_like(bad)
    want[2, 64 + 40] = want[3, 64 + 63] = True
    assert torch.equal(bad, want)
    clean = torch.where(want, 1.0, x)
    ref = T.qk_norm_rope(clean, 2, 1, 64, r)
    assert torch.equal(out[~want], ref[~want])
    dx, _, _ = T.qk_norm_rope_backward(x, None, 2, 1, 64, r)
    assert torch.equal(~dx.isfinite(), want)
