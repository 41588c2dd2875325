"""The attention sublayer over packed sequences and over new tokens with a cache: training steps against float64
autograd of the formulas, prompts answered in pieces against the float64 forward of the whole sequences.

Tolerances are the bf16 ones of tests/_util.py.
"""
import pytest
import torch

from tests._util import compare, to_np
from tests.test_gpu_attn_serving import EPS, _inputs, _reference

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
MAIN = ("norm_w", "w_qkv", "w_o", "b_o")


def _cu(lens, first=0):
    return torch.tensor([first] + [first + int(x) for x in torch.tensor(lens).cumsum(0)], **I32)


def _want(x, p, lens, nq, nkv, d, rot, il):
    parts, at = [], 0
    for n in lens:
        if n:
            parts.append(_reference(x[at: at + n], p, 1, n, nq, nkv, d, rot, il))
        at += n
    parts.append(x[at:] + p["b_o"])  # rows of nobody: attention output 0
    return torch.cat(parts)


TRAIN = [  # lengths, rows of nobody, H, nq, nkv, d, rot, il, norm
    ([100, 1, 0, 61], 0, 256, 4, 2, 64, 64, False, True),
    ([300, 77, 130], 5, 512, 4, 1, 128, 128, False, True),
    ([90, 150], 3, 256, 3, 3, 128, 64, True, False),
    ([70, 33], 0, 128, 2, 1, 192, 96, True, True),
    ([70, 33, 140], 9, 128, 2, 2, 256, 0, False, True),
]


@pytest.mark.parametrize("lens,extra,H,nq,nkv,d,rot,il,norm", TRAIN)
def test_training_step(lens, extra, H, nq, nkv, d, rot, il, norm):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    N = sum(lens) + extra
    x, p = _inputs(1, N, H, nq, nkv, d, norm, N + d)
    g = torch.Generator().manual_seed(9)
    dy = (torch.randn(N, H, generator=g) * 0.01).to(torch.bfloat16)
    m = T.TPAttn(N, H, nq, nkv, d, 64, max_t=1)
    dev = {k: v.cuda() for k, v in p.items()}
    qk = m.set_qk(T.Rotary(rot, interleaved=il) if rot else None, dev.get("q_norm_w"), dev.get("k_norm_w"), EPS)
    y = m.forward_packed(x.cuda(), *(dev[k] for k in MAIN), EPS, 1, _cu(lens))
    dx, gr = m.backward(dy.cuda())
    m.sync()
    X = x.double().requires_grad_()
    P = {k: v.double().requires_grad_() for k, v in p.items()}
    Y = _want(X, P, lens, nq, nkv, d, rot, il)
    Y.backward(dy.double())
    compare("y", to_np(y), to_np(Y), "bf16")
    compare("dx", to_np(dx), to_np(X.grad), "bf16")
    for k in P:
        compare("d" + k, to_np({**gr, **qk}[k]), to_np(P[k].grad), "bf16")


@pytest.mark.parametrize("fused_only", [False, True])
def test_equal_sequences_and_both_forwards_in_turn(fused_only):
    """Packed sequences of equal length agree with the plain forward; the two take turns in one context."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 3, 128, 256, 4, 2, 128
    x, p = _inputs(B, S, H, nq, nkv, d, True, 3)
    dev = {k: v.cuda() for k, v in p.items()}
    w = [dev[k] for k in MAIN]
    m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1, fused_only=fused_only)
    m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
    dy = (torch.randn(B * S, H, generator=torch.Generator().manual_seed(1)) * 0.01).to(torch.bfloat16).cuda()
    xd = x.cuda()
    a = [m.forward(xd, *w, EPS, 1, B, S), *m.backward(dy)]
    b = [m.forward_packed(xd, *w, EPS, 1, _cu([S] * B)), *m.backward(dy)]
    c = [m.forward(xd, *w, EPS, 1, B, S), *m.backward(dy)]
    m.sync()
    assert torch.equal(a[0], c[0])
    for other in (b, c):
        compare("y", to_np(other[0]), to_np(a[0]), "bf16")
        compare("dx", to_np(other[1]), to_np(a[1]), "bf16")
        for k in a[2]:
            compare(k, to_np(other[2][k]), to_np(a[2][k]), "bf16")


def test_updates_follow_a_packed_step():
    """The update in backward, and SGD after it, with masters: the same bits."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    lens, H, nq, nkv, d = [100, 30], 256, 4, 2, 64
    N = sum(lens)
    got = []
    for inside in (False, True):
        x, p = _inputs(1, N, H, nq, nkv, d, False, 7)
        dev = {k: v.cuda() for k, v in p.items()}
        masters = {k: v.float() for k, v in dev.items()}
        m = T.TPAttn(N, H, nq, nkv, d, 64, max_t=1)
        m.bind_master(masters)
        m.set_update_in_backward(inside, 0.1)
        y = m.forward_packed(x.cuda(), *(dev[k] for k in MAIN), EPS, 1, _cu(lens))
        m.backward(y)
        if not inside:
            m.sgd_step(0.1)
        m.sync()
        got.append((dev, masters))
    for a, b in zip(*got):
        for k in a:
            assert torch.equal(a[k], b[k]), k


def _pages(pages, nkv, d, f8=False):
    k = torch.full((pages, nkv, 16, d), float("nan"), device="cuda").to(torch.float8_e4m3fn if f8 else torch.bfloat16)
    return k, k.clone()


@pytest.mark.parametrize("d,rot,norm", [(64, 64, True), (128, 128, True), (192, 96, False), (256, 0, True)])
def test_prompts_answered_in_pieces(d, rot, norm):
    """Packed prompts stored, two pieces of different lengths behind them, then single tokens."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, total = 256, 4, 2, [150, 41, 90]
    steps = [[100, 1, 30], [44, 33, 0], [5, 6, 59], [1, 1, 1]]
    x, p = _inputs(1, sum(total), H, nq, nkv, d, norm, 11 + d)
    starts = [0, 150, 191]
    X = [x[s: s + n] for s, n in zip(starts, total)]
    want = [_reference(v.double(), {k: t.double() for k, t in p.items()}, 1, n, nq, nkv, d, rot, False)
            for v, n in zip(X, total)]
    dev = {k: v.cuda() for k, v in p.items()}
    w = [dev[k] for k in MAIN]
    m = T.TPAttn(300, H, nq, nkv, d, 64, max_t=1)
    m.set_qk(T.Rotary(rot) if rot else None, dev.get("q_norm_w"), dev.get("k_norm_w"), EPS)
    kv = T.TPKV(*_pages(40, nkv, d), nq, max_batch=3)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(0)).to(torch.int32)[:33].reshape(3, 11).cuda()
    done = [0, 0, 0]
    for i, new in enumerate(steps):
        rows = torch.cat([v[a: a + n] for v, a, n in zip(X, done, new)]).cuda()
        past = torch.tensor(done, **I32)
        if i == 0:
            y = m.forward_packed(rows, *w, EPS, 1, _cu(new))
            m.append_kv(kv, table)
        elif i < 3:
            y = m.extend(kv, rows, *w, EPS, 1, past, table, cu_rows=_cu(new))
        else:
            y = m.decode(kv, rows, *w, EPS, 1, past, table)
        m.sync()
        kv.sync()
        ref = torch.cat([v[a: a + n] for v, a, n in zip(want, done, new)])
        compare(f"step {i}", to_np(y), to_np(ref), "bf16")
        done = [a + n for a, n in zip(done, new)]
    assert done == total


def test_extend_with_padding_and_inactive_sequences():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, d, per = 256, 4, 2, 128, 20
    new = [7, 20, 0, 11]
    x, p = _inputs(4, per, H, nq, nkv, d, True, 5)
    dev = {k: v.cuda() for k, v in p.items()}
    w = [dev[k] for k in MAIN]
    m = T.TPAttn(4 * per, H, nq, nkv, d, 64, max_t=1)
    m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
    kv = T.TPKV(*_pages(20, nkv, d), nq, max_batch=4)
    table = torch.arange(16, **I32).reshape(4, 4)
    past = torch.tensor([0, 0, 0, -1], **I32)
    m.workspace.fill_(0xFF)  # NaN wherever nothing is written
    T.lib().tpattn_bind_workspace(m.ctx, m.workspace.data_ptr(), m.workspace.numel())
    y = m.extend(kv, x.cuda(), *w, EPS, 1, past, table, new_lens=torch.tensor(new, **I32))
    m.sync()
    kv.sync()
    P = {k: v.double() for k, v in p.items()}
    for b, n in enumerate(new):
        rows = x[b * per: (b + 1) * per].double()
        ref = rows + P["b_o"]
        if n and b != 3:
            ref[:n] = _reference(rows[:n], P, 1, n, nq, nkv, d, d, False)
        compare(f"sequence {b}", to_np(y[b * per: (b + 1) * per]), to_np(ref), "bf16")


def test_extend_with_window_and_e4m3():
    """Window, sinks and an 8-bit cache agree with the operators called one by one on the same queries."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, d = 256, 4, 2, 128
    x, p = _inputs(1, 90, H, nq, nkv, d, False, 8)
    dev = {k: v.cuda() for k, v in p.items()}
    eye = torch.zeros(H, nq * d)
    eye[:, :H] = torch.eye(H)
    dev["w_o"], dev["b_o"] = eye.to(torch.bfloat16).cuda(), torch.zeros(H, dtype=torch.bfloat16, device="cuda")
    w = [dev[k] for k in MAIN]
    sc = torch.tensor([0.02, 0.03], device="cuda")
    ys = []
    for whole in (True, False):
        m = T.TPAttn(128, H, nq, nkv, d, 64, max_t=1)
        kv = T.TPKV(*_pages(12, nkv, d, True), nq, max_batch=2, k_inv_scale=sc, v_inv_scale=sc)
        table = torch.arange(12, **I32).reshape(2, 6)
        past, cu = torch.zeros(2, **I32), _cu([60, 30])
        xd = x.cuda()
        if whole:
            y = m.extend(kv, xd, *w, EPS, 1, past, table, cu_rows=cu, window=20, sinks=2)
        else:  # in two pieces
            a = m.extend(kv, torch.cat([xd[:40], xd[60:75]]), *w, EPS, 1, past, table, cu_rows=_cu([40, 15]), window=20,
                         sinks=2)
            b = m.extend(kv, torch.cat([xd[40:60], xd[75:]]), *w, EPS, 1, torch.tensor([40, 15], **I32), table,
                         cu_rows=_cu([20, 15]), window=20, sinks=2)
            y = torch.cat([a[:40], b[:20], a[40:], b[20:]])
        m.sync()
        kv.sync()
        ys.append(y)
    compare("y", to_np(ys[0]), to_np(ys[1]), "bf16")


def test_refusals_and_order():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, d = 256, 4, 2, 128
    x, p = _inputs(1, 64, H, nq, nkv, d, False, 1)
    dev = {k: v.cuda() for k, v in p.items()}
    w = [dev[k] for k in MAIN]
    m = T.TPAttn(64, H, nq, nkv, d, 64, max_t=1)
    kv = T.TPKV(*_pages(12, nkv, d), nq, max_batch=2)
    table = torch.arange(12, **I32).reshape(2, 6)
    xd, cu, past = x.cuda(), _cu([30, 34]), torch.zeros(2, **I32)
    for call, status in (
            (lambda: m.forward_packed(torch.cat([xd, xd]), *w, EPS, 1, cu), T.ERR_SHAPE),
            (lambda: m.forward_packed(xd, *w, EPS, 1, cu.long()), T.ERR_ARG),
            (lambda: m.forward_packed(xd, *w, EPS, 1, cu[:1]), T.ERR_SHAPE),
            (lambda: m.forward_packed(xd, *w, EPS, 2, cu), T.ERR_SHAPE),
            (lambda: m.forward_packed(xd, *w, -1.0, 1, cu), T.ERR_ARG),
            (lambda: m.extend(kv, torch.cat([xd, xd]), *w, EPS, 1, past, table, cu_rows=cu), T.ERR_SHAPE),
            (lambda: m.extend(kv, xd[:63], *w, EPS, 1, past, table), T.ERR_SHAPE),
            (lambda: m.extend(kv, xd, *w, EPS, 1, past, table, cu_rows=cu, new_lens=past), T.ERR_ARG),
            (lambda: m.extend(kv, xd, *w, EPS, 1, past, table, cu_rows=cu, window=-1), T.ERR_ARG),
            (lambda: m.extend(kv, xd, *w, EPS, 1, past, table[:1], cu_rows=cu), T.ERR_ARG)):
        with pytest.raises(T.TPMLPError) as e:
            call()
        assert e.value.status == status
    y = m.forward_packed(xd, *w, EPS, 1, cu)
    with pytest.raises(T.TPMLPError) as e:
        m.append_kv(kv, table, new_lens=past)
    assert e.value.status == T.ERR_ARG
    m.append_kv(kv, table)
    m.backward(y)
    m.extend(kv, xd, *w, EPS, 1, torch.tensor([30, 34], **I32), table, cu_rows=cu)
    with pytest.raises(T.TPMLPError) as e:  # its workspace is gone
        m.backward(y)
    assert e.value.status == T.ERR_ORDER
    m.sgd_step(0.1)
    m.sync()
    kv.sync()
    m.forward_packed(xd, *w, EPS, 1, torch.tensor([0, 40, 30], **I32))
    with pytest.raises(T.TPMLPError) as e:
        m.sync()
    assert e.value.status == T.ERR_ARG
    m.sync()


def test_captured_steps():
    """A packed training step and an extend step replay, with other lengths, as eager calls do."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, d, N = 256, 4, 2, 128, 200
    x, p = _inputs(1, N, H, nq, nkv, d, True, 4)
    dev = {k: v.cuda() for k, v in p.items()}
    w = [dev[k] for k in MAIN]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m = T.TPAttn(N, H, nq, nkv, d, 64, max_t=1)
        m.set_qk(T.Rotary(d), dev["q_norm_w"], dev["k_norm_w"], EPS)
        kv = T.TPKV(*_pages(60, nkv, d), nq, max_batch=2)
        xd, dy = x.cuda(), (x * 0.01).to(torch.bfloat16).cuda()
        cu, past = _cu([150, 50]), torch.zeros(2, **I32)
        table = torch.arange(60, **I32).reshape(2, 30)

        def step():
            y = m.forward_packed(xd, *w, EPS, 1, cu)
            dx, g = m.backward(dy)
            m.append_kv(kv, table)
            z = m.extend(kv, xd, *w, EPS, 1, past, table, cu_rows=cu)
            return [y, dx, z, *g.values()]

        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for lens in ([150, 50], [1, 199], [200, 0]):
        cu.copy_(_cu(lens))
        past.copy_(torch.tensor(lens, **I32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = step()
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    m.sync()
    kv.sync()
