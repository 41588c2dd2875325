"""The attention sublayer's calls captured into a graph and replayed on new inputs: the bits of the same calls made
eagerly.

Contractions of 4096 and more are split over idle CTAs that hand partial sums over under arrival flags; 1024 and
below are not.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-6
I32 = dict(dtype=torch.int32, device="cuda")


def _weights(g, H, nq, nkv, d):
    r = lambda *s, std=0.02: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    return 1 + r(H), r((nq + 2 * nkv) * d, H), r(H, nq * d), r(H)


SIZES = [(4096, 8, 2, 128, 5), (1024, 36, 4, 128, 3), (512, 4, 1, 64, 70)]  # H, nq, nkv, d, batch


@pytest.mark.parametrize("H,nq,nkv,d,B", SIZES)
def test_decode_replays(H, nq, nkv, d, B):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = torch.Generator().manual_seed(H)
    w, steps = _weights(g, H, nq, nkv, d), 6
    xs = torch.randn(steps, B, H, generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(B * 2, **I32).reshape(B, 2)
    got = []
    for captured in (False, True):
        m = T.TPAttn(256, H, nq, nkv, d, 128, max_t=1)
        m.set_qk(T.Rotary(d))
        k, v = (torch.zeros(B * 2, nkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        kv = T.TPKV(k, v, nq, max_batch=B)
        past = torch.arange(B, **I32) % 9
        x, y = xs[0].clone(), torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
        step = lambda: (m.decode(kv, x, *w, EPS, 1, past, table, y=y), past.add_(1))  # noqa: E731
        ys, graph = [], None
        for i in range(steps):
            x.copy_(xs[i])
            if captured and graph is None:
                torch.cuda.synchronize()
                graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                m = T.TPAttn(256, H, nq, nkv, d, 128, max_t=1, stream=side)  # the sublayer's stream is the captured one
                m.set_qk(T.Rotary(d))
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    step()
            graph.replay() if graph is not None else step()
            ys.append(y.clone())
        torch.cuda.synchronize()
        kv.sync()
        got.append((torch.stack(ys), k, v))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].isfinite().all()


@pytest.mark.parametrize("H,nq,nkv,d", [s[:4] for s in SIZES])
def test_forward_and_backward_replay(H, nq, nkv, d):
    """Forward and backward on the unfused path, whose gradients have the same bits every run."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = torch.Generator().manual_seed(H + 1)
    B, S, steps = 1, 64, 4
    w = _weights(g, H, nq, nkv, d)
    xs, dys = (torch.randn(steps, B * S, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    got = []
    for captured in (False, True):
        side = torch.cuda.Stream()
        m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1, stream=side)
        qw, kw = (torch.full((d,), 1.1, dtype=torch.bfloat16, device="cuda") for _ in "qk")
        qk = m.set_qk(T.Rotary(d), qw, kw, EPS)
        x, dy, y, dx, gr = xs[0].clone(), dys[0].clone(), xs[0].clone(), xs[0].clone(), m.new_grads()
        outs = [y, dx, *gr.values(), *qk.values()]

        def step():
            m.forward(x, *w, EPS, 1, B, S, y=y)
            m.backward(dy, dx, gr)

        torch.cuda.synchronize()
        graph, res = torch.cuda.CUDAGraph(), []
        if captured:
            with torch.cuda.graph(graph, stream=side):
                step()
        for i in range(steps):
            x.copy_(xs[i])
            dy.copy_(dys[i])
            torch.cuda.synchronize()
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            res.append([t.clone() for t in outs])
        m.sync()
        got.append(res)
    for a, b in zip(*got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
