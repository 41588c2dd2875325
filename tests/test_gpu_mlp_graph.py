"""The MLP's forward and backward captured into a graph and replayed on new inputs: the bits of the eager calls.

Its contractions of 4096 and more (the hidden and ffn sizes here) are split over idle CTAs that hand partial sums over
under arrival flags.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("tokens,H,F,t", [(64, 4096, 4608, 1), (200, 512, 4096, 4), (136, 256, 768, 2)])
def test_forward_and_backward_replay(tokens, H, F, t):
    from tensor_transformer_mlp_rmsnorm_gb300 import TPMLP
    g = torch.Generator().manual_seed(H)
    r = lambda *s, std=0.02: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    w = (1 + r(H), r(2, F, H), r(H, F), r(H))
    steps = 4
    xs, dys = r(steps, tokens, H, std=1.0), r(steps, tokens, H, std=1.0)
    got = []
    for captured in (False, True):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            m = TPMLP(tokens, H, F, max_t=t, dtype="bf16")
        x, dy, y, dx, gr = xs[0].clone(), dys[0].clone(), xs[0].clone(), xs[0].clone(), m.new_grads()

        def step():
            m.forward(x, *w, EPS, t, y=y)
            m.backward(dy, dx=dx, grads=gr)

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
            res.append([v.clone() for v in (y, dx, *gr.values())])
        m.sync()
        got.append(res)
    for a, b in zip(*got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
