"""Tensors of calls that run on another stream than the current one: dropped right after the call, while its kernels
still wait behind other work, their memory must not be handed out again before.

Each test holds the call's stream back by some 30 ms, drops what it can, and fills new tensors of the same sizes on
the current stream: the results are those of a run that holds everything, and the new tensors keep their contents.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS, LR = 1e-6, 0.1
SLEEP = 60_000_000
I32 = dict(dtype=torch.int32, device="cuda")


def _fill(sizes):
    """Tensors of these bytes, twice each, filled at once with a pattern that is neither a page nor a number."""
    return [torch.full((max(n, 1),), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]


def _kept(junk):
    return all(bool((t == 0x7F).all()) for t in junk)


def _sizes(*tensors):
    return [t.numel() * t.element_size() for t in tensors]


def _hold(stream):
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SLEEP)


def _weights(g, H, nq, nkv, d):
    r = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    return 1 + r(H), r((nq + 2 * nkv) * d, H), r(H, nq * d), r(H)


def test_workspace_of_the_norms():
    """clear_qk, and a second set_qk, while forward and backward of the first are queued."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 2, 128, 256, 4, 2, 64
    got = []
    for drop in (False, True):
        g = torch.Generator().manual_seed(3)
        w = _weights(g, H, nq, nkv, d)
        x, dy = (torch.randn(B * S, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        qw, kw = (torch.full((d,), 1.25, dtype=torch.bfloat16, device="cuda") for _ in "qk")
        side = torch.cuda.Stream()
        m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1, stream=side)
        res, junk = [], []
        for again in range(2):
            qk = m.set_qk(T.Rotary(d), qw, kw, EPS)
            y, dx, gr = torch.empty_like(x), torch.empty_like(x), m.new_grads()
            _hold(side)
            m.forward(x, *w, EPS, 1, B, S, y=y)
            m.backward(dy, dx, gr)
            if drop:
                n = m._qk[-1].numel()
                m.clear_qk() if again else m.set_qk(T.Rotary(d), qw, kw, EPS)
                junk += _fill([n])
            torch.cuda.synchronize()
            res += [t.clone() for t in (y, dx, *gr.values(), *qk.values())]
        assert _kept(junk)
        got.append(res)
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("drop", ["arguments", "all"])
def test_sublayer_calls(drop):
    """Prompts, append and decode with arguments that nobody else holds; with the cache's context dropped as well."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    B, S, H, nq, nkv, d = 2, 64, 256, 4, 2, 64
    got = []
    for dropped in (False, True):
        g = torch.Generator().manual_seed(6)
        w = _weights(g, H, nq, nkv, d)
        x = torch.randn(B * S, H, generator=g).to(torch.bfloat16).cuda()
        xt = torch.randn(B, H, generator=g).to(torch.bfloat16).cuda()
        k, v = (torch.zeros(16, nkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        side = torch.cuda.Stream()
        m = T.TPAttn(B * S, H, nq, nkv, d, S, max_t=1, stream=side)
        m.set_qk(T.Rotary(d))
        kv = T.TPKV(k, v, nq, max_batch=B)
        table, lens = torch.randperm(16, generator=g).to(torch.int32).reshape(B, 8).cuda(), torch.tensor([40, 64], **I32)
        y = torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
        _hold(side)
        m.forward(x, *w, EPS, 1, B, S)
        m.append_kv(kv, table, lens)
        m.decode(kv, xt, *w, EPS, 1, lens, table, y=y)
        junk = []
        if dropped:
            sizes = _sizes(x, xt, lens, table)
            del xt, lens, table, x
            if drop == "all":
                sizes += _sizes(kv.workspace, *w)
                m._fwd_tensors = m.params = None
                kv.close()
                del kv, w
            junk = _fill(sizes)
        torch.cuda.synchronize()
        m.sync()
        assert _kept(junk)
        got.append((y, k, v))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][0].isfinite().all()


def test_cache_and_row_calls_on_a_stream_of_their_own():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    nq, nkv, d, n = 4, 2, 64, 50
    got = []
    for drop in (False, True):
        g = torch.Generator().manual_seed(7)
        side = torch.cuda.Stream()
        k, v = (torch.zeros(8, nkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        qkv = torch.randn((n, (nq + 2 * nkv) * d), generator=g).to(torch.bfloat16).cuda()
        w = torch.full((d,), 1.5, dtype=torch.bfloat16, device="cuda")
        past, cu, lens = torch.zeros(1, **I32), torch.tensor([0, n], **I32), torch.tensor([n], **I32)
        table = torch.randperm(8, generator=g).to(torch.int32)[None, :].cuda()
        x = torch.randn((300, 3 * d), generator=g).cuda()
        kv = T.TPKV(k, v, nq, max_batch=1, stream=side)
        kv.set_rotary(T.Rotary(d), w, w, EPS)
        _hold(side)
        q = kv.append(qkv, past, table, cu_rows=cu)
        out = kv.decode(q[:1], lens, table)
        rows = T.qk_norm_rope(x, 2, 1, d, T.Rotary(d), stream=side)
        dx, _, _ = T.qk_norm_rope_backward(rows, None, 2, 1, d, T.Rotary(d), stream=side)
        junk = []
        if drop:
            sizes = _sizes(qkv, past, cu, lens, table, x, w, kv.workspace)
            kv.close()
            del qkv, past, cu, lens, table, x, w, kv
            junk = _fill(sizes)
        torch.cuda.synchronize()
        assert _kept(junk)
        got.append((q, out, rows, dx, k, v))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_arguments_are_checked_before_the_stream_is_told():
    """A CPU tensor where a device one belongs is refused as on the current stream."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    kv = T.TPKV(k, k.clone(), 1, max_batch=1, stream=torch.cuda.Stream())
    one = torch.ones(1, **I32)
    q, table = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, **I32)
    for call in (lambda: kv.decode(q, one, table.cpu()), lambda: kv.decode(q.cpu(), one, table),
                 lambda: kv.append(torch.zeros(1, 192, dtype=torch.bfloat16), one, table)):
        with pytest.raises(T.TPMLPError) as e:
            call()
        assert e.value.status == T.ERR_ARG
