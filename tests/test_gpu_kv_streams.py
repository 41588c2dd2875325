"""The cache context's workspace, cleared on one stream and used on another."""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-6
I32 = dict(dtype=torch.int32, device="cuda")
SLEEP = 60_000_000  # cycles, some 30 ms: what is queued behind it has not run when the host goes on


def _case():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn((200, 1, 16, 128), generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    kv = T.TPKV(k, v, 4, max_batch=2)
    q = torch.randn((2, 512), generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(200, **I32)[None, :].repeat(2, 1)
    args = (q, torch.tensor([3000, 77], **I32), table)
    ref = kv.decode(*args)
    torch.cuda.synchronize()
    return T, kv, args, ref


def _rebind(T, kv):
    """A workspace of old contents, its clear still queued when this returns."""
    ws = torch.full_like(kv.workspace, 0x5A)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    assert T.lib().tpkv_bind_workspace(kv.ctx, ws.data_ptr(), ws.numel()) == 0
    return ws


def test_first_launch_on_another_stream_waits_for_the_clear():
    T, kv, args, ref = _case()
    outs = [torch.full_like(ref, 7.0) for _ in range(4)]
    side = [torch.cuda.Stream() for _ in range(2)]
    ws = _rebind(T, kv)
    for i, out in enumerate(outs):  # one stream after the other, each waiting for the one before
        with torch.cuda.stream(side[i % 2]):
            side[i % 2].wait_stream(side[1 - i % 2])
            kv.decode(*args, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs) and ws.numel()
    kv.sync()


def test_capture_behind_a_clear_on_another_stream():
    T, kv, args, ref = _case()
    out, side, graph = torch.full_like(ref, 7.0), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    ws = _rebind(T, kv)
    with torch.cuda.stream(side):
        graph.capture_begin()
        kv.decode(*args, out=out)
        graph.capture_end()
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and ws.numel()


def test_errors_cleared_on_one_stream_are_not_lost_on_another():
    """sync reports and clears; a launch on another stream right behind it reports its own."""
    T, kv, args, ref = _case()
    long = (args[0], torch.tensor([3201, 0], **I32), args[2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for s in (torch.cuda.current_stream(), side):
            with torch.cuda.stream(s):
                kv.decode(*long)
                with pytest.raises(T.TPMLPError) as e:
                    kv.sync()
                assert e.value.status == T.ERR_ARG
    assert torch.equal(kv.decode(*args), ref)
    kv.sync()


def test_sublayer_on_its_own_stream():
    """A cache built on the current stream, the sublayer that decodes through it on another."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    H, nq, nkv, d, B, n = 256, 4, 1, 64, 2, 4000
    g = torch.Generator().manual_seed(8)
    r = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    w = (1 + r(H), r((nq + 2 * nkv) * d, H), r(H, nq * d), r(H))
    k, v = r(B * 251, nkv, 16, d, std=1.0), r(B * 251, nkv, 16, d, std=1.0)
    x, past = r(B, H, std=1.0), torch.full((B,), n, **I32)
    table = torch.arange(B * 251, **I32).reshape(B, 251)
    got = []
    for own in (False, True):
        kc, vc, y = k.clone(), v.clone(), torch.full((B, H), 7.0, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream() if own else torch.cuda.current_stream()
        m = T.TPAttn(64, H, nq, nkv, d, 64, max_t=1, stream=s)
        m.set_qk(T.Rotary(d))
        kv = T.TPKV(kc, vc, nq, max_batch=B)
        ws = _rebind(T, kv) if own else None
        m.decode(kv, x, *w, EPS, 1, past, table, y=y)
        m.sync()
        kv.sync()
        got.append((y, kc, vc, ws))
    assert all(torch.equal(a, b) for a, b in zip(got[0][:3], got[1][:3]))
