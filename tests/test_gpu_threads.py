"""Calls from a thread that has made no CUDA call yet, as a server's worker makes them: every tensor is there already,
so nothing before the call makes the device's context current."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
I32 = dict(dtype=torch.int32, device="cuda")


def _tp():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


def _in_a_thread(call):
    got = []

    def body():
        try:
            call()
        except BaseException as e:  # handed over
            got.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    if got:
        raise got[0]
    torch.cuda.synchronize()


def test_packed_attention():
    T = _tp()
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, dout = (torch.randn(300, n * 64, generator=g, device="cuda").to(BF) for n in (4, 2, 2, 4))
    cu = torch.tensor([0, 170, 300], **I32)
    word = torch.zeros(1, **I32)
    want = T.packed_attention(q, k, v, cu, 4, 2, return_lse=True, status=word)
    out, lse = torch.zeros_like(q), torch.zeros(300, 4, device="cuda")
    _in_a_thread(lambda: T.packed_attention(q, k, v, cu, 4, 2, out=out, lse=lse, status=word))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    want = T.packed_attention_backward(dout, q, k, v, out, lse, cu, 4, 2, status=word)
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    ws = torch.empty(300 * 4 * 8 + 256, dtype=torch.uint8, device="cuda")
    _in_a_thread(lambda: T.packed_attention_backward(dout, q, k, v, out, lse, cu, 4, 2, dq=dq, dk=dk, dv=dv, workspace=ws,
                                                     status=word))
    assert all(torch.equal(a, b) for a, b in zip(want, (dq, dk, dv))) and int(word) == 0


def test_cache_calls():
    T = _tp()
    g = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn(24, 2, 16, 64, generator=g, device="cuda").to(BF) for _ in "kv")
    kv = T.TPKV(kc, vc, 4, max_batch=2)
    table = torch.arange(24, **I32).view(2, 12)
    past, cu = torch.tensor([20, 100], **I32), torch.tensor([0, 9, 50], **I32)
    qkv = torch.randn(50, 8 * 64, generator=g, device="cuda").to(BF)
    q = torch.empty(50, 256, dtype=BF, device="cuda")
    _in_a_thread(lambda: kv.append(qkv, past, table, cu_rows=cu, q_out=q))
    assert torch.equal(q, qkv[:, :256])
    want = kv.extend(q, past, table, cu_rows=cu)
    out = torch.zeros_like(q)
    _in_a_thread(lambda: kv.extend(q, past, table, cu_rows=cu, out=out))
    assert torch.equal(out, want)
    want = kv.decode(q[:2], past, table)
    _in_a_thread(lambda: kv.decode(q[:2], past, table, out=out[:2]))
    assert torch.equal(out[:2], want)
    kv.sync()
    # a cache bound in a thread of its own
    ptrs = kc.data_ptr(), vc.data_ptr(), *kc.stride()[:3], None, None
    status = []
    _in_a_thread(lambda: status.append(T.lib().tpkv_bind_cache(kv.ctx, *ptrs)))
    assert status == [0]


def test_fp8_gemm():
    T = _tp()
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = (torch.randn(256, 512, generator=g, device="cuda").to(BF) for _ in "ab")
    (ac, _, ai), (bc, _, bi) = (T.fp8_quantize(x, transposed=False) for x in (a, b))
    want, _ = T.fp8_gemm(ac, bc, 512, ai, bi)
    c, word, status = torch.zeros_like(want), torch.zeros(1, **I32), []
    args = (ac.data_ptr(), 512, bc.data_ptr(), 512, 256, 256, 512, ai.data_ptr(), bi.data_ptr(), c.data_ptr(), 256,
            word.data_ptr(), None)
    _in_a_thread(lambda: status.append(T.lib().tpmlp_fp8_gemm(*args)))
    assert status == [0] and torch.equal(c, want) and int(word) == 0


@pytest.mark.parametrize("packed", [False, True])
def test_sublayer(packed):
    T = _tp()
    H, nq, nkv, d, n = 256, 4, 2, 128, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.05).to(BF)  # noqa: E731
    w = [rn(H).abs() + 1, rn((nq + 2 * nkv) * d, H), rn(H, nq * d), rn(H)]
    x, cu = rn(n, H) * 20, torch.tensor([0, 100, 256], **I32)
    m = T.TPAttn(n, H, nq, nkv, d, 128, max_t=1)
    y = torch.empty_like(x)
    run = lambda: (m.forward_packed(x, *w, 1e-6, 1, cu, y=y) if packed  # noqa: E731
                   else m.forward(x, *w, 1e-6, 1, 2, 128, y=y))
    run()
    m.sync()
    want = y.clone()
    y.zero_()
    _in_a_thread(run)
    m.sync()
    assert torch.equal(y, want)
