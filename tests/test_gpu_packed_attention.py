"""Causal attention over packed sequences of different lengths and its gradients, against float64 with derived bounds
(tests/_varlen_ops.py)."""
import pytest
import torch

from tests import _varlen_ops as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _tp():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


def _inputs(lens, nq, nkv, d, seed=0, extra=0, std=1.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = sum(lens) + extra
    qkv = (torch.randn(rows, (nq + 2 * nkv) * d, generator=g, device="cuda") * std).to(BF)
    dout = torch.randn(rows, nq * d, generator=g, device="cuda").to(BF)
    cu = torch.tensor([0] + list(torch.tensor(lens, dtype=torch.int64).cumsum(0)), dtype=torch.int32, device="cuda")
    q, k, v = qkv.split([nq * d, nkv * d, nkv * d], 1)
    return q, k, v, dout, cu


def _spans(lens):
    at = 0
    for n in lens:
        if n:
            yield at, at + n
        at += n


def _h(x, heads):
    return x.double().unflatten(1, (heads, -1))


def check(lens, nq, nkv, d, window=0, sinks=0, scale=None, seed=0, grads=True, std=1.2):
    T = _tp()
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, seed, std=std)
    sc = d ** -0.5 if scale is None else scale
    out, lse = T.packed_attention(q, k, v, cu, nq, nkv, scale=scale, window=window, sinks=sinks, return_lse=True)
    gr = None
    if grads:
        gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv, scale=scale, window=window, sinks=sinks)
    T.packed_attention_check()
    for lo, hi in _spans(lens):
        mask = R.seen(hi - lo, 0, window, sinks)
        Q, K, V, G = _h(q[lo:hi], nq), _h(k[lo:hi], nkv), _h(v[lo:hi], nkv), _h(dout[lo:hi], nq)
        o, z, ot, zt = R.forward(Q, K, V, mask, sc)
        R.close(_h(out[lo:hi], nq), o, ot, f"out of rows {lo}..{hi}")
        R.close(lse[lo:hi], z, zt, f"lse of rows {lo}..{hi}")
        if grads:
            want, tol = R.backward(Q, K, V, G, mask, sc)
            for name, x, w, t, heads in zip(("dq", "dk", "dv"), gr, want, tol, (nq, nkv, nkv)):
                R.close(_h(x[lo:hi], heads), w, t, f"{name} of rows {lo}..{hi}")
    return out, lse, gr


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("nq,nkv", [(4, 1), (3, 3), (14, 2), (16, 1)])
def test_heads(d, nq, nkv):
    check([1, 130, 0, 63, 64, 65, 257, 2, 33], nq, nkv, d, seed=d + nq)


@pytest.mark.parametrize("lens", [[1], [2], [1] * 40, [127], [128], [129], [0, 0, 5, 0], [511, 1, 512, 513], [1500],
                                  [17] * 70])
def test_lengths(lens):
    check(lens, 4, 2, 128, seed=len(lens))


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 7), (128, 130), (300, 64), (5000, 4)])
def test_windows(d, window, sinks):
    check([700, 1, 129, 400], 6, 2, d, window, sinks, seed=window)


@pytest.mark.parametrize("nq,nkv,d", [(40, 1, 64), (65, 1, 128), (100, 1, 64), (200, 1, 64), (260, 2, 128)])
def test_many_heads_a_key_head(nq, nkv, d):
    check([70, 3, 141], nq, nkv, d)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scale(scale):
    check([200, 5], 4, 2, 64, scale=scale, std=0.5)


def test_large_scores():
    """Softmax that is all but one token's."""
    check([300, 130], 4, 2, 128, scale=2.0)


def test_rows_of_nobody_stay():
    T = _tp()
    lens, nq, nkv, d = [30, 100], 4, 2, 128
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, 3, extra=50)
    cu = cu + 20  # rows before the first and behind the last sequence
    out, lse = torch.full_like(dout, 7.0), torch.full((180, nq), 7.0, device="cuda")
    T.packed_attention(q, k, v, cu, nq, nkv, out=out, lse=lse)
    gr = [torch.full((180, n * d), 7.0, dtype=BF, device="cuda") for n in (nq, nkv, nkv)]
    T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv, dq=gr[0], dk=gr[1], dv=gr[2])
    T.packed_attention_check()
    ref = T.packed_attention(q[20:150], k[20:150], v[20:150], cu - 20, nq, nkv, return_lse=True)
    refg = T.packed_attention_backward(dout[20:150], q[20:150], k[20:150], v[20:150], *ref, cu - 20, nq, nkv)
    for got, want in zip((out, lse, *gr), (*ref, *refg)):
        assert torch.equal(got[20:150], want)
        assert bool((got[:20] == 7.0).all()) and bool((got[150:] == 7.0).all())


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_other_sequences_do_not_matter(d, bad):
    """What is not finite in one sequence, or in rows of nobody, reaches no other."""
    T = _tp()
    lens, nq, nkv = [77, 50, 131, 9], 4, 2
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, 5, extra=30)
    run = lambda: T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True)  # noqa: E731
    out, lse = run()
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv)
    for lo, hi in ((77, 127), (267, 297)):
        for t in (q, k, v, dout):
            t[lo:hi] = bad
    out2, lse2 = run()
    out2[267:], lse2[267:] = bad, bad
    gr2 = T.packed_attention_backward(dout, q, k, v, out2, lse2, cu, nq, nkv)
    T.packed_attention_check()
    for a, b in zip((out, lse, *gr), (out2, lse2, *gr2)):
        for lo, hi in ((0, 77), (127, 267)):
            assert torch.equal(a[lo:hi], b[lo:hi])


def test_strides_and_places():
    """Separate tensors, columns of packed rows and rows of wider ones give the same bits."""
    T = _tp()
    lens, nq, nkv, d = [90, 200], 6, 3, 64
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, 8)
    out, lse = T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True)
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv)
    wide = lambda x: torch.cat([x, x, x[:, :8]], 1)[:, x.shape[1] + 0: 2 * x.shape[1]]  # noqa: E731
    q2, k2, v2, dout2, out2 = q.contiguous(), wide(k), wide(v), wide(dout), wide(out)
    dest = wide(torch.zeros_like(out))
    assert torch.equal(T.packed_attention(q2, k2, v2, cu, nq, nkv, out=dest), out)
    grads = torch.zeros(290, (nq + 2 * nkv) * d, dtype=BF, device="cuda")
    dq, dk, dv = grads.split([nq * d, nkv * d, nkv * d], 1)
    T.packed_attention_backward(dout2, q2, k2, v2, out2, lse, cu, nq, nkv, dq=dq, dk=dk, dv=dv)
    for a, b in zip((dq, dk, dv), gr):
        assert torch.equal(a, b)
    over = q.contiguous()  # out over q
    assert torch.equal(T.packed_attention(over, k, v, cu, nq, nkv, out=over), out)


def test_repeats_give_the_same_bits():
    T = _tp()
    lens = [900, 33, 1500]
    q, k, v, dout, cu = _inputs(lens, 8, 2, 128, 4)
    first = None
    for _ in range(4):
        out, lse = T.packed_attention(q, k, v, cu, 8, 2, return_lse=True)
        got = (out, lse, *T.packed_attention_backward(dout, q, k, v, out, lse, cu, 8, 2))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_gradient_against_differences():
    """The kernels' gradient along a direction against central differences of the float64 loss sum(dout . out)."""
    T = _tp()
    lens, nq, nkv, d = [60, 141], 4, 2, 64
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, 11, std=0.8)
    out, lse = T.packed_attention(q, k, v, cu, nq, nkv, window=50, sinks=3, return_lse=True)
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv, window=50, sinks=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    dirs = [torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64) for x in (q, k, v)]

    def loss(h):
        x = [a.double() + h * e for a, e in zip((q, k, v), dirs)]
        total = 0.0
        for lo, hi in _spans(lens):
            o = R.forward(x[0][lo:hi].unflatten(1, (nq, d)), x[1][lo:hi].unflatten(1, (nkv, d)),
                          x[2][lo:hi].unflatten(1, (nkv, d)), R.seen(hi - lo, 0, 50, 3), d ** -0.5)[0]
            total = total + (o.flatten(1) * dout[lo:hi].double()).sum()
        return total

    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    got = sum((a.double() * e).sum() for a, e in zip(gr, dirs))
    # the bounds of every element, each against its part of the direction
    tol = 0.0
    for lo, hi in _spans(lens):
        _, t = R.backward(_h(q[lo:hi], nq), _h(k[lo:hi], nkv), _h(v[lo:hi], nkv), _h(dout[lo:hi], nq),
                          R.seen(hi - lo, 0, 50, 3), d ** -0.5)
        tol = tol + sum((x.flatten(1) * e[lo:hi].abs()).sum() for x, e in zip(t, dirs))
    assert abs(got - want) <= tol + 1e-6 * abs(want)
    assert abs(got - want) < 0.02 * sum((a.double().norm() * e.norm()) for a, e in zip(gr, dirs))


def test_captured_with_other_lengths():
    """A captured forward and backward replays for whatever cu_rows then hold."""
    T = _tp()
    nq, nkv, d = 4, 2, 128
    q, k, v, dout, cu = _inputs([100, 200, 84], nq, nkv, d, 2)
    run = lambda: T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True)  # noqa: E731
    bwd = lambda o: T.packed_attention_backward(dout, q, k, v, *o, cu, nq, nkv)  # noqa: E731
    bwd(run())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run()
        gr = bwd(o)
    for lens in ([100, 200, 84], [384, 0, 0], [1, 2, 381], [128, 128, 128]):
        cu.copy_(torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = run()
        for a, b in zip((*o, *gr), (*ref, *bwd(ref))):
            assert torch.equal(a, b)
    T.packed_attention_check()


def test_another_stream():
    T = _tp()
    q, k, v, dout, cu = _inputs([300, 50], 4, 2, 64, 6)
    out, lse = T.packed_attention(q, k, v, cu, 4, 2, return_lse=True)
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, 4, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2 = T.packed_attention(q, k, v, cu, 4, 2, return_lse=True, stream=side)
    g2 = T.packed_attention_backward(dout, q, k, v, *o2, cu, 4, 2, stream=side)
    side.synchronize()
    for a, b in zip((out, lse, *gr), (*o2, *g2)):
        assert torch.equal(a, b)


def test_bad_rows_are_reported():
    """cu_rows that descend or leave the rows: nothing outside the tensors is touched, and the report comes once."""
    T = _tp()
    nq, nkv, d = 2, 1, 64
    q, k, v, dout, cu = _inputs([40, 60], nq, nkv, d, 7)
    guard = torch.full((300, nq * d), 5.0, dtype=BF, device="cuda")
    for cut in ([0, 60, 40], [-5, 50, 100], [0, 50, 1000], [2 ** 31 - 1, 0, 100]):
        bad = torch.tensor(cut, dtype=torch.int32, device="cuda")
        out, lse = T.packed_attention(q, k, v, bad, nq, nkv, out=guard[100:200], return_lse=True)
        with pytest.raises(T.TPMLPError) as e:
            T.packed_attention_check()
        assert e.value.status == T.ERR_ARG
        T.packed_attention_check()
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        T.packed_attention_backward(dout, q, k, v, out, lse, bad, nq, nkv, status=word)
        assert int(word) == 2
        T.packed_attention_check()
    assert bool((guard[:100] == 5.0).all()) and bool((guard[200:] == 5.0).all())


def test_empty_calls():
    T = _tp()
    q = torch.zeros(0, 128, dtype=BF, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert T.packed_attention(q, q, q, cu, 2, 2).shape == (0, 128)
    x = torch.ones(5, 128, dtype=BF, device="cuda")
    out = torch.full_like(x, 3.0)
    T.packed_attention(x, x, x.clone(), cu, 2, 2, out=out)  # no sequences: rows of nobody
    T.packed_attention(x, x, x.clone(), torch.zeros(4, dtype=torch.int32, device="cuda"), 2, 2, out=out)
    assert bool((out == 3.0).all())


def test_many_short_sequences():
    check([1, 2, 3, 4, 5, 0, 6, 7] * 60, 2, 1, 64, seed=1)


def test_offsets_beyond_32_bits():
    """Rows that lie more than 2^31 elements apart."""
    T = _tp()
    nq, nkv, d, rows = 2, 1, 64, 200
    ld = 1 << 24  # 200 rows of 16 Mi elements: 3.3e9 elements
    big = torch.empty(rows, ld, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    parts = {n: torch.randn(rows, w * d, generator=g, device="cuda").to(BF) for n, w in
             (("q", nq), ("k", nkv), ("v", nkv), ("dout", nq), ("out", nq), ("dq", nq), ("dk", nkv), ("dv", nkv))}
    at, view = 0, {}
    for n, x in parts.items():
        view[n] = big[:, at: at + x.shape[1]]
        view[n].copy_(x)
        at += x.shape[1]
    cu = torch.tensor([0, 70, 200], dtype=torch.int32, device="cuda")
    out, lse = T.packed_attention(parts["q"], parts["k"], parts["v"], cu, nq, nkv, return_lse=True)
    gr = T.packed_attention_backward(parts["dout"], parts["q"], parts["k"], parts["v"], out, lse, cu, nq, nkv)
    _, l2 = T.packed_attention(view["q"], view["k"], view["v"], cu, nq, nkv, out=view["out"], return_lse=True)
    T.packed_attention_backward(view["dout"], view["q"], view["k"], view["v"], view["out"], l2, cu, nq, nkv,
                                dq=view["dq"], dk=view["dk"], dv=view["dv"])
    T.packed_attention_check()
    for a, b in zip((out, lse, *gr), (view["out"], l2, view["dq"], view["dk"], view["dv"])):
        assert torch.equal(a, b)
