"""What the calls over sequences of different lengths promise beyond their formulas: which rows influence which, what
is reported, and calls at the ends of their ranges."""
import pytest
import torch

from tests import _varlen_ops as R
from tests.test_gpu_kv_extend import BF, F8, I32, Case, _tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,f8", [(64, False), (128, True), (192, False), (256, True)])
@pytest.mark.parametrize("new,past", [([5, 140, 3], [600, 900, 50]), ([2, 3, 1], [600, 900, 50])])
def test_the_first_page_past_the_end_is_reported(d, f8, new, past):
    """num_pages itself is no page; where no row sees it, it does not matter."""
    T = _tp()
    c = Case(new, past, 4, 2, d, 16, f8)
    want, wl = c.run()
    keep, pages = c.table.clone(), c.k.shape[0]
    for at in (0, 7, (past[1] + new[1] - 1) // 16):
        c.table[1, at] = pages
        out = c.kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu)
        with pytest.raises(T.TPMLPError) as e:
            c.kv.sync()
        assert e.value.status == T.ERR_ARG, at
        lo, hi = c.cul[1], c.cul[2]
        assert torch.equal(out[:lo], want[:lo]) and torch.equal(out[hi:], want[hi:]), at
        c.table.copy_(keep)
    c.table[1, (past[1] + new[1] + 15) // 16:] = pages
    assert all(torch.equal(a, b) for a, b in zip(c.run(), (want, wl)))




def _steep(q, k, spans, hot):
    """Scores whose maxima keep rising: keys grow along the rows; rows of q in `hot` are 40 times as large."""
    for lo, hi in spans:
        k[lo:hi] *= torch.linspace(0.5, 1.5, hi - lo, device="cuda")[:, None].to(k.dtype)
    for lo, hi in hot:
        q[lo:hi] *= 40.0


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("nq,nkv", [(4, 1), (3, 3), (6, 2), (5, 1)])
def test_finite_rows_of_others_do_not_matter(d, nq, nkv):
    """The bits of a sequence are the same whatever (finite) numbers its neighbours and rows of nobody hold: their
    queries lie in the same tiles, and their scores against its keys rise by more than its own."""
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    lens = [701, 50, 943, 9]
    q, k, v, dout, cu = _inputs(lens, nq, nkv, d, 5, extra=30)
    _steep(q, k, ((0, 701), (751, 1694)), ())
    run = lambda: T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True)  # noqa: E731
    out, lse = run()
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, nq, nkv)
    for lo, hi in ((701, 751), (1694, 1733)):
        for t in (q, k, v, dout):
            t[lo:hi] *= 40.0
    out2, lse2 = run()
    gr2 = T.packed_attention_backward(dout, q, k, v, out2, lse2, cu, nq, nkv)
    T.packed_attention_check()
    for a, b in zip((out, lse, *gr), (out2, lse2, *gr2)):
        for lo, hi in ((0, 701), (751, 1694)):
            assert torch.equal(a[lo:hi], b[lo:hi])


@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True), (192, True), (256, False)])
@pytest.mark.parametrize("per,new", [(70, [61, 5, 33]), (9, [5, 0, 3])])
def test_queries_of_padding_do_not_matter(d, f8, per, new):
    c = Case(new, [900, 500, 1300], 4, 2, d, 16, f8)
    kv, n = c.kv, len(new) * per
    q = torch.zeros(n, 4 * d, dtype=BF, device="cuda")
    mine = torch.zeros(n, dtype=torch.bool, device="cuda")
    for b, m in enumerate(new):
        q[b * per: b * per + m] = c.q[c.cul[b]: c.cul[b + 1]]
        mine[b * per: b * per + m] = True
    noise = torch.randn(n, 4 * d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    lens = torch.tensor(new, **I32)
    got = []
    for size in (0.0, 40.0):
        x = torch.where(mine[:, None], q, noise * size)
        got.append(kv.extend(x, c.past_dev, c.table, new_lens=lens, return_lse=True))
    kv.sync()
    for a, b in zip(*got):
        assert torch.equal(a[mine], b[mine])
    out, lse = (x[mine] for x in got[1])
    c.check(out, lse)


@pytest.mark.parametrize("nq", [3, 5, 7])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_shared_memory_of_earlier_kernels_does_not_matter(nq, d):
    """Groups that do not fill a tile: the rest of its rows hold what was in shared memory before."""
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    q, k, v, _, cu = _inputs([700, 1100], nq, 1, d, 3)
    _steep(q, k, ((0, 700), (700, 1800)), ())
    fill, kf, vf, _, cf = _inputs([4096 * 4], 8, 4, d, 4)
    want = None
    for size in (0.0, 1.0, 30.0, 1000.0):
        T.packed_attention(fill * size, kf, vf, cf, 8, 4)
        got = T.packed_attention(q, k, v, cu, nq, 1, return_lse=True)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got)), size
    T.packed_attention_check()


@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-40])
@pytest.mark.parametrize("f8", [None, False, True])
def test_a_scale_of_zero_with_large_scores(scale, f8):
    """Products of up to 2^126 count as the scale says: nothing, so that every visible token weighs the same; inverse
    scales of the cache that make it smaller still hide nothing and show nothing."""
    T = _tp()
    n, past, nq, nkv, d = 40, 200, 4, 2, 128
    c = Case([n], [past], nq, nkv, d, 16, bool(f8))
    c.q *= 2.0 ** 60
    sc = torch.tensor(scale, dtype=torch.float32).item()
    if f8 is None:
        g = torch.Generator(device="cuda").manual_seed(2)
        k, v = (torch.randn(n, nkv * d, generator=g, device="cuda").to(BF) for _ in "kv")
        k *= 2.0 ** 60
        out, lse = T.packed_attention(c.q, k, v, c.cu, nq, nkv, scale=scale, return_lse=True)
        T.packed_attention_check()
        K, V, past = k.double().unflatten(1, (nkv, d)), v.double().unflatten(1, (nkv, d)), 0
    else:
        if f8:
            c.ks *= 2.0 ** -20
            c.kd[0] *= 2.0 ** -20
        else:
            c.k *= 2.0 ** 60
            c.kd[0] *= 2.0 ** 60
        out, lse = c.run(scale=scale)
        K, V = c.kd[0], c.vd[0]
    o, z, ot, zt = R.forward(c.q.double().unflatten(1, (nq, d)), K, V, R.seen(n, past, 0, 0), sc)
    R.close(out.unflatten(1, (nq, d)), o, ot, "out")
    R.close(lse, z, zt, "lse")


@pytest.mark.parametrize("at", [0, 1 << 19, (1 << 20) - 3])
def test_many_empty_sequences_and_key_heads(at):
    """2^20 sequences, three of them with rows, and 256 key heads: nobody waits too long for the blocks."""
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    heads, d = 256, 64
    q, k, v, dout, cu = _inputs([70, 1, 229], heads, heads, d, 3)
    out, lse = T.packed_attention(q, k, v, cu, heads, heads, return_lse=True)
    gr = T.packed_attention_backward(dout, q, k, v, out, lse, cu, heads, heads)
    wide = torch.full(((1 << 20) + 1,), 300, **I32)
    wide[: at + 1] = 0
    wide[at + 1: at + 4] = cu[1:]
    out2, lse2 = T.packed_attention(q, k, v, wide, heads, heads, return_lse=True)
    gr2 = T.packed_attention_backward(dout, q, k, v, out2, lse2, wide, heads, heads)
    T.packed_attention_check()
    for a, b in zip((out, lse, *gr), (out2, lse2, *gr2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("padded", [False, True])
def test_many_sequences_without_new_tokens(padded):
    """2^20 sequences over a cache, few of them with new tokens, as row ranges and as padded rows."""
    T = _tp()
    n, nq, nkv, d = 1 << 20, 2, 2, 64
    c = Case([1] * 4, [5, 17, 40, 0], nq, nkv, d, 16)
    want, wl = c.run()
    mine = torch.tensor([0, 7, n // 2, n - 1], device="cuda")
    table = torch.zeros(n, c.table.shape[1], **I32)
    past = torch.zeros(n, **I32)
    table[mine], past[mine] = c.table, c.past_dev
    new = torch.zeros(n, **I32)
    new[mine] = 1
    kv = T.TPKV(c.k, c.v, nq, max_batch=n)
    if padded:
        q = torch.zeros(n, nq * d, dtype=BF, device="cuda")
        q[mine] = c.q
        out, lse = kv.extend(q, past, table, new_lens=new, return_lse=True)
        out, lse = out[mine], lse[mine]
    else:
        cu = torch.zeros(n + 1, **I32)
        cu[1:] = new.cumsum(0)
        out, lse = kv.extend(c.q, past, table, cu_rows=cu, return_lse=True)
    kv.sync()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_extend_over_too_many_blocks_is_refused():
    """2^20 sequences of 65536 key heads; nothing is launched, and the context goes on."""
    T = _tp()
    n, heads = 1 << 20, 65536
    k = torch.zeros(1, heads, 8, 64, dtype=BF, device="cuda")
    kv = T.TPKV(k, k.clone(), heads, max_batch=n)
    q = torch.zeros(1, heads * 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 3.0)
    zeros = torch.zeros(n + 1, **I32)
    with pytest.raises(T.TPMLPError) as e:
        kv.extend(q, zeros[:n], zeros[:n, None], cu_rows=zeros, out=out)
    assert e.value.status == T.ERR_SHAPE
    kv.sync()
    assert bool((out == 3.0).all())
    kv.extend(q, zeros[:1], zeros[:1, None], out=out)
    kv.sync()
    assert bool((out == 0.0).all())


def test_a_report_of_another_stream_is_waited_for():
    """The check sees a call that is still to come on another stream, once."""
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    q, k, v, dout, cu = _inputs([40, 60], 2, 1, 64, 7)
    bad = torch.tensor([0, 60, 40], **I32)
    T.packed_attention(q, k, v, cu, 2, 1)
    T.packed_attention_check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 0.1 s
    T.packed_attention(q, k, v, bad, 2, 1, stream=side)
    with pytest.raises(T.TPMLPError) as e:
        T.packed_attention_check()
    assert e.value.status == T.ERR_ARG
    side.synchronize()
    T.packed_attention_check()


def test_first_calls_of_two_threads_share_one_word(monkeypatch):
    import threading
    import time
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    q, k, v, dout, cu = _inputs([40, 60], 2, 1, 64, 7)
    T.packed_attention(q, k, v, cu, 2, 1)
    torch.cuda.synchronize()
    keep = dict(T.tpmlp._packed_words)
    T.tpmlp._packed_words.clear()
    made, zeros, start = [], torch.zeros, threading.Barrier(4)

    def slow(*a, **kw):
        made.append(1)
        time.sleep(0.05)
        return zeros(*a, **kw)

    rows = [cu] + [torch.tensor([0, 60, 40], **I32) for _ in range(3)]
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "zeros", slow)

    done = []

    def call(r):
        start.wait()
        T.packed_attention(q, k, v, r, 2, 1)
        done.append(1)

    threads = [threading.Thread(target=call, args=(r,)) for r in rows]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and len(done) == 4
    with pytest.raises(T.TPMLPError):
        T.packed_attention_check()
    T.packed_attention_check()
    T.tpmlp._packed_words.update(keep)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (100, 9)])
def test_how_far_a_value_that_is_not_finite_reaches(d, bad, window, sinks):
    """A value (v) of one token: its own key head and column, and tokens that see it or are less than 256 away from one
    that does; keys and queries: only tokens that see them, and their own."""
    T = _tp()
    from tests.test_gpu_packed_attention import _inputs
    nq, nkv, t = 4, 2, 700
    q, k, v, dout, cu = _inputs([300, 1500, 200], nq, nkv, d, 8)
    run = lambda: T.packed_attention(q, k, v, cu, nq, nkv, window=window, sinks=sinks, return_lse=True)  # noqa: E731
    want, wl = run()
    row, col = 300 + t, d + 5  # of key head 1
    last = 300 + t + window - 1 if window else 1799
    keep = v[row, col].clone()
    v[row, col] = bad
    out, lse = run()
    assert torch.equal(lse, wl)
    same = torch.ones_like(out, dtype=torch.bool)
    same[row - 255: min(last + 256, 1800), torch.tensor([2 * d + 5, 3 * d + 5], device="cuda")] = False
    assert torch.equal(out[same], want[same])
    sees = out[row: last + 1].unflatten(1, (nq, d))[:, 2:, 5]
    assert not bool(sees.isfinite().any())
    v[row, col] = keep
    for x, c in ((k, d + 5), (q, 2 * d + 5)):
        keep = x[row, c].clone()
        x[row, c] = bad
        out, lse = run()
        same = torch.ones(2000, nq, dtype=torch.bool, device="cuda")
        if x is k:
            same[row: last + 1, 2:] = False
        else:
            same[row, 2] = False
        # a warp's rows share the moves of their maxima, so the last bits of its others may change: both are within half
        # a step of every probability and of the result, and of the f32 sum of 1500 terms, of the same value
        assert bool(((lse[same] - wl[same]).abs() <= 2 * 1500 * R.HALF_F32 * (1 + wl[same].abs())).all())
        a, b = (y.double().unflatten(1, (nq, d))[same] for y in (out, want))
        assert bool(((a - b).abs() <= 2 * R.HALF_BF16 * 1.01 * (b.abs() + float(v.abs().max()))).all())
        x[row, c] = keep
    T.packed_attention_check()
