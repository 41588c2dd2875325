"""Attention of new tokens over a paged cache, against float64 with derived bounds (tests/_varlen_ops.py)."""
import pytest
import torch

from tests import _varlen_ops as R

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
I32 = dict(dtype=torch.int32, device="cuda")


def _tp():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


class Case:
    """A cache that holds past and new tokens of each sequence, in pages of random order; what is behind the last
    token, and every page that is nobody's, is NaN."""

    def __init__(self, new, past, nq, nkv, d, page, f8=False, seed=0, order="phsd", spare=3, share=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.past, self.nq, self.nkv, self.d, self.page = new, past, nq, nkv, d, page
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.total = [max(p, 0) + n if p >= 0 else 0 for n, p in zip(new, past)]
        need = [(t + page - 1) // page for t in self.total]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(new), max(need) + 2), -1, **I32)
        shape = (pages, nkv, page, d) if order == "phsd" else (pages, page, nkv, d)
        nan = torch.full(shape, float("nan"), device="cuda")
        self.k, self.v = ((nan.to(F8) if f8 else nan.to(BF)) for _ in "kv")
        if order != "phsd":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.ks = self.vs = None
        if f8:
            self.ks, self.vs = (torch.rand(nkv, generator=g, device="cuda") * 0.02 + 0.02 for _ in "kv")
        self.kd, self.vd, at = [], [], 0
        for b, (t, n) in enumerate(zip(self.total, need)):
            ids = perm[at: at + n]
            at += n
            self.table[b, :n] = ids
            for cache, scale, dest in ((self.k, self.ks, self.kd), (self.v, self.vs, self.vd)):
                x = (rn(t, nkv, d) * (30.0 if f8 else 1.0)).clamp(-448, 448).to(cache.dtype)
                raw, codes = (cache.view(torch.uint8), x.view(torch.uint8)) if f8 else (cache, x)
                pos = torch.arange(t, device="cuda")
                raw[ids[pos // page].long(), :, pos % page] = codes
                dest.append(x.double() * (scale.double()[:, None] if f8 else 1.0))
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu, self.rows = torch.tensor(cu, **I32), cu[-1]
        self.cul = cu
        self.q = (rn(self.rows, nq * d) * 1.3).to(BF)
        self.past_dev = torch.tensor(past, **I32)
        self.kv = _tp().TPKV(self.k, self.v, nq, max_batch=len(new), k_inv_scale=self.ks, v_inv_scale=self.vs)

    def run(self, **kw):
        out, lse = self.kv.extend(self.q, self.past_dev, self.table, cu_rows=self.cu, return_lse=True, **kw)
        self.kv.sync()
        return out, lse

    def check(self, out, lse, window=0, sinks=0, scale=None):
        sc = self.d ** -0.5 if scale is None else scale
        for b, (n, p) in enumerate(zip(self.new, self.past)):
            lo, hi = self.cul[b], self.cul[b + 1]
            if n == 0:
                continue
            if p < 0:
                assert bool((out[lo:hi] == 0).all()) and bool((lse[lo:hi] == float("-inf")).all())
                continue
            q = self.q[lo:hi].double().unflatten(1, (self.nq, self.d))
            o, z, ot, zt = R.forward(q, self.kd[b], self.vd[b], R.seen(n, p, window, sinks), sc)
            R.close(out[lo:hi].unflatten(1, (self.nq, self.d)), o, ot, f"out of sequence {b}")
            R.close(lse[lo:hi], z, zt, f"lse of sequence {b}")


NEW = [1, 5, 0, 130, 64, 3, 257, 33]
PAST = [0, 700, 12, 0, 64, -1, 129, 2000]


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("nq,nkv", [(8, 2), (3, 3), (14, 2), (16, 1)])
def test_heads_and_types(d, f8, nq, nkv):
    c = Case(NEW, PAST, nq, nkv, d, 16, f8, seed=d + nq)
    c.check(*c.run())


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 200, 1024])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("order", ["phsd", "pshd"])
def test_pages(page, f8, order):
    c = Case(NEW, PAST, 4, 2, 128, page, f8, seed=page, order=order)
    c.check(*c.run())


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (64, 0), (100, 7), (129, 200), (1000, 64), (9000, 4)])
@pytest.mark.parametrize("f8", [False, True])
def test_windows(d, window, sinks, f8):
    c = Case([3, 300, 40, 700], [1500, 700, 90, 0], 6, 2, d, 24, f8, seed=window)
    c.check(*c.run(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [5000]), ([16], [484]), ([64], [9000]), ([7], [30000]),
                                      ([300], [12000]), ([1, 1, 1], [1, 20000, 127]), ([2] * 30, [999] * 30),
                                      ([5] * 3, [8192, 10, 3000]), ([1] * 90, [300] * 90)])
@pytest.mark.parametrize("d,f8", [(128, False), (128, True), (64, False), (192, False), (256, True)])
def test_few_rows_over_long_caches(new, past, d, f8):
    c = Case(new, past, 8, 2, d, 64, f8, seed=len(new))
    c.check(*c.run())


@pytest.mark.parametrize("nq,nkv,d", [(40, 1, 64), (65, 1, 128), (100, 1, 64), (200, 1, 64), (260, 2, 128), (160, 1, 256)])
def test_many_heads_a_key_head(nq, nkv, d):
    c = Case([70, 3, 141], [5, 600, 0], nq, nkv, d, 32)
    c.check(*c.run())


@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_scale(scale):
    c = Case([200, 5], [30, 400], 4, 2, 128, 16)
    c.check(*c.run(scale=scale), scale=scale)


def test_freed_pages_before_a_window_are_not_read():
    """Table entries of pages that every row's window has left may be anything."""
    c = Case([40, 3], [3000, 1000], 4, 2, 128, 16)
    want = c.run(window=100, sinks=5)
    for b, (n, p) in enumerate(zip(c.new, c.past)):
        c.table[b, 1: (p + 1 - 100) // 16] = torch.tensor([-7, 10 ** 9] * 100, **I32)[: (p + 1 - 100) // 16 - 1]
    got = c.run(window=100, sinks=5)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_padded_rows_stay():
    """Without cu_rows, each sequence has the same number of rows, new_lens of them tokens."""
    new, past, per = [5, 0, 9, 2], [100, 3, 0, 77], 9
    c = Case(new, past, 4, 2, 128, 16)
    want, wl = c.run()
    q = torch.full((4 * per, 512), float("nan"), dtype=BF, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((4 * per, 4), 7.0, device="cuda")
    for b, n in enumerate(new):
        q[b * per: b * per + n] = c.q[c.cul[b]: c.cul[b + 1]]
    c.kv.extend(q, c.past_dev, c.table, new_lens=torch.tensor(new, **I32), out=out, lse=lse)
    c.kv.sync()
    for b, n in enumerate(new):
        lo = b * per
        assert torch.equal(out[lo: lo + n], want[c.cul[b]: c.cul[b + 1]])
        assert torch.equal(lse[lo: lo + n], wl[c.cul[b]: c.cul[b + 1]])
        assert bool((out[lo + n: lo + per] == 7.0).all()) and bool((lse[lo + n: lo + per] == 7.0).all())


def test_rows_of_nobody_stay():
    c = Case([30, 100], [7, 400], 4, 2, 64, 16)
    want, wl = c.run()
    q = torch.cat([c.q[:20] * float("nan"), c.q, c.q[:9] * float("nan")])
    out, lse = torch.full_like(q, 7.0), torch.full((159, 4), 7.0, device="cuda")
    c.kv.extend(q, c.past_dev, c.table, cu_rows=c.cu + 20, out=out, lse=lse)
    c.kv.sync()
    assert torch.equal(out[20:150], want) and torch.equal(lse[20:150], wl)
    for x in (out, lse):
        assert bool((x[:20] == 7.0).all()) and bool((x[150:] == 7.0).all())


def test_in_place_and_strides():
    c = Case([30, 100], [7, 400], 4, 2, 128, 16)
    want, _ = c.run()
    wide = torch.cat([c.q, c.q], 1)
    c.kv.extend(wide[:, :512], c.past_dev, c.table, cu_rows=c.cu, out=wide[:, :512])
    assert torch.equal(wide[:, :512], want) and torch.equal(wide[:, 512:], c.q)


def test_agrees_with_decode():
    """One new token a sequence, against the one-token operator: both within their bounds of the same value."""
    c = Case([1] * 6, [0, 15, 16, 500, 4000, 129], 8, 2, 128, 16)
    out, lse = c.run()
    c.check(out, lse)
    o, z = c.kv.decode(c.q, c.past_dev, c.table, len_add=1, return_lse=True)
    c.kv.sync()
    c.check(o, z)


def test_bad_pages_and_lengths_are_reported():
    T = _tp()
    for spoil in ("page", "negative", "capacity", "huge"):
        c = Case([5, 140, 3], [600, 900, 50], 4, 2, 128, 16)
        want = c.run()[0]
        keep_table, keep_past = c.table.clone(), c.past_dev.clone()
        if spoil == "page":
            c.table[1, 7] = 10 ** 8
        elif spoil == "negative":
            c.table[1, 60] = -3
        elif spoil == "capacity":
            c.past_dev[1] = c.table.shape[1] * 16 - 100
        else:
            c.past_dev[1] = 2 ** 31 - 1
        out = c.kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu)
        with pytest.raises(T.TPMLPError) as e:
            c.kv.sync()
        assert e.value.status == T.ERR_ARG, spoil
        assert torch.equal(out[:5], want[:5]) and torch.equal(out[145:], want[145:]), spoil
        c.table.copy_(keep_table)
        c.past_dev.copy_(keep_past)
        assert torch.equal(c.run()[0], want), spoil


def test_bad_cu_rows_are_reported():
    T = _tp()
    c = Case([5, 140, 3], [600, 900, 50], 4, 2, 128, 16)
    for cut in ([0, 5, 2, 148], [0, 5, 145, 1000], [-9, 5, 145, 148]):
        guard = torch.full((400, 512), 5.0, dtype=BF, device="cuda")
        c.kv.extend(c.q, c.past_dev, c.table, cu_rows=torch.tensor(cut, **I32), out=guard[100:248])
        with pytest.raises(T.TPMLPError) as e:
            c.kv.sync()
        assert e.value.status == T.ERR_ARG
        assert bool((guard[:100] == 5.0).all()) and bool((guard[248:] == 5.0).all())
    c.check(*c.run())


def test_captured_with_grown_lengths():
    """A captured step replays with lengths and tables that have changed, split or not."""
    c = Case([16, 16], [3000, 40], 8, 2, 128, 16)
    run = lambda: c.kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu, return_lse=True)  # noqa: E731
    run()
    c.kv.sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for past in ([3000, 40], [0, 0], [100, 24], [2900, 39]):
        c.past_dev.copy_(torch.tensor(past, **I32))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.kv.sync()


def test_repeats_and_turns_with_decode_give_the_same_bits():
    """The two operators share the context's workspace, one call behind the other."""
    c = Case([16], [6000], 8, 2, 128, 16)
    first = None
    lens = torch.tensor([6016], **I32)
    for _ in range(5):
        got = [*c.run(), c.kv.decode(c.q[:1], lens, c.table)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_two_contexts_at_once():
    cs = [Case([16], [20000], 8, 2, 128, 16, seed=s) for s in range(2)]
    want = [c.run() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(c.kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu, return_lse=True))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_cache_beyond_32_bits():
    """Pages that lie more than 2^31 elements apart."""
    T = _tp()
    pages, page, nkv, d = 140, 64, 2, 128
    big = torch.empty(pages, 1 << 24, dtype=BF, device="cuda")  # 2.3e9 elements
    k = big[:, : nkv * page * d].unflatten(1, (nkv, page, d))
    v = big[:, nkv * page * d: 2 * nkv * page * d].unflatten(1, (nkv, page, d))
    g = torch.Generator(device="cuda").manual_seed(0)
    for x in (k, v):
        x.copy_(torch.randn(pages, nkv, page, d, generator=g, device="cuda"))
    q = torch.randn(50, 8 * d, generator=g, device="cuda").to(BF)
    table = torch.arange(pages, **I32).flip(0)[None]
    past = torch.tensor([pages * page - 50], **I32)
    got = T.TPKV(k, v, 8, max_batch=1).extend(q, past, table)
    kc, vc = k.contiguous(), v.contiguous()
    want = T.TPKV(kc, vc, 8, max_batch=1).extend(q, past, table)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool(got.isfinite().all())


def test_shared_pages_and_values_that_are_the_keys():
    """Two sequences with the same beginning; a cache whose values are its keys."""
    T = _tp()
    c = Case([6, 9], [64, 64], 4, 2, 128, 16)
    c.table[1, :4] = c.table[0, :4]
    c.kd[1][:64], c.vd[1][:64] = c.kd[0][:64], c.vd[0][:64]
    c.check(*c.run())
    kv = T.TPKV(c.k, c.k, 4, max_batch=2)
    out, lse = kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu, return_lse=True)
    c.vd = c.kd
    c.check(out, lse)


def _inf_keys(c):
    """Keys of sequence 0 whose first value is -inf, the last token's of key head 1 NaN."""
    n = c.total[0]
    raw = torch.full((n, 2, 128), 0.5, dtype=BF, device="cuda")
    raw[:, :, 0] = float("-inf")
    raw[n - 1, 1, 0] = float("nan")
    pos = torch.arange(n, device="cuda")
    c.k[c.table[0][pos // 16].long(), :, pos % 16] = raw


def test_scores_of_infinity():
    """All scores -inf: out NaN, lse -inf; a NaN score: both NaN; as for one token."""
    c = Case([3], [20], 4, 2, 128, 16)
    _inf_keys(c)
    q = c.q.zero_().unflatten(1, (4, 128))
    q[:, :, 0] = 1.0
    out, lse = c.run()
    o = out.unflatten(1, (4, 128))
    assert bool(o.isnan().all())
    assert bool((lse[:, :2] == float("-inf")).all()) and bool((lse[:2, 2:] == float("-inf")).all())
    assert bool(lse[2, 2:].isnan().all())


def test_scores_of_zero_times_infinity():
    """One head's scores are all -inf, the others' 0 times -inf: NaN."""
    c = Case([3], [20], 4, 2, 128, 16)
    c.q[:] = 0
    c.q[:, 0] = 1.0
    _inf_keys(c)
    out, lse = c.run()
    assert bool(out.isnan().all())
    assert bool((lse[:, 0] == float("-inf")).all()) and bool(lse[:, 1:].isnan().all())
