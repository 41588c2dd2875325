"""The paged key/value cache: append and one-token attention against the formulas in float64."""
import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np

pytestmark = pytest.mark.gpu

EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _table(g, lens, page, spare=2, width=None):
    """Pages in random order, -1 behind each sequence's last page (CPU int32)."""
    need = [(max(n, 0) + page - 1) // page for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    width = width if width is not None else max(need) + 1
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at: at + n]
        at += n
    return t, total


def _caches(g, pages, nkv, page, d, kind, layout="hnd", poison=False):
    """k, v as [pages, nkv, page, d] views on the GPU; `poison` fills them with NaN."""
    shape = (pages, nkv, page, d) if layout == "hnd" else (pages, page, nkv, d)
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g)
        if poison:
            t.fill_(float("nan"))
        t = t.to(torch.bfloat16) if kind == "bf16" else (t * 30).clamp(-448, 448).to(E4M3)
        t = t.cuda()
        out.append(t if layout == "hnd" else t.transpose(1, 2))
    return out


def _scales(g, nkv, kind):
    return (None, None) if kind == "bf16" else tuple((torch.rand(nkv, generator=g) * 0.02 + 0.02).cuda() for _ in "kv")


def _values(cache, scale):
    """float64 values [pages, nkv, page, d] of a cache."""
    v = cache.float().cpu().numpy().astype(np.float64)
    return v if scale is None else v * scale.cpu().numpy().astype(np.float64)[None, :, None, None]


def _tokens(vals, table, n, page):
    """[n, nkv, d] of a sequence's first n tokens."""
    t = np.arange(n)
    return vals[table[t // page], :, t % page]


APPENDS = [  # mode, past, new, nq, nkv, d, rot, kind, norm, interleaved, page, layout
    ("one", [5], [1], 32, 8, 128, 128, "bf16", True, False, 16, "hnd"),
    ("one", [0, 15, 16, -1, 300], [1] * 5, 4, 2, 64, 64, "e4m3", True, False, 16, "nhd"),
    ("ragged", [0, 7, 100, 3, 0], [3, 0, 40, 1, 129], 6, 3, 192, 96, "bf16", True, True, 24, "hnd"),
    ("ragged", [33, 0], [500, 77], 8, 1, 128, 128, "e4m3", False, False, 64, "nhd"),
    ("padded", [0, 4, 9, 2], [6, 0, 17, 3], 2, 2, 256, 256, "bf16", True, False, 8, "hnd"),
    ("ragged", [i % 11 for i in range(1200)], [(i * 7) % 3 for i in range(1200)], 2, 1, 64, 16, "bf16", True, True, 8, "hnd"),
]


@pytest.mark.parametrize("mode,past,new,nq,nkv,d,rot,kind,norm,il,page,layout", APPENDS)
def test_append(mode, past, new, nq, nkv, d, rot, kind, norm, il, page, layout):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(len(past) * 100 + d)
    batch, W = len(past), (nq + 2 * nkv) * d
    ends = [max(p, 0) + n for p, n in zip(past, new)]
    table, pages = _table(g, ends, page)
    k, v = _caches(g, pages, nkv, page, d, kind, layout)
    ks, vs = _scales(g, nkv, kind)
    per = max(new)
    if mode == "ragged":
        off = np.concatenate([[2], 2 + np.cumsum(new)])  # two rows before the first sequence, three behind the last
        rows, cu, nl = int(off[-1]) + 3, torch.tensor(off, dtype=torch.int32).cuda(), None
        owner = [(b, i, off[b] + i) for b in range(batch) for i in range(new[b])]
    else:
        rows, cu = batch * per, None
        nl = torch.tensor(new, dtype=torch.int32).cuda() if mode == "padded" else None
        owner = [(b, i, b * per + i) for b in range(batch) for i in range(new[b])]
    owner = [o for o in owner if past[o[0]] >= 0]
    x = (torch.randn((rows, W + 8), generator=g) * 1.5).to(torch.bfloat16)
    qw, kw = ((torch.randn(d, generator=g) * 0.1 + 1).to(torch.bfloat16) if norm else None for _ in range(2))
    kv = T.TPKV(k, v, nq, max_batch=batch, k_inv_scale=ks, v_inv_scale=vs)
    kv.set_rotary(T.Rotary(rot, interleaved=il), None if qw is None else qw.cuda(), None if kw is None else kw.cuda(), EPS)
    k0, v0 = k.clone(), v.clone()
    q_out = torch.full((rows, nq * d), 3.0, dtype=torch.bfloat16, device="cuda")
    kv.append(x.cuda(), torch.tensor(past, dtype=torch.int32).cuda(), table.cuda(), cu_rows=cu, new_lens=nl, q_out=q_out)
    kv.sync()
    X = to_np(x)
    idx = np.array([o[2] for o in owner])
    pos = np.array([past[b] + i for b, i, _ in owner])
    z, tol = R.rope(X[idx], nq, nkv, d, pos, rot, il, None if qw is None else to_np(qw), None if kw is None else to_np(kw),
                    EPS, "bf16")
    qn = to_np(q_out)
    R.within("q", qn[idx], z[:, : nq * d], tol[:, : nq * d])
    rest = np.setdiff1d(np.arange(rows), idx)
    assert (qn[rest] == 3.0).all()  # rows that are nobody's
    # keys: in code units with E4M3 (half an E4M3 step, plus what the rotation may be off, in code units)
    pg, slot = table.numpy()[[o[0] for o in owner], pos // page], pos % page
    zk, tk = z[:, nq * d:].reshape(-1, nkv, d), tol[:, nq * d:].reshape(-1, nkv, d)
    got = k.float().cpu().numpy().astype(np.float64)[pg, :, slot]
    zv = X[idx][:, (nq + nkv) * d: W].reshape(-1, nkv, d)
    gv = v.float().cpu().numpy().astype(np.float64)[pg, :, slot]
    if kind == "bf16":
        R.within("k", got, zk, tk)
        assert np.array_equal(gv, zv)
    else:
        sk, sv = (t.cpu().numpy().astype(np.float64)[:, None] for t in (ks, vs))
        u = (tk - 2.0 ** -8 * np.abs(zk)) / sk  # the float32 part alone
        R.within("k", got, np.clip(zk / sk, -448, 448), 2.0 ** -4 * np.abs(zk / sk) + 2.0 ** -10 + 2 * u)
        codes = torch.from_numpy((zv / sv).astype(np.float32)).clamp(-448, 448).to(E4M3).float().numpy()
        # zv / sv was rounded from float64: equal but where that lies on a step's border
        assert (codes != gv).mean() < 1e-4
    # everything else in the cache as it was
    keep = torch.ones(pages, page, dtype=torch.bool)
    keep[torch.from_numpy(pg.astype(np.int64)), torch.from_numpy(slot)] = False
    for now, before in ((k, k0), (v, v0)):
        a = now.transpose(1, 2).contiguous().view(torch.uint8).cpu()[keep]
        b = before.transpose(1, 2).contiguous().view(torch.uint8).cpu()[keep]
        assert torch.equal(a, b)


def test_append_reports_pages_outside_the_cache():
    """A page index outside the cache and a position behind the table: not stored, reported once by sync."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k, v = torch.zeros(2, 4, 1, 16, 64, dtype=torch.bfloat16, device="cuda").unbind(0)
    kv = T.TPKV(k, v, 1)
    x = torch.ones(3, 3 * 64, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[4], [2], [-1]], dtype=torch.int32, device="cuda")
    kv.append(x, torch.tensor([0, 16, 3], dtype=torch.int32, device="cuda"), table)
    with pytest.raises(T.TPMLPError) as e:
        kv.sync()
    assert e.value.status == T.ERR_ARG and not k.any() and not v.any()
    kv.append(x, torch.tensor([-1, 15, -5], dtype=torch.int32, device="cuda"), table)
    kv.sync()
    assert k[2, 0, 15].eq(1).all() and int(k.count_nonzero()) == 64


DECODES = [  # lens, nq, nkv, d, kind, page, layout, window, sinks
    ([1], 1, 1, 64, "bf16", 16, "hnd", 0, 0),
    ([500], 32, 8, 128, "bf16", 16, "hnd", 0, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 0, 127, 1000], 8, 2, 128, "bf16", 16, "nhd", 0, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 0, 127, 1000], 8, 2, 128, "e4m3", 24, "hnd", 0, 0),
    ([5000], 1, 1, 256, "bf16", 64, "hnd", 0, 0),          # one head over every CTA: groups of joins
    ([40000], 2, 1, 64, "e4m3", 128, "nhd", 0, 0),
    ([9000], 1, 1, 192, "bf16", 64, "hnd", 0, 0),          # more parts than one CTA joins, in each head tile
    ([9000, 5], 32, 1, 192, "e4m3", 64, "nhd", 0, 0),
    ([0, 9000], 12, 1, 128, "bf16", 16, "hnd", 0, 0),
    ([20000], 30, 1, 64, "bf16", 64, "hnd", 0, 0),
    ([9000], 16, 1, 256, "bf16", 64, "nhd", 0, 0),
    ([777, 64, 3], 48, 2, 64, "bf16", 8, "hnd", 0, 0),     # 24 heads a key head: two tiles of 16
    ([777, 64, 3], 36, 3, 192, "bf16", 48, "nhd", 0, 0),   # 12 heads a key head
    ([300, 2500], 33, 3, 256, "e4m3", 32, "hnd", 0, 0),    # 11 heads a key head
    ([130, 900, 70, 64], 21, 3, 192, "e4m3", 40, "nhd", 0, 0),
    ([1, 70, 200, 2000, 64, 128, 0], 6, 3, 128, "bf16", 16, "hnd", 64, 0),
    ([1, 70, 200, 2000, 64, 128, 0], 6, 3, 64, "bf16", 48, "hnd", 100, 4),
    ([1, 70, 200, 2000, 64, 128, 0], 16, 1, 128, "e4m3", 16, "nhd", 1, 70),
    ([3000, 10], 4, 4, 256, "bf16", 128, "hnd", 333, 129),
    ([(i * 37) % 150 for i in range(700)], 2, 1, 64, "bf16", 16, "hnd", 0, 0),
]


def _decode_case(lens, nq, nkv, d, kind, page, layout, window, sinks, seed=0):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(seed * 1000 + len(lens) + d + nq)
    batch = len(lens)
    table, pages = _table(g, lens, page)
    k, v = _caches(g, pages, nkv, page, d, kind, layout)
    ks, vs = _scales(g, nkv, kind)
    # tokens behind a sequence's last one, and pages that are nobody's, hold NaN
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        used[table[b][t // page].long(), t % page] = True
    for c in (k, v):
        flat = c.transpose(1, 2)
        raw = flat if kind == "bf16" else flat.view(torch.uint8)
        raw[(~used).cuda()] = float("nan") if kind == "bf16" else 0x7F
    q = (torch.randn((batch, nq * d + 8), generator=g) * 1.5).to(torch.bfloat16)
    kv = T.TPKV(k, v, nq, max_batch=batch, k_inv_scale=ks, v_inv_scale=vs)
    return kv, q, table, k, v, ks, vs


def _check_decode(out, lse, q, table, lens, k, v, ks, vs, nq, d, page, kind, window, sinks):
    Q, K, V, tb = to_np(q), _values(k, ks), _values(v, vs), table.numpy()
    for b, n in enumerate(lens):
        t = np.arange(n)
        if window:
            t = t[(t >= n - window) | (t < sinks)]
        kk, vv = K[tb[b][t // page], :, t % page], V[tb[b][t // page], :, t % page]
        want, tol, wl, tl = R.decode(Q[b, : nq * d].reshape(nq, d), kk, vv, d ** -0.5, kind)
        R.within(f"out[{b}] of {n}", to_np(out[b]).reshape(nq, d), want, tol)
        R.within(f"lse[{b}] of {n}", to_np(lse[b]), wl, tl)


@pytest.mark.parametrize("lens,nq,nkv,d,kind,page,layout,window,sinks", DECODES)
def test_decode(lens, nq, nkv, d, kind, page, layout, window, sinks):
    kv, q, table, k, v, ks, vs = _decode_case(lens, nq, nkv, d, kind, page, layout, window, sinks)
    args = (q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    out, lse = kv.decode(*args, window=window, sinks=sinks, return_lse=True)
    kv.sync()
    _check_decode(out, lse, q, table, lens, k, v, ks, vs, nq, d, page, kind, window, sinks)
    for _ in range(3):  # the same bits, whatever CTA arrives last
        again = kv.decode(*args, window=window, sinks=sinks)
        assert torch.equal(again, out)
    kv.sync()


def test_decode_reports_pages_and_lengths_outside():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k, v = torch.ones(2, 4, 1, 16, 64, dtype=torch.bfloat16, device="cuda").unbind(0)
    kv = T.TPKV(k, v, 1)
    q = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for lens, table in (([20], [[0, 9]]), ([33], [[0, 1]]), ([20], [[-1, 1]])):
        kv.decode(q, torch.tensor(lens, **i32), torch.tensor(table, **i32))
        with pytest.raises(T.TPMLPError) as e:
            kv.sync()
        assert e.value.status == T.ERR_ARG
    out = kv.decode(q, torch.tensor([-7], **i32), torch.tensor([[0, 1]], **i32))
    kv.sync()
    assert not out.any()
    out = kv.decode(q, torch.tensor([32], **i32), torch.tensor([[0, 1]], **i32))
    kv.sync()
    assert out.eq(1).all()


def test_decode_infinite_and_nan_values_reach_their_heads_only():
    """A NaN among a sequence's own keys or values makes that head's result NaN, and no other's."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    lens = [100, 100, 100]
    kv, q, table, k, v, *_ = _decode_case(lens, 4, 2, 64, "bf16", 16, "hnd", 0, 0)
    k[int(table[0, 2]), 0, 3, 5] = float("nan")
    v[int(table[1, 1]), 1, 2, 7] = float("nan")
    out = kv.decode(q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    kv.sync()
    bad = out.view(3, 4, 64).isnan()
    assert bad[0, :2].all() and not bad[0, 2:].any()
    assert bad[1, 2:, 7].all() and int(bad[1].sum()) == 2
    assert not bad[2].any()


@pytest.mark.parametrize("kind,d,nq,nkv,il", [("bf16", 128, 8, 2, False), ("e4m3", 64, 6, 6, True)])
def test_prompt_then_tokens(kind, d, nq, nkv, il):
    """Prompts of different lengths appended at once, then four tokens each: every step's attention against the
    float64 form over the cache's own contents, with captured steps replayed."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(5)
    lens, page, steps = [40, 1, 130, 0], 16, 4
    batch, W = len(lens), (nq + 2 * nkv) * d
    table, pages = _table(g, [n + steps for n in lens], page)
    k, v = _caches(g, pages, nkv, page, d, kind, poison=True)
    ks, vs = _scales(g, nkv, kind)
    kv = T.TPKV(k, v, nq, max_batch=batch, k_inv_scale=ks, v_inv_scale=vs)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    kv.set_rotary(T.Rotary(d, interleaved=il), w, w, EPS)
    tb = table.cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    x = torch.randn((sum(lens), W), generator=g).to(torch.bfloat16).cuda()
    past = torch.zeros(batch, dtype=torch.int32, device="cuda")
    kv.append(x, past, tb, cu_rows=cu)
    past = torch.tensor(lens, dtype=torch.int32).cuda()
    xt = torch.empty(batch, W, dtype=torch.bfloat16, device="cuda")
    qo = torch.empty(batch, nq * d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(qo), torch.empty(batch, nq, dtype=torch.float32, device="cuda")

    def step():
        kv.append(xt, past, tb, q_out=qo)
        kv.decode(qo, past, tb, len_add=1, out=out, lse=lse)
        past.add_(1)

    graph = None
    for i in range(steps):
        xt.copy_(torch.randn((batch, W), generator=g).to(torch.bfloat16))
        if i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        _check_decode(out, lse, qo, table, [n + i + 1 for n in lens], k, v, ks, vs, nq, d, page, kind, 0, 0)
    kv.sync()
    assert past.tolist() == [n + steps for n in lens]


def test_append_writes_queries_in_place():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(3)
    nq, nkv, d, n = 6, 2, 128, 77
    table, pages = _table(g, [n], 16)
    (k, v), (k2, v2) = _caches(g, pages, nkv, 16, d, "bf16"), _caches(g, pages, nkv, 16, d, "bf16")
    x = torch.randn((n, (nq + 2 * nkv) * d), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    cu, past = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for kc, vc, inplace in ((k, v, False), (k2, v2, True)):
        kv = T.TPKV(kc, vc, nq, max_batch=1)
        kv.set_rotary(T.Rotary(d), w, w, EPS)
        rows = x.clone()
        got.append(kv.append(rows, past, table.cuda(), cu_rows=cu, q_out=rows if inplace else None))
        kv.sync()
    assert torch.equal(got[0], got[1][:, : nq * d])
    t = torch.arange(n)
    at = table[0][t // 16].long(), slice(None), t % 16
    assert torch.equal(k[at], k2[at]) and torch.equal(v[at], v2[at])


def test_refusals_of_a_context():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k = torch.zeros(1, 1, 65536, 64, dtype=torch.bfloat16, device="cuda")
    kv = T.TPKV(k, k.clone(), 2, max_batch=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    one, table = torch.ones(1, **i32), torch.zeros(1, 2, **i32)

    def refused(status, f):
        with pytest.raises(T.TPMLPError) as e:
            f()
        assert e.value.status == status

    refused(T.ERR_SHAPE, lambda: kv.decode(q, one, torch.zeros(1, 16385, **i32)))     # above 2^30 tokens a sequence
    refused(T.ERR_SHAPE, lambda: kv.decode(q.expand(3, 128).contiguous(), torch.ones(3, **i32), torch.zeros(3, 2, **i32)))
    refused(T.ERR_ARG, lambda: kv.decode(q, one, table, window=-1))
    refused(T.ERR_ARG, lambda: kv.decode(q, one, table, scale=float("nan")))
    refused(T.ERR_ARG, lambda: kv.decode(q.float(), one, table))
    refused(T.ERR_ARG, lambda: kv.decode(q, one.long(), table))
    refused(T.ERR_ARG, lambda: kv.decode(q, one, table.cpu()))
    refused(T.ERR_ARG, lambda: kv.decode(q[:, :64], one, table))
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    refused(T.ERR_SHAPE, lambda: kv.append(x, torch.zeros(2, **i32), torch.zeros(2, 2, **i32)))  # 3 rows for 2 sequences
    cu = torch.zeros(2, **i32)
    refused(T.ERR_ARG, lambda: kv.append(x, one, table, cu_rows=cu, new_lens=one))
    refused(T.ERR_ARG, lambda: T.TPKV(k, k[:, :, ::2], 2))
    refused(T.ERR_SHAPE, lambda: T.TPKV(k[:, :, :100], k[:, :, :100], 2))                # 100 tokens a page
    refused(T.ERR_SHAPE, lambda: T.TPKV(k[..., :32], k[..., :32], 2))                    # heads of 32
    refused(T.ERR_UNSUPPORTED, lambda: T.TPKV(k.float(), k.float(), 2))
    refused(T.ERR_ARG, lambda: T.TPKV(k, k, 2, k_inv_scale=torch.ones(1, device="cuda")))  # scales without E4M3
    kv.decode(q, one, table)
    kv.sync()


def test_fixed_stream():
    """A context on a stream of its own, called while another one is current: the same bits."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    lens = [700, 64, 1, 3000]
    kv, q, table, k, v, *_ = _decode_case(lens, 8, 2, 128, "bf16", 16, "hnd", 0, 0)
    args = (q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    ref = kv.decode(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    own = T.TPKV(k, v, 8, max_batch=4, stream=side)
    outs = [own.decode(*args) for _ in range(5)]
    x = torch.randn(9, 3 * 128, device="cuda")
    torch.cuda.synchronize()
    a = T.qk_norm_rope(x, 2, 1, 128, T.Rotary(128), stream=side)
    own.sync()
    side.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert torch.equal(a, T.qk_norm_rope(x, 2, 1, 128, T.Rotary(128)))
