"""The cache calls over what the other tests leave out: more query heads a key head than one tile holds, tables that
share and repeat pages or lie in wider ones, caches of more than 2^31 elements, and the log-sum-exp by itself."""
import math

import numpy as np
import pytest
import torch

from tests._util import to_np
from tests.test_gpu_kv_cache import _check_decode, _decode_case, _gen

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
I32 = dict(dtype=torch.int32, device="cuda")

MANY_HEADS = [  # lens, nq, nkv, d, kind, page, layout, window, sinks
    ([500, 1, 0, 64, 2100], 40, 1, 64, "bf16", 16, "hnd", 0, 0),      # 32 + 8 heads
    ([300, 77], 130, 2, 128, "e4m3", 32, "nhd", 0, 0),                # 32 + 32 + 1
    ([9000], 100, 1, 128, "bf16", 64, "hnd", 0, 0),                   # joins over many CTAs in each chunk
    ([700, 129], 66, 2, 192, "e4m3", 48, "hnd", 100, 4),              # 32 + 1, windowed
    ([2000, 3], 64, 1, 256, "bf16", 16, "nhd", 0, 0),                 # 32 + 32
]


@pytest.mark.parametrize("lens,nq,nkv,d,kind,page,layout,window,sinks", MANY_HEADS)
def test_more_query_heads_than_a_tile(lens, nq, nkv, d, kind, page, layout, window, sinks):
    kv, q, table, k, v, ks, vs = _decode_case(lens, nq, nkv, d, kind, page, layout, window, sinks, seed=3)
    args = (q.cuda(), torch.tensor(lens, **I32), table.cuda())
    out, lse = kv.decode(*args, window=window, sinks=sinks, return_lse=True)
    kv.sync()
    _check_decode(out, lse, q, table, lens, k, v, ks, vs, nq, d, page, kind, window, sinks)
    rows = args[0].clone()  # in place, the same bits: a chunk's queries are read before another's output is written
    assert torch.equal(kv.decode(rows, *args[1:], window=window, sinks=sinks, out=rows)[:, : nq * d], out)
    kv.sync()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 64)])
def test_tables_that_share_and_repeat_pages(kind, d):
    """A prefix shared by all sequences, a page that one of them has twice, and a table in the columns of a wider one."""
    lens, nq, nkv, page = [300, 170, 96, 500], 8, 2, 16
    kv, q, table, k, v, ks, vs = _decode_case([500], nq, nkv, d, kind, page, "hnd", 0, 0, seed=5)
    g = _gen(9)
    one = table[0, :32]
    shared = torch.stack([torch.cat([one[:4], one[torch.randint(0, 31, (28,), generator=g)]]) for _ in lens])
    shared[1, 5] = shared[1, 2]
    wide = torch.full((4, 50), 1 << 30, dtype=torch.int32)
    wide[:, 9:41] = shared
    q = torch.randn((4, nq * d), generator=g).to(torch.bfloat16)
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    kv = T.TPKV(k, v, nq, max_batch=4, k_inv_scale=ks, v_inv_scale=vs)
    n = torch.tensor(lens, **I32)
    out, lse = kv.decode(q.cuda(), n, wide.cuda()[:, 9:41], return_lse=True)
    kv.sync()
    _check_decode(out, lse, q, shared, lens, k, v, ks, vs, nq, d, page, kind, 0, 0)
    assert torch.equal(out, kv.decode(q.cuda(), n, shared.cuda()))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_caches_of_more_than_2_31_elements(kind):
    """Appends and decodes over pages at both ends of a large cache: the bits of a small one with the same pages."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    nq, nkv, d, page, few = 4, 2, 128, 64, 12
    dt = torch.bfloat16 if kind == "bf16" else E4M3
    pages = (1 << 31) // (nkv * page * d) + 40
    g = _gen(11)
    lens, new = [150, 64, 0, 5], [40, 3, 130, 1]
    small = torch.randperm(few, generator=g).to(torch.int32).reshape(4, 3)
    large = torch.where(small < few // 2, small, pages - few + small)
    x = torch.randn((sum(new), (nq + 2 * nkv) * d), generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **I32)
    past, q = torch.tensor(lens, **I32), torch.randn((4, nq * d), generator=g).to(torch.bfloat16).cuda()
    fill = torch.randn((2, few, nkv, page, d), generator=g).to(dt).cuda()
    got = []
    for n, table in ((few, small), (pages, large)):
        at = torch.arange(few, device="cuda") if n == few else torch.arange(few, device="cuda") + torch.where(
            torch.arange(few, device="cuda") < few // 2, 0, pages - few)
        caches = []
        for i in range(2):
            c = torch.zeros((n, nkv, page, d), dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device="cuda")
            c[at] = fill[i] if kind == "bf16" else fill[i].view(torch.uint8)
            caches.append(c.view(dt))
        kv = T.TPKV(*caches, nq, max_batch=4)
        kv.set_rotary(T.Rotary(d))
        qo = kv.append(x, past, table.cuda(), cu_rows=cu)
        out, lse = kv.decode(q, past + torch.tensor(new, **I32), table.cuda(), return_lse=True)
        kv.sync()
        raw = [c if kind == "bf16" else c.view(torch.uint8) for c in caches]
        got.append((qo, out, lse, *[r[at] for r in raw], *[torch.count_nonzero(r[few // 2: n - few // 2]) for r in raw]))
        del caches, raw, kv
    assert all(torch.equal(a, b) for a, b in zip(got[0][:5], got[1][:5]))
    assert got[1][5] == 0 and got[1][6] == 0  # nothing between the two ends
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [1, 31, 1000, 6000])
@pytest.mark.parametrize("kind,d,nq", [("bf16", 64, 8), ("bf16", 256, 20), ("e4m3", 128, 3), ("e4m3", 192, 33)])
def test_lse_of_exact_scores(n, kind, d, nq):
    """Queries and keys of small whole numbers and a scale of 1/8: the products are exact, so lse has only its own
    roundings.

    |err| <= 2^-22 |s| (the score times log2 e) + 2^-20 (the exponential of a difference below 16) + 120 2^-24 (the
    longest chain of sums: a lane's 17 a tile over four tiles, the shuffles, warps and parts) + 2^-21 (|lse| + 24)
    (the logarithm of the sum, its sum with the maximum and the change of base)."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(n + d)
    page, dt = 16, torch.bfloat16 if kind == "bf16" else E4M3
    pages = (n + page - 1) // page
    k, v = (torch.randint(-2, 3, (pages, 1, page, d), generator=g).float() for _ in "kv")
    q = torch.randint(-2, 3, (1, nq * d), generator=g).to(torch.bfloat16)
    kv = T.TPKV(k.to(dt).cuda(), v.to(dt).cuda(), nq, max_batch=1)
    out, lse = kv.decode(q.cuda(), torch.tensor([n], **I32), torch.arange(pages, **I32)[None, :], scale=0.125,
                         return_lse=True)
    kv.sync()
    s = to_np(q).reshape(nq, d) @ to_np(k).transpose(0, 2, 1, 3).reshape(-1, d)[:n].T * 0.125
    top = s.max(1)
    want = top + np.log(np.exp(s - top[:, None]).sum(1))
    tol = 2.0 ** -22 * np.abs(s).max(1) + 2.0 ** -20 + 120 * 2.0 ** -24 + 2.0 ** -21 * (np.abs(want) + 24)
    err = np.abs(to_np(lse)[0] - want)
    assert (err <= tol).all(), (err / tol).max()
    assert math.isfinite(float(out.float().sum()))


@pytest.mark.parametrize("B", [1, 129, 257])
def test_sublayer_decode_of_any_batch(B):
    """One, and more sequences than rows of a GEMM tile, against float64 attention over the cache's own contents."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    from tests._util import compare
    H, nq, nkv, d, page, n = 256, 4, 2, 64, 16, 40
    g = _gen(B)
    r = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    w = (1 + r(H), r((nq + 2 * nkv) * d, H), r(H, nq * d), r(H))
    k, v = r(B * 3, nkv, page, d, std=1.0), r(B * 3, nkv, page, d, std=1.0)
    table = torch.randperm(B * 3, generator=g).to(torch.int32).reshape(B, 3)
    lens = torch.randint(-1, n, (B,), generator=g).to(torch.int32)
    x = r(B, H, std=1.0)
    m = T.TPAttn(B, H, nq, nkv, d, 64, max_t=1)
    kv = T.TPKV(k, v, nq, max_batch=B)
    y = m.decode(kv, x, *w, 1e-6, 1, lens.cuda(), table.cuda())
    m.sync()
    kv.sync()
    W, K, V, X = [to_np(t) for t in w], to_np(k), to_np(v), to_np(x)
    nrm = X / np.sqrt((X * X).mean(1, keepdims=True) + 1e-6) * W[0]
    q = (nrm @ W[1].T)[:, : nq * d].reshape(B, nq, d)
    z = np.zeros((B, nq, d))
    for b in range(B):
        t = np.arange(int(lens[b]) + 1)  # the token's own key and value are in the cache by now
        if t.size:
            kk, vv = (c[table.numpy()[b][t // page], :, t % page].repeat(nq // nkv, 1) for c in (K, V))
            s = np.einsum("hd,thd->ht", q[b], kk) / d ** 0.5
            pr = np.exp(s - s.max(1, keepdims=True))
            z[b] = np.einsum("ht,thd->hd", pr / pr.sum(1, keepdims=True), vv)
    compare("y", to_np(y), X + z.reshape(B, nq * d) @ W[2].T + W[3], "bf16")
