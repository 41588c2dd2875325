"""Every variant of the decode and append kernels over page sizes and ragged lengths, large rows, and two contexts at
once."""
import itertools

import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np
from tests.test_gpu_kv_cache import _caches, _check_decode, _decode_case, _gen, _scales, _table

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
DIMS, KINDS = (64, 128, 192, 256), ("bf16", "e4m3")


@pytest.mark.parametrize("page", [8, 24, 64, 128, 256])
@pytest.mark.parametrize("d,kind,heads", list(itertools.product(DIMS, KINDS, (3, 12, 27))))
def test_decode(d, kind, heads, page):
    nkv, layout = 1 + heads % 2, "hnd" if (page + heads) % 2 else "nhd"
    lens = [0, 1, 2 * page - 1, 131, 1500, 64]
    window, sinks = ((0, 0), (70, 9))[(d + page) // 8 % 2]
    kv, q, table, k, v, ks, vs = _decode_case(lens, heads * nkv, nkv, d, kind, page, layout, window, sinks, seed=page)
    out, lse = kv.decode(q.cuda(), torch.tensor(lens, **I32), table.cuda(), window=window, sinks=sinks, return_lse=True)
    kv.sync()
    _check_decode(out, lse, q, table, lens, k, v, ks, vs, heads * nkv, d, page, kind, window, sinks)


@pytest.mark.parametrize("d,kind,il,rot", [(d, k, il, r) for d, k, il in itertools.product(DIMS, KINDS, (False, True))
                                           for r in (16, d // 2, d - 16, d)])
def test_append(d, kind, il, rot):
    """Ragged rows of three sequences; norm weights by turns."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    g = _gen(d + rot)
    nq, nkv, page, past, new = 6, 2, 24, [0, 23, 100], [30, 1, 47]
    ends = [p + n for p, n in zip(past, new)]
    table, pages = _table(g, ends, page)
    k, v = _caches(g, pages, nkv, page, d, kind, "nhd" if il else "hnd")
    ks, vs = _scales(g, nkv, kind)
    x = (torch.randn((sum(new), (nq + 2 * nkv) * d), generator=g) * 1.5).to(torch.bfloat16)
    w = (torch.randn(d, generator=g) * 0.1 + 1).to(torch.bfloat16)
    qw, kw = w if rot != d else None, w if rot != 16 else None
    kv = T.TPKV(k, v, nq, max_batch=3, k_inv_scale=ks, v_inv_scale=vs)
    kv.set_rotary(T.Rotary(rot, interleaved=il), None if qw is None else qw.cuda(), None if kw is None else kw.cuda(), 1e-6)
    off = np.concatenate([[0], np.cumsum(new)])
    q = kv.append(x.cuda(), torch.tensor(past, **I32), table.cuda(), cu_rows=torch.tensor(off, **I32))
    kv.sync()
    X, pos = to_np(x), np.concatenate([np.arange(p, e) for p, e in zip(past, ends)])
    seq = np.repeat(np.arange(3), new)
    z, tol = R.rope(X, nq, nkv, d, pos, rot, il, None if qw is None else to_np(qw), None if kw is None else to_np(kw), 1e-6,
                    "bf16")
    R.within("q", to_np(q), z[:, : nq * d], tol[:, : nq * d])
    at = table.numpy()[seq, pos // page], slice(None), pos % page
    zk, tk = z[:, nq * d:].reshape(-1, nkv, d), tol[:, nq * d:].reshape(-1, nkv, d)
    gk, gv = (c.float().cpu().numpy().astype(np.float64)[at[0], :, at[2]] for c in (k, v))
    zv = X[:, (nq + nkv) * d:].reshape(-1, nkv, d)
    if kind == "bf16":
        R.within("k", gk, zk, tk)
        assert np.array_equal(gv, zv)
    else:  # in code units, as the tests of append have it
        sk, sv = (t.cpu().numpy().astype(np.float64)[:, None] for t in (ks, vs))
        u = (tk - 2.0 ** -8 * np.abs(zk)) / sk
        R.within("k", gk, np.clip(zk / sk, -448, 448), 2.0 ** -4 * np.abs(zk / sk) + 2.0 ** -10 + 2 * u)
        R.within("v", gv, np.clip(zv / sv, -448, 448), 2.0 ** -4 * np.abs(zv / sv) + 2.0 ** -10)


def test_rows_beyond_2_31_elements():
    """Packed rows of more than 2^31 elements: the last rows get the bits that they get alone."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    nq, nkv, d = 2, 1, 128
    W = (nq + 2 * nkv) * d
    rows = (1 << 31) // W + 300
    x = torch.zeros((rows, W), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((400, W), generator=_gen(1)).to(torch.bfloat16).cuda()
    x[-400:] = tail
    k, v = (torch.zeros(40, nkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.arange(40, **I32)[None, :]
    kv = T.TPKV(k, v, nq, max_batch=1)
    kv.set_rotary(T.Rotary(d))
    q = kv.append(x, torch.tensor([7], **I32), table, cu_rows=torch.tensor([rows - 400, rows], **I32))
    kv.sync()
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    kv2 = T.TPKV(k2, v2, nq, max_batch=1)
    kv2.set_rotary(T.Rotary(d))
    q2 = kv2.append(tail, torch.tensor([7], **I32), table, cu_rows=torch.tensor([0, 400], **I32))
    kv2.sync()
    assert torch.equal(q[-400:], q2) and torch.equal(k, k2) and torch.equal(v, v2) and bool(k.any())
    del q
    torch.cuda.empty_cache()


def test_two_contexts_on_one_cache_at_once():
    """A context a stream: decodes that overlap on the GPU, replayed and eager, have the bits of one alone."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    lens, nq, nkv, d = [7000, 300, 0, 2500], 8, 2, 128
    kv, q, table, k, v, *_ = _decode_case(lens, nq, nkv, d, "bf16", 16, "hnd", 0, 0)
    args = (q.cuda(), torch.tensor(lens, **I32), table.cuda())
    want = kv.decode(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    ctx = [T.TPKV(k, v, nq, max_batch=4, stream=s) for s in streams]
    graph, replayed = torch.cuda.CUDAGraph(), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[0]):
        ctx[0].decode(*args, out=replayed)
    outs = []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        outs += [c.decode(*args) for c in ctx[1:]]
    torch.cuda.synchronize()
    assert torch.equal(replayed, want) and all(torch.equal(o, want) for o in outs)
    for c in ctx:
        c.sync()
