"""The cache calls where the formulas meet NaN, infinities and extreme weights, and their smallest calls."""
import math

import numpy as np
import pytest
import torch

from tests import _attn_ops as R
from tests._util import to_np

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
I32 = dict(dtype=torch.int32, device="cuda")


def _cache(n, nkv, d, kind, page=16, seed=1):
    """Key and value pages of one sequence of n tokens in order, and its table."""
    pages = max(1, (n + page - 1) // page)
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn((pages, nkv, page, d), generator=g).to(torch.bfloat16 if kind == "bf16" else E4M3).cuda()
          for _ in "kv"]
    return kv[0], kv[1], torch.arange(pages, **I32)[None, :]


def _set_keys(k, first, last, value):
    """Every component of the keys of tokens [first, last) of the only sequence."""
    raw = k.view(torch.uint8) if k.dtype == E4M3 else k
    t = torch.arange(first, last, device="cuda")
    raw[t // k.shape[2], :, t % k.shape[2]] = value


# n tokens: one part; several joined at once; groups of parts and then their leaders
@pytest.mark.parametrize("n", [100, 2000, 9000])
@pytest.mark.parametrize("kind,d,nq", [("bf16", 64, 2), ("e4m3", 128, 12), ("bf16", 192, 3), ("e4m3", 256, 20)])
def test_nan_scores_reach_the_lse(n, kind, d, nq):
    """A head whose scores hold a NaN has NaN for its log-sum-exp, as for its output; the others are as without it."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k, v, table = _cache(n, 1, d, kind)
    kv = T.TPKV(k, v, nq, max_batch=1)
    q = torch.randn(1, nq * d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    lens = torch.tensor([n], **I32)
    ref, ref_lse = kv.decode(q, lens, table, return_lse=True)
    assert ref_lse.isfinite().all()
    # a NaN in one query: every one of its scores
    bad = q.clone()
    bad[0, d + 5] = float("nan")
    out, lse = kv.decode(bad, lens, table, return_lse=True)
    kv.sync()
    keep = torch.arange(nq, device="cuda") != 1
    assert out.view(nq, d)[1].isnan().all() and lse[0, 1].isnan()
    assert torch.equal(out.view(nq, d)[keep], ref.view(nq, d)[keep]) and torch.equal(lse[0, keep], ref_lse[0, keep])
    # NaN keys in the first part of the sequence, wherever it is split: every head
    nan = 0x7F if kind == "e4m3" else float("nan")
    _set_keys(k, 0, min(n, 600), nan)
    out, lse = kv.decode(q, lens, table, return_lse=True)
    kv.sync()
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("n", [100, 2000, 9000])
@pytest.mark.parametrize("d,nq", [(64, 2), (128, 20), (256, 9)])
def test_scores_of_minus_infinity(n, d, nq):
    """softmax of scores that are all -inf is NaN, as the formula has it; one finite score takes all the weight; a
    sequence without tokens keeps its 0."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k, v, table = _cache(n, 1, d, "bf16")
    k.zero_()
    k[..., 3] = float("-inf")
    kv = T.TPKV(k, v, nq, max_batch=1)
    q = torch.ones(1, nq * d, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n], **I32)
    out, lse = kv.decode(q, lens, table, return_lse=True)
    kv.sync()
    assert out.isnan().all() and torch.equal(lse, torch.full_like(lse, float("-inf")))
    at = n - 7
    k[at // 16, 0, at % 16, 3] = 0.0
    out, lse = kv.decode(q, lens, table, return_lse=True)
    kv.sync()
    assert torch.equal(out.view(nq, d), v[at // 16, 0, at % 16].expand(nq, d)) and not lse.any()
    out, lse = kv.decode(q, torch.zeros(1, **I32), table, return_lse=True)
    kv.sync()
    assert not out.any() and torch.equal(lse, torch.full_like(lse, float("-inf")))


@pytest.mark.parametrize("inplace", ["rows", "columns"])
@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("transform", [True, False])
def test_append_in_place_of_one_row(n, inplace, transform):
    """Queries written over their own columns, for a single row too."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    nq, nkv, d = 6, 2, 128
    x = torch.randn((n, (nq + 2 * nkv) * d), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    past, table = torch.full((n,), 5, **I32), torch.arange(n, **I32)[:, None]
    got = []
    for where in ("apart", inplace):
        k, v = (torch.zeros(n, nkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        kv = T.TPKV(k, v, nq, max_batch=n)
        kv.set_rotary(T.Rotary(d), w, w, 1e-6)
        rows = x.clone()
        q_out = {"apart": None, "rows": rows, "columns": rows[:, : nq * d]}[where]
        q = kv.append(rows, past, table, q_out=q_out, transform=transform)
        kv.sync()
        got.append((q[:, : nq * d].clone(), k, v))
        if where != "apart":
            assert torch.equal(rows[:, nq * d:], x[:, nq * d:])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].any()


def test_strides_of_a_single_row_do_not_matter():
    """The C calls in place with one row: its strides are of no use, so they may differ."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    d, nq = 64, 2
    L, s = T.lib(), torch.cuda.current_stream().cuda_stream
    x = torch.randn(1, 512, device="cuda").to(torch.bfloat16)
    r = T.Rotary(d)
    want = T.qk_norm_rope(x, nq, 1, d, r, torch.tensor([9], **I32))
    pos = torch.tensor([9], **I32)
    desc = T.tpmlp.QkDesc(1, nq, 1, d, T.BF16, pos.data_ptr(), 0, None, None, 1e-6, 0)
    y = x.clone()
    assert L.tpattn_qk_rope_forward(desc, r.spec, y.data_ptr(), 256, y.data_ptr(), 192, s) == 0
    assert torch.equal(y[:, :192], want) and torch.equal(y[:, 192:], x[:, 192:])
    wdx = T.qk_norm_rope_backward(want, None, nq, 1, d, r, pos)[0]
    z = want.clone()
    assert L.tpattn_qk_rope_backward(desc, r.spec, None, 0, z.data_ptr(), 192, z.data_ptr(), 256, None, None, None, 0,
                                     s) == 0
    assert torch.equal(z, wdx)
    k, v, table = _cache(50, 1, d, "bf16")
    kv = T.TPKV(k, v, nq, max_batch=1)
    q, lens = x[:, : nq * d].contiguous(), torch.tensor([50], **I32)
    out = kv.decode(q, lens, table)
    assert L.tpkv_decode(kv.ctx, 1, q.data_ptr(), 128, lens.data_ptr(), 0, table.data_ptr(), table.shape[1],
                         table.shape[1], d ** -0.5, 0, 0, q.data_ptr(), 256, None) == 0
    kv.sync()
    assert torch.equal(q, out)


@pytest.mark.parametrize("n", [300, 20000])
@pytest.mark.parametrize("d,nq", [(64, 1), (128, 9), (256, 17)])
def test_many_small_weights_of_an_e4m3_cache(n, d, nq):
    """A page's first token has value 0 and weight 1, its others value 1 and weight e^-18, below 2^-25: together they
    are the output.

    Tolerance, relative: the output's rounding 2^-8, a weight's in f16 2^-11, the exponential and the sums 2^-14."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k, v, table = _cache(n, 1, d, "e4m3")
    k.view(torch.uint8).zero_()
    v.copy_(torch.ones_like(v, dtype=torch.float32).to(E4M3))
    k[:, 0, 0, 0] = torch.tensor(18.0, device="cuda").to(E4M3)
    v.view(torch.uint8)[:, 0, 0] = 0
    kv = T.TPKV(k, v, nq, max_batch=1)
    q = torch.zeros(1, nq * d, dtype=torch.bfloat16, device="cuda")
    q.view(nq, d)[:, 0] = 1.0
    out, lse = kv.decode(q, torch.tensor([n], **I32), table, scale=1.0, return_lse=True)
    kv.sync()
    first = (n + 15) // 16
    rest = (n - first) * math.exp(-18.0)
    assert np.abs(to_np(out) / (rest / (first + rest)) - 1.0).max() <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14
    # the scores are exact; the sum, its logarithm and 18 round a few times each
    assert np.abs(to_np(lse) - (18.0 + math.log(first + rest))).max() <= 28 * 2.0 ** -22 + 2.0 ** -18


@pytest.mark.parametrize("log_q", [10, 14, 20, 40, 100])
@pytest.mark.parametrize("d,nq", [(64, 1), (128, 9)])
def test_scores_of_any_size(log_q, d, nq):
    """Scores up to 448 x 2^100: the greatest takes all the weight (the next is 32 x 2^10 below it), exactly."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    n = 3000
    k, v, table = _cache(n, 1, d, "e4m3")
    g = torch.Generator().manual_seed(log_q)
    codes = torch.tensor([-448.0, -20.0, 0.0, 1.0, 2.0, 256.0, 416.0])[torch.randint(0, 7, (k.shape[0], 16), generator=g)]
    k.view(torch.uint8).zero_()
    k[:, 0, :, 0] = codes.cuda().to(E4M3)
    at = 1777
    k[at // 16, 0, at % 16, 0] = torch.tensor(448.0, device="cuda").to(E4M3)
    kv = T.TPKV(k, v, nq, max_batch=1)
    q = torch.zeros(1, nq * d, dtype=torch.bfloat16, device="cuda")
    q.view(nq, d)[:, 0] = 2.0 ** log_q
    out, lse = kv.decode(q, torch.tensor([n], **I32), table, scale=1.0, return_lse=True)
    kv.sync()
    assert torch.equal(out.view(nq, d), v[at // 16, 0, at % 16].to(torch.bfloat16).expand(nq, d))
    assert np.abs(to_np(lse) / (448.0 * 2.0 ** log_q) - 1.0).max() <= 2.0 ** -21
