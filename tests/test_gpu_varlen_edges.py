"""Attention over packed sequences and over new tokens with a cache, where blocks of different lengths follow one
another on a multiprocessor and where arguments are as large as they may be: against float64 with derived bounds
(tests/_varlen_ops.py)."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_kv_extend import Case
from tests.test_gpu_packed_attention import _inputs, _tp
from tests.test_gpu_packed_attention import check as check_packed

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


def _lens(n, most, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, most + 1, (n,), generator=g).tolist()


@pytest.mark.parametrize("window,sinks", [(TOP, 0), (TOP, TOP), (TOP - 1, 3), (128, TOP), (1, TOP), (1 << 20, 1 << 20)])
def test_largest_windows_packed(window, sinks):
    check_packed([300, 1, 129], 4, 2, 64, window, sinks)


@pytest.mark.parametrize("window,sinks", [(TOP, 0), (TOP, TOP), (TOP - 1, 3), (128, TOP), (1, TOP), (1 << 20, 1 << 20)])
def test_largest_windows_extend(window, sinks):
    for new, past in (([40, 3, 1], [300, 9, 5000]), ([5], [7000])):  # the second over a split cache
        c = Case(new, past, 4, 2, 64, 16)
        c.check(*c.run(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("n,most", [(40, 300), (100, 300)])  # ordered by length, and by place
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_many_blocks_packed(d, n, most, window, sinks):
    check_packed(_lens(n, most, d + n), 16, 8, d, window, sinks, seed=d)


@pytest.mark.parametrize("d,f8", [(64, True), (128, False), (128, True), (192, False), (256, True), (256, False)])
@pytest.mark.parametrize("n", [30, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_many_blocks_extend(d, f8, n, window, sinks):
    past = [p - 20 if p < 20 else p for p in _lens(n, 400, n)]  # some inactive
    c = Case(_lens(n, 200, d), past, 16, 8, d, 16, f8, seed=d)
    c.check(*c.run(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True), (192, True), (256, False)])
@pytest.mark.parametrize("new,past", [([6, 1, 3], [9000, -1, 2000]), ([64], [20000]), ([2, 0, 200], [12000, 4, 300])])
@pytest.mark.parametrize("window,sinks", [(3000, 0), (3000, 200), (6000, 2500)])
def test_windows_over_long_caches(d, f8, new, past, window, sinks):
    c = Case(new, past, 8, 2, d, 64, f8, seed=d)
    c.check(*c.run(window=window, sinks=sinks), window, sinks)


def test_sequences_none_of_which_is_active():
    c = Case([3, 140, 1], [-1, -5, -(2 ** 31)], 4, 2, 128, 16)
    c.check(*c.run())


def test_packed_calls_on_two_streams_at_once():
    """Calls with workspaces of their own side by side."""
    T = _tp()
    nq, nkv, d = 8, 2, 128
    jobs = [(_inputs([700, 129, 1, 60 + s], nq, nkv, d, s), torch.cuda.Stream()) for s in range(2)]

    def step(t, stream=None):
        q, k, v, dout, cu = t
        o = T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True, stream=stream)
        return (*o, *T.packed_attention_backward(dout, q, k, v, *o, cu, nq, nkv, stream=stream))

    want = [step(t) for t, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for t, s in jobs:
            with torch.cuda.stream(s):
                got.append(step(t))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    T.packed_attention_check()


def test_two_captured_steps_replayed_in_turn():
    T = _tp()
    nq, nkv, d = 4, 2, 64
    jobs = []
    for s in range(2):
        q, k, v, dout, cu = _inputs([200, 33 + s], nq, nkv, d, s)

        def step(q=q, k=k, v=v, dout=dout, cu=cu):
            o = T.packed_attention(q, k, v, cu, nq, nkv, return_lse=True)
            return (*o, *T.packed_attention_backward(dout, q, k, v, *o, cu, nq, nkv))

        want = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        jobs.append((graph, got, want, step))  # a graph reads its inputs where they lie: they are kept
    for _ in range(3):
        for graph, got, _, _ in jobs:
            for x in got:
                x.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in jobs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True), (192, False), (192, True), (256, True)])
@pytest.mark.parametrize("new,past,nq,nkv", [
    ([256] * 20, [3900] * 20, 8, 8), ([128] * 22, [5000] + [3300] * 21, 16, 8),  # a last turn of 8 to 24 blocks
    ([200, 300, 90, 256] * 5, [4000, 3500, 5100, -1] * 5, 8, 8), ([100] * 70, [3400, 10] * 35, 8, 8),
    ([2] * 40, [4100] * 40, 16, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2600, 100)])
def test_last_turns_over_long_caches(d, f8, new, past, nq, nkv, window, sinks):
    c = Case(new, past, nq, nkv, d, 64, f8, seed=len(new))
    c.check(*c.run(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("d,f8", [(64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("new,past,nq,nkv", [([2] * 40, [4100] * 40, 16, 4), ([2] * 36, [4100] * 36, 16, 4),
                                             ([5] * 48, [2500] * 48, 8, 2)])
def test_values_that_arrive_after_later_keys(d, f8, new, past, nq, nkv):
    """Many copies in flight land in any order: each is waited for, so that repeats give the same bits."""
    c = Case(new, past, nq, nkv, d, 64, f8, seed=len(new))
    out, lse = c.run()
    c.check(out, lse)
    for _ in range(20):
        again, _ = c.run()
        assert torch.equal(again, out)


def test_more_rows_than_there_may_be_are_refused():
    T = _tp()
    c = Case([3], [20], 4, 2, 128, 16)
    q, out = c.q, torch.empty_like(c.q)
    status = T.lib().tpkv_extend(c.kv.ctx, 2 ** 28 + 1, 1, q.data_ptr(), 512, c.cu.data_ptr(), None,
                                 c.past_dev.data_ptr(), c.table.data_ptr(), c.table.shape[1], c.table.shape[1], 0.1, 0, 0,
                                 out.data_ptr(), 512, None)
    assert status == T.ERR_SHAPE


FIRST_CALLS = """
import torch, tensor_transformer_mlp_rmsnorm_gb300 as T
g = torch.Generator(device="cuda").manual_seed(0)
q, k, v, dout = (torch.randn(300, n * 64, generator=g, device="cuda").bfloat16() for n in (4, 2, 2, 4))
cu = torch.tensor([0, 170, 300], dtype=torch.int32, device="cuda")
past = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12)
kc, vc = (torch.zeros(24, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
for b, (lo, hi) in enumerate(((0, 170), (170, 300))):
    for cache, x in ((kc, k), (vc, v)):
        pos = torch.arange(hi - lo, device="cuda")
        cache[table[b][pos // 16].long(), :, pos % 16] = x[lo:hi].view(-1, 2, 64)
kv = T.TPKV(kc, vc, 4, max_batch=2)
word = torch.zeros(1, dtype=torch.int32, device="cuda")
def step():
    out, lse = T.packed_attention(q, k, v, cu, 4, 2, return_lse=True, status=word)
    return (out, lse, *T.packed_attention_backward(dout, q, k, v, out, lse, cu, 4, 2, status=word),
            kv.extend(q, past, table, cu_rows=cu))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert int(word) == 0
print("same")
"""


def test_captured_before_any_other_call():
    """A process whose first calls are captured: what a kernel's first launch sets up is no work of a stream."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
