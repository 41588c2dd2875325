"""Attention over packed sequences and over new tokens with a cache, where blocks of different lengths follow one
another on a multiprocessor and where arguments are as large as they may be: against float64 with derived bounds
(tests/_varlen_ops.py)."""
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
