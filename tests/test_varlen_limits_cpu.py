"""Calls over more blocks than are numbered are refused on the host, before anything is launched."""
import pytest

from tests.test_varlen_refusals_cpu import T, _backward, _desc, _forward  # noqa: F401


# sequences, heads, key heads, rows: just beyond 2^30 blocks
@pytest.mark.parametrize("batch,nq,nkv,rows", [(1 << 20, 65536, 65536, 1), (1 << 20, 4096, 1024, 1),
                                               (1 << 14, 65536, 65536, 5), (1, 65536, 65536, 1 << 21)])
def test_too_many_blocks(T, batch, nq, nkv, rows):  # noqa: F811
    d = _desc(T, rows=rows, batch=batch, n_heads=nq, n_kv_heads=nkv)
    wide = nq * 64
    assert _forward(T, d, ld_q=wide, ld_k=wide, ld_v=wide, ld_out=wide) == T.ERR_SHAPE
    assert b"too many blocks" in T.lib().tpmlp_last_error(None)
    assert _backward(T, d) == T.ERR_SHAPE
    assert b"too many blocks" in T.lib().tpmlp_last_error(None)


@pytest.mark.parametrize("batch,nq,nkv,rows", [(1 << 20, 1023, 1023, 1), (1 << 13, 65536, 65536, 5), (3, 4096, 64, 1 << 20)])
def test_as_many_as_there_may_be(T, batch, nq, nkv, rows):  # noqa: F811
    d = _desc(T, rows=rows, batch=batch, n_heads=nq, n_kv_heads=nkv)
    assert _forward(T, d, q=None, ld_q=nq * 64, ld_k=nkv * 64, ld_v=nkv * 64, ld_out=nq * 64) == T.ERR_ARG
    assert b"NULL" in T.lib().tpmlp_last_error(None)


def test_sizes_of_the_cache_scratch(T):  # noqa: F811
    """What append and decode need is as small as two partial results of a query-head tile for each of 512 workers."""
    import ctypes
    L = T.lib()
    assert L.tpkv_least_workspace_bytes(None) == 0
    for d in (64, 128, 192, 256):
        for hpg, tile in ((1, 8), (8, 8), (16, 16), (32, 32), (200, 32)):
            c = T.tpmlp.KvConfig(16, 16, 4, 2 * hpg, 2, d, 0, 0)
            least, most = (f(ctypes.byref(c)) for f in (L.tpkv_least_workspace_bytes, L.tpkv_workspace_bytes))
            need = 2 * 512 * tile * (d + 2) * 4
            assert need <= least <= need + 8192 and least < most
    c = T.tpmlp.KvConfig(16, 16, 4, 7, 2, 64, 0, 0)
    assert L.tpkv_least_workspace_bytes(ctypes.byref(c)) == 0
