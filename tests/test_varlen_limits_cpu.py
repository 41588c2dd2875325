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
