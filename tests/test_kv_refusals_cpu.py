"""Refusals of the query/key rotation and cache calls that are decided on the host: no device is needed."""
import ctypes
import math
import re
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def T():
    from tensor_transformer_mlp_rmsnorm_gb300 import build
    build.build()
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


def test_header_library_and_binding_agree(T):
    from tensor_transformer_mlp_rmsnorm_gb300 import tpmlp
    text = open(os.path.join(ROOT, "include", "tpmlp.h")).read()
    names = set(re.findall(r"^TPMLP_API\s+[\w\s\*]+?\b(tpkv_\w+)\(", text, flags=re.M))
    assert {"tpkv_create", "tpkv_append", "tpkv_decode", "tpkv_sync"} <= names
    L = ctypes.CDLL(T.LIB_PATH)
    assert all(hasattr(L, n) for n in names) and names <= set(tpmlp._SIGNATURES)


def test_rotary_init(T):
    L, S = T.lib(), T.tpmlp.RotarySpec
    d = (ctypes.c_double * 128)(*([1.0] * 128))

    def init(rot, il=0, f=d):
        return L.tpattn_rotary_init(ctypes.byref(S()), rot, il, f)

    assert init(0) == 0 and init(16) == 0 and init(256, 1) == 0
    assert init(8) == T.ERR_SHAPE and init(-16) == T.ERR_SHAPE and init(272) == T.ERR_SHAPE
    assert init(16, 2) == T.ERR_ARG and init(16, 0, None) == T.ERR_ARG
    for bad in (math.nan, math.inf, 2.0 ** 21):
        assert init(16, 0, (ctypes.c_double * 8)(*([1.0] * 7 + [bad]))) == T.ERR_ARG
    assert L.tpattn_rotary_init(None, 16, 0, d) == T.ERR_ARG
    with pytest.raises(T.TPMLPError):
        T.Rotary(32, inv_freq=[1.0])


def test_rotary_turns_are_the_frequencies(T):
    """turn / 2^64 = inv_freq / 2 pi mod 1, to 2^-60 (from 50 digits of pi)."""
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    freq = [1.0, 10000.0 ** (-2 / 64), 1e-7, -0.5, 6.283185307179586, 12345.678, -1e-18, 0.0]
    r = T.Rotary(16, inv_freq=freq)
    for f, t in zip(freq, r.spec.turn):
        want = Fraction(f) / (2 * pi)
        off = (Fraction(t, 1 << 64) - want) % 1
        assert min(off, 1 - off) < Fraction(1, 1 << 60) * max(1, abs(int(f))), f


def _desc(T, **kw):
    a = dict(rows=4, n_heads=2, n_kv_heads=1, head_dim=64, dtype=T.BF16, positions=None, seq=0, q_norm_w=None,
             k_norm_w=None, eps=1e-6, reserved=0)
    a.update(kw)
    return T.tpmlp.QkDesc(*a.values())


def test_row_calls(T):
    L = T.lib()
    rot = T.Rotary(64)
    big = T.Rotary(128)

    def fwd(x=1024, ldx=192, out=2048, ldo=192, r=rot, **kw):
        return L.tpattn_qk_rope_forward(ctypes.byref(_desc(T, **kw)), r.ref if r else None, x, ldx, out, ldo, None)

    def bwd(x=1024, ldx=192, g=2048, ldg=192, dx=4096, ldd=192, dq=None, dk=None, ws=None, wb=0, r=rot, **kw):
        return L.tpattn_qk_rope_backward(ctypes.byref(_desc(T, **kw)), r.ref if r else None, x, ldx, g, ldg, dx, ldd,
                                         dq, dk, ws, wb, None)

    for call in (fwd, bwd):
        for status, kw in ((T.ERR_SHAPE, dict(head_dim=96)), (T.ERR_SHAPE, dict(head_dim=0)),
                           (T.ERR_SHAPE, dict(rows=-1)), (T.ERR_SHAPE, dict(n_heads=-1)),
                           (T.ERR_SHAPE, dict(seq=-2)), (T.ERR_UNSUPPORTED, dict(dtype=5)),
                           (T.ERR_ARG, dict(eps=math.nan)), (T.ERR_ARG, dict(eps=-1.0)), (T.ERR_ARG, dict(reserved=1)),
                           (T.ERR_ARG, dict(positions=2)), (T.ERR_ARG, dict(q_norm_w=8)), (T.ERR_SHAPE, dict(r=big)),
                           (T.ERR_SHAPE, dict(rows=1 << 33))):
            assert call(**kw) == status, (call, kw)
    assert fwd(ldx=191) == T.ERR_SHAPE and fwd(ldx=184) == T.ERR_SHAPE and fwd(ldo=184) == T.ERR_SHAPE
    assert fwd(x=None) == T.ERR_ARG and fwd(out=None) == T.ERR_ARG and fwd(x=1032) == T.ERR_ARG
    assert fwd(out=1024, ldo=200) == T.ERR_ARG  # in place with another stride
    assert fwd(rows=0, x=None, out=None) == 0
    assert bwd(g=None) == T.ERR_ARG and bwd(dx=None) == T.ERR_ARG and bwd(g=4096, ldg=200) == T.ERR_ARG
    assert bwd(dq=64) == T.ERR_ARG                                # a gradient without its weight
    assert bwd(q_norm_w=64) == T.ERR_ARG                          # a weight without its gradient
    assert bwd(q_norm_w=64, dq=128) == T.ERR_ARG                  # no workspace
    need = L.tpattn_qk_rope_workspace_bytes(64)
    assert bwd(q_norm_w=64, dq=128, ws=256, wb=need - 1) == T.ERR_ARG
    assert bwd(q_norm_w=64, dq=128, ws=256, wb=need, x=None) == T.ERR_ARG
    assert need > 0 and L.tpattn_qk_rope_workspace_bytes(100) == 0
    assert L.tpattn_qk_rope_forward(None, None, 16, 192, 16, 192, None) == T.ERR_ARG


def test_cache_config(T):
    L = T.lib()
    good = dict(num_pages=16, page_size=16, max_batch=4, n_heads=8, n_kv_heads=2, head_dim=128, cache_dtype=0, reserved=0)

    def both(**kw):
        c = T.tpmlp.KvConfig(*{**good, **kw}.values())
        out = ctypes.c_void_p()
        n = L.tpkv_workspace_bytes(ctypes.byref(c))
        return n, L.tpkv_create(ctypes.byref(c), None, ctypes.byref(out)) if n == 0 else None

    assert both()[0] > 0 and both()[0] % 256 == 0
    for status, kw in ((T.ERR_SHAPE, dict(num_pages=0)), (T.ERR_SHAPE, dict(page_size=0)), (T.ERR_SHAPE, dict(page_size=12)),
                       (T.ERR_SHAPE, dict(page_size=65544)), (T.ERR_SHAPE, dict(max_batch=0)),
                       (T.ERR_SHAPE, dict(n_heads=7)), (T.ERR_SHAPE, dict(n_kv_heads=0)), (T.ERR_SHAPE, dict(head_dim=80)),
                       (T.ERR_UNSUPPORTED, dict(cache_dtype=2)), (T.ERR_ARG, dict(reserved=3))):
        assert both(**kw) == (0, status), kw
        assert L.tpkv_last_error(None)
    assert L.tpkv_workspace_bytes(None) == 0 and L.tpkv_create(None, None, None) == T.ERR_ARG


def test_null_context(T):
    L = T.lib()
    assert L.tpkv_bind_workspace(None, None, 0) == T.ERR_ARG
    assert L.tpkv_set_stream(None, None) == T.ERR_ARG
    assert L.tpkv_bind_cache(None, None, None, 0, 0, 0, None, None) == T.ERR_ARG
    assert L.tpkv_set_rotary(None, None, None, None, 0.0) == T.ERR_ARG
    assert L.tpkv_append(None, 0, 0, None, 0, None, None, None, None, 0, 0, 0, None, 0) == T.ERR_ARG
    assert L.tpkv_decode(None, 0, None, 0, None, 0, None, 0, 0, 0.0, 0, 0, None, 0, None) == T.ERR_ARG
    assert L.tpkv_sync(None) == T.ERR_ARG and L.tpkv_launch_count(None) == 0
    L.tpkv_destroy(None)
