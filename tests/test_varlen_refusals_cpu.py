"""Refusals of the packed-sequence and extend calls that are decided on the host: no device is needed."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is aligned and never followed: the call is refused, or there is no device


@pytest.fixture(scope="module")
def T():
    from tensor_transformer_mlp_rmsnorm_gb300 import build
    build.build()
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    return T


def _desc(T, **kw):
    a = dict(rows=10, batch=2, n_heads=4, n_kv_heads=2, head_dim=64, cu_rows=P, scale=0.1, window=0, sinks=0, reserved=0)
    a.update(kw)
    return T.tpmlp.PackedDesc(*a.values())


def _forward(T, desc=None, q=P, ld_q=512, k=2 * P, ld_k=512, v=3 * P, ld_v=512, out=4 * P, ld_out=256, lse=None,
             status=5 * P):
    d = _desc(T) if desc is None else desc
    return T.lib().tpattn_packed_forward(ctypes.byref(d), q, ld_q, k, ld_k, v, ld_v, out, ld_out, lse, status, None)


def _backward(T, desc=None, q=P, k=2 * P, v=3 * P, out=4 * P, lse=5 * P, dout=6 * P, ld_dout=256, dq=7 * P, dk=8 * P,
              dv=9 * P, ld_dq=512, ld_dk=512, ws=10 * P, nbytes=1 << 20, status=11 * P):
    d = _desc(T) if desc is None else desc
    return T.lib().tpattn_packed_backward(ctypes.byref(d), q, 512, k, 512, v, 512, out, 256, lse, dout, ld_dout, dq, ld_dq,
                                          dk, ld_dk, dv, 512, ws, nbytes, status, None)


BAD_DESC = [(dict(rows=-1), "SHAPE"), (dict(rows=(1 << 28) + 1), "SHAPE"), (dict(batch=-1), "SHAPE"),
            (dict(batch=(1 << 20) + 1), "SHAPE"), (dict(n_heads=0), "SHAPE"), (dict(n_kv_heads=0), "SHAPE"),
            (dict(n_kv_heads=3), "SHAPE"), (dict(n_heads=65538), "SHAPE"), (dict(head_dim=96), "SHAPE"),
            (dict(head_dim=0), "SHAPE"), (dict(head_dim=320), "SHAPE"), (dict(cu_rows=None), "ARG"),
            (dict(cu_rows=P + 2), "ARG"), (dict(scale=float("nan")), "ARG"), (dict(scale=float("inf")), "ARG"),
            (dict(window=-1), "ARG"), (dict(sinks=-1), "ARG"), (dict(reserved=1), "ARG")]


@pytest.mark.parametrize("kw,kind", BAD_DESC)
def test_descriptor(T, kw, kind):
    want = getattr(T, "ERR_" + kind)
    assert _forward(T, _desc(T, **kw)) == want
    assert _backward(T, _desc(T, **kw)) == want
    assert T.lib().tpmlp_last_error(None)


def test_forward_tensors(T):
    for name in ("q", "k", "v", "out", "status"):
        assert _forward(T, **{name: None}) == T.ERR_ARG, name
    for name in ("q", "k", "v", "out"):
        assert _forward(T, **{name: P + 8}) == T.ERR_ARG, name
    for name in ("ld_q", "ld_k", "ld_v", "ld_out"):
        assert _forward(T, **{name: 260}) == T.ERR_SHAPE and _forward(T, **{name: 64}) == T.ERR_SHAPE, name
    assert _forward(T, lse=P + 2) == T.ERR_ARG and _forward(T, status=P + 1) == T.ERR_ARG
    assert _forward(T, out=P) == T.ERR_ARG  # over q with another stride
    assert _forward(T, out=2 * P) == T.ERR_ARG and _forward(T, out=3 * P) == T.ERR_ARG
    assert T.lib().tpattn_packed_forward(None, *[P, 512] * 4, None, P, None) == T.ERR_ARG
    for kw in (dict(rows=0), dict(batch=0)):  # nothing to do
        assert _forward(T, _desc(T, **kw), q=None, out=None) == 0


def test_backward_tensors(T):
    for name in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws", "status"):
        assert _backward(T, **{name: None}) == T.ERR_ARG, name
    for name in ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "ws"):
        assert _backward(T, **{name: P + 8}) == T.ERR_ARG, name
    for name in ("ld_dout", "ld_dq", "ld_dk"):
        assert _backward(T, **{name: 260}) == T.ERR_SHAPE and _backward(T, **{name: 64}) == T.ERR_SHAPE, name
    for name in ("dq", "dk", "dv"):
        for at in (1, 2, 3, 4, 6):  # q, k, v, out, dout
            assert _backward(T, **{name: at * P}) == T.ERR_ARG, (name, at)
    assert _backward(T, dk=9 * P) == T.ERR_ARG and _backward(T, dq=8 * P) == T.ERR_ARG
    need = T.lib().tpattn_packed_workspace_bytes(10, 4)
    assert need >= 10 * 4 * 8 and _backward(T, nbytes=need - 1) == T.ERR_ARG
    for rows, heads in ((-1, 4), ((1 << 28) + 1, 4), (4, 0), (4, 65537)):
        assert T.lib().tpattn_packed_workspace_bytes(rows, heads) == 0


def test_null_contexts(T):
    L = T.lib()
    assert L.tpkv_extend(None, 1, 1, *[None, 8, None, None, None, None, 1, 1, 1.0, 0, 0, None, 8, None]) == T.ERR_ARG
    assert L.tpattn_forward_packed(None, 1, 1, *[None] * 6, 1e-6, 1, None) == T.ERR_ARG
    assert L.tpattn_extend(None, None, 1, 1, *[None] * 5, 1e-6, 1, None, None, None, None, 1, 1, 0, 0, None) == T.ERR_ARG


def test_header_and_binding_agree(T):
    text = open(os.path.join(ROOT, "include", "tpmlp.h")).read()
    args = dict(re.findall(r"TPMLP_API\s+[\w\s\*]+?\b(tp\w+)\(([^)]*)\)", text))
    for name in ("tpkv_extend", "tpattn_packed_forward", "tpattn_packed_backward", "tpattn_packed_workspace_bytes",
                 "tpattn_forward_packed", "tpattn_extend"):
        assert len(args[name].split(",")) == len(T.tpmlp._SIGNATURES[name][1]), name
    fields = re.search(r"typedef struct \{([^}]*)\} tpattn_packed_desc;", text).group(1)
    names = re.findall(r"(\w+)(?=[,;])", re.sub(r"/\*.*?\*/", "", fields, flags=re.S))
    assert names == [f[0] for f in T.tpmlp.PackedDesc._fields_]


def test_binding_refuses_what_is_no_cuda_tensor(T):
    import torch
    q = torch.zeros(4, 128, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(T.TPMLPError):
        T.packed_attention(q, q, q, cu, 2, 2)
    with pytest.raises(T.TPMLPError):
        T.packed_attention(q, q, q, cu, 2, 1 << 31)
    assert T.packed_attention_check is not None
