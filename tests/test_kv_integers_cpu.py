"""Whole numbers that do not fit the C ABI's 32 bits: ctypes would mask them (a window of 2^32 + 5 became 5); the
binding refuses them before the library is called.  No device is needed: the argument checks of a CPU stand-in pass,
and the library would refuse its NULL context with another message.
"""
import pytest
import torch

BIG = (1 << 32) + 5


@pytest.fixture
def T(monkeypatch):
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    monkeypatch.setattr(T.tpmlp, "_stream_of", lambda *a: None)
    return T


@pytest.fixture
def kv(T):
    k = object.__new__(T.TPKV)
    k.ctx = None
    k.index, k.device, k._fixed, k._stream = -1, torch.device("cpu"), None, None
    k.nq, k.nkv, k.d = 2, 1, 64
    return k


@pytest.mark.parametrize("kw", [dict(window=BIG), dict(sinks=BIG), dict(len_add=BIG), dict(window=-BIG),
                                dict(window=1 << 31)])
def test_decode(T, kv, kw):
    q, lens, table = torch.zeros(1, 128, dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32), torch.zeros(
        1, 1, dtype=torch.int32)
    with pytest.raises(T.TPMLPError) as e:
        kv.decode(q, lens, table, **kw)
    assert e.value.status == T.ERR_ARG and "32 bits" in str(e.value) and next(iter(kw)) in str(e.value)


@pytest.mark.parametrize("kw", [dict(window=BIG), dict(sinks=BIG), dict(t=BIG)])
def test_sublayer_decode(T, kv, kw):
    m = object.__new__(T.TPAttn)
    m.ctx, m.device = None, torch.device("cpu")
    m.H, m.nq, m.nkv, m.d, m.W = 128, 2, 1, 64, 256
    m._t = lambda *a, **k: None
    m.device = type("D", (), {"index": -1})()
    b = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(T.TPMLPError) as e:
        m.decode(kv, b, b, b, b, b, 1e-6, kw.pop("t", 1), torch.ones(1, dtype=torch.int32),
                 torch.zeros(1, 1, dtype=torch.int32), **kw)
    assert e.value.status == T.ERR_ARG and "32 bits" in str(e.value)


def test_context(T):
    k = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    k.get_device = lambda: 0  # past the check that it is a device tensor
    for kw in (dict(n_heads=BIG), dict(n_heads=1, max_batch=BIG)):
        with pytest.raises(T.TPMLPError) as e:
            T.TPKV(k, k, **kw)
        assert e.value.status == T.ERR_ARG and "32 bits" in str(e.value)
