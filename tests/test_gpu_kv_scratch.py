"""The cache context's scratch: the size that the one-token calls need serves every call."""
import ctypes

import pytest
import torch

from tests.test_gpu_kv_extend import Case, _tp

pytestmark = pytest.mark.gpu


def _sizes(T, cfg):
    return (int(T.lib().tpkv_least_workspace_bytes(ctypes.byref(cfg))), int(T.lib().tpkv_workspace_bytes(ctypes.byref(cfg))))


@pytest.mark.parametrize("d,f8,nq,nkv", [(64, False, 8, 2), (128, True, 8, 2), (128, False, 64, 2), (256, False, 4, 4)])
@pytest.mark.parametrize("extra", [0, 140_000, 3_000_000])
def test_extend_in_less(d, f8, nq, nkv, extra):
    """Few rows over a long cache, cut into as many parts as there is room for; nothing behind the scratch is written."""
    T = _tp()
    c = Case([16, 3], [6000, 9000], nq, nkv, d, 64, f8)
    least, most = _sizes(T, c.kv.cfg)
    assert least <= 2 ** 25 and least + extra < most
    buf = torch.full((least + extra + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert T.lib().tpkv_bind_workspace(c.kv.ctx, buf.data_ptr(), least - 1) == T.ERR_ARG
    assert T.lib().tpkv_bind_workspace(c.kv.ctx, buf.data_ptr(), least + extra) == 0
    got = c.run()
    c.check(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, c.run()))
    out, lse = c.kv.decode(c.q[:2], c.past_dev, c.table, return_lse=True)
    c.kv.sync()
    assert bool(out.isfinite().all())
    assert bool((buf[least + extra:] == 0x5A).all())


def test_binding_chooses():
    T = _tp()
    c = Case([16, 3], [6000, 9000], 8, 2, 128, 64)
    small = T.TPKV(c.k, c.v, 8, max_batch=2, extend_scratch=False)
    assert (small.workspace.numel(), c.kv.workspace.numel()) == _sizes(T, c.kv.cfg)
    out, lse = small.extend(c.q, c.past_dev, c.table, cu_rows=c.cu, return_lse=True)
    small.sync()
    c.check(out, lse)
    a, b = (kv.decode(c.q[:2], c.past_dev, c.table) for kv in (small, c.kv))
    assert torch.equal(a, b)
