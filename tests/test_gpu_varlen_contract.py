"""What the calls over sequences of different lengths promise beyond their formulas: which rows influence which, what
is reported, and calls at the ends of their ranges."""
import pytest
import torch

from tests import _varlen_ops as R
from tests.test_gpu_kv_extend import BF, F8, I32, Case, _tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,f8", [(64, False), (128, True), (192, False), (256, True)])
@pytest.mark.parametrize("new,past", [([5, 140, 3], [600, 900, 50]), ([2, 3, 1], [600, 900, 50])])
def test_the_first_page_past_the_end_is_reported(d, f8, new, past):
    """num_pages itself is no page; where no row sees it, it does not matter."""
    T = _tp()
    c = Case(new, past, 4, 2, d, 16, f8)
    want, wl = c.run()
    keep, pages = c.table.clone(), c.k.shape[0]
    for at in (0, 7, (past[1] + new[1] - 1) // 16):
        c.table[1, at] = pages
        out = c.kv.extend(c.q, c.past_dev, c.table, cu_rows=c.cu)
        with pytest.raises(T.TPMLPError) as e:
            c.kv.sync()
        assert e.value.status == T.ERR_ARG, at
        lo, hi = c.cul[1], c.cul[2]
        assert torch.equal(out[:lo], want[:lo]) and torch.equal(out[hi:], want[hi:]), at
        c.table.copy_(keep)
    c.table[1, (past[1] + new[1] + 15) // 16:] = pages
    assert all(torch.equal(a, b) for a, b in zip(c.run(), (want, wl)))


