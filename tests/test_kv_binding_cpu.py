"""What the cache binding passes on for strides, decided on the host: no device is needed.

The binding's checks take the device's index from the tensor, -1 on the CPU, so its pure-Python part runs on CPU
tensors; no call reaches the library.
"""
import pytest
import torch


@pytest.fixture(scope="module")
def kv():
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    k = object.__new__(T.TPKV)  # without a context
    k.index = -1
    return k


def _reach(t, ld, rows, width):
    """Elements of t's storage that `rows` rows of `width` at stride ld would reach from its start."""
    return t.storage_offset() + (rows - 1) * ld + width <= t.untyped_storage().size() // 4


def test_block_tables_whose_rows_overlap_are_refused(kv):
    """A table that shares one stored row (expand) or overlaps rows: its real stride is below its width, and any other
    would read behind it."""
    import tensor_transformer_mlp_rmsnorm_gb300 as T
    one = torch.arange(5, dtype=torch.int32)
    for t in (one.expand(3, 5), one[:1].expand(4, 1), one.as_strided((3, 3), (1, 1))):
        with pytest.raises(T.TPMLPError) as e:
            kv._table(t, t.shape[0])
        assert e.value.status == T.ERR_ARG


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(3, 7, dtype=torch.int32),
    lambda: torch.zeros(3, 12, dtype=torch.int32)[:, 2:9],       # columns of a wider table
    lambda: torch.zeros(6, 7, dtype=torch.int32)[::2],           # every other row
    lambda: torch.zeros(1, 7, dtype=torch.int32).expand(1, 7),
    lambda: torch.zeros(7, dtype=torch.int32).expand(1, 7),      # one row: its stride is of no use
    lambda: torch.zeros(2, 1, dtype=torch.int32),
    lambda: torch.zeros(3, 0, dtype=torch.int32),
    lambda: torch.zeros(0, 4, dtype=torch.int32),
])
def test_block_tables_keep_their_stride(kv, make):
    t = make()
    _, ld, pages = kv._table(t, t.shape[0])
    assert pages == t.shape[1] and ld >= pages
    if t.shape[0] > 1 and pages:
        assert ld == t.stride(0) and _reach(t, ld, *t.shape)
