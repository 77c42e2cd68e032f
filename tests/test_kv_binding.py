"""What the Python binding of the KV cache calls takes and refuses before the
library is called; no device is needed."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from fp4_fp8_quant_gb300 import iq

HERE = SimpleNamespace(device=torch.device("cpu"))


def _one_column(n, stride):
    return torch.arange(n * max(1, stride), dtype=torch.int32).as_strided((n, 1), (max(1, stride), stride))


@pytest.mark.parametrize("stride", [0, 1, 7])
def test_a_table_of_one_column_has_any_column_stride(stride):
    row_start, kv_len = torch.arange(4, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    b = iq._kv_batch(HERE, 3, _one_column(3, stride), row_start, kv_len)
    assert (b.max_pages, b.table_ld, b.num_seqs) == (1, max(1, stride), 3)
    columns = torch.from_numpy(np.arange(3, dtype=np.int32)[:, None])
    assert iq._kv_batch(HERE, 3, columns, row_start, kv_len).table_ld == columns.stride(0)
    with pytest.raises(ValueError, match="unit column stride"):
        iq._kv_batch(HERE, 3, torch.zeros((3, 8), dtype=torch.int32)[:, ::2], row_start, kv_len)


@pytest.mark.parametrize("stride", [0, 1, 7])
def test_lists_of_one_entry_have_any_column_stride(stride, monkeypatch):
    monkeypatch.setattr(iq, "_require", lambda *a, **k: None)        # (wants a GPU's tensor)
    assert iq._kv_indices(_one_column(3, stride), 3) == (1, max(1, stride))
    with pytest.raises(ValueError, match="unit column stride"):
        iq._kv_indices(torch.zeros((3, 8), dtype=torch.int32)[:, ::2], 3)
