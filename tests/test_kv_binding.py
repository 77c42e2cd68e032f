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
    assert iq._kv_indices(_one_column(3, stride), HERE, 3) == (1, max(1, stride))
    with pytest.raises(ValueError, match="unit column stride"):
        iq._kv_indices(torch.zeros((3, 8), dtype=torch.int32)[:, ::2], HERE, 3)


class _Elsewhere:
    """Stands for a contiguous tensor on another GPU."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st = [1] * len(self.shape)
        for d in range(len(self.shape) - 2, -1, -1):
            st[d] = st[d + 1] * self.shape[d + 1]
        return tuple(st) if i is None else st[i]

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()


def test_a_cache_on_another_gpu_than_the_current_one_is_refused(monkeypatch):
    cache = SimpleNamespace(device=torch.device("cuda", 1))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for stream in (None, 77):
        with pytest.raises(ValueError, match="not the current GPU"):
            iq._kv_stream(cache, stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    assert iq._kv_stream(cache, None) == 101 and iq._kv_stream(cache, 77) == 77


def test_lists_and_a_workspace_on_another_gpu_are_refused(monkeypatch):
    with pytest.raises(ValueError, match="indices must be on the cache's GPU"):
        iq._kv_indices(_Elsewhere((3, 4), torch.int32), SimpleNamespace(device=torch.device("cuda", 0)), 3)
    # The rest of a call on the cache's GPU, up to the workspace.
    cache = SimpleNamespace(device=torch.device("cuda", 0), kv_heads=1, head_dim=64)
    monkeypatch.setattr(iq, "_kv_batch", lambda *a: None)
    monkeypatch.setattr(iq, "_kv_rows", lambda *a: 64)
    monkeypatch.setattr(iq, "lib", lambda: None)
    monkeypatch.setattr(iq, "kv_attention_workspace_bytes", lambda *a: 256)
    with pytest.raises(ValueError, match="workspace must be on the cache's GPU"):
        iq.kv_attention(cache, _Elsewhere((3, 1, 64), torch.bfloat16), None, None, None,
                        out=_Elsewhere((3, 1, 64), torch.bfloat16), workspace=_Elsewhere((256,), torch.uint8))
