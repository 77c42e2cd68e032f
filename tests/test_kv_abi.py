"""Refusals of the KV cache calls: status codes of the C entries (before any
CUDA call, so no device is needed) and the Python binding's checks."""

import ctypes

import pytest
import torch

from fp4_fp8_quant_gb300 import build as B

ARG, ALIGN, SHAPE, WORKSPACE = -1, -2, -3, -6
ENOUGH = 1 << 40


@pytest.fixture(scope="module")
def iq():
    B.build()
    from fp4_fp8_quant_gb300 import iq
    iq.lib()
    return iq


def _cache(iq, **kw):
    d = dict(k_codes=256, v_codes=256, k_sf=1, v_sf=1, num_pages=10, kv_heads=2, page_size=64, head_dim=128) | kw
    return ctypes.byref(iq._KVCacheStruct(**d))


def _batch(iq, **kw):
    d = dict(block_table=4, table_ld=5, max_pages=5, row_start=4, kv_len=4, num_seqs=2, num_rows=3) | kw
    return ctypes.byref(iq._KVBatchStruct(**d))


BAD_CACHES = [(dict(k_codes=None), ARG), (dict(v_codes=None), ARG), (dict(k_sf=None), ARG), (dict(v_sf=None), ARG),
              (dict(num_pages=-1), ARG), (dict(num_pages=0), ARG), (dict(kv_heads=0), SHAPE), (dict(kv_heads=70000), SHAPE),
              (dict(page_size=48), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=256), SHAPE),
              (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE), (dict(k_codes=264), ALIGN),
              (dict(v_codes=257), ALIGN), (dict(num_pages=1 << 24), ARG)]
BAD_BATCHES = [(dict(block_table=None), ARG), (dict(row_start=None), ARG), (dict(kv_len=None), ARG),
               (dict(num_seqs=-1), ARG), (dict(num_seqs=0), ARG), (dict(num_rows=-1), ARG), (dict(max_pages=-1), ARG),
               (dict(table_ld=4), ARG), (dict(block_table=6), ALIGN), (dict(row_start=5), ALIGN), (dict(kv_len=2), ALIGN)]


def _calls(iq):
    L = iq.lib()
    return [
        lambda c, b: L.iq_kv_cache_write(c, b, 16, 256, 16, 256, None),
        lambda c, b: L.iq_kv_cache_read(c, b, 16, 256, 16, 256, None),
        lambda c, b: L.iq_kv_attention(c, b, 16, 1024, 8, 0.1, 16, 1024, 256, ENOUGH, None),
        lambda c, b: L.iq_kv_attention_topk(c, b, 16, 1024, 8, 4, 7, 7, 0.1, 16, 1024, 256, ENOUGH, None),
    ]


def test_bad_caches_and_batches(iq):
    for call in _calls(iq):
        assert call(None, _batch(iq)) == ARG and call(_cache(iq), None) == ARG
        for kw, want in BAD_CACHES:
            assert call(_cache(iq, **kw), _batch(iq)) == want, kw
        for kw, want in BAD_BATCHES:
            assert call(_cache(iq), _batch(iq, **kw)) == want, kw


def test_no_rows_is_no_work(iq):
    for call in _calls(iq):
        assert call(_cache(iq), _batch(iq, num_rows=0)) == 0
        assert call(_cache(iq), _batch(iq, num_rows=0, num_seqs=0, block_table=None, row_start=None, kv_len=None)) == 0
        assert call(_cache(iq, page_size=48), _batch(iq, num_rows=0)) == SHAPE


def test_bad_rows(iq):
    L, c, b = iq.lib(), _cache(iq), _batch(iq)
    for f in (L.iq_kv_cache_write, L.iq_kv_cache_read):
        assert f(c, b, None, 256, 16, 256, None) == ARG
        assert f(c, b, 16, 256, None, 256, None) == ARG
        assert f(c, b, 16, 255, 16, 256, None) == ARG
        assert f(c, b, 16, 256, 16, 248, None) == ARG
        assert f(c, b, 24, 256, 16, 256, None) == ALIGN
        assert f(c, b, 16, 256, 18, 256, None) == ALIGN
        assert f(c, b, 16, 260, 16, 256, None) == ALIGN


def test_bad_attention_arguments(iq):
    L, c, b = iq.lib(), _cache(iq), _batch(iq)

    def call(q=16, ldq=1024, heads=8, scale=0.1, out=16, ldo=1024, ws=256, ws_bytes=ENOUGH):
        return L.iq_kv_attention(c, b, q, ldq, heads, scale, out, ldo, ws, ws_bytes, None)

    for kw, want in [(dict(q=None), ARG), (dict(out=None), ARG), (dict(ldq=1016), ARG), (dict(ldo=1000), ARG),
                     (dict(ldq=1028), ALIGN), (dict(ldo=1025), ALIGN), (dict(q=8), ALIGN), (dict(out=20), ALIGN),
                     (dict(heads=0), SHAPE), (dict(heads=7), SHAPE), (dict(heads=-2), SHAPE),
                     (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG), (dict(scale=3e38), ARG),
                     (dict(ws=None), ARG), (dict(ws=128), ALIGN),
                     (dict(ws_bytes=iq.kv_attention_workspace_bytes(3, 8, 2, 128) - 1), WORKSPACE)]:
        assert call(**kw) == want, kw

    def topk(idx=4, ld=7, k=7):
        return L.iq_kv_attention_topk(c, b, 16, 1024, 8, idx, ld, k, 0.1, 16, 1024, 256, 0, None)

    assert topk(idx=None) == ARG and topk(k=0) == ARG and topk(ld=6) == ARG and topk(idx=6) == ALIGN
    assert topk() == WORKSPACE


def test_workspace_sizes(iq):
    f = iq.kv_attention_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(-1, 8, 2, 128) == 0 and f(4, 7, 2, 128) == 0 and f(4, 8, 0, 128) == 0
    assert f(4, 8, 2, 96) == 0
    for rows in (1, 64, 5000):
        for heads in (1, 8, 64, 128):
            assert 0 < f(rows, heads, 1, 128) < 1 << 28


def test_python_checks(iq):
    """The binding's own checks; CPU tensors never reach the library."""
    z = torch.zeros((4, 2, 64, 128), dtype=torch.uint8)
    sf = torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        iq.KVCache(z, z, sf, sf)
    with pytest.raises(ValueError, match="num_pages"):
        iq.KVCache(z[0], z, sf, sf)


@pytest.mark.gpu
def test_python_checks_on_gpu_tensors(cuda_device):
    from fp4_fp8_quant_gb300 import iq
    c = iq.KVCache.empty(4, 2, 64, 128)
    z, sf = c.k_codes, c.k_sf
    for bad in ((z, z[:3], sf, sf), (z, z, sf[:, :1], sf), (z, z, sf, sf.int()), (z.transpose(0, 1), z, sf, sf)):
        with pytest.raises(ValueError):
            iq.KVCache(*bad)
    tab = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    rs, n = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    for k, v, b in [(x.half(), x, (tab, rs, n)), (x, x[:2], (tab, rs, n)), (x[:, :1], x, (tab, rs, n)),
                    (x.cpu(), x, (tab, rs, n)), (x.transpose(0, 1).contiguous().transpose(0, 1), x, (tab, rs, n)),
                    (x, x, (tab.long(), rs, n)), (x, x, (tab, rs[:1], n)), (x, x, (tab[0], rs, n)),
                    (x, x, (tab.cpu(), rs, n)), (x, x, (tab, rs, n.float()))]:
        with pytest.raises(ValueError):
            iq.kv_cache_write(c, k, v, *b)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((3, 5), dtype=torch.int32, device="cuda")
    for bad in (q[:, :, :64], q[0], q.float()):
        with pytest.raises(ValueError):
            iq.kv_attention(c, bad, tab, rs, n)
    with pytest.raises(iq.IQError) as e:
        iq.kv_attention(c, q[:, :7], tab, rs, n)
    assert e.value.code == SHAPE
    for bad in (idx[:2], idx.long(), idx[0], idx.t().contiguous().t()):
        with pytest.raises(ValueError):
            iq.kv_attention_topk(c, q, bad, tab, rs, n)
    with pytest.raises(ValueError):
        iq.kv_attention(c, q, tab, rs, n, workspace=torch.empty(1 << 20, device="cuda"))
    with pytest.raises(iq.IQError) as e:
        iq.kv_attention(c, q, tab, rs, n, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.code in (ARG, WORKSPACE)
