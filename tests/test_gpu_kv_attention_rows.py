"""Attention of items with many rows (prompts, and selected keys under many
query heads) where its way of working could go wrong: scores that grow along
the keys, lists that begin with nothing, many items of one tile, other scales."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from tests.kv_cases import bf16, dev, gaussian_cache, make_batch
from tests.test_gpu_kv_attention import _check, _gpu_cache, _indices, _iq

pytestmark = pytest.mark.gpu


def _growing(rng, kc, batch, G, D, hot):
    """Queries of which every third prefers one key, far ahead of all others:
    row r of those the key at position hot[r]."""
    T = int(batch[1][-1])
    _, qt = bf16(rng, (T, G, D), 2.0)
    keys, _ = K.gather(kc, batch[0], 0, np.array(hot))
    for r in range(0, T * G, 3):
        qt[r // G, r % G] = torch.from_numpy(keys[r % len(hot), 0] * 20).to(torch.bfloat16)
    return qt.to(torch.float64).numpy(), qt


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,T", [(1500, 2), (9000, 3)])
def test_scores_that_grow_along_the_keys(cuda_device, n, T, D):
    """The largest weight is 2^100 times the first tile's, in a later tile of
    the same block or of another one."""
    rng = np.random.default_rng(n + D)
    page, G = 64, 64
    batch, P = make_batch(rng, [T], [n], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    q, qt = _growing(rng, kc, batch, G, D, [20, 130, 700, n // 2, n - T - 1])
    cache = _gpu_cache(kc, vc)
    _check(_iq().kv_attention(cache, dev(qt), *map(dev, batch)), kc, vc, q, batch, D ** -0.5)
    idx = _indices(rng, batch, 1400, "sorted")
    _check(_iq().kv_attention_topk(cache, dev(qt), dev(idx), *map(dev, batch)), kc, vc, q, batch, D ** -0.5, idx)


def test_growing_scores_beside_ordinary_items(cuda_device):
    """Only some of a block's items are of that kind; the others' bits are
    those of a batch without any."""
    rng = np.random.default_rng(5)
    page, G, D, B = 32, 64, 128, 400
    kv_len = [int(x) for x in rng.integers(1, 400, B)]
    batch, P = make_batch(rng, [1] * B, kv_len, page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    q, qt = bf16(rng, (B, G, D), 2.0)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    plain = _iq().kv_attention(cache, dev(qt), *args)
    _check(plain, kc, vc, q, batch, D ** -0.5)
    hot = [b for b in range(0, B, 7) if kv_len[b] > 200]
    for b in hot:
        keys, _ = K.gather(kc, batch[0], b, np.array([kv_len[b] - 1]))
        qt[b, 5] = torch.from_numpy(keys[0, 0] * 20).to(torch.bfloat16)
    got = _iq().kv_attention(cache, dev(qt), *args)
    _check(got, kc, vc, qt.to(torch.float64).numpy(), batch, D ** -0.5)
    same = [b for b in range(B) if b not in hot]
    assert hot and torch.equal(got[same], plain[same])


@pytest.mark.parametrize("nothing", [1, 128, 200, 300])
def test_lists_that_begin_with_nothing(cuda_device, nothing):
    """The first entries of some lists are no position, all of them in one."""
    rng = np.random.default_rng(nothing)
    page, G, D, k = 64, 64, 128, 300
    batch, P = make_batch(rng, [5, 1], [500, 301], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    q, qt = bf16(rng, (6, G, D), 2.0)
    idx = _indices(rng, batch, k, "sorted")
    idx[::2, :nothing] = -1
    got = _iq().kv_attention_topk(_gpu_cache(kc, vc), dev(qt), dev(idx), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5, idx)


@pytest.mark.parametrize("H,G,T", [(1, 64, 1), (2, 40, 1), (1, 3, 11)])
def test_many_items_of_one_tile(cuda_device, H, G, T):
    rng = np.random.default_rng(G)
    page, D, B = 16, 64, 900
    kv_len = [int(x) for x in rng.integers(T, 129, B)]
    batch, P = make_batch(rng, [T] * B, kv_len, page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (B * T, H * G, D), 2.0)
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scales(cuda_device, scale, D):
    rng = np.random.default_rng(11)
    batch, P = make_batch(rng, [3], [400], 64)
    kc, vc = gaussian_cache(rng, P, 1, 64, D), gaussian_cache(rng, P, 1, 64, D)
    q, qt = bf16(rng, (3, 64, D))
    cache = _gpu_cache(kc, vc)
    _check(_iq().kv_attention(cache, dev(qt), *map(dev, batch), scale=scale), kc, vc, q, batch, scale)
    idx = _indices(rng, batch, 200)
    got = _iq().kv_attention_topk(cache, dev(qt), dev(idx), *map(dev, batch), scale=scale)
    _check(got, kc, vc, q, batch, scale, idx)


@pytest.mark.parametrize("G", [8, 64])
def test_a_nan_query_stays_in_its_row(cuda_device, G):
    rng = np.random.default_rng(21)
    page, D, T = 64, 128, 2
    batch, P = make_batch(rng, [T], [700], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    _, qt = bf16(rng, (T, G, D), 2.0)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    bad = qt.clone()
    bad[1, 3, 5] = float("nan")
    want, got = _iq().kv_attention(cache, dev(qt), *args), _iq().kv_attention(cache, dev(bad), *args)
    assert torch.all(torch.isnan(got[1, 3]))
    keep = torch.ones(T, G, dtype=torch.bool)
    keep[1, 3] = False
    torch.testing.assert_close(got[keep].float(), want[keep].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert _iq().device_status() == 0
