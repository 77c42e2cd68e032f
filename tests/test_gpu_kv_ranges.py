"""What the cache calls do with values at the ends of their ranges: batches that
name rows that are not there, the largest scores, dominant keys, scale bytes."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from tests.kv_cases import bf16, dev, gaussian_cache, make_batch, make_cache
from tests.test_gpu_kv_attention import _check, _gpu_cache, _indices, _iq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G", [(2, 4), (1, 64)])
@pytest.mark.parametrize("first,last", [(0, 5), (-3, 0), (-3, 5)])
def test_rows_that_are_not_there_are_not_touched(cuda_device, H, G, first, last):
    """row_start begins `first` rows before 0 and ends `last` rows past the
    last one: the rows that exist keep their positions, and the rows of the
    wider tensors around them stay as they are."""
    rng = np.random.default_rng(G + last)
    page, D, new, kv_len = 64, 128, [3, 9, 40], [300, 9, 170]
    T, pad = sum(new), 8
    batch, P = make_batch(rng, new, kv_len, page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (T + 2 * pad, H * G, D), 2.0)
    out = torch.full(qt.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    row_start, length = batch[1].copy(), batch[2].copy()
    row_start[0] += first
    row_start[-1] += last
    length[-1] += last                                   # row t is at kv_len - row_start[b + 1] + t
    cache, inner = _gpu_cache(kc, vc), slice(pad, pad + T)
    _iq().kv_attention(cache, dev(qt)[inner], dev(batch[0]), dev(row_start), dev(length), out=out[inner])
    _check(out[inner], kc, vc, q[inner], batch, D ** -0.5)
    assert torch.all(out[:pad] == 5.0) and torch.all(out[pad + T:] == 5.0)


@pytest.mark.parametrize("first,last", [(0, 5), (-3, 0), (-3, 5)])
def test_rows_that_are_not_there_are_not_written_or_read(cuda_device, first, last):
    rng = np.random.default_rng(31)
    page, D, H, new, kv_len = 16, 64, 2, [3, 9, 40], [300, 9, 170]
    T = sum(new)
    batch, P = make_batch(rng, new, kv_len, page)
    kc, vc = make_cache(rng, P, H, page, D), make_cache(rng, P, H, page, D)
    x, xt = bf16(rng, (T, H, D))
    row_start, length = batch[1].copy(), batch[2].copy()
    row_start[0] += first
    row_start[-1] += last
    length[-1] += last
    args = dev(batch[0]), dev(row_start), dev(length)
    cache = _gpu_cache(kc, vc)
    _iq().kv_cache_write(cache, dev(xt), dev(-xt), *args)
    k, v = _iq().kv_cache_read(cache, T, *args)
    kc, vc = K.write(kc, x, batch), K.write(vc, -x, batch)
    assert np.array_equal(cache.k_codes.cpu().numpy(), kc["codes"]) and np.array_equal(cache.v_sf.cpu().numpy(), vc["sf"])
    assert np.array_equal(k.double().cpu().numpy(), K.read(kc, batch, T))
    assert np.array_equal(v.double().cpu().numpy(), K.read(vc, batch, T))


def _large_scores(rng, G, D, n, lists):
    """Rows whose query is a multiple of one key, 2^22 to 2^29 times it: its
    score is far ahead of every other's by more than float32 rounds it, so the
    output is that key's value, which BF16 holds."""
    page = 64
    batch, P = make_batch(rng, [2], [n], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    every, _ = K.gather(kc, batch[0], 0, np.arange(n))
    dots = every[:, 0] @ every[:, 0].T
    order = np.sort(dots, axis=1)
    clear = [s for s in range(n - 2) if dots[s, s] == order[s, -1] and order[s, -1] - order[s, -2] > 5]
    hot = rng.choice(clear, (2, G))
    keys, _ = K.gather(kc, batch[0], 0, hot.ravel())
    values, _ = K.gather(vc, batch[0], 0, hot.ravel())
    q = keys[:, 0].reshape(2, G, D) * 2.0 ** np.linspace(22, 29, 2 * G).reshape(2, G, 1)
    qt = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    score = np.einsum("tgd,nd->tgn", qt.to(torch.float64).numpy(), every[:, 0]) * D ** -0.5
    ahead = np.sort(score, axis=2)
    assert np.all(ahead[:, :, -1] - ahead[:, :, -2] > 1000) and np.all(score.argmax(axis=2) == hot)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    if lists:
        idx = np.stack([rng.permutation(n - 2) for _ in range(2)]).astype(np.int32)
        got = _iq().kv_attention_topk(cache, dev(qt), dev(idx), *args)
    else:
        got = _iq().kv_attention(cache, dev(qt), *args)
    assert _iq().device_status() == 0
    assert np.array_equal(got.double().cpu().numpy(), values[:, 0].reshape(2, G, D))


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("G,D", [(5, 128), (8, 64), (16, 128)])
def test_the_largest_scores_settle(cuda_device, G, D, lists):
    """(For two tokens: up to 32 rows per item.)"""
    _large_scores(np.random.default_rng(G + D), G, D, 700, lists)
