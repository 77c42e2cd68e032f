"""The KV cache kernels against the oracle: every byte of codes and scales
after a write, every value of a read."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from tests.kv_cases import bf16, dev, make_batch, make_cache

pytestmark = pytest.mark.gpu


def _iq():
    from fp4_fp8_quant_gb300 import iq
    return iq


def _gpu_cache(kc, vc):
    return _iq().KVCache(dev(kc["codes"]), dev(vc["codes"]), dev(kc["sf"]), dev(vc["sf"]))


def _same(cache, kc, vc):
    torch.cuda.synchronize()
    assert np.array_equal(cache.k_sf.cpu().numpy(), kc["sf"]) and np.array_equal(cache.v_sf.cpu().numpy(), vc["sf"])
    assert np.array_equal(cache.k_codes.cpu().numpy(), kc["codes"])
    assert np.array_equal(cache.v_codes.cpu().numpy(), vc["codes"])


SHAPES = [(16, 64), (32, 128), (64, 64), (64, 128), (128, 128), (128, 64), (16, 128), (32, 64)]


@pytest.mark.parametrize("page,D", SHAPES)
@pytest.mark.parametrize("H,new,kv_len", [
    (1, [1], [1]),                                        # the first token of all
    (3, [1, 1, 1, 1, 1], [1, 16, 17, 128, 129]),          # decode on page boundaries
    (2, [5, 0, 1, 130, 0, 33], [5, 7, 64, 391, 0, 40]),   # ragged, sequences without rows
    (8, [257], [300]),
    (1, [3] * 50, list(range(3, 53))),                    # many short runs in one window
])
def test_write_is_exact(cuda_device, page, D, H, new, kv_len):
    rng = np.random.default_rng(page * 1000 + D + H)
    batch, P = make_batch(rng, new, kv_len, page, ld_pad=2)
    kc, vc = make_cache(rng, P, H, page, D, 100, 124), make_cache(rng, P, H, page, D, 100, 124)
    T = int(batch[1][-1])
    scale = np.exp2(rng.uniform(-6, 6, (T, 1, 1)))
    x, xt = bf16(rng, (T, H, D), scale)
    y, yt = bf16(rng, (T, H, D), scale[::-1])
    cache = _gpu_cache(kc, vc)
    _iq().kv_cache_write(cache, dev(xt), dev(yt), *map(dev, batch))
    _same(cache, K.write(kc, x, batch), K.write(vc, y, batch))


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128)])
def test_write_token_by_token(cuda_device, page, D):
    """Decoding 40 tokens one at a time, magnitudes rising and falling: the
    older codes are rounded again whenever the page's exponent grows."""
    rng = np.random.default_rng(5)
    H, steps = 2, 40
    (table, _, _), P = make_batch(rng, [1, 1], [60, 45], page)
    kc, vc = make_cache(rng, P, H, page, D, 90, 95), make_cache(rng, P, H, page, D, 90, 95)
    cache = _gpu_cache(kc, vc)
    for i in range(steps):
        batch = (table, np.array([0, 1, 2], np.int32), np.array([20 + i, 5 + i], np.int32))
        x, xt = bf16(rng, (2, H, D), 2.0 ** rng.integers(-8, 9))
        y, yt = bf16(rng, (2, H, D), 2.0 ** rng.integers(-30, 30))
        kc, vc = K.write(kc, x, batch), K.write(vc, y, batch)
        _iq().kv_cache_write(cache, dev(xt), dev(yt), *map(dev, batch))
    _same(cache, kc, vc)


def test_write_extremes(cuda_device):
    """Zeros, values under the floor, the largest BF16 values, signed zeros."""
    rng = np.random.default_rng(6)
    page, D, H = 32, 128, 4
    batch, P = make_batch(rng, [4, 4], [4, 36], page)
    kc, vc = make_cache(rng, P, H, page, D), make_cache(rng, P, H, page, D)
    x = torch.zeros((8, H, D), dtype=torch.bfloat16)
    x[:, 1] = 1e-7
    x[:, 2] = torch.finfo(torch.bfloat16).max
    x[1, 2] = -torch.finfo(torch.bfloat16).max
    x[:, 3] = -0.0
    x[5, 3, 7] = 1e-40
    cache = _gpu_cache(kc, vc)
    _iq().kv_cache_write(cache, dev(x), dev(-x), *map(dev, batch))
    xd = x.to(torch.float64).numpy()
    _same(cache, K.write(kc, xd, batch), K.write(vc, -xd, batch))


def test_write_rows_of_a_wider_tensor(cuda_device):
    """K and V as slices of one projection output, and a table with a row stride."""
    rng = np.random.default_rng(7)
    page, D, H, T = 64, 128, 2, 70
    batch, P = make_batch(rng, [T], [T + 30], page)
    kc, vc = make_cache(rng, P, H, page, D), make_cache(rng, P, H, page, D)
    f, ft = bf16(rng, (T, 7 * H, D))
    fd = dev(ft)
    cache = _gpu_cache(kc, vc)
    wide = torch.full((1, batch[0].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :-5] = dev(batch[0])
    _iq().kv_cache_write(cache, fd[:, 3 * H:4 * H], fd[:, 5 * H:6 * H], wide[:, :-5], dev(batch[1]), dev(batch[2]))
    _same(cache, K.write(kc, f[:, 3 * H:4 * H], batch), K.write(vc, f[:, 5 * H:6 * H], batch))


def test_rows_without_a_page_are_left_out(cuda_device):
    """Negative positions, positions past the table, page numbers outside the pool."""
    rng = np.random.default_rng(8)
    page, D, H = 16, 64, 2
    table = np.array([[0, 3, -1], [99, 2, 1]], np.int32)
    batch = (table, np.array([0, 60, 110], np.int32), np.array([56, 50], np.int32))
    kc, vc = make_cache(rng, 4, H, page, D), make_cache(rng, 4, H, page, D)
    x, xt = bf16(rng, (110, H, D))
    cache = _gpu_cache(kc, vc)
    _iq().kv_cache_write(cache, dev(xt), dev(-xt), *map(dev, batch))
    kc, vc = K.write(kc, x, batch), K.write(vc, -x, batch)
    _same(cache, kc, vc)
    k, v = _iq().kv_cache_read(cache, 110, *map(dev, batch))
    assert np.array_equal(k.double().cpu().numpy(), K.read(kc, batch, 110))
    assert np.array_equal(v.double().cpu().numpy(), K.read(vc, batch, 110))


@pytest.mark.parametrize("page,D", SHAPES)
@pytest.mark.parametrize("H,new,kv_len", [(1, [1], [1]), (5, [7, 0, 200, 1], [7, 3, 500, 129]), (8, [333], [333])])
def test_read_is_exact(cuda_device, page, D, H, new, kv_len):
    rng = np.random.default_rng(page + D + H)
    batch, P = make_batch(rng, new, kv_len, page)
    kc, vc = make_cache(rng, P, H, page, D, 60, 200), make_cache(rng, P, H, page, D, 60, 200)
    T = int(batch[1][-1])
    out = torch.full((2, T, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")   # rows of a wider tensor
    _iq().kv_cache_read(_gpu_cache(kc, vc), T, *map(dev, batch), k=out[0, :, :H], v=out[1, :, :H])
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert np.array_equal(got[0, :, :H], K.read(kc, batch, T)) and np.array_equal(got[1, :, :H], K.read(vc, batch, T))
    assert np.all(got[:, :, H] == 7.0)


def test_offsets_past_32_bits(cuda_device):
    """A pool whose last pages lie more than 2^32 bytes in."""
    page, D, H = 128, 128, 8
    P = (1 << 32) // (H * page * D) + 3
    cache = _iq().KVCache.empty(P, H, page, D)
    rng = np.random.default_rng(9)
    x, xt = bf16(rng, (150, H, D))
    batch = [dev(np.array(a, np.int32)) for a in ([[P - 1, P - 2]], [0, 150], [150])]
    _iq().kv_cache_write(cache, dev(xt), dev(-xt), *batch)
    k, v = _iq().kv_cache_read(cache, 150, *batch)
    small = {"codes": np.zeros((2, H, page, D), np.uint8), "sf": np.zeros((2, H), np.uint8)}
    sb = (np.array([[1, 0]]), np.array([0, 150]), np.array([150]))
    want = K.read(K.write(small, x, sb), sb, 150)
    assert np.array_equal(k.double().cpu().numpy(), want) and np.array_equal(v.double().cpu().numpy(), -want)


def test_write_then_read_on_another_stream(cuda_device):
    """The calls run on the stream they are given, in its order."""
    rng = np.random.default_rng(10)
    page, D, H, T = 64, 128, 4, 500
    batch, P = make_batch(rng, [T], [T], page)
    cache = _iq().KVCache.empty(P, H, page, D)
    x, xt = bf16(rng, (T, H, D))
    xd, b = dev(xt), [dev(a) for a in batch]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _iq().kv_cache_write(cache, xd, xd, *b, stream=st)
    k, v = _iq().kv_cache_read(cache, T, *b, stream=st.cuda_stream)
    st.synchronize()
    empty = {"codes": np.zeros((P, H, page, D), np.uint8), "sf": np.zeros((P, H), np.uint8)}
    want = K.read(K.write(empty, x, batch), batch, T)
    assert np.array_equal(k.double().cpu().numpy(), want) and torch.equal(k, v)
