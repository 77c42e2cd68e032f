"""What the cache calls do with values at the ends of their ranges: batches that
name rows that are not there, the largest scores, dominant keys, scale bytes."""

import numpy as np
import pytest
import torch

from oracle import iq_oracle as O
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


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("G,D", [(64, 128), (40, 64), (64, 64)])
def test_the_largest_scores_many_rows(cuda_device, G, D, lists):
    _large_scores(np.random.default_rng(G + D), G, D, 700, lists)


def _quantised(x, page):
    """A cache of one head whose pages 0, 1, ... hold the rows x, each page
    under the scale of its largest value."""
    n, D = x.shape
    P = -(-n // page)
    full = np.zeros((P * page, D))
    full[:n] = x
    full = full.reshape(P, 1, page, D)
    e = O.ue8m0_exponent(np.abs(full).max(axis=(2, 3)), 448.0, 1e-4).astype(np.int64)
    return {"codes": O.round_to_e4m3_codes(full * np.exp2(-e.astype(np.float64))[:, :, None, None]).astype(np.uint8),
            "sf": (e + 127).astype(np.uint8)}


def _dominant_first_key(rng, n, D, share, scale_up):
    """Keys of which the first has about `share` of every row's weight and the
    others, within an octave of one another, the rest.  The values have a common
    part, the first key's is small; in dimension 3 one value of the first page
    is 2^scale_up times the others."""
    k = rng.standard_normal((n, D)) * 0.05
    k[:, 0] = 0.0
    k[0] = 0.0
    k[0, 0] = 1.0
    v = 1.0 + 0.25 * rng.standard_normal((n, D))
    v[0] = 0.0625
    if scale_up:
        v[:16] = 0.0
        v[5, 3] = 2.0 ** scale_up
    return k, v, np.log((n - 1) * share / (1 - share)) * np.sqrt(D)


def _check_weights(got, kc, vc, q, batch, indices=None):
    """The bound: a result and a weight rounded to BF16 (2^-8 of themselves, the
    weights alike in the sum), float32 sums and exponentials (2^-12), and scores
    as float32 sums (tests/kv_cases.py).  It does not grow with the keys."""
    D = q.shape[2]
    out, mag, _, dot = K.attention(kc, vc, q, batch, D ** -0.5, indices)
    err = np.abs(got.double().cpu().numpy() - out)
    bound = 2.0 ** -8 * (2 * np.abs(out) + mag) + (2.0 ** -12 + 2 * 2.0 ** -15 * dot[:, :, None]) * mag
    worst = np.unravel_index(np.argmax(err / bound), err.shape)
    assert np.all(err <= bound), f"at {worst}: error {err[worst]:.3g}, allowed {bound[worst]:.3g}, exact {out[worst]:.3g}"
    assert _iq().device_status() == 0


def _first_key_case(G, D, n, share, scale_up, lists, seqs=1):
    """`seqs` sequences over the same pages, each with one token; with many of
    them an item is not divided between blocks.  Four are compared."""
    rng = np.random.default_rng(n + D)
    page = 16
    k, v, top = _dominant_first_key(rng, n, D, share, scale_up)
    kc, vc = _quantised(k, page), _quantised(v, page)
    pages = np.arange(-(-n // page), dtype=np.int32)[None]
    batch = (np.repeat(pages, seqs, 0), np.arange(seqs + 1, dtype=np.int32), np.full(seqs, n, np.int32))
    q = rng.standard_normal((seqs, G, D))
    q[:, :, 0] = top * rng.uniform(0.98, 1.02, (seqs, G))
    qt = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    q, cache, args = qt.to(torch.float64).numpy(), _gpu_cache(kc, vc), [dev(a) for a in batch]
    idx = np.concatenate([[0], 1 + rng.permutation(n - 1)]).astype(np.int32)[None] if lists else None
    if lists:
        got = _iq().kv_attention_topk(cache, dev(qt), dev(np.repeat(idx, seqs, 0)), *args)
    else:
        got = _iq().kv_attention(cache, dev(qt), *args)
    for s in sorted({0, seqs // 3, seqs // 2, seqs - 1}):
        one = (pages, np.array([0, 1], np.int32), np.array([n], np.int32))
        _check_weights(got[s:s + 1], kc, vc, q[s:s + 1], one, idx)


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("n,share", [(4632, 0.9), (4632, 0.5), (33000, 0.9), (33000, 0.99)])
@pytest.mark.parametrize("G,D", [(64, 64), (40, 128)])
def test_a_dominant_first_key_does_not_hide_the_others_many_rows(cuda_device, G, D, n, share, lists):
    _first_key_case(G, D, n, share, 0, lists, 310)


def test_a_dominant_first_key_of_a_long_context(cuda_device):
    _first_key_case(64, 64, 131072, 0.9, 0, False, 155)


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("scale_up", [12, 24, 40])
@pytest.mark.parametrize("n,share", [(3000, 0.0005), (33000, 0.9)])
def test_a_first_page_of_large_values_does_not_hide_the_others_many_rows(cuda_device, n, share, scale_up, lists):
    _first_key_case(64, 128, n, share, scale_up, lists)


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("G", [8, 32])
@pytest.mark.parametrize("n,share,scale_up", [(4632, 0.9, 0), (33000, 0.99, 0), (3000, 0.0005, 12), (3000, 0.0005, 24),
                                              (33000, 0.9, 12), (33000, 0.9, 40)])
def test_a_dominant_first_key_or_page_few_rows(cuda_device, n, share, scale_up, G, lists):
    """310 sequences: items are whole in a block; one: they are divided."""
    _first_key_case(G, 128, n, share, scale_up, lists, 310 if n < 10000 else 1)


@pytest.mark.parametrize("G", [8, 64])
def test_equal_scores_of_any_size_under_different_value_scales(cuda_device, G):
    """Two keys are the same, far ahead of the rest, and lie in pages whose
    value scales differ by 2^6: they count alike however large the score."""
    rng = np.random.default_rng(G)
    page, D, n = 16, 64, 300
    k, v = rng.standard_normal((n, D)) * 0.1, rng.standard_normal((n, D))
    k[[5, 250], :4] = 3.0
    v[240:256] *= 64.0
    v[[5, 250], 0] = 1.0, 3.0
    k[250] = k[5]
    kc, vc = _quantised(k, page), _quantised(v, page)
    batch = (np.arange(-(-n // page), dtype=np.int32)[None], np.array([0, 1], np.int32), np.array([n], np.int32))
    q = np.zeros((1, G, D))
    q[:, :, :4] = 2.0 ** np.linspace(4, 30, G)[None, :, None]
    qt = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    values, _ = K.gather(vc, batch[0], 0, np.array([5, 250]))
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *[dev(a) for a in batch]).double().cpu().numpy()
    want = np.broadcast_to(values[:, 0].mean(axis=0), got.shape)
    other = want == 0                                    # (what is left there is the other keys')
    assert np.all((np.abs(got - want) <= 2.0 ** -7 * np.abs(want)) | other)


@pytest.mark.parametrize("grow", [False, True])
def test_thousands_of_segments_per_block(cuda_device, grow):
    """48000 tokens with a list each under 4 KV heads: some 1260 segments for
    each block of the many-rows kernel.  With `grow` the later lists end with a
    key far ahead of their first tile's."""
    rng = np.random.default_rng(40)
    T, H, G, D, page, k, n = 48000, 4, 33, 64, 16, 140, 400
    table, P = make_batch(rng, [1], [n], page)
    table = table[0]
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    batch = (np.repeat(table, T, 0), np.arange(T + 1, dtype=np.int32), np.full(T, n, np.int32))
    lists = np.stack([rng.permutation(n)[:k] for _ in range(50)]).astype(np.int32)
    _, some = bf16(rng, (50, H * G, D), 2.0)
    if grow:
        for t in range(25, 50):                          # (tokens 25 .. 49 of every 50)
            hot, _ = K.gather(kc, table, 0, lists[t, -1:])
            some[t, 3::G] = torch.from_numpy(hot[0] * 20).to(torch.bfloat16)
    idx, qt = dev(lists).repeat(T // 50, 1), dev(some).repeat(T // 50, 1, 1)
    got = _iq().kv_attention_topk(_gpu_cache(kc, vc), qt, idx, *[dev(a) for a in batch])
    one = (np.repeat(table, 50, 0), np.arange(51, dtype=np.int32), np.full(50, n, np.int32))
    _check_weights(got[:50], kc, vc, some.to(torch.float64).numpy(), one, lists)
    rounds = got.view(T // 50, 50, H * G, D).float()
    torch.testing.assert_close(rounds, rounds[:1].expand_as(rounds), rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("G", [8, 64])
def test_an_infinite_query_gives_nan_in_its_row(cuda_device, G, value):
    rng = np.random.default_rng(22)
    page, D, T = 64, 128, 2
    batch, P = make_batch(rng, [T], [700], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    kc["sf"] -= 8                                        # keys so small that 448 times 2^120 would give finite scores
    _, qt = bf16(rng, (T, G, D), 2.0)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    bad = qt.clone()
    bad[1, 3, 5] = value
    idx = dev(_indices(rng, batch, 300))
    for call in (lambda q: _iq().kv_attention(cache, dev(q), *args), lambda q: _iq().kv_attention_topk(cache, dev(q), idx, *args)):
        want, got = call(qt), call(bad)
        assert torch.all(torch.isnan(got[1, 3]))
        keep = torch.ones(T, G, dtype=torch.bool)
        keep[1, 3] = False
        torch.testing.assert_close(got[keep].float(), want[keep].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert _iq().device_status() == 0


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("G", [8, 64])
def test_scores_near_the_lowest_float(cuda_device, G, lists):
    """All scores lie around -2^110 and below; the one nearest to zero counts."""
    rng = np.random.default_rng(23)
    page, D, n = 64, 128, 300
    batch, P = make_batch(rng, [1], [n], page)
    k = np.abs(rng.standard_normal((P * page, D))) + 1.0
    k[::7] *= 0.25
    kc, vc = _quantised(k, page), gaussian_cache(rng, P, 1, page, D)
    q = np.full((1, G, D), -2.0 ** 103) * (1.0 + rng.integers(0, 4, (1, G, 1)) / 4)
    qt = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    keys, _ = K.gather(kc, batch[0], 0, np.arange(n))
    score = np.einsum("gd,nd->gn", q[0], keys[:, 0])
    best = score.argmax(axis=1)
    assert np.all(np.sort(score, axis=1)[:, -1] - np.sort(score, axis=1)[:, -2] > 2.0 ** 90)
    values, _ = K.gather(vc, batch[0], 0, best)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    if lists:
        got = _iq().kv_attention_topk(cache, dev(qt), dev(rng.permutation(n).astype(np.int32)[None]), *args)
    else:
        got = _iq().kv_attention(cache, dev(qt), *args)
    assert np.array_equal(got[0].double().cpu().numpy(), values[:, 0])
    assert _iq().device_status() == 0


def test_read_with_every_scale_byte(cuda_device):
    """All 254 finite codes under every byte: exact where BF16 holds the value,
    else rounded to nearest even or infinite; 255 gives NaN."""
    page, D = 16, 64
    every = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    codes = np.zeros((256, 1, page * D), np.uint8)
    codes[:, 0, :254] = every
    c = {"codes": codes.reshape(256, 1, page, D), "sf": np.arange(256, dtype=np.uint8)[:, None]}
    batch = (np.arange(256, dtype=np.int32).reshape(256, 1), page * np.arange(257, dtype=np.int32), np.full(256, page, np.int32))
    got, _ = _iq().kv_cache_read(_gpu_cache(c, c), 256 * page, *[dev(a) for a in batch])
    exact = O.decode_e4m3(codes.reshape(256, -1)) * 2.0 ** (np.arange(256.0) - 127)[:, None]
    with np.errstate(over="ignore"):
        want = torch.from_numpy(exact.astype(np.float32)).to(torch.bfloat16)     # (float32 is exact here, or 2^128 and more)
    got = got.cpu().reshape(256, -1)
    assert torch.equal(got[:255], want[:255]) and torch.all(torch.isnan(got[255]))
    held = want[:255].double().numpy() == exact[:255]
    assert np.all(held[3:247]) and not np.all(held[2]) and not np.all(held[247])


@pytest.mark.parametrize("G", [8, 64])
@pytest.mark.parametrize("k_lo,v_lo", [(100, 64), (118, 236), (20, 100)])
def test_attention_under_scale_bytes_far_from_127(cuda_device, G, k_lo, v_lo):
    rng = np.random.default_rng(G + v_lo)
    page, D, n = 16, 64, 500
    batch, P = make_batch(rng, [3], [n], page)
    kc, vc = make_cache(rng, P, 1, page, D, k_lo, k_lo + 3), make_cache(rng, P, 1, page, D, v_lo, v_lo + 3)
    q, qt = bf16(rng, (3, G, D), 2.0 ** (118 - k_lo - 5))
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    _check_weights(_iq().kv_attention(cache, dev(qt), *args), kc, vc, q, batch)
    idx = _indices(rng, batch, 200)
    _check_weights(_iq().kv_attention_topk(cache, dev(qt), dev(idx), *args), kc, vc, q, batch, idx)


@pytest.mark.parametrize("n", [200, 20000])
@pytest.mark.parametrize("G", [8, 64])
def test_the_mean_of_the_largest_values(cuda_device, G, n):
    """20000 values of 1.5 * 2^126 with equal weights: their sum leaves float32,
    their mean does not."""
    page, D = 64, 128
    P = -(-n // page)
    c = {"codes": np.full((P, 1, page, D), 0x3C, np.uint8), "sf": np.full((P, 1), 253, np.uint8)}
    args = dev(np.arange(P, dtype=np.int32)[None]), dev(np.array([0, 1], np.int32)), dev(np.array([n], np.int32))
    q = torch.zeros((1, G, D), dtype=torch.bfloat16, device="cuda")
    k = dict(c, sf=np.full((P, 1), 127, np.uint8))
    got = _iq().kv_attention(_gpu_cache(k, c), q, *args)
    assert torch.all(got.double() == 1.5 * 2.0 ** 126) and _iq().device_status() == 0


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("G,D", [(4, 64), (16, 128), (32, 128)])
def test_weights_of_few_rows_keep_sixteen_bits(cuda_device, G, D, lists):
    """The bound of _check_weights with 2^-14 for a weight: two BF16 terms leave
    2^-17 of it, and the float32 sums add the unrounded ones."""
    rng = np.random.default_rng(G + D)
    page, n = 64, 5000
    batch, P = make_batch(rng, [1], [n], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    q, qt = bf16(rng, (1, G, D), 2.0)
    cache, args = _gpu_cache(kc, vc), [dev(a) for a in batch]
    idx = _indices(rng, batch, 1500) if lists else None
    got = _iq().kv_attention_topk(cache, dev(qt), dev(idx), *args) if lists else _iq().kv_attention(cache, dev(qt), *args)
    out, mag, _, dot = K.attention(kc, vc, q, batch, D ** -0.5, idx)
    err = np.abs(got.double().cpu().numpy() - out)
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -14 + 2.0 ** -12 + 2 * 2.0 ** -15 * dot[:, :, None]) * mag
    assert np.all(err <= bound) and _iq().device_status() == 0


@pytest.mark.parametrize("row_start", [[2 ** 31 - 1, -2 ** 31], [-2 ** 31, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1], [7, 2]])
@pytest.mark.parametrize("G", [8, 64])
def test_a_batch_that_names_no_row_touches_nothing(cuda_device, G, row_start):
    rng = np.random.default_rng(50)
    page, D, T = 64, 128, 5
    batch, P = make_batch(rng, [T], [300], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    _, qt = bf16(rng, (T, G, D), 2.0)
    out = torch.full((T, G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), dev(batch[0]), dev(np.array(row_start, np.int32)), dev(batch[2]), out=out)
    assert torch.all(out == 5.0) and _iq().device_status() == 0
