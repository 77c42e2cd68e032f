"""Pins of the KV cache oracle to things other than itself: hand-written pages,
closed forms of the scale rule and of the softmax, and planted mistakes that
must be seen."""

import numpy as np
import pytest

from oracle import iq_oracle as O
from oracle import kv_oracle as K


def _cache(P, H, page, D, sf=127):
    return {"codes": np.zeros((P, H, page, D), np.uint8), "sf": np.full((P, H), sf, np.uint8)}


def _batch(table, row_start, kv_len):
    return (np.array(table, np.int32), np.array(row_start, np.int32), np.array(kv_len, np.int32))


def test_rows_are_the_newest_positions():
    batch = _batch([[0], [1], [2]], [0, 2, 2, 5], [7, 9, 3])
    assert list(K.rows_of(batch)) == [(0, 0, 5), (1, 0, 6), (2, 2, 0), (3, 2, 1), (4, 2, 2)]


def test_write_places_and_scales_by_hand():
    """Two rows crossing a page boundary: each lands in its own page with the
    scale of what that page received."""
    page, D = 16, 64
    c = _cache(4, 1, page, D, sf=7)
    batch = _batch([[3, 1]], [0, 2], [17])               # positions 15 and 16
    x = np.zeros((2, 1, D))
    x[0, 0, 0], x[1, 0, 5] = 448.0, -1.0
    out = K.write(c, x, batch)
    assert out["codes"][3, 0, 15, 0] == 0x7E and out["sf"][3, 0] == 127      # 448 * 2^0; old exponent 7 - 127 is below
    assert out["sf"][1, 0] == 127 - 8                                        # 1 = 256 * 2^-8
    assert O.decode_e4m3(out["codes"][1, 0, 0, 5:6])[0] == -256.0
    changed = np.argwhere(out["codes"] != c["codes"])
    assert sorted(map(tuple, changed)) == [(1, 0, 0, 5), (3, 0, 15, 0)]
    assert out["sf"][0, 0] == 7 and out["sf"][2, 0] == 7


def test_growing_exponent_rounds_the_older_codes():
    page, D = 16, 64
    c = _cache(1, 1, page, D, sf=127)
    vals = np.array([448.0, 3.5, 2.0 ** -9, 3 * 2.0 ** -9, -13.0])
    c["codes"][0, 0, 0, :5] = O.round_to_e4m3_codes(vals)
    x = np.full((1, 1, D), 449.0)                         # needs exponent 1
    out = K.write(c, x, _batch([[0]], [0, 1], [2]))
    assert out["sf"][0, 0] == 128
    # halves; 2^-10 ties to the even 0, 3 * 2^-10 ties to the even 2 * 2^-9
    assert list(O.decode_e4m3(out["codes"][0, 0, 0, :5])) == [224.0, 1.75, 0.0, 2 * 2.0 ** -9, -6.5]
    assert O.decode_e4m3(out["codes"][0, 0, 1, :1])[0] == 224.0
    small = K.write(c, x / 4, _batch([[0]], [0, 1], [2]))  # a smaller row keeps the exponent and the codes
    assert small["sf"][0, 0] == 127 and np.array_equal(small["codes"][0, 0, 0], c["codes"][0, 0, 0])
    fresh = K.write(c, x / 4, _batch([[0]], [0, 1], [1]))  # a page's first row sets the exponent anew
    assert fresh["sf"][0, 0] == 126


def test_read_inverts_write_on_representable_values():
    rng = np.random.default_rng(0)
    page, D, H = 16, 64, 3
    batch = _batch([[5, 0, 2], [1, 4, 3]], [0, 33, 38], [40, 5])
    x = O.decode_e4m3(rng.integers(0, 0x78, (38, H, D)).astype(np.uint8)) * 2.0 ** -3
    x[:, :, 0] = 448.0 * 2.0 ** -3
    got = K.read(K.write(_cache(6, H, page, D, sf=0), x, batch), batch, 38)
    assert np.array_equal(got, x)


def test_missing_pages_read_as_zeros_and_are_not_written():
    c = _cache(2, 1, 16, 64)
    c["codes"][:] = 0x38
    batch = _batch([[-1, 2, 1]], [0, 50], [49])           # position -1, pages -1, 2 (of 2), 1, and past the table
    out = K.read(c, batch, 50)
    assert not out[:33].any() and np.all(out[33:49] == 1.0) and not out[49:].any()
    w = K.write(c, np.ones((50, 1, 64)), batch)
    assert np.array_equal(w["codes"][0], c["codes"][0])


def _random(seed, T, B, kv_len, H=2, Hq=6, page=16, D=64):
    rng = np.random.default_rng(seed)
    W = max(1, max(-(-n // page) for n in kv_len))
    P = B * W + 1
    kc, vc = _cache(P, H, page, D), _cache(P, H, page, D)
    for c in (kc, vc):
        c["codes"] = rng.integers(0, 0x60, c["codes"].shape).astype(np.uint8) | (
            rng.integers(0, 2, c["codes"].shape) << 7).astype(np.uint8)
        c["sf"] = rng.integers(118, 122, c["sf"].shape).astype(np.uint8)
    table = rng.permutation(P)[:B * W].reshape(B, W)
    row_start = np.concatenate([[0], np.cumsum(T)])
    q = rng.standard_normal((row_start[-1], Hq, D))
    return kc, vc, q, _batch(table, row_start, kv_len)


def _brute(kc, vc, q, batch, scale, indices=None, shift=0, drop_sf=False, head_shift=0):
    """Explicit loops over rows, heads and keys."""
    table, row_start, kv_len = batch
    T, Hq, D = q.shape
    H, page = kc["sf"].shape[1], kc["codes"].shape[2]
    out = np.zeros((T, Hq, D))
    for b in range(len(kv_len)):
        for t in range(row_start[b], row_start[b + 1]):
            pos = kv_len[b] - row_start[b + 1] + t + shift
            keys = range(pos + 1) if indices is None else [s for s in indices[t] if 0 <= s <= pos]
            for hq in range(Hq):
                h = (hq // (Hq // H) + head_shift) % H
                num, den = np.zeros(D), 0.0
                for s in keys:
                    p, slot = table[b, s // page], s % page
                    k = O.decode_e4m3(kc["codes"][p, h, slot]) * (1.0 if drop_sf else 2.0 ** (int(kc["sf"][p, h]) - 127))
                    v = O.decode_e4m3(vc["codes"][p, h, slot]) * 2.0 ** (int(vc["sf"][p, h]) - 127)
                    w = np.exp(scale * float(np.dot(q[t, hq], k)))
                    num += w * v
                    den += w
                if den > 0:
                    out[t, hq] = num / den
    return out


@pytest.mark.parametrize("sparse", [False, True])
def test_attention_equals_explicit_loops(sparse):
    kc, vc, q, batch = _random(1, [1, 0, 5], 3, [37, 3, 20])
    idx = None
    if sparse:
        idx = np.array([[0, 5, 36, -1], [-1, -1, -1, -1], [3, 15, 16, 19], [17, 2, 900, 0], [4, 4, 4, 5], [0, -1, 1, -1]])
    got = K.attention(kc, vc, q, batch, 0.125, idx)[0]
    assert np.allclose(got, _brute(kc, vc, q, batch, 0.125, idx), rtol=1e-12, atol=1e-13)
    if sparse:
        assert not got[1].any()                           # a row whose list is empty


def test_attention_closed_forms():
    kc, vc, q, batch = _random(2, [3], 1, [3])
    out = K.attention(kc, vc, q, batch, 0.125)[0]
    V, _ = K.gather(vc, batch[0], 0, np.arange(3))
    assert np.allclose(out[0], np.repeat(V[0], 3, axis=0))          # the first row sees one key: its value
    same = K.attention(kc, vc, np.zeros_like(q), batch, 0.125)[0]
    assert np.allclose(same[2], np.repeat(V.mean(axis=0), 3, axis=0))   # no preference: the mean
    empty = K.attention(kc, vc, q, (batch[0], batch[1], np.array([2])), 0.125)[0]
    assert not empty[0].any() and empty[1].any()                     # position -1 sees nothing


@pytest.mark.parametrize("mistake", [dict(shift=1), dict(drop_sf=True), dict(head_shift=1), dict(scale=0.25)])
def test_planted_mistakes_are_seen(mistake):
    kc, vc, q, batch = _random(3, [2, 4], 2, [20, 30])
    kw = dict(mistake)
    scale = kw.pop("scale", 0.125)
    if "shift" in kw:
        batch = (batch[0], batch[1], batch[2] - 1)
    got = K.attention(kc, vc, q, batch, 0.125)[0]
    assert not np.allclose(got, _brute(kc, vc, q, batch, scale, **kw), rtol=1e-3, atol=1e-4)
