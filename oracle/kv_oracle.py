"""CPU oracle of the paged 8-bit KV cache and its attention (test
infrastructure only): plain numpy in float64, one loop per definition.

A cache is a dict {"codes": uint8 [P, H, page, D], "sf": uint8 [P, H]} for K and
another for V; a batch is (block_table [B, W], row_start [B + 1], kv_len [B]).
"""

from __future__ import annotations

import numpy as np

from .iq_oracle import AMAX_FLOOR, E4M3_MAX, decode_e4m3, decode_ue8m0, round_to_e4m3_codes, ue8m0_exponent


def rows_of(batch):
    """(row, sequence, position) of every packed row."""
    _, row_start, kv_len = batch
    for b in range(len(kv_len)):
        for t in range(row_start[b], row_start[b + 1]):
            yield t, b, int(kv_len[b]) - int(row_start[b + 1]) + t


def page_of(table, b, pos, page, num_pages):
    """Page of a position, or None when the batch does not have it."""
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    p = int(table[b, pos // page])
    return p if 0 <= p < num_pages else None


def write(cache, x, batch):
    """Quantises rows x float64 [T, H, D] into (a copy of) the cache."""
    codes, sf = cache["codes"].copy(), cache["sf"].copy()
    P, H, page, _ = codes.shape
    units = {}                                   # page -> [(slot, row)], in row order
    for t, b, pos in rows_of(batch):
        p = page_of(batch[0], b, pos, page, P)
        if p is not None:
            units.setdefault(p, []).append((pos % page, t))
    for p, members in units.items():
        first = members[0][0]
        rows = [t for _, t in members]
        for h in range(H):
            e = int(ue8m0_exponent(np.array(np.abs(x[rows, h]).max()), E4M3_MAX, AMAX_FLOOR))
            if first > 0:
                old = int(sf[p, h]) - 127
                e = max(e, old)
                if e > old:
                    codes[p, h, :first] = round_to_e4m3_codes(decode_e4m3(codes[p, h, :first]) * 2.0 ** (old - e))
            for slot, t in members:
                codes[p, h, slot] = round_to_e4m3_codes(x[t, h] * 2.0 ** -e)
            sf[p, h] = e + 127
    return {"codes": codes, "sf": sf}


def read(cache, batch, T):
    """float64 [T, H, D] values of the batch's rows (zeros where there is no page)."""
    P, H, page, D = cache["codes"].shape
    out = np.zeros((T, H, D))
    for t, b, pos in rows_of(batch):
        p = page_of(batch[0], b, pos, page, P)
        if p is not None:
            out[t] = decode_e4m3(cache["codes"][p, :, pos % page]) * decode_ue8m0(cache["sf"][p])[:, None]
    return out


def gather(cache, table, b, positions):
    """(values [n, H, D], found [n]) of positions of sequence b."""
    P, H, page, D = cache["codes"].shape
    pids = [page_of(table, b, int(s), page, P) for s in positions]
    found = np.array([p is not None for p in pids], dtype=bool)
    p = np.array([0 if p is None else p for p in pids], dtype=np.int64)
    slot = np.asarray(positions, dtype=np.int64) % page
    val = decode_e4m3(cache["codes"][p, :, slot]) * decode_ue8m0(cache["sf"][p])[:, :, None]
    return np.where(found[:, None, None], val, 0.0), found


def attention(kc, vc, q, batch, scale, indices=None):
    """Causal attention, out float64 [T, Hq, D], and what its error bound needs:
    mag [T, Hq, D] = sum p |v| / sum p, top [T, Hq, D] = max p sum |v| / sum p,
    dot [T, Hq] = the largest |scale| sum_d |q k| among the row's keys."""
    T, Hq, D = q.shape
    H = kc["sf"].shape[1]
    g = Hq // H
    out, mag, top = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    dot = np.zeros((T, Hq))
    for t, b, pos in rows_of(batch):
        if indices is None:
            cand = np.arange(max(pos + 1, 0))
        else:
            cand = np.array([s for s in indices[t] if 0 <= s <= pos], dtype=np.int64)
        if len(cand) == 0:
            continue
        K, found = gather(kc, batch[0], b, cand)
        V, _ = gather(vc, batch[0], b, cand)
        K, V = K[found], V[found]
        if len(K) == 0:
            continue
        for h in range(H):
            qh = q[t, h * g:(h + 1) * g]                            # [g, D]
            s = scale * (qh @ K[:, h].T)                            # [g, n]
            p = np.exp(s - s.max(axis=1, keepdims=True))
            total = p.sum(axis=1, keepdims=True)
            out[t, h * g:(h + 1) * g] = p @ V[:, h] / total
            mag[t, h * g:(h + 1) * g] = p @ np.abs(V[:, h]) / total
            top[t, h * g:(h + 1) * g] = np.abs(V[:, h]).sum(axis=0) / total
            dot[t, h * g:(h + 1) * g] = abs(scale) * (np.abs(qh) @ np.abs(K[:, h]).T).max(axis=1)
    return out, mag, top, dot
