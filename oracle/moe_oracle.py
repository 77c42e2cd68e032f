"""CPU oracle of the experts' feed-forward block and of the adapters (test
infrastructure only): plain numpy in float64, one loop per definition."""

from __future__ import annotations

import numpy as np

from .iq_oracle import decode_e4m3, decode_ue8m0


def route(logits, k, score="softmax", normalize=False, scale=1.0):
    """(weights, experts, slots, rows, row_start) of float logits [T, E]."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64)) + 0.0
    T, E = l.shape
    w, experts = np.zeros((T, k)), np.zeros((T, k), np.int32)
    for t in range(T):
        chosen = sorted(range(E), key=lambda e: (-l[t, e], e))[:k]
        experts[t] = chosen
        top = l[t, chosen]
        if score == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-top))
            if normalize:
                p = p / p.sum() if p.sum() > 0 else 0.0 * p
        elif top[0] == -np.inf:
            p = np.zeros(k)
        else:
            with np.errstate(invalid="ignore"):
                rel = np.where(l[t] == top[0], 0.0, l[t] - top[0])
            every = np.exp(rel)
            p = every[chosen] / (every[chosen].sum() if normalize else every.sum())
        w[t] = p * scale
    pairs = sorted((int(experts[t, j]), t, j) for t in range(T) for j in range(k))
    slots, rows = np.zeros((T, k), np.int32), np.zeros(T * k, np.int32)
    for s, (_, t, j) in enumerate(pairs):
        slots[t, j] = s
        rows[s] = t
    row_start = np.array([sum(1 for p in pairs if p[0] < e) for e in range(E + 1)], np.int32)
    return w, experts, slots, rows, row_start


def unpack_scales(words, K):
    """UE8M0 bytes [M_al, K / 128] of the packed words [ceil(K / 512), M_al]."""
    b = np.ascontiguousarray(words).view(np.uint8).reshape(words.shape[0], words.shape[1], 4)
    return b.transpose(1, 0, 2).reshape(words.shape[1], -1)[:, :K // 128]


def silu(g):
    return g / (1.0 + np.exp(-np.clip(g, -700, None)))


def grouped(x, words, w, w_sf, row_start, gated=False):
    """(out, magnitude) float64 [M, .] of grouped products and a bool [M]: the
    rows that belong to a group.  Magnitude: what the sums' errors scale with."""
    M, K = x.shape
    G, N, _ = w.shape
    xs = decode_ue8m0(unpack_scales(words, K))[:M]
    xv = decode_e4m3(x) * np.repeat(xs, 128, axis=1)
    y, mag, there = np.zeros((M, N)), np.zeros((M, N)), np.zeros(M, bool)
    for g in range(G):
        lo = min(max(int(row_start[g]), 0), M)
        hi = min(max(int(row_start[g + 1]), lo), M)
        if lo == hi:
            continue
        f = np.repeat(np.repeat(decode_ue8m0(w_sf[g]), 128, axis=0)[:N], 128, axis=1)
        wv = decode_e4m3(w[g]) * f
        y[lo:hi] = xv[lo:hi] @ wv.T
        mag[lo:hi] = np.abs(xv[lo:hi]) @ np.abs(wv).T
        there[lo:hi] = True
    if gated:
        gate, up, mg, mu = y[:, :N // 2], y[:, N // 2:], mag[:, :N // 2], mag[:, N // 2:]
        return silu(gate) * up, 1.1 * np.abs(up) * mg + np.abs(silu(gate)) * mu, there
    return y, mag, there


def combine(y, slots, weights, add=None):
    """(out, magnitude) of the weighted sums."""
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if add is None else add.astype(np.float64)
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                out[t] = out[t] + float(weights[t, j]) * y[slots[t, j]]
                mag[t] = mag[t] + np.abs(float(weights[t, j]) * y[slots[t, j]])
    return out, mag


def adapters(x, base, a, b, scale, row_start, adapter):
    """(out, magnitude of the low-rank term's sums, rows of some request)."""
    T, N = x.shape[0], b.shape[1]
    out = np.zeros((T, N)) if base is None else base.astype(np.float64).copy()
    mag, there, covered = np.zeros((T, N)), np.zeros(T, bool), 0
    for i in range(len(adapter)):
        end = min(max(int(row_start[i + 1]), 0), T)
        lo = max(min(max(int(row_start[i]), 0), T), covered)
        hi = max(end, lo)
        covered = max(covered, end)
        there[lo:hi] = True
        j = int(adapter[i])
        if 0 <= j < len(scale) and hi > lo:
            s = float(scale[j])
            out[lo:hi] += s * ((x[lo:hi] @ a[j].T) @ b[j].T)
            mag[lo:hi] = abs(s) * ((np.abs(x[lo:hi]) @ np.abs(a[j]).T) @ np.abs(b[j]).T)
    return out, mag, there
