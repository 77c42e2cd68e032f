"""Seeded inputs of the KV cache tests, and the error bound of the attention."""

import numpy as np
import torch

from oracle import iq_oracle as O


def make_batch(rng, new, kv_len, page, spare=3, ld_pad=0):
    """Block table over a shuffled pool (unused entries -1), row_start, kv_len
    and the pool's size."""
    B = len(new)
    need = [max(0, -(-n // page)) for n in kv_len]
    W = max(1, max(need))
    P = sum(need) + spare
    perm = rng.permutation(P)
    table = np.full((B, W + ld_pad), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    row_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return (table, row_start, np.array(kv_len, np.int32)), P


def make_cache(rng, P, H, page, D, sf_lo=115, sf_hi=122):
    """Finite random codes of all magnitudes and scales spread over 2^7."""
    c = {"codes": rng.integers(0, 0x7F, (P, H, page, D)).astype(np.uint8),
         "sf": rng.integers(sf_lo, sf_hi, (P, H)).astype(np.uint8)}
    c["codes"] |= (rng.integers(0, 2, c["codes"].shape) << 7).astype(np.uint8)
    return c


def gaussian_cache(rng, P, H, page, D):
    """Codes of normal values: K . q then looks like real scores."""
    x = rng.standard_normal((P, H, page, D)) * np.exp2(rng.uniform(-1, 1, (P, H, 1, 1)))
    e = O.ue8m0_exponent(np.abs(x).max(axis=(2, 3)), 448.0, 1e-4).astype(np.int64)
    return {"codes": O.round_to_e4m3_codes(x * np.exp2(-e.astype(np.float64))[:, :, None, None]).astype(np.uint8),
            "sf": (e + 127).astype(np.uint8)}


def bf16(rng, shape, scale=1.0):
    """(float64 values, BF16 tensor) of normal draws."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t.to(torch.float64).numpy(), t


def dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).cuda()


def attention_bound(out, mag, top, dot):
    """Largest allowed |kernel - exact| per output.

    - the result is rounded to BF16: 2^-9 |out| (2^-8 allows for the half ulp
      of a value just above a power of two);
    - a score is a float32 sum of D <= 128 exact products, scaled: its error is
      at most 128 * 2^-23 * dot with truncated additions, so 2^-15 * dot
      covers it with the few roundings of the scaling; a score error d changes
      a weight by the factor exp(d), in numerator and denominator: 2 d mag;
    - a weight enters the second product with at least 8 significant bits
      (2^-8 of itself) or, far below the largest weight, with an absolute
      error of 2^-18 of the largest one: 2^-8 mag + 2^-18 top;
    - exp2, the float32 sums over n keys and the final division stay below
      2^-12 for n < 2^11 keys per partial sum and pairwise joining.
    """
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -12) * mag + 2 * 2.0 ** -15 * dot[:, :, None] * mag \
        + 2.0 ** -18 * top + 1e-30
