"""The attention block's operators from their definitions, in float64.

bf16 arrays are uint16 bit patterns. A batch is ragged: sequence b owns rows
``cu_q[b] .. cu_q[b+1]-1`` of the new tokens and ``kv_lens[b]`` keys, the new
tokens' among them; position j of it is token ``j % page_size`` of page
``table[b, j // page_size]`` of the cache ``[pages, page_size, heads, D]``.
"""

from __future__ import annotations

import numpy as np

BF16_HALF_STEP = 2.0 ** -8   # largest relative error of one rounding to bf16
FP32_HALF_STEP = 2.0 ** -24


def bf16_f64(bits: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def rope(x: np.ndarray, positions, inv_freq, interleaved: bool = False, amplitude: float = 1.0):
    """x float64 [T, H, D] -> (y, size): y exact, size = |x1| + |x2| of the pair that gives each element (0 where copied)."""
    f = np.asarray(inv_freq, np.float32).astype(np.float64)
    n = f.size
    ang = np.asarray(positions, np.float64)[:, None] * f[None, :]
    c, s = amplitude * np.cos(ang)[:, None, :], amplitude * np.sin(ang)[:, None, :]
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y, size = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., first], x[..., second]
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., first] = size[..., second] = np.abs(x1) + np.abs(x2)
    return y, size


def rope_tolerance(y, size, amplitude: float = 1.0):
    """One rounding to bf16, and in fp32: the angle (in units of pi, at most 1, rounded to fp32: pi 2^-25, and the sine's
    and cosine's own few units), the factor, two products and a sum: below 2^-20 of |x1| + |x2| in all."""
    return BF16_HALF_STEP * np.abs(y) + (1 + BF16_HALF_STEP) * 2.0 ** -20 * abs(amplitude) * size


def positions(cu_q, kv_lens):
    """(sequence, position) of each row of the batch."""
    seq, pos = [], []
    for b in range(len(kv_lens)):
        n = cu_q[b + 1] - cu_q[b]
        seq += [b] * n
        pos += [kv_lens[b] - n + i for i in range(n)]
    return np.array(seq, np.int64), np.array(pos, np.int64)


def paged_attention(q, k_cache, v_cache, table, cu_q, kv_lens, scale: float, window: int = 0):
    """q float64 [T, Hq, D], caches float64 -> dict of out [T, Hq, D], lse [T, Hq], and for the tolerance abs = sum p |v|,
    score = the largest scale * sum |q k| of a row's keys, keys = how many a row sees. Rows of no sequence are NaN."""
    T, Hq, D = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    g = Hq // Hkv
    out, ab = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, score = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    keys = np.zeros((T,), np.int64)
    for b in range(len(kv_lens)):
        r0, r1, m = int(cu_q[b]), int(cu_q[b + 1]), int(kv_lens[b])
        if r1 == r0:
            continue
        pages = np.asarray(table[b, : -(-m // page)], np.int64)
        k = k_cache[pages].reshape(-1, Hkv, D)[:m]
        v = v_cache[pages].reshape(-1, Hkv, D)[:m]
        pos = m - (r1 - r0) + np.arange(r1 - r0)
        j = np.arange(m)
        seen = j[None, :] <= pos[:, None]
        if window > 0:
            seen &= j[None, :] > pos[:, None] - window
        keys[r0:r1] = seen.sum(1)
        for h in range(Hq):
            if m == 0:
                out[r0:r1, h], ab[r0:r1, h], lse[r0:r1, h], score[r0:r1, h] = 0, 0, -np.inf, 0
                continue
            # keys that nobody of the sequence sees may hold anything
            live = seen.any(0)
            kh, vh = np.where(live[:, None], k[:, h // g], 0), np.where(live[:, None], v[:, h // g], 0)
            s = np.where(seen, scale * (q[r0:r1, h] @ kh.T), -np.inf)
            top = s.max(1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0)
            p = np.exp(s - top)
            l = p.sum(1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[r0:r1, h] = (np.log(l) + top)[:, 0]
            p = p / np.where(l > 0, l, 1)
            out[r0:r1, h] = p @ vh
            ab[r0:r1, h] = p @ np.abs(vh)
            score[r0:r1, h] = np.where(seen, scale * (np.abs(q[r0:r1, h]) @ np.abs(kh).T), 0).max(1)
    return {"out": out, "lse": lse, "abs": ab, "score": score, "keys": keys}


def attention_tolerance(ref, D: int):
    """(for out, for lse). A score is a sum of D exact products in fp32 in any order, the tensor core's adds being off by a
    whole step each at most: D 2^-23 of scale sum |q k|, and its scaling and shift for the exponential 4 steps more: ds. A
    probability is then off by 2 ds (its own score and the maximum or the sum), by its exponential (2^-21) and by its
    rounding to bf16 (2^-8); the sums over n keys by n 2^-23; out by one rounding to bf16."""
    ds = (D + 4) * 2.0 ** -23 * ref["score"]
    n = (ref["keys"][:, None] + 64) * 2.0 ** -23
    rel = BF16_HALF_STEP + 2 * ds + 2 * n + 2.0 ** -20
    out = rel[..., None] * ref["abs"] * (1 + BF16_HALF_STEP) + BF16_HALF_STEP * np.abs(ref["out"]) + 1e-37
    finite = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0)
    return out, ds + n + 2.0 ** -20 + 4 * FP32_HALF_STEP * finite
