"""The 4-bit cache format and the attention over it in 64 bits, code by code (numpy).

Its own words of include/dflash_mx4_cache.h, for the tests: blocks of 32 elements with a scale byte s
(power 2^(s - 127)), sizes GRID in the order of their codes.
"""
import numpy as np

D, BLOCK, TOKENS, CODE_BYTES, CHUNK_BYTES = 256, 32, 16, 2048, 2176
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def least_scale(top):
    """The scale byte of blocks whose largest size is top."""
    s = np.zeros(np.shape(top), dtype=np.int64)
    for i in range(254):  # 7 * 2^(i - 127) is below top: a larger one is needed
        s += np.asarray(top) > np.ldexp(7.0, i - 127)
    return s


def quantise(x):
    """(codes, scale bytes) of x [..., 256]: nearest size, ties to the even code."""
    x = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (D // BLOCK, BLOCK))
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    s = least_scale(np.abs(x).max(-1))
    y = np.abs(np.ldexp(x, (127 - s)[..., None]))
    best = np.zeros(y.shape, dtype=np.uint8)
    for c in range(1, 8):
        mid = (GRID[c - 1] + GRID[c]) / 2
        best = np.where((y > mid) | ((y == mid) & (c % 2 == 0)), c, best)
    codes = best.astype(np.uint8) | np.where(x < 0, 8, 0).astype(np.uint8)
    return (codes.reshape(codes.shape[:-2] + (D,)), np.where(bad, 255, s).astype(np.uint8))


def numbers(codes, scales):
    """Values [..., 256] of codes and scale bytes."""
    x = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    power = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return x * np.repeat(power, BLOCK, axis=-1)


def empty_pool(num_pages, page, Hkv):
    return np.zeros((num_pages, page // TOKENS, Hkv, CHUNK_BYTES), dtype=np.uint8)


def put(pool, slots, codes, scales, of_v):
    """Write rows [T, Hkv, .] at slots [T]."""
    flat = pool.reshape((-1,) + pool.shape[2:])
    for r, s in enumerate(slots):
        if s < 0:
            continue
        c, t = flat[s // TOKENS], s % TOKENS
        for d in range(D):
            at, high = (16 * (d % 128) + t, d >= 128) if of_v else (
                256 * (d // 32) + 16 * t + d % 32 // 2, d % 2 == 1)
            old = c[:, at]
            c[:, at] = (old & 0x0F) | (codes[r, :, d] << 4) if high else (
                (old & 0xF0) | codes[r, :, d])
        c[:, CODE_BYTES + 8 * t:CODE_BYTES + 8 * t + 8] = scales[r]


def get(pool, slots, of_v):
    """(codes [T, Hkv, 256], scales [T, Hkv, 8]) at slots [T]."""
    slots = np.asarray(slots, dtype=np.int64)
    c, t = pool.reshape((-1,) + pool.shape[2:])[slots // TOKENS], slots % TOKENS
    d = np.arange(D)
    at = 16 * (d % 128) + t[:, None] if of_v else 256 * (d // 32) + 16 * t[:, None] + d % 32 // 2
    byte = np.take_along_axis(c, at[:, None], axis=2)
    codes = np.where(d >= 128 if of_v else d % 2 == 1, byte >> 4, byte & 15).astype(np.uint8)
    sc = CODE_BYTES + 8 * t[:, None] + np.arange(8)
    return codes, np.take_along_axis(c, sc[:, None], axis=2)


def attention(q, k_pool, v_pool, table, lens, page):
    """(out, lse, spread, weight) in 64 bits. weight: sum of p |v| per output; spread: the largest
    sum |q_d k_d| / 16 of a row's visible keys."""
    B, q_len, Hq, _ = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    spread = np.zeros(q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pos = np.arange(n)
        slots = table[b, pos // page].astype(np.int64) * page + pos % page
        k, v = (numbers(*get(p, slots, of_v)) for p, of_v in ((k_pool, False), (v_pool, True)))
        for i in range(q_len):
            seen = n - q_len + i + 1
            if seen <= 0:
                continue
            for hq in range(Hq):
                h, x = hq // G, q[b, i, hq].astype(np.float64)
                s = k[:seen, h] @ x / 16.0
                m = s.max()
                p = np.exp(s - m)
                lse[b, i, hq] = m + np.log(p.sum())
                p /= p.sum()
                out[b, i, hq] = p @ v[:seen, h]
                weight[b, i, hq] = p @ np.abs(v[:seen, h])
                spread[b, i, hq] = (np.abs(k[:seen, h]) @ np.abs(x)).max() / 16.0
    return out, lse, spread, weight
