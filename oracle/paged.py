"""CPU oracle of the paged MXFP4 KV cache and of attention over it (fp64, numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with the CUDA sources.
The cache is a uint8 array [n_pages, Hkv, 2 (K, V), P, 17 d / 32]; the P rows of one chunk are its
P * d/2 code bytes and then its P * d/32 scale bytes, interleaved as include/mxattn.h's entry points
write them: word w (4 bytes) of block b of a K row at byte w * d/8 + 4 b of the row, half-word h
(2 bytes) of block b of a V row at byte h * d/16 + 2 b; scale rows ordered within 16 tokens.
"""
from __future__ import annotations

import numpy as np

from . import mxfp4 as mx


def scale_row(i: int, which: int) -> int:
    """Row of token i (of 16) among their scale rows. K: tokens g, g + 8 are neighbours. V: tokens
    2c, 2c + 1, 2c + 8, 2c + 9 are."""
    if which == 0:
        return [0, 2, 4, 6, 8, 10, 12, 14, 1, 3, 5, 7, 9, 11, 13, 15][i]
    return [0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15][i]


def byte_of(x: int, d: int, which: int) -> int:
    """Place in a cache row of byte x of a row in the canonical layout."""
    b, y = divmod(x, 16)
    part = 4 if which == 0 else 2
    return (y // part) * (part * (d // 32)) + part * b + y % part


def _views(cache):
    n, H, _, P, row = cache.shape
    flat = cache.reshape(n, H, 2, P * row)
    nb = row // 17
    return flat[..., : P * nb * 16].reshape(n, H, 2, P, nb * 16), flat[..., P * nb * 16:].reshape(n, H, 2, P, nb)


def append(cache, k, v, slots, mode):
    """Write the MXFP4 rows of k, v [T, Hkv, d] (fp64) into the slots of `cache` (in place)."""
    n, H, _, P, row = cache.shape
    d = row // 17 * 32
    codes_of, scales_of = _views(cache)
    for which, x in ((0, k), (1, v)):
        codes, scales = mx.quantize_rows(x, mode)
        at = [byte_of(i, d, which) for i in range(d // 2)]
        for t, s in enumerate(np.asarray(slots)):
            if not 0 <= s < n * P:
                continue
            page, off = divmod(int(s), P)
            codes_of[page, :, which, off, at] = codes[t].T
            scales_of[page, :, which, off - off % 16 + scale_row(off % 16, which)] = scales[t]


def read(cache, slots):
    """k, v [T, Hkv, d] (fp64) held by the slots; zeros for slots outside the cache."""
    n, H, _, P, row = cache.shape
    d = row // 17 * 32
    codes_of, scales_of = _views(cache)
    out = []
    for which in (0, 1):
        at = [byte_of(i, d, which) for i in range(d // 2)]
        x = np.zeros((len(slots), H, d))
        for t, s in enumerate(np.asarray(slots)):
            if not 0 <= s < n * P:
                continue
            page, off = divmod(int(s), P)
            c = codes_of[page, :, which, off][:, at]
            val = np.empty((H, d))
            val[:, 0::2], val[:, 1::2] = mx.e2m1_decode(c & 15), mx.e2m1_decode(c >> 4)
            sc = scales_of[page, :, which, off - off % 16 + scale_row(off % 16, which)].astype(np.float64)
            x[t] = val * np.repeat(np.exp2(sc - 127), 32, axis=-1)
        out.append(x)
    return out[0], out[1]


def plan(ctx, new, table, free, P, max_tokens):
    """(table, q_start, kv_len, slots, info), one request after another."""
    table = np.array(table, dtype=np.int64)
    start, kv, taken, refused = [0], [], 0, 0
    slots = np.full(max_tokens, -1, dtype=np.int64)
    tokens, wanted = 0, 0      # wanted: pages asked for so far, those of refused requests included
    for r, (c, n0) in enumerate(zip(ctx, new)):
        n = max(n0, 0)
        ok = c >= 0 and n0 >= 0 and tokens + n <= max_tokens and -(-(c + n) // P) <= table.shape[1]
        if ok:
            held, full = -(-c // P), -(-(c + n) // P)
            end = wanted + full - held
            if full > held and end > len(free):
                ok = False
            else:
                table[r, held:full] = free[wanted:end]
                taken = max(taken, end) if full > held else taken
            wanted = end
        if ok:
            for i in range(n):
                page = table[r, (c + i) // P]
                slots[tokens + i] = page * P + (c + i) % P if page >= 0 else -1
        refused += not ok
        kv.append(c + n if ok else max(c, 0))
        tokens += n
        start.append(min(tokens, max_tokens))
    return table, np.array(start), np.array(kv), slots, np.array([start[-1], taken, refused, 0])


def _heads(q, cache, table, q_start, kv_len, causal, max_kv):
    """(rows, head, q rows, k, v, seen, p before the division, its sums, top) of each request's rows and head."""
    T, Hq, d = q.shape
    n_pages, H, _, P, _ = cache.shape
    for r in range(len(kv_len)):
        a, n = int(q_start[r]), int(q_start[r + 1] - q_start[r])
        if n <= 0:
            continue
        L = min(max(int(kv_len[r]), 0), table.shape[1] * P, 1 << 62 if max_kv is None else max_kv)
        pos = np.arange(L)
        page = np.asarray(table)[r, pos // P]
        there = (page >= 0) & (page < n_pages)
        k, v = read(cache, np.where(there, page * P + pos % P, -1))
        for h in range(Hq):
            kh, vh, qh = k[:, h // (Hq // H)], v[:, h // (Hq // H)], q[a:a + n, h]
            seen = np.broadcast_to(there, (n, L)).copy()
            if causal:
                seen &= pos[None] <= (int(kv_len[r]) - n + np.arange(n))[:, None]
            x = np.where(seen, qh @ kh.T / np.sqrt(d), -np.inf)
            top = x.max(axis=1, initial=-np.inf, keepdims=True)
            e = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
            yield slice(a, a + n), h, qh, kh, vh, seen, e, e.sum(axis=1, keepdims=True), top


def attention(q, cache, table, q_start, kv_len, causal, max_kv=None):
    """(out, lse, spread, mass) of the requests' rows: out [T, Hq, d] fp64 and lse [T, Hq], and for tolerances
    spread = sum_j p_j |v_j| and mass = max_j sum_c |q_c k_jc| / sqrt(d). NaN in rows of no request."""
    T, Hq, d = q.shape
    out = np.full((T, Hq, d), np.nan)
    lse = np.full((T, Hq), np.nan)
    spread, mass = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for rows, h, qh, kh, vh, seen, e, tot, top in _heads(q, cache, table, q_start, kv_len, causal, max_kv):
        p = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
        out[rows, h] = p @ vh
        spread[rows, h] = p @ np.abs(vh)
        with np.errstate(divide="ignore"):
            lse[rows, h] = (np.where(np.isfinite(top), top, 0.0) + np.log(tot))[:, 0]
        if len(kh):
            mass[rows, h] = np.where(seen, np.abs(qh) @ np.abs(kh).T, 0).max(axis=1) / np.sqrt(d)
    return out, lse, spread, mass


def attention_weights(q, cache, table, q_start, kv_len, causal, max_kv=None):
    """(square, share, apart, others) [T, Hq, d] for tolerances: square = sum_j p_j^2 v_j^2, share = max_j p_j times the
    sum of |v_j| over the keys that the row sees, apart = sum_j p_j |v_j - out|, others = square without the largest p_j."""
    square, share, apart, others = (np.zeros(q.shape) for _ in range(4))
    for rows, h, _, _, vh, seen, e, tot, _ in _heads(q, cache, table, q_start, kv_len, causal, max_kv):
        p = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
        square[rows, h] = p ** 2 @ vh ** 2
        share[rows, h] = p.max(axis=1, initial=0.0, keepdims=True) * (seen.astype(float) @ np.abs(vh))
        for i, row in zip(range(rows.start, rows.stop), p):
            apart[i, h] = row @ np.abs(vh - row @ vh)
            if len(row):
                most = np.argmax(row)
                others[i, h] = np.delete(row, most) ** 2 @ np.delete(vh, most, axis=0) ** 2
    return square, share, apart, others
