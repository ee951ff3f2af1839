"""fp64 CPU oracle of the calls around the DSA path: rotary positions, new tokens into
the two caches, the attention mass of cached tokens, and trimming the caches by it.

TEST INFRASTRUCTURE ONLY (see ``dsa_oracle``): plain loops and numpy, written from the
definitions in include/dsa.h. Cache arrays are numpy arrays in their paged or contiguous
shape; a row (b, slot) is addressed through ``cache_at``.
"""

from __future__ import annotations

import numpy as np

from .dsa_oracle import E4M3_MAX, QSCALE_FLOOR, e4m3_encode


def cache_at(b, slot, block_table=None, page_size=64):
    """Index of the cache row of slot `slot` of sequence b (leading two axes)."""
    if block_table is None:
        return b, slot
    return int(block_table[b][slot // page_size]), slot % page_size


def rope_rows(x, positions, freqs, magnitude=1.0, *, rot_begin=0, interleaved=False,
              backward=False):
    """x [rows, heads, dim] with dims [rot_begin, rot_begin + 2 len(freqs)) turned, fp64."""
    x = np.array(x, dtype=np.float64)
    half = len(freqs)
    for t in range(x.shape[0]):
        for i in range(half):
            a = float(positions[t]) * float(freqs[i])
            c, s = np.cos(a) * magnitude, np.sin(a) * magnitude * (-1.0 if backward else 1.0)
            d0 = rot_begin + (2 * i if interleaved else i)
            d1 = rot_begin + (2 * i + 1 if interleaved else i + half)
            u, v = x[t, :, d0].copy(), x[t, :, d1].copy()
            x[t, :, d0] = u * c - v * s
            x[t, :, d1] = u * s + v * c
    return x


def append_token(latent, key, position, freqs, magnitude=1.0, *, interleaved=True,
                 idx_interleaved=False):
    """(latent row [576] fp64, key [128] fp64, scale fp32) of one new token."""
    lat = rope_rows(np.asarray(latent)[None, None], [position], freqs, magnitude, rot_begin=512,
                    interleaved=interleaved)[0, 0]
    k = np.asarray(key, dtype=np.float64)
    if idx_interleaved is not None:
        k = rope_rows(k[None, None], [position], freqs, magnitude,
                      interleaved=idx_interleaved)[0, 0]
    scale = np.float32(max(np.max(np.abs(k)), QSCALE_FLOOR)) / np.float32(E4M3_MAX)
    return lat, k, scale


def key_codes(key32, scale):
    """E4M3 codes of an fp32 key for its fp32 scale."""
    return e4m3_encode(np.asarray(key32, np.float32) / np.float32(scale))


def attn_weight(q_t, rows, scale, lse_t):
    """(p [n], its per-head terms [heads, n]) of one query row over latent rows [n, 576]."""
    z = scale * (np.asarray(q_t, np.float64) @ np.asarray(rows, np.float64).T)
    a = np.exp(z - np.asarray(lse_t, np.float64)[:, None])
    return a.mean(axis=0), a


def evict_select(mass, n, keep, sink, recent):
    """Kept slots (ascending) of one sequence of n tokens."""
    if n <= keep:
        return list(range(n))
    order = []
    for s in range(sink, n - recent):
        m = float(mass[s])
        order.append((0, 0.0, s) if np.isnan(m) else (1, m + 0.0, s))
    order.sort(key=lambda o: (-o[0], -o[1], o[2]))
    middle = [o[2] for o in order[: keep - sink - recent]]
    return sorted(list(range(sink)) + middle + list(range(n - recent, n)))
