"""Definitions of the calls on ragged batches in 64 bits (TEST INFRASTRUCTURE): norm and
rotation of head rows, where a batch's tokens stand, their encodings, and attention of
ragged query rows.  Nothing here is shared with the library."""

from __future__ import annotations

import numpy as np

from .whole_cache import DIM, PAGE, bf16, e4m3, e2m1, rows

E4M3_VALUES = np.array([e4m3(c) for c in range(127)])  # ascending
E2M1_VALUES = np.array([e2m1(c) for c in range(8)])


def turned(x, weight, positions, radians, rotary_dim, interleaved=False, scale=1.0, eps=1e-6, offset=0.0):
    """Rows x (bf16 bits [T, H, 128]) after norm and rotation, and the size of what each element was
    added up from (for tolerances)."""
    x = bf16(x)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (bf16(weight) + offset)
    out, size = x.copy(), np.abs(x)
    if rotary_dim:
        half = np.arange(rotary_dim // 2)
        a, b = (2 * half, 2 * half + 1) if interleaved else (half, half + rotary_dim // 2)
        t = np.asarray(positions, np.float64)[:, None] * np.asarray(radians, np.float64)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * t)[:, None] * scale
        out[..., a], out[..., b] = z.real, z.imag
        size[..., a] = size[..., b] = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, size


def places(offsets, seq_lens, num_tokens):
    """Request and position of every token, -1 for rows behind the last request's."""
    req, pos = np.full(num_tokens, -1), np.full(num_tokens, -1)
    for r in range(len(seq_lens)):
        t = np.arange(offsets[r], offsets[r + 1])
        req[t], pos[t] = r, int(seq_lens[r]) - 1 + t - offsets[r]
    return req, pos


def to_codes(x, values):
    """The nearest of `values` (ascending from 0, even codes win ties), with the sign in the bit above; +0 for zeros."""
    a = np.minimum(np.abs(x), values[-1])
    up = np.clip(np.searchsorted(values, a), 1, len(values) - 1)
    lo, hi = values[up - 1], values[up]
    near = np.where((a - lo < hi - a) | ((a - lo == hi - a) & (up % 2 == 1)), up - 1, up)
    near = np.where(a == 0, 0, near)
    return np.where((x < 0) & (near > 0), near + (128 if len(values) > 8 else 8), near).astype(np.uint8)


def attention(pb, q, offsets, seq_lens, causal, distances=True):
    """out, lse of ragged query rows (bf16 bits [T, Hq, 128]) over pb's pages, NaN in rows of no request; for tolerances
    the values' weighted mean distance from each output, and the largest sums of |q||k| scale and |v|."""
    T, Hq = q.shape[:2]
    G = Hq // pb.num_kv_heads
    out, lse, far = np.full((T, Hq, DIM), np.nan), np.full((T, Hq), np.nan), np.zeros((T, Hq, DIM))
    big_s = big_v = 0.0
    for r in range(len(seq_lens)):
        n, L = int(offsets[r + 1] - offsets[r]), int(seq_lens[r])
        if n == 0:
            continue
        at = slice(int(offsets[r]), int(offsets[r + 1]))
        if L == 0:
            out[at], lse[at] = 0, -np.inf
            continue
        total = L + (n - 1 if causal else 0)
        for g in range(pb.num_kv_heads):
            heads = slice(g * G, (g + 1) * G)
            k, v = rows(pb, r, 0, g, total), rows(pb, r, 1, g, total)
            qq = bf16(q[at, heads])
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.einsum("jgd,pd->jgp", qq, k) * float(np.float32(pb.softmax_scale))
            size = (np.abs(qq) @ np.abs(np.where(np.isfinite(k), k, 0)).T).max() * abs(pb.softmax_scale)
            big_s, big_v = max(big_s, float(size)), max(big_v, float(np.abs(v[np.isfinite(v)]).max(initial=0)))
            for j in range(n):
                seen = L + (j if causal else 0)
                x = s[j, :, :seen]
                m = x.max(-1, keepdims=True)
                p = np.exp(x - m)
                p /= (total_p := p.sum(-1, keepdims=True))
                with np.errstate(invalid="ignore"):
                    o = out[at, heads][j] = p @ v[:seen]
                    far[at, heads][j] = np.sum(p[:, :, None] * np.abs(v[:seen] - o[:, None]), 1) if distances else 0
                lse[at, heads][j] = (m + np.log(total_p))[:, 0]
    return out, lse, far, big_s, big_v
