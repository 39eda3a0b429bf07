"""Definitions of the whole-cache operators in 64 bits (TEST INFRASTRUCTURE).

Plain numpy, one query row at a time: attention over every position a token
sees, the attention weight accumulated per position, and which positions an
eviction keeps.  Pools are decoded from their bit fields; nothing here is
shared with the library.
"""

from __future__ import annotations

import numpy as np

PAGE = 128
DIM = 128


def bf16(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3(codes):
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m / 512)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7 == 1, -v, v)


def e2m1(codes):
    return np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])[np.asarray(codes) & 15]


def rows(pb, r, which, g, n):
    """The first n rows of K (0) or V (1) of KV head g of request r, as values."""
    pages = pb.block_table[r, : -(-n // PAGE)]
    x = pb.kv_pool[pages, which, g]
    if pb.kv_dtype == "bf16":
        return bf16(x).reshape(-1, DIM)[:n]
    scale = float(np.float32(pb.v_scale if which else pb.k_scale))
    if pb.kv_dtype == "fp8":
        return e4m3(x).reshape(-1, DIM)[:n] * scale
    codes = x[:, :8192].reshape(-1, 64)
    v = np.stack([e2m1(codes), e2m1(codes >> 4)], -1).reshape(-1, DIM)
    return (v * np.repeat(e4m3(x[:, 8192:]).reshape(-1, 8), 16, axis=1))[:n] * scale


def _requests(pb):
    nq = pb.q_per_req
    for r in range(pb.num_requests):
        n = int(pb.seq_lens[r]) + nq - 1
        if pb.seq_lens[r] > 0:
            yield r, n


def _logits(pb, q, r, g, n, sel=None):
    """[nq, G, n] logits of KV head g, -inf where a row does not look."""
    nq, Hkv = pb.q_per_req, pb.num_kv_heads
    G = q.shape[1] // Hkv
    k = rows(pb, r, 0, g, n)
    qq = bf16(q[r * nq:(r + 1) * nq, g * G:(g + 1) * G])
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.einsum("jgd,pd->jgp", qq, k) * float(np.float32(pb.softmax_scale))
    size = float((np.abs(qq) @ np.abs(np.where(np.isfinite(k), k, 0)).T).max() * abs(pb.softmax_scale)) if n else 0.0
    p = np.arange(n)
    for j in range(nq):
        hide = p >= int(pb.seq_lens[r]) + j
        if sel is not None:
            hide |= ~np.isin(p // PAGE, sel[r * nq + j, g if sel.shape[1] > 1 else 0])
        s[j, :, hide] = -np.inf
    return s, size


def dense_decode(pb, q):
    """out [T, Hq, 128], lse [T, Hq] and, for tolerances, the largest sum of |q||k| scale and |v|."""
    T, Hq = q.shape[:2]
    nq, Hkv = pb.q_per_req, pb.num_kv_heads
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, DIM)), np.full((T, Hq), -np.inf)
    big_s = big_v = 0.0
    for r, n in _requests(pb):
        for g in range(Hkv):
            s, size = _logits(pb, q, r, g, n)
            v = rows(pb, r, 1, g, n)
            big_s, big_v = max(big_s, size), max(big_v, float(np.abs(v[np.isfinite(v)]).max(initial=0)))
            for j in range(nq):
                seen = int(pb.seq_lens[r]) + j
                x, t = s[j, :, :seen], slice(g * G, (g + 1) * G)
                m = x.max(-1, keepdims=True)
                p = np.exp(x - m)
                out[r * nq + j, t] = (p @ v[:seen]) / p.sum(-1, keepdims=True)
                lse[r * nq + j, t] = (m + np.log(p.sum(-1, keepdims=True)))[:, 0]
    return out, lse, big_s, big_v


def weights(pb, q, lse, before=None, decay=1.0, selected=None, after=None):
    """The accumulated weights [R, Hkv, max_blocks * 128]; elements behind the cache as in `after`."""
    nq, Hkv = pb.q_per_req, pb.num_kv_heads
    G = q.shape[1] // Hkv
    out = np.zeros((pb.num_requests, Hkv, pb.max_blocks * PAGE)) if after is None else after.astype(np.float64)
    for r, n in _requests(pb):
        for g in range(Hkv):
            s, _ = _logits(pb, q, r, g, n, selected)
            e = lse[r * nq:(r + 1) * nq, g * G:(g + 1) * G].astype(np.float64)[..., None]
            with np.errstate(invalid="ignore"):
                w = np.where(np.isneginf(e) | np.isneginf(s), 0.0, np.exp(s - e)).sum((0, 1))
            old = np.zeros(n) if before is None else before[r, g, :n].astype(np.float64) * decay
            old[int(pb.seq_lens[r]) - 1:] = 0.0
            out[r, g, :n] = old + w
    return out


def evict_lists(seq_lens, q_per_req, w, heads, keep, first, last):
    """kept [R, heads, keep] and the new lengths: heads = 1 ranks by the maximum over KV heads."""
    R = len(seq_lens)
    kept, lens = np.full((R, heads, keep), -1, np.int32), np.zeros(R, np.int32)
    per = w.shape[1] // heads
    for r in range(R):
        if seq_lens[r] == 0:
            continue
        n = int(seq_lens[r]) + q_per_req - 1
        lens[r] = min(n, keep) - q_per_req + 1
        for h in range(heads):
            x = w[r, h * per:(h + 1) * per, :n]
            nan = np.isnan(x).any(0)
            x = np.where(nan, 0, np.where(np.isnan(x), 0, x).max(0))
            p = np.arange(n)
            forced = (p < first) | (p >= n - last)
            order = np.lexsort((p, -x, ~nan, ~forced))[:keep]
            kept[r, h, :len(order)] = np.sort(order)
    return kept, lens


def evict(pb, kept, new_table, w, new_w, Hi=1):
    """Pools and weights after the rows of `kept` went to new_table's pages."""
    kv, idxk = pb.kv_pool.copy(), pb.idxk_pool.copy()
    scales = None if pb.idxk_scales is None else pb.idxk_scales.copy()
    new_w = new_w.copy()
    R, Hs, _ = kept.shape
    Hkv = pb.num_kv_heads
    for r in range(R):
        for h in range(Hs):
            at = kept[r, h][kept[r, h] >= 0]
            i = np.arange(len(at))
            a, b = pb.block_table[r, at // PAGE], at % PAGE
            c, d = new_table[r, i // PAGE], i % PAGE
            for g in range(h * Hkv // Hs, (h + 1) * Hkv // Hs):
                new_w[r, g, i] = w[r, g, at]
                for v in (0, 1):
                    if pb.kv_dtype == "nvfp4":
                        for lo, width in ((0, 64), (8192, 8)):
                            span = lambda row: lo + row[:, None] * width + np.arange(width)  # noqa: E731
                            kv[c[:, None], v, g, span(d)] = pb.kv_pool[a[:, None], v, g, span(b)]
                    else:
                        kv[c, v, g, d] = pb.kv_pool[a, v, g, b]
            for k in range(h * Hi // Hs, (h + 1) * Hi // Hs):
                idxk[c, k, d] = pb.idxk_pool[a, k, b]
                if scales is not None:
                    scales[c, k, d] = pb.idxk_scales[a, k, b]
    return kv, idxk, scales, new_w
