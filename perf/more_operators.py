"""Cases and plain forms of the operators that bring tokens into the cache and let any number of
them attend: norm and rotation of queries and keys (rope), keys and values appended to their
pages with norm and rotation on the way (append), and attention of ragged query rows over paged
states, causal or to all of them (attend).

Layouts are those of include/msa.h: a pool of 128-token pages reached through a block table,
query heads in groups of G per KV head.  The tokens of request r are rows offsets[r] ..
offsets[r + 1] - 1; token j of them stands at position seq_lens[r] - 1 + j and sees
seq_lens[r] + j positions (causal) or seq_lens[r] (all).
"""

import math

import numpy as np
import torch

own = False

PAGE = 128
DIM = 128
SCALE = DIM ** -0.5
EPS = 1e-6
ROW_BYTES = {"bf16": 256, "fp8": 128, "nvfp4": 72}  # one K or V row of one head
FP8_SCALE = 2.0 ** -6     # E4M3 values of N(0,1) data divided by this stay below 448
NVFP4_SCALE = 0.25        # tensor scale of the NVFP4 pools


def _rope(name, T, Hq, Hk, rot, interleaved=False, norm="shared", fused=True, far=131072):
    return dict(name=name, op="rope", T=T, Hq=Hq, Hk=Hk, rot=rot, interleaved=interleaved, norm=norm, fused=fused, far=far)


def _append(name, kv, R, nlo, nhi, Hkv, lo, hi, G=16, Hi=1, queries=True, rot=128, norm="shared", fused=True):
    return dict(name=name, op="append", kv=kv, R=R, nlo=nlo, nhi=nhi, Hkv=Hkv, G=G, Hi=Hi, lo=lo, hi=hi, queries=queries, rot=rot,
                interleaved=False, norm=norm, fused=fused)


def _attend(name, kv, R, nlo, nhi, Hkv, lo, hi, causal, G=16):
    return dict(name=name, op="attend", kv=kv, R=R, nlo=nlo, nhi=nhi, Hkv=Hkv, G=G, lo=lo, hi=hi, causal=causal)


def listed():
    return [
        # one token of one request: the latency of a lone user's step
        _rope("rope-step", 1, 64, 4, 128),
        # a prompt's projections: half of each head rotated, norm weights for each head
        _rope("rope-prompt", 8192, 64, 4, 64, norm="heads"),
        # an odd number of index queries and keys, pairs next to one another, far positions, no norm
        _rope("rope-index", 5001, 4, 1, 128, interleaved=True, norm="none", fused=False, far=1000000),
        # a decode step of 48 requests into an E4M3 cache: queries, keys, values, index queries and keys
        _append("append-step", "fp8", 48, 1, 1, 4, 2048, 65536, Hi=4),
        # ragged prompts, queries and index keys in the same pass
        _append("append-prompts", "bf16", 8, 700, 3500, 4, 0, 5000),
        # more requests than usual, keys and values alone, E4M3, half of each head rotated
        _append("append-values", "fp8", 19, 1, 2500, 8, 0, 20000, G=8, Hi=0, queries=False, rot=64),
        # a few tokens over a short text's states
        _attend("cross-tiny", "bf16", 1, 7, 7, 2, 200, 200, False, G=8),
        # one token each over an encoder's states
        _attend("cross-step", "bf16", 64, 1, 1, 8, 1500, 1500, False, G=4),
        # ragged texts over ragged states, E4M3
        _attend("cross-ragged", "fp8", 16, 1, 300, 8, 64, 2000, False, G=4),
        # ragged prompts without a cached beginning
        _attend("prompt-ragged", "bf16", 4, 1500, 4096, 4, 1, 1, True),
        # a chunk of a prompt over a long cached beginning, E4M3
        _attend("prompt-chunk", "fp8", 1, 512, 512, 4, 65536, 65536, True),
        # short chunks over a 4-bit cache, odd lengths
        _attend("chunk-nvfp4", "nvfp4", 5, 33, 100, 4, 5001, 20001, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    if op == "rope":
        Hq, Hk = rng.choice([1, 2, 4, 5, 8, 16, 32, 64]), rng.choice([0, 1, 2, 4, 8])
        c = _rope("", _log_int(rng, 1, 550000 // (Hq + Hk)), Hq, Hk, rng.choice([16, 32, 64, 96, 128, 128]), rng.random() < 0.5,
                  rng.choice(["none", "shared", "heads"]), rng.random() < 0.5, _log_int(rng, 100, 2000000))
    elif op == "append":
        R, Hkv, G = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8, 16])
        most = max(1, min(65536, 1000000 // (Hkv * (2 + G))) // R)
        nhi = _log_int(rng, 1, most)
        hi = _log_int(rng, 1, max(1, 1000000 // (R * Hkv)))
        c = _append("", rng.choice(["bf16", "fp8"]), R, rng.choice([0, nhi, _log_int(rng, 1, nhi)]), nhi, Hkv, rng.choice([0, _log_int(rng, 1, hi)]),
                    hi, G, rng.choice([0, 1, Hkv]), rng.random() < 0.5, rng.choice([32, 64, 128, 128]), rng.choice(["none", "shared", "heads"]),
                    rng.random() < 0.5)
    else:
        R, Hkv, G = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16, 16])
        hi = _log_int(rng, 1, min(65536, 4000000 // (R * Hkv)))
        causal = rng.random() < 0.5
        most = max(1, min(4096, 1800000000 // (R * Hkv * G * hi), 1500000 // (R * Hkv * G)))
        if causal:  # the tokens themselves are positions too
            most = max(1, min(most, int(math.sqrt(1800000000 / (R * Hkv * G)))))
            hi = max(1, min(hi, 1800000000 // (R * Hkv * G * most) - most))
        nhi = _log_int(rng, 1, most)
        c = _attend("", rng.choice(["bf16", "bf16", "fp8", "nvfp4"]), R, rng.choice([0, nhi, _log_int(rng, 1, nhi)]), nhi, Hkv,
                    rng.choice([1, hi, _log_int(rng, 1, hi)]), hi, causal, G)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# what a case's sizes are (no random values)

def _spread(lo, hi, R, step):
    """R numbers spread over lo .. hi, both ends among them where there are two."""
    f = [((r + 1) * step) % 1.0 for r in range(R)]
    f[-1] = 1.0
    if R > 1:
        f[R // 2] = 0.0
    return np.array([lo + round(x * (hi - lo)) for x in f], dtype=np.int64)


def _sizes(c):
    """New tokens of each request, and the positions that its first token sees."""
    n = _spread(c["nlo"], c["nhi"], c["R"], 0.6180339887498949)
    lens = _spread(c["lo"], c["hi"], c["R"], 0.7548776662466927)
    return n, lens + 1 if c["op"] == "append" else lens


def _seen(c):
    """Positions that exist after the call, for each request."""
    n, lens = _sizes(c)
    return lens if c["op"] == "attend" and not c["causal"] else lens + np.maximum(n - 1, 0)


def work(case):
    c = case
    if c["op"] == "rope":
        weights = {"none": 0, "shared": 2, "heads": c["Hq"] + c["Hk"]}[c["norm"]]
        return {"bytes": c["T"] * ((c["Hq"] + c["Hk"]) * 512 + 4) + 256 * weights, "flops": 8 * DIM * c["T"] * (c["Hq"] + c["Hk"])}
    n, lens = _sizes(c)
    T, Hq, row = int(n.sum()), c["Hkv"] * c["G"], ROW_BYTES[c["kv"]]
    if c["op"] == "append":
        rows = T * (2 * c["Hkv"] * (256 + row) + c["Hi"] * 512 + (512 * (Hq + c["Hi"]) if c["queries"] else 0))
        return {"bytes": rows + 8 * c["R"], "flops": 8 * rows // 4}
    pairs = sum(int(a) * int(s) + (int(a) * (int(a) - 1) // 2 if c["causal"] else 0) for a, s in zip(n, lens))
    read = int(_seen(c)[n > 0].sum()) * 2 * row * c["Hkv"]
    return {"bytes": read + T * Hq * (2 * 256 + 4), "flops": 4 * DIM * Hq * pairs}


# ---------------------------------------------------------------------------
# inputs

def _nvfp4_pool(g, pages, Hkv, dev):
    pool = torch.randint(0, 256, (pages, 2, Hkv, 9216), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.rand((pages, 2, Hkv, 1024), generator=g, device=dev) * 2 + 0.5
    pool[..., 8192:] = scales.to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def _normal(g, shape, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)


def _rows(g, T, heads, fused, dev):
    """bf16 [T, h, 128] for each h of `heads`: parts of one projection's output, or tensors of their own."""
    if fused:
        x = _normal(g, (T, sum(heads) + 1, DIM), dev)
        at = np.cumsum([0] + list(heads))
        return [x[:, a:a + h] for a, h in zip(at, heads)]
    return [_normal(g, (T, h, DIM), dev) for h in heads]


def _norm_weight(g, c, heads, dev):
    if c["norm"] == "none" or heads == 0:
        return None
    shape = (heads, DIM) if c["norm"] == "heads" else (DIM,)
    return (1 + torch.randn(shape, generator=g, device=dev) / 8).to(torch.bfloat16)


def _inv_freq(c):
    return 10000.0 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])


def _paged(s, g, dev):
    """Block table, lengths and offsets of a ragged batch, pages in random order."""
    c = s["c"]
    n, lens = _sizes(c)
    nb = -(-_seen(c) // PAGE)
    B, used = max(1, int(nb.max())), max(1, int(nb.sum()))
    perm = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["R"], B), -1, dtype=torch.int32, device=dev)
    has = torch.arange(B, device=dev)[None] < torch.from_numpy(nb).to(dev)[:, None]
    table[has] = perm[: int(nb.sum())]
    offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s |= {"table": table, "pages": used, "B": B, "T": int(offsets[-1]), "longest": int(n.max()), "offsets": torch.from_numpy(offsets).to(dev),
          "seq_lens": torch.from_numpy(lens.astype(np.int32)).to(dev)}


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "rope":
        s["q"], s["k"] = _rows(g, c["T"], [c["Hq"], c["Hk"]], c["fused"], dev)
        s["positions"] = torch.randint(0, c["far"], (c["T"],), generator=g, device=dev, dtype=torch.int32)
        s["q_weight"], s["k_weight"] = _norm_weight(g, c, c["Hq"], dev), _norm_weight(g, c, c["Hk"], dev)
        s["inv_freq"] = torch.from_numpy(_inv_freq(c)).to(dev)
        s["q_out"] = torch.empty((c["T"], c["Hq"], DIM), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((c["T"], c["Hk"], DIM), dtype=torch.bfloat16, device=dev)
        return s
    _paged(s, g, dev)
    Hkv, Hq, T, kv = c["Hkv"], c["Hkv"] * c["G"], s["T"], c["kv"]
    s["k_scale"] = s["v_scale"] = {"bf16": 1.0, "fp8": FP8_SCALE, "nvfp4": NVFP4_SCALE}[kv]
    if c["op"] == "append":
        Hi = c["Hi"]
        heads = [Hq if c["queries"] else 0, Hkv, Hkv, Hi if c["queries"] else 0, Hi]
        s["q"], s["k"], s["v"], s["q_idx"], s["idxk"] = _rows(g, T, heads, c["fused"], dev)
        for name, h in (("q", heads[0]), ("k", Hkv), ("q_idx", heads[3]), ("idxk", Hi)):
            s[name + "_weight"] = _norm_weight(g, c, h, dev)
        s["inv_freq"] = torch.from_numpy(_inv_freq(c)).to(dev)
        s["q_out"], s["q_idx_out"] = (torch.empty((T, h, DIM), dtype=torch.bfloat16, device=dev) for h in (heads[0], heads[3]))
        s["pool"] = torch.zeros((s["pages"], 2, Hkv, PAGE, DIM), dtype=torch.uint8 if kv == "fp8" else torch.bfloat16, device=dev)
        s["idx_pool"] = torch.zeros((s["pages"], Hi, PAGE, DIM), dtype=torch.bfloat16, device=dev)
        return s
    if kv == "nvfp4":
        s["pool"] = _nvfp4_pool(g, s["pages"], Hkv, dev)
    elif kv == "fp8":
        s["pool"] = torch.empty((s["pages"], 2, Hkv, PAGE, DIM), dtype=torch.uint8, device=dev)
        for i in range(0, s["pages"], 4096):  # the values before their rounding need not all be held at once
            x = _normal(g, s["pool"][i:i + 4096].shape, dev).float() / FP8_SCALE
            s["pool"][i:i + 4096] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["pool"] = _normal(g, (s["pages"], 2, Hkv, PAGE, DIM), dev)
    s["q"] = _normal(g, (T, Hq, DIM), dev)
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, Hq), device=dev)
    return s


# ---------------------------------------------------------------------------
# the plain forms: 32-bit torch operations

def _turned(s, x, weight, positions):
    """RMS norm and rotation of rows [T, heads, 128], in 32 bits; the angles in 64."""
    c = s["c"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = torch.remainder(positions.double()[:, None] * s["inv_freq"], 2 * math.pi).float()[:, None]
    cos, sin = angle.cos(), angle.sin()
    rot = x[..., : c["rot"]]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot.chunk(2, -1)
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, x[..., c["rot"]:]], -1)


def _plain_rope(s):
    out = {"q": _turned(s, s["q"], s["q_weight"], s["positions"]).to(torch.bfloat16)}
    if s["c"]["Hk"]:
        out["k"] = _turned(s, s["k"], s["k_weight"], s["positions"]).to(torch.bfloat16)
    return out


def _places(s):
    """Request and position of every new token."""
    t = torch.arange(s["T"], device="cuda")
    r = torch.searchsorted(s["offsets"], t.int(), right=True) - 1
    return r, s["seq_lens"][r] - 1 + (t - s["offsets"][r])


def _stored(kv, x, scale):
    if kv == "fp8":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(torch.bfloat16)


def _appended(s):
    pool = s["pool"].view(torch.float8_e4m3fn) if s["c"]["kv"] == "fp8" else s["pool"]
    out = {"pool": pool}
    if s["c"]["Hi"]:
        out["index_keys"] = s["idx_pool"]
    if s["c"]["queries"]:
        out["q"] = s["q_out"]
        if s["c"]["Hi"]:
            out["q_idx"] = s["q_idx_out"]
    return out


def _plain_append(s):
    c = s["c"]
    r, pos = _places(s)
    page, row = s["table"][r, pos // PAGE].long(), pos % PAGE
    s["pool"][page, 0, :, row] = _stored(c["kv"], _turned(s, s["k"], s["k_weight"], pos), s["k_scale"])
    s["pool"][page, 1, :, row] = _stored(c["kv"], s["v"].float(), s["v_scale"])
    if c["Hi"]:
        s["idx_pool"][page, :, row] = _turned(s, s["idxk"], s["idxk_weight"], pos).to(torch.bfloat16)
    if c["queries"]:
        s["q_out"].copy_(_turned(s, s["q"], s["q_weight"], pos))
        if c["Hi"]:
            s["q_idx_out"].copy_(_turned(s, s["q_idx"], s["q_idx_weight"], pos))
    return _appended(s)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _values(kv, x):
    """Rows of the pool, gathered as stored, in 32 bits (without the tensor scale)."""
    if kv == "bf16":
        return x.float()
    if kv == "fp8":
        return x.view(torch.float8_e4m3fn).float()
    codes = x[..., :8192].reshape(*x.shape[:-1], PAGE, 64)
    scales = x[..., 8192:].reshape(*x.shape[:-1], PAGE, 8).contiguous().view(torch.float8_e4m3fn).float()
    value = torch.tensor(_E2M1, device=x.device)
    both = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1)
    return (both.reshape(*scales.shape, 16) * scales[..., None]).reshape(*scales.shape[:-1], DIM)


def _states(s, which):
    """K (0) or V (1) of every position, [R, Hkv, B * 128, 128]."""
    x = s["pool"][:, which][s["table"].clamp(min=0)]
    x = _values(s["c"]["kv"], x).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, DIM)


def _plain_attend(s):
    c = s["c"]
    R, Hkv, G, N, C = c["R"], c["Hkv"], c["G"], max(1, s["longest"]), s["B"] * PAGE
    j = torch.arange(N, device="cuda")
    first, count = s["offsets"][:-1, None], (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    at = (first + torch.minimum(j, (count - 1).clamp(min=0))).clamp(max=max(0, s["T"] - 1))  # rows of the padded batch
    q = s["q"][at].float().reshape(R, N, Hkv, G, DIM).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, DIM)
    x = (q @ _states(s, 0).transpose(2, 3)).mul_(SCALE * s["k_scale"])
    seen = s["seq_lens"][:, None] + (j if c["causal"] else 0 * j)
    hidden = torch.arange(C, device="cuda") >= seen[..., None]
    x = x.reshape(R, Hkv, N, G, C).masked_fill_(hidden[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    v = _states(s, 1)
    v = v.masked_fill_((torch.arange(C, device="cuda") >= seen.amax(1, keepdim=True))[:, None, :, None], 0)
    out = (x.reshape(R, Hkv, N * G, C) @ v).reshape(R, Hkv, N, G, DIM) / total * s["v_scale"]
    lse = (m + total.log())[..., 0]
    real = j < count
    out = out.permute(0, 2, 1, 3, 4).reshape(R, N, Hkv * G, DIM)[real].to(torch.bfloat16)
    return out, lse.permute(0, 2, 1, 3).reshape(R, N, Hkv * G)[real]


# ---------------------------------------------------------------------------
# the framework's calls

def _plan(s):
    """What a serving loop keeps between steps: shapes, the rotation and the workspace."""
    if "plan" not in s:
        import sparse_attention_decode_msa_gb300 as msa

        c, kept = s["c"], {"msa": msa}
        if c["op"] != "attend":
            stride = lambda name: s[name].stride(0) if name in s else 0  # noqa: E731
            kept["rope"] = msa.make_rope(rotary_dim=c["rot"], interleaved=c["interleaved"], norm_eps=EPS, per_head_weights=c["norm"] == "heads",
                                         q_stride=stride("q"), k_stride=stride("k"), v_stride=stride("v"), q_idx_stride=stride("q_idx"),
                                         idxk_stride=stride("idxk"))
            kept["freqs"] = msa.rope_frequencies(s["inv_freq"])
        if c["op"] != "rope":
            kept["shape"] = shape = msa.make_shape(
                num_requests=c["R"], q_per_req=1, num_kv_heads=c["Hkv"], num_q_heads=c["G"] * c["Hkv"], num_pages=s["pages"],
                max_blocks_per_seq=s["B"], topk=1, kv_dtype=c["kv"], softmax_scale=SCALE, k_scale=s["k_scale"], v_scale=s["v_scale"],
                num_index_heads=max(1, c.get("Hi", 1)))
            kept["size"] = msa.msa_ragged_workspace_bytes(shape)
            kept["ws"] = torch.empty(kept["size"], dtype=torch.uint8, device="cuda")
            msa.msa_workspace_init(kept["ws"], kept["size"])
        s["plan"] = kept
    return s["plan"]


def _own(s):
    p, c = _plan(s), s["c"]
    if c["op"] == "rope":
        if c["Hk"]:
            p["msa"].msa_qk_norm_rope(p["rope"], p["freqs"], c["T"], s["positions"], c["Hq"], s["q"], s["q_weight"], s["q_out"],
                                      c["Hk"], s["k"], s["k_weight"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        p["msa"].msa_qk_norm_rope(p["rope"], p["freqs"], c["T"], s["positions"], c["Hq"], s["q"], s["q_weight"], s["q_out"])
        return {"q": s["q_out"]}
    if c["op"] == "append":
        index, queries = c["Hi"] > 0, c["queries"]
        q = (s["q"], s["q_weight"], s["q_out"]) if queries else (None, None, None)
        q_idx = (s["q_idx"], s["q_idx_weight"], s["q_idx_out"]) if queries and index else (None, None, None)
        idxk = (s["idxk"], s["idxk_weight"]) if index else (None, None)
        p["msa"].msa_kv_append(p["shape"], p["rope"], p["freqs"], s["T"], s["offsets"], s["k"], s["k_weight"], s["v"], *idxk, *q, *q_idx,
                               s["table"], s["seq_lens"], s["pool"], s["idx_pool"] if index else None, None, p["ws"], p["size"])
        return _appended(s)
    p["msa"].msa_ragged_attention(p["shape"], s["T"], c["causal"], s["q"], s["offsets"], s["pool"], s["table"], s["seq_lens"], s["out"],
                                  s["lse"], p["ws"], p["size"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(c, x, weight, positions):
    """Each pair as a complex number times e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / DIM + EPS).sqrt() * weight.double()
    out, rot = x.clone(), c["rot"]
    half = np.arange(rot // 2)
    one, two = (2 * half, 2 * half + 1) if c["interleaved"] else (half, half + rot // 2)
    angle = positions.double()[:, None] * torch.from_numpy(_inv_freq(c)).cuda()
    z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    out[..., one], out[..., two] = z.real, z.imag
    return out


def _power(e):
    """2^e in 64 bits, from the exponent's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_e4m3(x):
    """The nearest E4M3 values, ties to even, largest 448 (1.75 x 2^8, smallest step 2^-9)."""
    step = _power(torch.frexp(x)[1].clamp(min=-5) - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _decoded(kv, x):
    """Stored rows of one head, [blocks, ...] -> [blocks * 128, 128] in 64 bits, from the formats' bit fields."""
    if kv == "bf16":
        return x.double().reshape(-1, DIM)

    def e4m3(b):
        b = b.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(e > 0, (1 + m / 8) * _power(e - 7), m / 512)
        return torch.where(b >> 7 > 0, -v, v)

    if kv == "fp8":
        return e4m3(x).reshape(-1, DIM)
    b = x[:, :8192].reshape(-1, 64).long()
    code = torch.stack([b % 16, b // 16], -1).reshape(-1, DIM)
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * _power(e - 1), m / 2)
    v = torch.where(code >> 3 > 0, -v, v)
    return v * e4m3(x[:, 8192:]).reshape(-1, 8).repeat_interleave(16, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        out = {"q": _exact_rows(c, s["q"], s["q_weight"], s["positions"])}
        return out | ({"k": _exact_rows(c, s["k"], s["k_weight"], s["positions"])} if c["Hk"] else {})
    n, lens = _sizes(c)
    if c["op"] == "append":
        pool = torch.zeros((s["pages"], 2, c["Hkv"], PAGE, DIM), dtype=torch.float64, device="cuda")
        idx = torch.zeros((s["pages"], c["Hi"], PAGE, DIM), dtype=torch.float64, device="cuda")
        req = np.repeat(np.arange(c["R"]), n)
        pos = np.concatenate([np.arange(a) + b - 1 for a, b in zip(n, lens)])
        pos, req = torch.from_numpy(pos).cuda(), torch.from_numpy(req).cuda()
        page = s["table"].long()[req, pos // PAGE]
        k, v = _exact_rows(c, s["k"], s["k_weight"], pos), s["v"].double()
        if c["kv"] == "fp8":
            k, v = _to_e4m3(k / s["k_scale"]), _to_e4m3(v / s["v_scale"])
        for h in range(c["Hkv"]):
            pool[page, 0, h, pos % PAGE], pool[page, 1, h, pos % PAGE] = k[:, h], v[:, h]
        out = {"pool": pool}
        if c["Hi"]:
            idx[page, :, pos % PAGE] = _exact_rows(c, s["idxk"], s["idxk_weight"], pos)
            out["index_keys"] = idx
        if c["queries"]:
            out["q"] = _exact_rows(c, s["q"], s["q_weight"], pos)
            if c["Hi"]:
                out["q_idx"] = _exact_rows(c, s["q_idx"], s["q_idx_weight"], pos)
        return out
    Hkv, G = c["Hkv"], c["G"]
    out = torch.zeros((s["T"], Hkv * G, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["T"], Hkv * G), dtype=torch.float64, device="cuda")
    total = _seen(c)
    at = np.concatenate([[0], np.cumsum(n)])
    for r in range(c["R"]):
        L = int(total[r])
        pages = s["table"][r, : -(-L // PAGE)].long()
        for h in range(Hkv if n[r] else 0):
            heads = slice(h * G, (h + 1) * G)
            k = _decoded(c["kv"], s["pool"][pages, 0, h])[:L] * s["k_scale"]
            v = _decoded(c["kv"], s["pool"][pages, 1, h])[:L] * s["v_scale"]
            chunk = max(1, 400_000_000 // (G * L))
            for j0 in range(0, int(n[r]), chunk):
                j1 = min(int(n[r]), j0 + chunk)
                tokens = slice(int(at[r]) + j0, int(at[r]) + j1)
                x = torch.einsum("jgd,pd->jgp", s["q"][tokens, heads].double(), k) / math.sqrt(DIM)
                if c["causal"]:
                    for j in range(j0, j1) if L - int(lens[r]) < 64 else ():
                        x[j - j0, :, int(lens[r]) + j:] = -math.inf
                    if L - int(lens[r]) >= 64:
                        late = torch.arange(L, device="cuda")[None] >= int(lens[r]) + torch.arange(j0, j1, device="cuda")[:, None]
                        x.masked_fill_(late[:, None], -math.inf)
                top = torch.logsumexp(x, -1)
                lse[tokens, heads] = top
                out[tokens, heads] = torch.einsum("jgp,pd->jgd", torch.exp(x - top[..., None]), v)
    return out, lse
