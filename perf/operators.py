"""Cases and plain forms of the whole-cache operators: attention over every cached
position (decode), the attention weight accumulated per position (weights), and
the eviction of positions by that weight (evict).

Layouts are those of include/msa.h: a pool of 128-token pages reached through a
block table, query heads in groups of G per KV head, token t = r * nq + j of
request r seeing positions 0 .. seq_lens[r] + j - 1.
"""

import math
import statistics

import numpy as np
import torch

own = False

PAGE = 128
DIM = 128
SCALE = DIM ** -0.5
ROW_BYTES = {"bf16": 256, "fp8": 128, "nvfp4": 72}  # one K or V row of one head
FP8_SCALE = 2.0 ** -6     # E4M3 values of N(0,1) data divided by this stay below 448
NVFP4_SCALE = 0.25        # tensor scale of the NVFP4 pools


def _case(name, op, kv, R, nq, Hkv, lo, hi, G=16, spread="even", **more):
    return dict(name=name, op=op, kv=kv, R=R, nq=nq, Hkv=Hkv, G=G, lo=lo, hi=hi, spread=spread, **more)


def listed():
    return [
        # one request, one KV head, a 4096-token cache: the latency of a lone user's step
        _case("decode-tiny", "decode", "bf16", 1, 1, 1, 4096, 4096),
        # speculative verification of 4 tokens a request over ragged contexts
        _case("decode-spec-verify", "decode", "bf16", 8, 4, 4, 8192, 32768),
        # a chunk of 48 tokens (tree verification, a prompt's last chunk) over two long contexts
        _case("decode-long-verify", "decode", "bf16", 2, 48, 4, 131072, 131072),
        # many requests, one token each, lognormal contexts, E4M3 cache
        _case("decode-high-concurrency", "decode", "fp8", 48, 1, 4, 2048, 65536, spread="lognormal"),
        # 4-bit cache, two tokens a request
        _case("decode-nvfp4", "decode", "nvfp4", 32, 2, 4, 65536, 65536),
        # 8 query heads a KV head (a tensor-parallel half), one token, odd contexts
        _case("decode-8-heads", "decode", "bf16", 16, 1, 2, 1, 20001, G=8),
        # every step's weights after a dense step, E4M3 cache
        _case("weights-decode", "weights", "fp8", 48, 1, 4, 2048, 65536, spread="lognormal", decay=1.0, topk=0, Hi=1),
        # after a block-sparse step: 16 selected blocks a token and KV head, fading weights
        _case("weights-sparse", "weights", "bf16", 8, 4, 4, 8192, 32768, decay=0.96875, topk=16, Hi=4),
        # a prompt's last 32 tokens weigh the prompt before it is cut
        _case("weights-window", "weights", "bf16", 2, 32, 4, 32768, 32768, decay=1.0, topk=0, Hi=1),
        # one request cut from 4096 to 1024 positions
        _case("evict-tiny", "evict", "bf16", 1, 1, 1, 4096, 4096, keep=1024, first=4, last=128, Hi=1),
        # prompts cut to 4096 positions, one list a request, index keys moved too
        _case("evict-prompts", "evict", "bf16", 8, 1, 4, 8192, 32768, keep=4096, first=4, last=256, Hi=1),
        # long E4M3 contexts cut to an eighth, one list a KV head
        _case("evict-long", "evict", "fp8", 8, 1, 4, 65536, 131072, keep=16384, first=16, last=1000, Hi=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "weights", "evict"])
    kv = rng.choice(["bf16", "fp8"] if op == "evict" else ["bf16", "fp8", "nvfp4"])
    R, Hkv = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8])
    nq = 1 if op == "evict" else rng.choice([1, 1, 2, 3, 4, 5, 8, rng.randint(9, 64)])
    G = rng.choice([1, 2, 4, 5, 8, 16, 16, 16])
    most = min(131072, 2_000_000 // (R * Hkv), 150_000_000 // (R * Hkv * G * nq))
    hi = _log_int(rng, nq, max(nq, most))
    lo = _log_int(rng, nq, hi)
    c = _case("", op, kv, R, nq, Hkv, lo, hi, G=G)
    del c["name"]
    if op == "weights":
        Hi = rng.choice([1, Hkv])
        c |= {"decay": rng.choice([1.0, 0.96875]), "topk": rng.choice([0, 0, rng.randint(1, 32)]), "Hi": Hi}
    if op == "evict":
        keep = _log_int(rng, 1, hi)
        first = rng.randint(0, min(16, keep))
        c |= {"keep": keep, "first": first, "last": rng.randint(0, min(256, keep - first)), "Hi": rng.choice([1, Hkv])}
    return c


# ---------------------------------------------------------------------------
# what a case's sizes are (no random values)

def _contexts(c):
    """Cached tokens of each request, spread over the case's range."""
    R, lo, hi = c["R"], c["lo"], c["hi"]
    f = [((r + 1) * 0.6180339887498949) % 1.0 for r in range(R)]
    if c["spread"] == "lognormal":  # median 16384, sigma 1, clipped to the range
        nd = statistics.NormalDist(math.log(16384), 1.0)
        return np.array([min(hi, max(lo, round(math.exp(nd.inv_cdf(min(0.999, max(0.001, x))))))) for x in f])
    return np.array([lo + round(x * (hi - lo)) for x in f])


def _selected(c):
    """Block tables of a sparse step: the first and the last visible block and others in between, ascending, -1 padded."""
    rng, n, nq, k = np.random.RandomState(7), _contexts(c), c["nq"], c["topk"]
    Hs = 1 if c["Hi"] == 1 else c["Hkv"]
    sel = np.full((c["R"] * nq, Hs, k), -1, dtype=np.int32)
    for r in range(c["R"]):
        for h in range(Hs):
            near = rng.permutation(-(-int(n[r]) // PAGE))  # the tokens of a step look at much the same blocks
            for j in range(nq):
                nb = -(-(int(n[r]) - nq + 1 + j) // PAGE)
                few = near[near < nb][: max(1, k + k // 4)]
                few = few[rng.permutation(len(few))][:k]
                few[0] = 0
                few = np.unique(np.concatenate([few[: k - 1], [nb - 1]]) if k > 1 else np.array([nb - 1]))
                sel[r * nq + j, h, : len(few)] = few
    return sel


def work(case):
    c, n = case, _contexts(case)
    R, nq, Hkv, G = c["R"], c["nq"], c["Hkv"], c["G"]
    row, T, pos = ROW_BYTES[c["kv"]], c["R"] * c["nq"], int(n.sum())
    seen = sum(int(x) - nq + 1 + j for x in n for j in range(nq))  # (token, visible position) pairs
    table = 4 * sum(-(-int(x) // PAGE) for x in n) + 4 * R
    qb = T * Hkv * G * DIM * 2
    if c["op"] == "decode":
        return {"bytes": 2 * row * Hkv * pos + 2 * qb + 4 * T * Hkv * G + table, "flops": 4 * DIM * Hkv * G * seen}
    if c["op"] == "weights":
        read, flops = row * Hkv * pos, 2 * DIM * Hkv * G * seen
        if c["topk"]:
            sel = _selected(c)
            Hs = sel.shape[1]
            size = lambda r, j, b: min(PAGE, int(n[r]) - nq + 1 + j - b * PAGE)  # noqa: E731
            read, flops = 0, 0
            for r in range(R):
                for h in range(Hs):
                    rows = {}
                    for j in range(nq):
                        for b in sel[r * nq + j, h]:
                            if b >= 0:
                                rows[b] = max(rows.get(b, 0), size(r, j, b))
                                flops += 2 * DIM * G * size(r, j, b) * (Hkv // Hs)
                    read += row * (Hkv // Hs) * sum(rows.values())
            read += 4 * sel.size
        return {"bytes": int(read + 8 * Hkv * pos + qb + 4 * T * Hkv * G + table), "flops": int(flops)}
    kept = int(np.minimum(n, c["keep"]).sum())
    Hs = 1 if c["Hi"] == 1 else Hkv
    return {"bytes": 4 * Hkv * pos + kept * (2 * (2 * Hkv * row + 256 * c["Hi"]) + 8 * Hkv + 4 * Hs) + table, "flops": 0}


# ---------------------------------------------------------------------------
# inputs

def _nvfp4_pool(g, pages, Hkv, dev):
    pool = torch.randint(0, 256, (pages, 2, Hkv, 9216), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.rand((pages, 2, Hkv, 1024), generator=g, device=dev) * 2 + 0.5
    pool[..., 8192:] = scales.to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def _normal(g, shape, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    R, nq, Hkv, G, kv = c["R"], c["nq"], c["Hkv"], c["G"], c["kv"]
    n = _contexts(c)
    nb = -(-n // PAGE)
    B, used = int(nb.max()), int(nb.sum())
    new_blocks = -(-c["keep"] // PAGE) if c["op"] == "evict" else 0
    pages = used + R * new_blocks
    perm = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    table = torch.full((R, B), -1, dtype=torch.int32, device=dev)
    has = torch.arange(B, device=dev)[None] < torch.from_numpy(nb).to(dev)[:, None]
    table[has] = perm
    s = {"c": c, "table": table, "seq_lens": torch.from_numpy((n - nq + 1).astype(np.int32)).to(dev), "pages": pages, "used": used, "B": B}
    if kv == "nvfp4":
        s["pool"], s["k_scale"], s["v_scale"] = _nvfp4_pool(g, pages, Hkv, dev), NVFP4_SCALE, NVFP4_SCALE
    elif kv == "fp8":
        s["pool"] = torch.empty((pages, 2, Hkv, PAGE, DIM), dtype=torch.uint8, device=dev)
        for i in range(0, pages, 4096):  # the values before their rounding need not all be held at once
            x = _normal(g, s["pool"][i:i + 4096].shape, dev).float() / FP8_SCALE
            s["pool"][i:i + 4096] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_scale"], s["v_scale"] = FP8_SCALE, FP8_SCALE
    else:
        s["pool"], s["k_scale"], s["v_scale"] = _normal(g, (pages, 2, Hkv, PAGE, DIM), dev), 1.0, 1.0
    T, Hq = R * nq, Hkv * G
    if c["op"] == "evict":
        new = torch.randperm(R * new_blocks, generator=g, device=dev) + used
        s["new_table"] = new.to(torch.int32).reshape(R, new_blocks)
        s["idxk"] = _normal(g, (pages, c["Hi"], PAGE, DIM), dev)
        s["pool"][used:] = 0
        s["idxk"][used:] = 0
        # heavy-tailed weights, many positions that nothing attended to
        w = torch.exp(2 * torch.randn((R, Hkv, B * PAGE), generator=g, device=dev)) / 1024
        s["weights"] = w * (torch.rand(w.shape, generator=g, device=dev) < 0.75)
        s["new_weights"] = torch.zeros((R, Hkv, new_blocks * PAGE), device=dev)
        s["kept"] = torch.full((R, 1 if c["Hi"] == 1 else Hkv, c["keep"]), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(R, dtype=torch.int32, device=dev)
        return s
    s["q"] = _normal(g, (T, Hq, DIM), dev)
    if c["op"] == "decode":
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, Hq), device=dev)
        return s
    s["selected"] = torch.from_numpy(_selected(c)).to(dev) if c["topk"] else None
    p = _logits(s)
    s["lse"] = torch.logsumexp(p, -1).reshape(R, Hkv, nq, G).permute(0, 2, 1, 3).reshape(T, Hq).contiguous()
    del p
    s["weights_in"] = torch.rand((R, Hkv, B * PAGE), generator=g, device=dev)
    s["weights"] = torch.zeros_like(s["weights_in"])
    return s


# ---------------------------------------------------------------------------
# the plain forms: 32-bit torch operations on the padded batch

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


def _rows(s, which):
    """K (0) or V (1) of every cached position, [R, Hkv, B * 128, 128]."""
    x = s["pool"][:, which][s["table"].clamp(min=0)]
    x = _values(s["c"]["kv"], x).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, DIM)


def _visible(s):
    """[R, 1, nq * G, B * 128]: whether a row sees a position."""
    c = s["c"]
    seen = s["seq_lens"][:, None] + torch.arange(c["nq"], device="cuda")
    ok = torch.arange(s["B"] * PAGE, device="cuda") < seen[..., None]
    return ok.repeat_interleave(c["G"], 1)[:, None]


def _chosen(s):
    """[R, Hs, nq * G, B * 128]: whether a position lies in a block that a row's token selected."""
    c, sel = s["c"], s["selected"]
    T, Hs, _ = sel.shape
    hit = torch.zeros((T, Hs, s["B"] + 1), dtype=torch.bool, device="cuda")
    hit.scatter_(2, torch.where(sel < 0, s["B"], sel).long(), True)
    hit = hit[..., : s["B"]].reshape(c["R"], c["nq"], Hs, s["B"]).transpose(1, 2)
    return hit.repeat_interleave(c["G"], 2).repeat_interleave(PAGE, 3)


def _queries(s):
    c = s["c"]
    q = s["q"].float().reshape(c["R"], c["nq"], c["Hkv"], c["G"], DIM).transpose(1, 2)
    return q.reshape(c["R"], c["Hkv"], c["nq"] * c["G"], DIM)


def _logits(s):
    x = (_queries(s) @ _rows(s, 0).transpose(2, 3)) * (SCALE * s["k_scale"])
    ok = _visible(s)
    if s.get("selected") is not None:
        ok = ok & _chosen(s)
    return x.masked_fill_(~ok, -math.inf)


def _by_token(s, x):
    """[R, Hkv, nq * G, ...] -> [T, Hq, ...]."""
    c = s["c"]
    x = x.reshape(c["R"], c["Hkv"], c["nq"], c["G"], *x.shape[3:]).transpose(1, 2)
    return x.reshape(c["R"] * c["nq"], c["Hkv"] * c["G"], *x.shape[4:])


def _plain_decode(s):
    x = _logits(s)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ _rows(s, 1)) / total * s["v_scale"]
    lse = (m + total.log())[..., 0]
    return _by_token(s, out).to(torch.bfloat16), _by_token(s, lse)


def _plain_weights(s):
    c = s["c"]
    lse = s["lse"].reshape(c["R"], c["nq"], c["Hkv"], c["G"]).transpose(1, 2).reshape(c["R"], c["Hkv"], -1, 1)
    w = _logits(s).sub_(lse).exp_().sum(2)
    at = torch.arange(s["B"] * PAGE, device="cuda")
    first_new = s["seq_lens"][:, None, None] - 1
    before = torch.where(at < first_new, s["weights_in"] * c["decay"], torch.zeros((), device="cuda"))
    return torch.where(at < first_new + c["nq"], before + w, s["weights"])


def _plain_evict(s):
    c = s["c"]
    R, Hkv, keep = c["R"], c["Hkv"], c["keep"]
    n = s["seq_lens"][:, None, None].long()
    w = s["weights"]
    C = w.shape[2]
    at = torch.arange(C, device="cuda")
    score = w.amax(1, keepdim=True) if c["Hi"] == 1 else w
    Hs = score.shape[1]
    score = score.masked_fill((at < c["first"]) | (at >= n - c["last"]), math.inf)
    score = score.masked_fill(at >= n, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    if order.shape[-1] < keep:  # a budget larger than the cache
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=C)
    kept = torch.where(torch.arange(keep, device="cuda") < n, order, C).sort(-1).values
    real = kept < C
    new_lens = n[:, 0, 0].clamp(max=keep).to(torch.int32)
    src = kept.clamp(max=C - 1)
    i = torch.arange(keep, device="cuda")
    r = torch.arange(R, device="cuda")[:, None, None]
    from_page = s["table"].long()[r, src // PAGE]
    to_page = s["new_table"].long()[r, (i // PAGE).expand(R, Hs, keep)]

    def move(pool):  # [pages, heads, 128, ...], heads in the order of the kept lists
        per = pool.shape[1] // Hs
        pick = lambda x: x[:, :, None].expand(R, Hs, per, keep)  # noqa: E731
        h = torch.arange(pool.shape[1], device="cuda").reshape(1, Hs, per, 1).expand(R, Hs, per, keep)
        ok = pick(real)
        rows = pool[pick(from_page)[ok], h[ok], pick(src % PAGE)[ok]]
        pool[pick(to_page)[ok], h[ok], pick((i % PAGE).expand(R, Hs, keep))[ok]] = rows

    move(s["pool"][:, 0])
    move(s["pool"][:, 1])
    move(s["idxk"])
    each = src.expand(R, Hkv, keep)
    s["new_weights"][..., :keep] = torch.where(real, w.gather(2, each), s["new_weights"][..., :keep])
    return _evicted(s, torch.where(real, kept, -1).to(torch.int32), new_lens)


def _evicted(s, kept, new_lens):
    pages = s["pool"][s["used"]:]
    return {"kept": kept, "new_lens": new_lens, "weights": s["new_weights"], "index_keys": s["idxk"][s["used"]:],
            "pages": pages.view(torch.float8_e4m3fn) if s["c"]["kv"] == "fp8" else pages}


# ---------------------------------------------------------------------------
# the framework's calls

def _plan(s):
    """The shape and the workspace that a serving loop keeps between steps."""
    if "plan" not in s:
        import sparse_attention_decode_msa_gb300 as msa

        c = s["c"]
        shape = msa.make_shape(
            num_requests=c["R"], q_per_req=c["nq"], num_kv_heads=c["Hkv"], num_q_heads=c["G"] * c["Hkv"], num_pages=s["pages"],
            max_blocks_per_seq=s["B"], topk=c.get("topk") or 1, kv_dtype=c["kv"], softmax_scale=SCALE, k_scale=s["k_scale"],
            v_scale=s["v_scale"], num_index_heads=c.get("Hi", 1))
        size = msa.msa_cache_workspace_bytes(shape)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        msa.msa_workspace_init(ws, size)
        s["plan"] = msa, shape, ws, size
    return s["plan"]


def run(state):
    s, op = state, state["c"]["op"]
    if own:
        msa, shape, ws, size = _plan(s)
        c = s["c"]
        if op == "decode":
            msa.msa_dense_decode(shape, s["q"], s["pool"], s["table"], s["seq_lens"], s["out"], s["lse"], ws, size)
            return s["out"], s["lse"]
        if op == "weights":
            msa.msa_weight_accumulate(shape, s["q"], s["pool"], s["table"], s["seq_lens"], s["selected"], s["lse"], c["decay"],
                                      s["weights_in"], s["weights"], ws, size)
            return s["weights"]
        msa.msa_cache_evict(shape, c["keep"], c["first"], c["last"], s["weights"], s["table"], s["seq_lens"], s["new_table"], s["pool"],
                            s["idxk"], None, s["new_weights"], s["kept"], s["new_lens"], ws, size)
        return _evicted(s, s["kept"], s["new_lens"])
    if op == "decode":
        return _plain_decode(s)
    if op == "weights":
        return _plain_weights(s)
    return _plain_evict(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one request and KV head at a time

def _decoded(kv, x):
    """Stored rows of one head, [blocks, ...] -> [blocks * 128, 128] in 64 bits, from the formats' bit fields."""
    if kv == "bf16":
        return x.double().reshape(-1, DIM)

    def e4m3(b):
        b = b.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 512)
        return torch.where(b >> 7 > 0, -v, v)

    if kv == "fp8":
        return e4m3(x).reshape(-1, DIM)
    b = x[:, :8192].reshape(-1, 64).long()
    code = torch.stack([b % 16, b // 16], -1).reshape(-1, DIM)
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
    v = torch.where(code >> 3 > 0, -v, v)
    return v * e4m3(x[:, 8192:]).reshape(-1, 8).repeat_interleave(16, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    R, nq, Hkv, G = c["R"], c["nq"], c["Hkv"], c["G"]
    n = _contexts(c)
    if c["op"] == "evict":
        return _exact_evict(c, s, n)
    T, Hq, C = R * nq, Hkv * G, s["B"] * PAGE
    out = torch.zeros((T, Hq, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    w = torch.zeros((R, Hkv, C), dtype=torch.float64, device="cuda")
    for r in range(R):
        N, first_new = int(n[r]), int(n[r]) - nq
        pages = s["table"][r, : -(-N // PAGE)].long()
        for h in range(Hkv):
            tokens, heads = slice(r * nq, (r + 1) * nq), slice(h * G, (h + 1) * G)
            k = _decoded(c["kv"], s["pool"][pages, 0, h])[:N] * s["k_scale"]
            x = torch.einsum("jgd,pd->jgp", s["q"][tokens, heads].double(), k) / math.sqrt(DIM)
            for j in range(nq):
                x[j, :, first_new + 1 + j:] = -math.inf
                if s.get("selected") is not None:
                    blocks = s["selected"][r * nq + j, h if s["selected"].shape[1] > 1 else 0].tolist()
                    not_in = [b for b in range(-(-N // PAGE)) if b not in blocks]
                    x[j].index_fill_(1, torch.tensor([p for b in not_in for p in range(b * PAGE, min(N, b * PAGE + PAGE))],
                                                     dtype=torch.long, device="cuda"), -math.inf)
            if c["op"] == "weights":
                w[r, h, :N] = torch.exp(x - s["lse"][tokens, heads].double()[..., None]).sum((0, 1))
                w[r, h, :first_new] += s["weights_in"][r, h, :first_new].double() * c["decay"]
                continue
            v = _decoded(c["kv"], s["pool"][pages, 1, h])[:N] * s["v_scale"]
            top = torch.logsumexp(x, -1)
            lse[tokens, heads] = top
            out[tokens, heads] = torch.einsum("jgp,pd->jgd", torch.exp(x - top[..., None]), v)
    return w if c["op"] == "weights" else (out, lse)


def _exact_evict(c, s, n):
    R, Hkv, keep = c["R"], c["Hkv"], c["keep"]
    kept, w = s["kept"].clone(), s["weights"].cpu().numpy().astype(np.float64)
    new_w = s["new_weights"].double()
    Hs = kept.shape[1]
    for r in range(R):
        N = int(n[r])
        for h in range(Hs):
            score = w[r].max(0)[:N] if Hs == 1 else w[r, h, :N].copy()
            p = np.arange(N)
            forced = (p < c["first"]) | (p >= N - c["last"])
            best = np.lexsort((p, -score, ~forced))[:keep]  # forced ones first, then by weight, then by position
            best = torch.from_numpy(np.sort(best)).cuda()
            k = len(best)
            kept[r, h, :k] = best.to(torch.int32)
            old = s["table"][r].long()[best // PAGE], best % PAGE
            new = s["new_table"][r].long()[torch.arange(k, device="cuda") // PAGE], torch.arange(k, device="cuda") % PAGE
            for g in range(Hkv) if Hs == 1 else (h,):
                for which in (0, 1):
                    s["pool"][new[0], which, g, new[1]] = s["pool"][old[0], which, g, old[1]]
                new_w[r, g, :k] = s["weights"][r, g, best].double()
            per = c["Hi"] // Hs
            for i in range(h * per, (h + 1) * per):
                s["idxk"][new[0], i, new[1]] = s["idxk"][old[0], i, old[1]]
    got = _evicted(s, kept, torch.from_numpy(np.minimum(n, keep)).to("cuda", torch.int32))
    return {**got, "weights": new_w}
