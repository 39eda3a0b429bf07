"""Norm and rotation of head rows and the append to the paged cache, on the GPU against their
64-bit definitions.

Tolerance of a value before its rounding: with u = 2^-24 and s the size of what it was added up
from (|a| + |b| of its pair), the norm's sum of 128 squares takes at most 19 roundings, halved by
the root, its reciprocal root 2 ulp (4 u), three products 3 u and the weight's sum 1 u: 17.5 u.
The angle is a float of a turn (u of at most pi: 3.2 u), its sine and cosine 2 ulp (4 u), the scale
u, two products and a difference 3 u: 11.2 u.  Together under 32 u = 2^-19 of s.  Stored values
are the rounding of a number that near: bf16 adds 2^-8 of itself, codes are monotone in theirs."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import ragged as ref
from oracle.whole_cache import bf16, e4m3
from sparse_attention_decode_msa_gb300 import synth

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -19


def dev(a):
    import torch

    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def freqs_of(rotary_dim, base=10000.0):
    return base ** (-np.arange(0, rotary_dim, 2) / max(1, rotary_dim))


def weights_of(rng, heads, norm):
    if norm == "none":
        return None
    shape = (heads, 128) if norm == "heads" else (128,)
    return synth.f32_to_bf16_bits((1 + rng.standard_normal(shape) / 4).astype(np.float32))


def fused(rng, T, *heads):
    """Rows of each kind as parts of one [T][sum + 1][128] tensor: host bits, device views, the stride."""
    total = sum(heads) + 1
    x = synth.normal_bf16(rng, (T, total, 128))
    d, at = dev(x), np.cumsum((0,) + heads)
    return [x[:, a:a + h] for a, h in zip(at, heads)], [d[:, a:a + h] for a, h in zip(at, heads)], total * 128


def is_near(got_bits, want, size):
    got = bf16(got_bits.view(np.uint16))
    return np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + NEAR * 1.01 * size


def host(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("norm", ["none", "shared", "heads"])
@pytest.mark.parametrize("T,Hq,Hk,rot,interleaved,far", [
    (1, 1, 0, 128, False, 10), (1, 64, 4, 128, False, 1000000), (7, 5, 1, 64, True, 131072), (33, 3, 2, 16, False, 5000),
    (130, 8, 8, 96, False, 2000000), (129, 2, 1, 112, True, 70000), (5, 6, 5, 48, False, 999), (9, 4, 4, 0, False, 9), (2000, 16, 2, 32, True, 2 ** 31 - 1),
])
def test_norm_and_rotation(torch_cuda, T, Hq, Hk, rot, interleaved, far, norm):
    torch = torch_cuda
    rng = np.random.default_rng(T + Hq)
    (q, k), (dq, dk), stride = fused(rng, T, Hq, Hk)
    pos = rng.integers(0, far, T).astype(np.int32)
    qw, kw, rad = weights_of(rng, Hq, norm), weights_of(rng, Hk, norm), freqs_of(rot)
    more = dict(scale=1.25, norm_eps=1e-3, norm_offset=1.0) if T % 2 else {}
    rope = msa.make_rope(rotary_dim=rot, interleaved=interleaved, per_head_weights=norm == "heads", q_stride=stride, k_stride=stride, **more)
    q_out = torch.full((T, Hq, 128), 7, dtype=torch.int16, device="cuda")
    k_out = torch.full((T, Hk, 128), 7, dtype=torch.int16, device="cuda")
    d = lambda w: None if w is None else dev(w)  # noqa: E731
    ks = (Hk, dk, d(kw), k_out) if Hk else ()
    msa.msa_qk_norm_rope(rope, msa.rope_frequencies(rad, "cuda") if rot else None, T, dev(pos), Hq, dq, d(qw), q_out, *ks)
    named = dict(scale=more.get("scale", 1.0), eps=float(np.float32(more.get("norm_eps", 1e-6))), offset=more.get("norm_offset", 0.0))
    for x, w, y in ((q, qw, q_out), (k, kw, k_out)):
        want, size = ref.turned(x, w, pos, rad, rot, interleaved, **named)
        assert np.all(is_near(host(y), want, size))
        if norm == "none" and rot < 128:  # what neither turns nor is normed is copied
            assert np.array_equal(host(y).view(np.uint16)[..., rot:], x[..., rot:])


def test_far_positions_turn_exactly(torch_cuda):
    # angles whose 32-bit products are off by whole radians: pairs (1, 0) become (cos, sin)
    torch = torch_cuda
    pos = np.array([0, 1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -5], np.int32)
    rad = np.linspace(0.01, 3.0, 64)
    x = np.zeros((6, 1, 128), np.uint16)
    x[..., :64] = 0x3F80
    y = torch.empty((6, 1, 128), dtype=torch.bfloat16, device="cuda")
    msa.msa_qk_norm_rope(msa.make_rope(), msa.rope_frequencies(rad, "cuda"), 6, dev(pos), 1, dev(x), None, y)
    t = np.asarray(pos, np.longdouble)[:, None] * rad.astype(np.longdouble)
    want = np.concatenate([np.cos(t), np.sin(t)], -1).astype(np.float64)[:, None]
    # the table keeps 2^-56 of a turn: 2^-25 of one at 2^31
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + NEAR * 2 + 2.0 ** -22)


def test_in_place_and_dense(torch_cuda):
    rng = np.random.default_rng(3)
    q, k = synth.normal_bf16(rng, (77, 6, 128)), synth.normal_bf16(rng, (77, 2, 128))
    pos, rad = rng.integers(0, 9999, 77).astype(np.int32), freqs_of(128)
    dq, dk, w = dev(q), dev(k), weights_of(rng, 1, "shared")
    msa.msa_qk_norm_rope(msa.make_rope(), msa.rope_frequencies(rad, "cuda"), 77, dev(pos), 6, dq, dev(w), dq, 2, dk, None, dk)
    for x, wt, y in ((q, w, dq), (k, None, dk)):
        want, size = ref.turned(x, wt, pos, rad, 128)
        assert np.all(is_near(host(y), want, size))


# ---------------------------------------------------------------------------

class Batch:
    """Ragged new tokens and the pools that take them."""

    def __init__(self, counts, first, Hkv=2, G=4, Hi=1, kv="bf16", index="bf16", rot=128, interleaved=False, norm="shared", seed=1, behind=0,
                 queries=True, scale=0.75):
        rng = np.random.default_rng(seed)
        self.counts, self.first = np.array(counts), np.array(first)  # new tokens, cached before
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.seq_lens = (self.first + 1).astype(np.int32)
        self.T, self.R, self.Hkv, self.Hi, self.Hq = int(self.offsets[-1]) + behind, len(counts), Hkv, Hi, Hkv * G
        self.kv, self.index, self.rot, self.interleaved, self.norm, self.queries = kv, index, rot, interleaved, norm, queries
        blocks = [max(1, -(-(c + f) // 128)) for c, f in zip(counts, first)]
        self.B, self.pages = max(blocks) + 1, sum(blocks) + 2
        perm = rng.permutation(self.pages - 1) + 1
        self.table, i = np.full((self.R, self.B), -1, np.int32), 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = perm[i:i + b]
            i += b
        heads = (self.Hq, Hi, Hkv, Hkv, Hi)
        self.host, self.dev, stride = fused(rng, self.T, *heads)
        self.w = [weights_of(rng, h, norm) for h in heads]
        self.w[3] = None  # values
        self.rad = freqs_of(rot)
        per = {"bf16": 256, "fp8": 128}
        self.pool = rng.integers(0, 256, (self.pages, 2, Hkv, 9216 if kv == "nvfp4" else 128 * per[kv]), dtype=np.uint8)
        self.idx_pool = rng.integers(0, 256, (self.pages, Hi, 128, 64 if index == "nvfp4" else 256), dtype=np.uint8)
        self.idx_scales = rng.integers(0, 256, (self.pages, Hi, 128, 8), dtype=np.uint8)
        self.k_scale, self.v_scale = (1.0, 1.0) if kv == "bf16" else (scale / 64, 2.0 ** -6) if kv == "fp8" else (scale, 0.5)
        self.shape = msa.make_shape(num_requests=self.R, q_per_req=1, num_kv_heads=Hkv, num_q_heads=self.Hq, num_pages=self.pages, max_blocks_per_seq=self.B,
                                    topk=1, kv_dtype=kv, index_dtype=index, k_scale=self.k_scale, v_scale=self.v_scale, num_index_heads=Hi)
        self.rope = msa.make_rope(rotary_dim=rot, interleaved=interleaved, per_head_weights=norm == "heads", q_stride=stride, k_stride=stride,
                                  v_stride=stride, q_idx_stride=stride, idxk_stride=stride)

    def run(self, torch, table=None, seq_lens=None, offsets=None, stream=None):
        d = lambda x: None if x is None else dev(x)  # noqa: E731
        self.nbytes = msa.msa_ragged_workspace_bytes(self.shape)
        self.ws = torch.zeros(self.nbytes, dtype=torch.uint8, device="cuda")
        self.d_pool, self.d_idx, self.d_sc = dev(self.pool), dev(self.idx_pool), dev(self.idx_scales)
        self.q_out = torch.full((self.T, self.Hq, 128), 7, dtype=torch.int16, device="cuda")
        self.qi_out = torch.full((self.T, self.Hi, 128), 7, dtype=torch.int16, device="cuda")
        q, qi, k, v, ik = self.dev
        qs = (q, d(self.w[0]), self.q_out, qi, d(self.w[1]), self.qi_out) if self.queries else (None,) * 6
        freqs = msa.rope_frequencies(self.rad, "cuda") if self.rot else None
        torch.cuda.synchronize()
        msa.msa_kv_append(self.shape, self.rope, freqs, self.T, dev(self.offsets if offsets is None else offsets), k, d(self.w[2]), v, ik,
                          d(self.w[4]), *qs, dev(self.table if table is None else table), dev(self.seq_lens if seq_lens is None else seq_lens),
                          self.d_pool, self.d_idx, self.d_sc, self.ws, self.nbytes, stream)
        torch.cuda.synchronize()
        return msa.msa_check_device_status(self.ws)

    def turned(self, i):
        req, pos = ref.places(self.offsets, self.seq_lens, self.T)
        if i == 3:
            x = bf16(self.host[3])
            return x, 0 * x
        return ref.turned(self.host[i], self.w[i], pos, self.rad, self.rot, self.interleaved, eps=float(np.float32(1e-6)))

    def check(self):
        req, pos = ref.places(self.offsets, self.seq_lens, self.T)
        real = req >= 0
        for i, y in ((0, self.q_out), (1, self.qi_out)):
            got = host(y)
            if self.queries:
                want, size = self.turned(i)
                assert np.all(is_near(got, want, size)[real])
                assert np.all(got[req < 0] == 7)
            else:
                assert np.all(got == 7)
        t = np.nonzero(real)[0]
        page, row = self.table[req[t], pos[t] // 128], pos[t] % 128
        pool, idx, sc = host(self.d_pool), host(self.d_idx), host(self.d_sc)
        untouched = [pool.copy(), idx.copy(), sc.copy()]
        for which, i, scale in ((0, 2, self.k_scale), (1, 3, self.v_scale)):
            want, size = self.turned(i)
            for g in range(self.Hkv):
                tile = pool[page, which, g]
                self.check_rows(tile, row, self.kv, want[t, g], size[t, g], float(np.float32(scale)))
                for a, at in zip(page, row):
                    for lo, n in self.spans(self.kv, at):
                        untouched[0][a, which, g, lo:lo + n] = self.pool[a, which, g, lo:lo + n]
        want, size = self.turned(4)
        for h in range(self.Hi):
            if self.index == "bf16":
                assert np.all(is_near(idx[page, h, row].view(np.uint16), want[t, h], size[t, h]))
            else:
                self.check_nvfp4(idx[page, h, row], sc[page, h, row], want[t, h], size[t, h])
                untouched[2][page, h, row] = self.idx_scales[page, h, row]
            untouched[1][page, h, row] = self.idx_pool[page, h, row]
        # no other row changed
        assert np.array_equal(untouched[0], self.pool) and np.array_equal(untouched[1], self.idx_pool) and np.array_equal(untouched[2], self.idx_scales)

    @staticmethod
    def spans(kv, row):
        return ((64 * row, 64), (8192 + 8 * row, 8)) if kv == "nvfp4" else ((row * (256 if kv == "bf16" else 128), 256 if kv == "bf16" else 128),)

    def check_rows(self, tile, row, kv, want, size, scale):
        i = np.arange(len(row))
        if kv == "bf16":
            got = tile.reshape(len(row), 128, 256)[i, row].view(np.uint16)
            assert np.all(is_near(got, want, size))
        elif kv == "fp8":
            got = tile.reshape(len(row), 128, 128)[i, row]
            lo, hi = ((want - NEAR * size) / scale, (want + NEAR * size) / scale)
            e = 2.0 ** -23 * np.abs(want / scale)  # the quotient
            v = e4m3(got)
            assert np.all(e4m3(ref.to_codes(lo - e, ref.E4M3_VALUES)) <= v) and np.all(v <= e4m3(ref.to_codes(hi + e, ref.E4M3_VALUES)))
            assert not np.any(got == 0x80)
        else:
            codes = np.stack([tile[i, 64 * row + b] for b in range(64)], -1)
            self.check_nvfp4(codes, np.stack([tile[i, 8192 + 8 * row + b] for b in range(8)], -1), want / scale, size / scale)

    @staticmethod
    def check_nvfp4(codes, scales, want, size):
        tol = NEAR * size + 2.0 ** -23 * np.abs(want)
        group = lambda a: a.reshape(len(a), 8, 16)  # noqa: E731
        S = e4m3(scales)
        lo = (np.abs(group(want)) - group(tol)).max(-1) / 6 * (1 - 2.0 ** -22)
        hi = (np.abs(group(want)) + group(tol)).max(-1) / 6 * (1 + 2.0 ** -22)
        assert np.all(e4m3(ref.to_codes(np.maximum(lo, 0), ref.E4M3_VALUES)) <= S) and np.all(S <= e4m3(ref.to_codes(hi, ref.E4M3_VALUES)))
        nib = np.stack([codes & 15, codes >> 4], -1).reshape(len(codes), 128)
        v = np.repeat(S, 16, -1)
        got = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])[nib]
        safe = np.where(v > 0, v, 1)
        e2 = lambda x: np.where(x < 0, -1, 1) * ref.E2M1_VALUES[ref.to_codes(np.abs(x), ref.E2M1_VALUES) & 7]  # noqa: E731
        e = 2.0 ** -22 * np.abs(want / safe)
        ok = (e2((want - tol) / safe - e) <= got) & (got <= e2((want + tol) / safe + e))
        assert np.all(np.where(v > 0, ok, nib == 0)) and not np.any(nib == 8)


@pytest.mark.parametrize("kv,index", [("bf16", "bf16"), ("fp8", "nvfp4"), ("nvfp4", "nvfp4"), ("nvfp4", "bf16")])
@pytest.mark.parametrize("counts,first,Hkv,G,Hi,rot,interleaved,norm", [
    ([1], [0], 1, 16, 1, 128, False, "shared"),
    ([1, 1, 1], [127, 128, 4095], 4, 16, 4, 128, False, "heads"),
    ([0, 5, 0, 130, 1], [9, 126, 3, 0, 255], 2, 5, 1, 64, True, "heads"),
    ([300, 7], [1000, 5], 3, 1, 6, 48, False, "none"),
    ([64] * 40, list(range(40)), 1, 2, 1, 16, False, "shared"),
    ([33, 100], [0, 77], 1, 4, 1, 0, False, "shared"),
])
def test_append(torch_cuda, kv, index, counts, first, Hkv, G, Hi, rot, interleaved, norm):
    b = Batch(counts, first, Hkv, G, Hi, kv, index, rot, interleaved, norm, seed=sum(counts) + rot, behind=3, queries=rot != 48)
    assert b.run(torch_cuda) == msa.MSA_OK
    b.check()


def test_many_requests(torch_cuda):
    # the search over offsets: every number of rounds, runs of requests without tokens
    for R, seed in ((31, 1), (33, 2), (1025, 3), (8192, 4)):
        rng = np.random.default_rng(seed)
        b = Batch(rng.integers(0, 3, R).tolist(), rng.integers(0, 300, R).tolist(), Hkv=1, G=1, rot=16, seed=seed, behind=1)
        assert b.run(torch_cuda) == msa.MSA_OK
        b.check()


@pytest.mark.parametrize("kv,index", [("bf16", "bf16"), ("fp8", "bf16"), ("fp8", "nvfp4"), ("nvfp4", "nvfp4")])
def test_append_as_it_is_gives_the_bytes_of_the_update(torch_cuda, kv, index):
    torch = torch_cuda
    pb = synth.make_problem(name="append", contexts=[700, 129, 1000, 128], q_per_req=4, num_kv_heads=2, topk=2, kv_dtype=kv, index_dtype=index, seed=21)
    upd = synth.make_update(pb)
    for x in (upd["k_new"], upd["v_new"], upd["idxk_new"]):
        x.reshape(-1)[:9] = [0x7F80, 0xFF80, 0x7FC1, 0x8000, 0x0001, 0x7F7F, 0xFF7F, 0x0000, 0x3F80]  # infinities, NaN, zeros, a subnormal, the largest
    bufs = {n: None if getattr(pb, n) is None else dev(getattr(pb, n)) for n in ("kv_pool", "idxk_pool", "idxk_scales")}
    direct = {n: None if x is None else x.clone() for n, x in bufs.items()}
    k, v, ik = (dev(upd[n]) for n in ("k_new", "v_new", "idxk_new"))
    shape = msa.make_shape(num_requests=4, q_per_req=4, num_kv_heads=2, num_pages=pb.num_pages, max_blocks_per_seq=pb.max_blocks, topk=2, kv_dtype=kv,
                           index_dtype=index, k_scale=pb.k_scale, v_scale=pb.v_scale)
    n = msa.msa_ragged_workspace_bytes(shape)
    ws = torch.zeros(max(n, 1 << 16), dtype=torch.uint8, device="cuda")
    table, lens = dev(pb.block_table), dev(pb.seq_lens)
    msa.msa_kv_append(shape, msa.make_rope(rotary_dim=0), None, 16, dev(np.arange(0, 20, 4, dtype=np.int32)), k, None, v, ik, None, None, None, None, None,
                      None, None, table, lens, *bufs.values(), ws, n)
    big = torch.zeros(msa.msa_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    msa.msa_kv_update(shape, k, v, ik, table, lens, *direct.values(), big, big.numel())
    assert msa.msa_check_device_status(ws) == msa.MSA_OK
    for name, x in bufs.items():
        if x is not None:
            assert torch.equal(x, direct[name]), name


def test_bad_lengths_and_pages_are_reported_and_skipped(torch_cuda):
    b = Batch([2, 3, 130], [100, 10, 50], seed=9)
    for bad in (0, -4, b.B * 128 + 1, 2 ** 31 - 1):  # none, and beyond the table
        lens = b.seq_lens.copy()
        lens[1] = bad
        assert b.run(torch_cuda, seq_lens=lens) == msa.MSA_ERR_DEVICE_CHECK
        pool = host(b.d_pool)
        req, pos = ref.places(b.offsets, b.seq_lens, b.T)
        for t in (2, 3, 4):  # their rows are as they were
            page, row = b.table[1, pos[t] // 128], pos[t] % 128
            assert np.array_equal(pool[page, :, :, 256 * row:256 * row + 256], b.pool[page, :, :, 256 * row:256 * row + 256])
    b = Batch([2, 3, 130], [100, 10, 50], seed=9)
    for bad in (-1, b.pages, 2 ** 31 - 1):
        table = b.table.copy()
        table[2, 1] = bad
        assert b.run(torch_cuda, table=table) == msa.MSA_ERR_DEVICE_CHECK
        pool = host(b.d_pool)
        assert np.array_equal(pool[b.table[2, 1]], b.pool[b.table[2, 1]])
        assert np.array_equal(pool[0], b.pool[0])


def test_offsets_out_of_order_write_nothing_outside(torch_cuda):
    # refused by nothing on the host: every row goes to a request that has it, or nowhere
    b = Batch([4, 4, 4], [10, 10, 10], seed=5)
    for offsets in ([0, 9, 3, 12], [5, 4, 3, 2], [0, 2 ** 31 - 1, -7, 12]):
        b.run(torch_cuda, offsets=np.array(offsets, np.int32))
        assert np.array_equal(host(b.d_pool)[0], b.pool[0])  # the page of no request


def test_streams_and_graphs(torch_cuda):
    torch = torch_cuda
    b = Batch([3, 0, 140], [5, 9, 0], seed=12, kv="fp8")
    side = torch.cuda.Stream()
    assert b.run(torch, stream=side) == msa.MSA_OK
    b.check()
    q, qi, k, v, ik = b.dev
    freqs, offsets, table, lens = msa.rope_frequencies(b.rad, "cuda"), dev(b.offsets), dev(b.table), dev(b.seq_lens)
    ws = [None if w is None else dev(w) for w in b.w]
    b.d_pool, b.d_idx, b.d_sc = dev(b.pool), dev(b.idx_pool), dev(b.idx_scales)
    b.q_out.fill_(7)
    b.qi_out.fill_(7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_kv_append(b.shape, b.rope, freqs, b.T, offsets, k, ws[2], v, ik, ws[4], q, ws[0], b.q_out, qi, ws[1], b.qi_out, table, lens,
                          b.d_pool, b.d_idx, b.d_sc, b.ws, b.nbytes)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    b.check()


def test_offsets_below_zero_are_reported_and_write_nothing(torch_cuda):
    b = Batch([4, 4, 4], [10, 10, 10], seed=5)
    for first in (-1, -2 ** 31):
        offsets = b.offsets.copy()
        offsets[0] = first
        assert b.run(torch_cuda, offsets=offsets) == msa.MSA_ERR_DEVICE_CHECK
        pool = host(b.d_pool)
        assert np.array_equal(pool[0], b.pool[0]) and np.array_equal(pool[b.table[0, 0]], b.pool[b.table[0, 0]])
