"""Attention of ragged query rows on the GPU against its 64-bit definition.

Tolerances, from the number formats (half a step: bf16 2^-8, fp16 2^-11, fp32 2^-24).  With S the
largest scale * sum |q||k| of a row, a logit is off by at most d = 32 * 2^-23 S + 4 * 2^-24 S (an
fp32 sum of 128 exact products in at most 32 roundings or cuts of one step; the scale, the
subtraction), and exp2's hardware form by 2^-22 relative.
  lse  d + 2^-22 + n 2^-24 (sum of n terms) + 2^-22 (1 + |lse|) (log2, the two products)
  out  2^-8 |o| for its storage; max |v| times 2 (d + 2^-22) and n 2^-23 for the sums; and for P
       fp16: 2^-11 max |v|
       bf16: p (1 + e) with |e| <= 2^-8, divided by their own sum: o is off by sum p e (v - o) / sum p (1 + e),
       at most 2^-8 / (1 - 2^-8) times the weighted mean of |v - o|"""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import ragged as ref
from sparse_attention_decode_msa_gb300 import synth

pytestmark = pytest.mark.gpu

KV = ["bf16", "fp8", "nvfp4"]


class Ragged:
    """A batch of `counts` tokens over pages that hold seq_lens (+ the tokens themselves, causal) positions."""

    def __init__(self, counts, lens, causal, Hkv=1, G=16, kv="bf16", seed=1, ctas=0, behind=0, scale=None):
        import torch

        self.torch, self.causal, self.Hkv, self.G = torch, causal, Hkv, G
        self.counts, self.seq_lens = np.array(counts), np.array(lens, np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.T = int(self.offsets[-1]) + behind
        total = [max(1, length + (max(0, n - 1) if causal and length > 0 else 0)) for n, length in zip(counts, lens)]
        self.pb = synth.make_problem(name="ragged", contexts=total, q_per_req=1, num_kv_heads=Hkv, topk=1, kv_dtype=kv, seed=seed)
        if kv == "nvfp4":
            self.pb.k_scale, self.pb.v_scale = 0.75, 0.5
        if scale is not None:
            self.pb.softmax_scale = scale
        self.q = synth.normal_bf16(np.random.default_rng(seed + 7), (self.T, Hkv * G, 128))
        self.ctas = ctas
        self.upload()

    def dev(self, a):
        a = np.ascontiguousarray(a)
        return self.torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()

    def upload(self):
        pb, torch = self.pb, self.torch
        self.dq, self.kv, self.table = self.dev(self.q), self.dev(pb.kv_pool), self.dev(pb.block_table)
        self.d_offsets, self.lens = self.dev(self.offsets), self.dev(self.seq_lens)
        self.out = torch.full((self.T, self.Hkv * self.G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, self.Hkv * self.G), 7.0, device="cuda")
        self.shape = msa.make_shape(num_requests=pb.num_requests, q_per_req=1, num_kv_heads=self.Hkv, num_q_heads=self.Hkv * self.G, num_pages=pb.num_pages,
                                    max_blocks_per_seq=pb.max_blocks, topk=1, kv_dtype=pb.kv_dtype, softmax_scale=pb.softmax_scale, k_scale=pb.k_scale,
                                    v_scale=pb.v_scale, decode_ctas=self.ctas)
        self.nbytes = msa.msa_ragged_workspace_bytes(self.shape)
        assert self.nbytes > 0
        self.ws = torch.full((self.nbytes,), 0xFF, dtype=torch.uint8, device="cuda")  # only the error word is initialised
        self.ws[:256] = 0

    def run(self, stream=None):
        msa.msa_ragged_attention(self.shape, self.T, self.causal, self.dq, self.d_offsets, self.kv, self.table, self.lens, self.out, self.lse, self.ws,
                                 self.nbytes, stream)
        return self

    def status(self):
        return msa.msa_check_device_status(self.ws)

    def result(self):
        self.torch.cuda.synchronize()
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self):
        assert self.status() == msa.MSA_OK
        out, lse = self.result()
        real = int(self.offsets[-1])
        want, want_lse, far, S, V = ref.attention(self.pb, self.q, self.offsets, self.seq_lens, self.causal)
        assert np.all(out[real:] == 7) and np.all(lse[real:] == 7)  # rows behind the last request's
        check(out[:real], lse[:real], want[:real], want_lse[:real], far[:real], S, V, int(self.seq_lens.max()) + int(self.counts.max()),
              self.pb.kv_dtype)
        return out, lse


def check(out, lse, want, want_lse, far, S, V, n, kv):
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(out[empty] == 0)
    top = np.abs(np.where(empty, 0, want_lse)).max(initial=0)
    d = 36 * 2.0 ** -23 * S
    assert np.all(np.abs(lse[~empty] - want_lse[~empty]) <= d + 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -22 * (1 + top))
    p = 2.0 ** -8 / (1 - 2.0 ** -8) * far if kv == "bf16" else 2.0 ** -11 * V
    tol = 2.0 ** -8 * np.abs(want) + p + V * (2 * (d + 2.0 ** -22) + n * 2.0 ** -23)
    assert np.all(np.abs(out - want) <= tol), np.abs(out - want).max()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("counts,lens,Hkv,G", [
    ([1], [1], 1, 16), ([1], [200], 1, 1), ([7], [200], 2, 8), ([1, 1, 1], [127, 128, 129], 2, 16), ([3, 0, 5], [1000, 77, 1], 1, 5),
    ([17, 16, 15], [300, 1, 128], 2, 16), ([300], [1], 1, 16), ([129, 400, 2], [513, 1, 2000], 2, 4), ([700, 1], [5, 900], 1, 1),
    ([64] * 5, [1] * 5, 2, 2), ([9, 33], [250, 640], 1, 64), ([40], [100], 1, 48), ([1] * 70, list(range(1, 71)), 1, 3),
])
def test_ragged_attention(torch_cuda, kv, causal, counts, lens, Hkv, G):
    Ragged(counts, lens, causal, Hkv, G, kv, seed=sum(counts) + sum(lens), behind=2).run().check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 37, 152, 400])
def test_the_split_does_not_matter(torch_cuda, kv, causal, ctas):
    Ragged([5, 0, 90, 1], [1500, 40, 900, 3000], causal, 2, 16, kv, seed=ctas, ctas=ctas).run().check()


def test_one_long_unit_over_all_ctas(torch_cuda):
    # 300 pages of one unit: every CTA has a part, the join adds them with all of its warps
    for n in (1, 16):
        Ragged([n], [300 * 128 - 40], False, 1, 16, seed=n).run().check()
        Ragged([n], [300 * 128 - 40], False, 1, 16, seed=n, ctas=9).run().check()


def test_requests_without_states(torch_cuda):
    for causal in (True, False):
        for kv in KV:
            c = Ragged([3, 40, 1, 0], [0, 0, 130, 0], causal, 2, 8, kv, seed=4, behind=1)
            c.run().check()
        c = Ragged([3, 2], [0, 0], causal)
        c.run().check()


@pytest.mark.parametrize("kv", KV)
def test_the_same_bits_again(torch_cuda, kv):
    c = Ragged([100, 3, 500], [700, 4000, 1], True, 2, 16, kv, seed=9)
    a = [x.copy() for x in c.run().result()]
    for _ in range(5):
        c.out.fill_(0)
        b = c.run().result()
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("kv", KV)
def test_uniform_batches_agree_with_the_dense_decode(torch_cuda, kv):
    torch = torch_cuda
    c = Ragged([5] * 6, [1000, 1, 300, 128, 77, 2049], True, 2, 16, kv, seed=5)
    out, lse = c.run().check()
    shape = msa.make_shape(num_requests=6, q_per_req=5, num_kv_heads=2, num_pages=c.pb.num_pages, max_blocks_per_seq=c.pb.max_blocks, topk=1,
                           kv_dtype=kv, k_scale=c.pb.k_scale, v_scale=c.pb.v_scale)
    n = msa.msa_cache_workspace_bytes(shape)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    o, e = torch.empty_like(c.out), torch.empty_like(c.lse)
    msa.msa_dense_decode(shape, c.dq, c.kv, c.table, c.lens, o, e, ws, n)
    assert np.abs(e.double().cpu().numpy() - lse).max() < 1e-4
    assert np.abs(o.double().cpu().numpy() - out).max() < 2.0 ** -7 * max(1, np.abs(out).max())


# ---------------------------------------------------------------------------
# logits at odds with the references: rows whose later pages pass the first's maximum

@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", ["late", "early", "rising", "one row", "equal", "negative scale", "no scale", "low first page"])
def test_references(torch_cuda, kv, causal, shape):
    c = Ragged([40, 3], [900, 1500], causal, 1, 4, kv, seed=3, ctas=3)
    q = c.q
    big = synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(q) * 40)
    if shape == "late":      # the heaviest position is the last page's
        q[:] = big
        place(c, 0, 899, 24.0)
        place(c, 1, 1499, 24.0)
    elif shape == "early":
        q[:] = big
        place(c, 0, 0, 24.0)
    elif shape == "rising":  # every page holds a heavier one: each asks for a new reference
        q[:] = big
        for page in range(7):
            place(c, 0, 128 * page + 5, 2.0 + 3 * page)
    elif shape == "one row":  # one row of a warp's rises, the others stay
        q[7] = big[7]
        place(c, 0, 700, 30.0)
    elif shape == "equal":    # all logits alike, and in later pages alike but larger
        q[:] = 0x3F80
        for r in (0, 1):
            for g in (0,):
                fill_keys(c, r, 0, 300, 0)
                fill_keys(c, r, 300, 10000, 1)
    elif shape == "negative scale":
        c.pb.softmax_scale = -0.25
    elif shape == "no scale":
        c.pb.softmax_scale = 0.0
    else:                     # a first page far below all others
        q[:] = 0x3F80
        fill_keys(c, 0, 0, 128, 2)
        fill_keys(c, 1, 0, 300, 2)
    c.upload()
    c.run().check()


def stored(c, v):
    """The code of an element in the pool's format, near v."""
    if c.pb.kv_dtype == "bf16":
        return synth.f32_to_bf16_bits(np.array([v], np.float32))[0]
    if c.pb.kv_dtype == "fp8":
        return ref.to_codes(np.array([v / c.pb.k_scale]), ref.E4M3_VALUES)[0]
    return ref.to_codes(np.array([v]), ref.E2M1_VALUES)[0]


def rows_of(c, r, lo, hi, which):
    """(page, row) of positions lo .. hi - 1 that the batch has."""
    total = int(c.seq_lens[r]) + (int(c.counts[r]) - 1 if c.causal else 0)
    for p in range(lo, min(hi, total)):
        yield c.pb.block_table[r, p // 128], p % 128


def set_row(c, page, which, row, code, scale=None):
    if c.pb.kv_dtype == "nvfp4":
        c.pb.kv_pool[page, which, :, 64 * row:64 * row + 64] = code | code << 4
        if scale is not None:
            c.pb.kv_pool[page, which, :, 8192 + 8 * row:8192 + 8 * row + 8] = scale
    else:
        c.pb.kv_pool[page, which, :, row] = code


def place(c, r, pos, size):
    """A key of `size` in every dimension at a position."""
    for page, row in rows_of(c, r, pos, pos + 1, 0):
        set_row(c, page, 0, row, stored(c, min(size, 5.0) if c.pb.kv_dtype != "bf16" else size), 0x38)


def fill_keys(c, r, lo, hi, kind):
    """All keys alike: 0 small, 1 a little larger, 2 far below 0."""
    v = (0.5, 1.0, -6.0)[kind]
    for page, row in rows_of(c, r, lo, hi, 0):
        set_row(c, page, 0, row, stored(c, v), 0x38)


# ---------------------------------------------------------------------------
# values that are not finite

def bad_codes(kv):
    return {"bf16": (0x7F80, 0xFF80, 0x7FC0), "fp8": (0x7F, 0xFF), "nvfp4": (0x7F, 0xFF)}[kv]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("counts,lens,G", [([30, 5], [200, 1], 4), ([300], [1], 1), ([40], [120], 48), ([3, 3], [126, 255], 16)])
def test_values_that_are_not_finite_reach_those_who_see_them(torch_cuda, kv, counts, lens, G):
    # at cached positions, at the tokens' own and behind the last: what a row's outputs are not finite of is known
    for ctas in (0, 3):
        c = Ragged(counts, lens, True, 1, G, kv, seed=8, ctas=ctas)
        rng = np.random.default_rng(4)
        spots = []  # (request, position, dimensions)
        for r, (n, length) in enumerate(zip(counts, lens)):
            for pos in sorted(set(rng.integers(0, length + n - 1, 3).tolist() + [length, length + n - 2])):
                if pos < length + n - 1:
                    spots.append((r, pos, rng.integers(0, 8) * 16))
        v = c.pb.kv_pool
        for i, (r, pos, d) in enumerate(spots):
            page, row, code = c.pb.block_table[r, pos // 128], pos % 128, bad_codes(kv)[i % len(bad_codes(kv))]
            if kv == "nvfp4":  # a scale that is NaN: its 16 dimensions
                v[page, 1, 0, 8192 + 8 * row + d // 16] = code
            else:
                v[page, 1, 0, row, d] = code
        c.upload()
        out, lse = c.run().result()
        assert c.status() == msa.MSA_OK and np.all(np.isfinite(lse))
        clean = Ragged(counts, lens, True, 1, G, kv, seed=8, ctas=ctas)
        width = 16 if kv == "nvfp4" else 1
        for r, pos, d in spots:
            page, row = clean.pb.block_table[r, pos // 128], pos % 128
            if kv == "nvfp4":
                clean.pb.kv_pool[page, 1, 0, 8192 + 8 * row + d // 16] = 0
            else:
                clean.pb.kv_pool[page, 1, 0, row, d] = 0
        want, want_lse, far, S, V = ref.attention(clean.pb, clean.q, clean.offsets, clean.seq_lens, True)
        hit = np.zeros(out.shape, bool)
        for r, pos, d in spots:
            for j in range(counts[r]):
                if lens[r] + j > pos:
                    hit[c.offsets[r] + j, :, d:d + width] = True
        assert np.array_equal(~np.isfinite(out), hit)
        check(np.where(hit, want, out), lse, want, want_lse, far, S, V, 1000, kv)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv", KV)
def test_what_lies_behind_the_last_position_is_not_looked_at(torch_cuda, kv, causal):
    c = Ragged([20, 1, 7], [100, 129, 300], causal, 2, 8, kv, seed=6)
    for r in range(3):
        total = int(c.seq_lens[r]) + (int(c.counts[r]) - 1 if causal else 0)
        page = c.pb.block_table[r, (total - 1) // 128]
        for row in range((total - 1) % 128 + 1, 128):
            for which in (0, 1):
                if kv == "nvfp4":
                    c.pb.kv_pool[page, which, :, 8192 + 8 * row:8192 + 8 * row + 8] = 0x7F
                else:
                    c.pb.kv_pool[page, which, :, row] = bad_codes(kv)[row % len(bad_codes(kv))]
    c.upload()
    c.run().check()


def test_rows_with_infinite_logits_are_alone(torch_cuda):
    c = Ragged([20, 9], [300, 500], True, 1, 16, seed=2)
    c.q[3, 5, 0] = 0x7FC0  # a NaN, an infinity: in one row each
    c.q[4, 2, 1] = 0x7F80
    c.upload()
    out, lse = c.run().result()
    hit = np.zeros(lse.shape, bool)
    hit[3, 5] = hit[4, 2] = True
    assert np.array_equal(~np.isfinite(lse), hit) and np.array_equal(~np.isfinite(out).all(-1), hit)
    c.q[3, 5, 0] = c.q[4, 2, 1] = 0
    want, want_lse, far, S, V = ref.attention(c.pb, c.q, c.offsets, c.seq_lens, True)
    check(np.where(hit[..., None], want, out), np.where(hit, want_lse, lse), want, want_lse, far, S, V, 600, "bf16")


# ---------------------------------------------------------------------------
# inputs that only the device can see, and the ways of calling

def test_bad_inputs_are_reported_and_the_others_are_right(torch_cuda):
    torch = torch_cuda
    good = Ragged([5, 40, 7], [300, 200, 100], True, 1, 16, seed=5)
    want, want_lse, far, S, V = ref.attention(good.pb, good.q, good.offsets, good.seq_lens, True)
    others = np.r_[0:5, 45:52]
    for lens in (-1, good.pb.max_blocks * 128 + 1, 2 ** 31 - 1):
        c = Ragged([5, 40, 7], [300, 200, 100], True, 1, 16, seed=5)
        c.lens[1] = lens
        out, lse = c.run().result()
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK
        check(out[others], lse[others], want[others], want_lse[others], far[others], S, V, 400, "bf16")
        assert np.all(out[5:45] == 7)  # the refused request's rows are left
    for offsets in ([0, 5, 3, 52], [0, 5, 45, 60], [-4, 5, 45, 52], [0, 2 ** 31 - 1, 45, 52]):
        c = Ragged([5, 40, 7], [300, 200, 100], True, 1, 16, seed=5)
        c.d_offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        c.run()
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK
    for page in (-1, good.pb.num_pages, 2 ** 31 - 1):
        c = Ragged([5, 40, 7], [300, 200, 100], True, 1, 16, seed=5)
        c.table[1, 1] = page
        c.run()
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK
        assert c.status() == msa.MSA_OK  # reported once
    good.run().check()


@pytest.mark.parametrize("kv", KV)
def test_a_wait_that_runs_out_reports_timeout_and_the_next_call_is_exact(torch_cuda, kv):
    c = Ragged([100, 5, 30], [900, 2000, 1], True, 2, 16, kv, seed=7)
    c.run().check()
    msa.msa_set_decode_wait_limit(1)
    try:
        c.run()
        assert c.status() == msa.MSA_ERR_TIMEOUT
    finally:
        msa.msa_set_decode_wait_limit(0)
    c.run().check()


def test_page_offsets_beyond_32_bits(torch_cuda):
    # 75000 pages of 64 KiB; the request's pages are the last ones
    torch = torch_cuda
    c = Ragged([9], [700], True, 1, 16, seed=31)
    pages, n = 75000, c.pb.num_pages
    pool = torch.zeros((pages, 2, 1, 128, 128), dtype=torch.int16, device="cuda")
    pool[pages - n:] = c.kv
    c.kv = pool
    c.table += pages - n
    c.shape.num_pages = pages
    c.run().check()


def test_streams_graphs_and_two_calls_at_once(torch_cuda):
    torch = torch_cuda
    a, b = Ragged([50, 3], [700, 2000], True, 2, 16, seed=11), Ragged([200], [900], False, 1, 4, "fp8", seed=12)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):  # a workspace each: they may overlap
        a.run()
        b.run(side)
    a.check()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
        b.run()
    a.out.zero_()
    b.out.zero_()
    # a graph's replay sees the lengths that are there then
    a.seq_lens[:] = [333, 1999]
    a.lens.copy_(torch.from_numpy(a.seq_lens))
    graph.replay()
    graph.replay()
    a.check()
    b.check()


def test_a_batch_without_tokens_or_requests(torch_cuda):
    c = Ragged([0, 0], [5, 300], True, 1, 16, seed=1, behind=3)
    c.run()
    out, lse = c.result()
    assert np.all(out == 7) and np.all(lse == 7) and c.status() == msa.MSA_OK
    c.shape.num_requests = 0
    c.run()
    c.T = 0
    c.run()
    assert np.all(c.result()[0] == 7)


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,index", [("bf16", "bf16"), ("fp8", "nvfp4"), ("nvfp4", "nvfp4")])
def test_prompts_and_steps_through_the_cache(torch_cuda, kv, index):
    """Prompts appended in ragged chunks and attended causally, an encoder's states beside them, then decode steps
    on the same cache: dense, and block-sparse over the selected pages."""
    torch = torch_cuda
    rng = np.random.default_rng(17)
    R, Hkv, G, B = 3, 2, 16, 8
    Hq, pages = Hkv * G, R * B + 1
    rope = msa.make_rope(rotary_dim=64)
    rad = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    freqs = msa.rope_frequencies(rad, "cuda")
    elems = {"bf16": 128 * 256, "fp8": 128 * 128, "nvfp4": 9216}[kv]
    pool = torch.zeros((pages, 2, Hkv, elems), dtype=torch.uint8, device="cuda")
    idx_pool = torch.zeros((pages, 1, 128, 64 if index == "nvfp4" else 256), dtype=torch.uint8, device="cuda")
    idx_scales = torch.zeros((pages, 1, 128, 8), dtype=torch.uint8, device="cuda")
    table = torch.from_numpy((rng.permutation(pages - 1) + 1).astype(np.int32).reshape(R, B)).cuda()
    scales = dict(k_scale=1.0, v_scale=1.0) if kv == "bf16" else dict(k_scale=1 / 64, v_scale=1 / 64) if kv == "fp8" else dict(k_scale=0.5, v_scale=0.5)
    common = dict(num_requests=R, num_kv_heads=Hkv, num_pages=pages, max_blocks_per_seq=B, topk=8, kv_dtype=kv, index_dtype=index, **scales)
    shape = msa.make_shape(q_per_req=1, **common)
    nbytes = msa.msa_ragged_workspace_bytes(shape)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")

    def dev(a, dtype=None):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    class Pb:  # the pools as the definitions read them
        kv_dtype, num_kv_heads, softmax_scale = kv, Hkv, float(np.float32(128 ** -0.5))
        k_scale, v_scale = scales["k_scale"], scales["v_scale"]
        block_table = table.cpu().numpy()

    def host_pool():
        a = pool.cpu().numpy()
        return a.view(np.uint16).reshape(pages, 2, Hkv, 128, 128) if kv == "bf16" else a.reshape(pages, 2, Hkv, 128, 128) if kv == "fp8" else a

    cached = np.zeros(R, np.int64)
    for counts in ([300, 17, 0], [140, 0, 129], [1, 1, 1], [5, 5, 5]):
        T = sum(counts)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        lens = (cached + 1).astype(np.int32)
        rows = [synth.normal_bf16(rng, (T, h, 128)) for h in (Hq, Hkv, Hkv, 1, 1)]
        q, k, v, q_idx, idxk = (dev(x.view(np.int16)) for x in rows)
        d_offsets, d_lens = dev(offsets), dev(lens)
        msa.msa_kv_append(shape, rope, freqs, T, d_offsets, k, None, v, idxk, None, q, None, q, q_idx, None, q_idx, table, d_lens, pool, idx_pool,
                          idx_scales, ws, nbytes)
        out, lse = torch.empty((T, Hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((T, Hq), device="cuda")
        msa.msa_ragged_attention(shape, T, True, q, d_offsets, pool, table, d_lens, out, lse, ws, nbytes)
        assert msa.msa_check_device_status(ws) == msa.MSA_OK
        pb = Pb()
        pb.kv_pool = host_pool()
        q_bits = q.cpu().numpy().view(np.uint16)  # what the append left in place
        _, pos = ref.places(offsets, lens, T)
        want, size = ref.turned(rows[0], None, pos, rad, 64)
        assert np.all(np.abs(ref.bf16(q_bits) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size)
        want, want_lse, far, S, V = ref.attention(pb, q_bits, offsets, lens, True)
        o, e = out.double().cpu().numpy(), lse.double().cpu().numpy()
        check(o, e, want, want_lse, far, S, V, 1024, kv)
        if len(set(counts)) == 1:  # a decode step: the dense decode agrees, and the sparse one over all blocks does
            n = counts[0]
            s2 = msa.make_shape(q_per_req=n, **common)
            o2, e2 = torch.empty_like(out), torch.empty_like(lse)
            cw = msa.msa_cache_workspace_bytes(s2)
            wsc = torch.zeros(cw, dtype=torch.uint8, device="cuda")
            msa.msa_dense_decode(s2, q, pool, table, d_lens, o2, e2, wsc, cw)
            check(o2.double().cpu().numpy(), e2.double().cpu().numpy(), want, want_lse, far + 2.0 ** -2, S, V, 1024, kv)
            ds = msa.msa_workspace_bytes(s2)
            wsd = torch.zeros(ds, dtype=torch.uint8, device="cuda")
            msa.msa_decode_step(s2, q_idx, idx_pool, idx_scales, q, pool, table, d_lens, None, None, o2, e2, wsd, ds)
            assert msa.msa_check_device_status(wsd) == msa.MSA_OK
            assert np.abs(e2.double().cpu().numpy() - want_lse).max() < 1e-3 and np.abs(o2.double().cpu().numpy() - want).max() < 2e-2
        cached += counts
    # cross attention: each request's tokens to all that is cached of it, ragged queries
    counts = [7, 0, 200]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q_bits = synth.normal_bf16(rng, (207, Hq, 128))
    out, lse = torch.empty((207, Hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((207, Hq), device="cuda")
    msa.msa_ragged_attention(shape, 207, False, dev(q_bits.view(np.int16)), dev(offsets), pool, table, dev(cached.astype(np.int32)), out, lse, ws, nbytes)
    want, want_lse, far, S, V = ref.attention(pb, q_bits, offsets, cached, False)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, want_lse, far, S, V, 1024, kv)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("counts,lens,Hkv,G", [([70, 1], [300, 140], 2, 4), ([1, 200], [900, 1], 1, 5)])
def test_outputs_that_begin_at_any_multiple_of_16_bytes(torch_cuda, kv, counts, lens, Hkv, G):
    c = Ragged(counts, lens, True, Hkv, G, kv, seed=3).run()
    out, lse = c.check()
    room = c.torch.full((c.T * Hkv * G * 128 + 16,), 7.0, dtype=c.torch.bfloat16, device="cuda")
    c.out = room[8:-8].view(c.T, Hkv * G, 128)
    assert c.out.data_ptr() % 32 == 16
    again, again_lse = c.run().check()
    assert np.array_equal(out, again) and np.array_equal(lse, again_lse)
    assert bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())
