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
