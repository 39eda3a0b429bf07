"""The whole-cache operators on the GPU against their 64-bit definitions:
dense decode, accumulated weights, eviction, and a run of them together.

Tolerances, from the number formats (u = half a step: bf16 2^-8, fp16 2^-11,
fp32 2^-24).  With S the largest scale * sum |q||k| of a row, a logit is off by
at most d = 32 * 2^-23 * S + 4 * 2^-24 * |x| (an fp32 sum of 128 exact
products, in at most 32 roundings or cuts of one step; the scale, the subtraction), and
exp2's hardware form by 2^-22 relative.
  lse      d + 2^-22 + n 2^-24 (sum of n terms) + 2^-22 (1 + |lse|) (log2, the two products)
  out      2^-8 |o| for its storage, and max |v| times: 2^-11 for P, 2 (d + 2^-22), n 2^-23 for the
           sums.  P is fp16 (2^-11 of each p) or a bf16 pair (2^-16), or bf16 alone where each p is at
           most l / 64: then its errors, independent and 2^-8 / sqrt(3) p (rms) at most, add up to
           2^-8 / sqrt(3) sqrt(sum p^2) / l <= 2^-8 / sqrt(3) / 8 = 2^-11.8 (rms) of max |v|, and of the
           rms of v, a quarter of its maximum here, 5 sigma are 2^-11.5
           (that last case no longer occurs: equal logits round alike, so bf16 P is the pair in every step)
  weights  relative d + 2^-22 + 2^-23 |lse| a term, rows 2^-24 for the sum, 2^-23 for decay
"""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import whole_cache as ref
from sparse_attention_decode_msa_gb300 import synth

pytestmark = pytest.mark.gpu

KV = ["bf16", "fp8", "nvfp4"]


class Cache:
    """A problem on the GPU with the buffers of the whole-cache operators."""

    def __init__(self, contexts, nq=1, Hkv=1, G=16, kv="bf16", seed=1, idle=(), extra_pages=0, Hi=1, index="bf16", ctas=0, pb=None):
        import torch

        self.torch = torch
        need = sum(-(-c // 128) for c in contexts)
        self.pb = pb or synth.make_problem(name="cache", contexts=contexts, q_per_req=nq, num_kv_heads=Hkv, topk=4, kv_dtype=kv,
                                           index_dtype=index, seed=seed, num_index_heads=Hi, num_pages=need + 1 + extra_pages)
        if kv == "nvfp4":
            self.pb.k_scale, self.pb.v_scale = 0.75, 0.5
        for r in idle:
            self.pb.seq_lens[r] = 0
        self.G, self.Hkv, self.nq, self.ctas, self.Hi = G, Hkv, nq, ctas, Hi
        self.q = synth.normal_bf16(np.random.default_rng(seed + 77), (self.pb.num_tokens, Hkv * G, 128))
        self.upload()

    def upload(self):
        pb, torch = self.pb, self.torch

        def dev(a):
            a = np.ascontiguousarray(a)
            return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()

        self.dq, self.kv, self.idxk = dev(self.q), dev(pb.kv_pool), dev(pb.idxk_pool)
        self.scales = None if pb.idxk_scales is None else dev(pb.idxk_scales)
        self.table, self.lens = dev(pb.block_table), dev(pb.seq_lens)
        T, Hq = self.q.shape[:2]
        self.out = torch.full((T, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, Hq), float("nan"), device="cuda")
        self.shape = msa.make_shape(
            num_requests=pb.num_requests, q_per_req=self.nq, num_kv_heads=self.Hkv, num_q_heads=Hq, num_pages=pb.num_pages,
            max_blocks_per_seq=pb.max_blocks, topk=pb.topk, kv_dtype=pb.kv_dtype, index_dtype=pb.index_dtype, softmax_scale=pb.softmax_scale,
            k_scale=pb.k_scale, v_scale=pb.v_scale, decode_ctas=self.ctas, num_index_heads=self.Hi)
        self.nbytes = msa.msa_cache_workspace_bytes(self.shape)
        assert self.nbytes > 0
        self.ws = torch.empty(self.nbytes, dtype=torch.uint8, device="cuda")
        msa.msa_workspace_init(self.ws, self.nbytes)

    def decode(self, stream=None):
        msa.msa_dense_decode(self.shape, self.dq, self.kv, self.table, self.lens, self.out, self.lse, self.ws, self.nbytes, stream)

    def accumulate(self, lse, w_in, w_out, decay=1.0, selected=None):
        msa.msa_weight_accumulate(self.shape, self.dq, self.kv, self.table, self.lens, selected, lse, decay, w_in, w_out, self.ws, self.nbytes)

    def status(self):
        return msa.msa_check_device_status(self.ws)

    def result(self):
        self.torch.cuda.synchronize()
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check_decode(self):
        out, lse = self.result()
        want, want_lse, S, V = ref.dense_decode(self.pb, self.q)
        check_attention(out, lse, want, want_lse, S, V, int(self.pb.seq_lens.max()) + self.nq)
        assert self.status() == msa.MSA_OK
        return out, lse


def logit_error(S, x):
    return 32 * 2.0 ** -23 * S + 4 * 2.0 ** -24 * x


def check_attention(out, lse, want, want_lse, S, V, n):
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(out[empty] == 0)
    top = np.abs(np.where(empty, 0, want_lse)).max() if want_lse.size else 0.0
    d = logit_error(S, S)
    assert np.all(np.abs(lse[~empty] - want_lse[~empty]) <= d + 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -22 * (1 + top))
    tol = 2.0 ** -8 * np.abs(want) + V * (2.0 ** -11 + 2 * (d + 2.0 ** -22) + n * 2.0 ** -23)
    assert np.all(np.abs(out - want) <= tol), np.abs(out - want).max()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("contexts,nq,Hkv,G", [
    ([1], 1, 1, 16), ([127, 128, 129], 1, 2, 16), ([1000, 1, 300], 1, 1, 1), ([513, 77], 1, 2, 5), ([640, 2, 1111], 2, 2, 8),
    ([900, 4, 129], 4, 1, 16), ([700, 333], 3, 1, 7), ([1025, 48], 48, 2, 16), ([260, 64], 64, 1, 64), ([2000, 131], 5, 1, 64),
])
def test_dense_decode(torch_cuda, kv, contexts, nq, Hkv, G):
    c = Cache(contexts, nq, Hkv, G, kv, seed=sum(contexts) + nq)
    c.decode()
    c.check_decode()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", [1, 3, 20])  # 16, 48 and 320 query rows
@pytest.mark.parametrize("ctas", [1, 2, 5, 37, 152, 400])
def test_dense_decode_does_not_depend_on_the_split(torch_cuda, kv, nq, ctas):
    c = Cache([3000, 129, 1500, nq, 20], nq, 2, 16, kv, seed=5, ctas=ctas)
    c.decode()
    c.check_decode()


@pytest.mark.parametrize("nq,idle", [(1, (0, 2)), (3, (1,)), (2, (0, 1, 2, 3)), (48, (3,))])
def test_idle_slots_of_a_padded_batch(torch_cuda, nq, idle):
    c = Cache([400, 130, 700, 64], nq, 2, 8, idle=idle, seed=9)
    c.pb.block_table[list(idle)] = -1
    c.upload()
    c.decode()
    c.check_decode()
    w = c.torch.full((4, 2, c.pb.max_blocks * 128), 7.0, device="cuda")
    c.accumulate(c.lse, None, w)
    assert c.status() == msa.MSA_OK
    assert bool((w[list(idle)] == 7.0).all())


def poison(pb, kv):
    """NaN and infinities behind the last position of every request, and in every page without owner."""
    used = set(pb.block_table[pb.block_table >= 0].tolist())
    for page in range(pb.num_pages):
        if page not in used:
            pb.kv_pool[page] = 0x7FC0 if kv == "bf16" else 0x7F
    for r in range(pb.num_requests):
        n = int(pb.seq_lens[r]) + pb.q_per_req - 1
        page, row = pb.block_table[r, (n - 1) // 128], n % 128
        if row == 0:
            continue
        if kv == "nvfp4":
            tile = pb.kv_pool[page]
            tile[..., 8192 + row * 8:] = 0x7F
            tile[..., row * 64:8192] = 0x77
        else:
            pb.kv_pool[page, :, :, row:] = 0x7F80 if kv == "bf16" else 0x7F


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq,G", [(1, 16), (2, 16), (4, 16), (48, 16), (3, 5)])
def test_what_lies_behind_the_cache_does_not_matter(torch_cuda, kv, nq, G):
    c = Cache([190, 1000, 65, 128], nq, 2, G, kv, seed=13)
    poison(c.pb, kv)
    c.upload()
    c.decode()
    c.check_decode()
    w = c.torch.full((4, 2, c.pb.max_blocks * 128), -1.0, device="cuda")
    c.accumulate(c.lse, None, w)
    check_weights(c, w, c.lse, None, 1.0, None)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("nq,G", [(2, 8), (4, 16), (5, 3), (40, 16)])
def test_an_infinite_value_reaches_only_the_tokens_that_see_it(torch_cuda, kv, nq, G):
    # the last token's own V row is not finite: the tokens before it do not see it
    c = Cache([300, 129], nq, 1, G, kv, seed=17)
    for r in range(2):
        last = int(c.pb.seq_lens[r]) + nq - 2
        c.pb.kv_pool[c.pb.block_table[r, last // 128], 1, 0, last % 128, 5] = 0x7F80 if kv == "bf16" else 0x7F
    c.upload()
    c.decode()
    out, lse = c.result()
    want, want_lse, S, V = ref.dense_decode(c.pb, c.q)
    fine = np.ones(c.pb.num_tokens, bool)
    fine[nq - 1::nq] = False
    check_attention(out[fine], lse[fine], want[fine], want_lse[fine], S, V, 400)
    assert not np.isfinite(out[~fine][:, :, 5]).any()
    others = np.arange(128) != 5
    check_attention(out[~fine][:, :, others], lse[~fine], want[~fine][:, :, others], want_lse[~fine], S, V, 400)


def test_dense_decode_equals_the_sparse_decode_of_all_blocks(torch_cuda):
    from sparse_attention_decode_msa_gb300.runner import DeviceProblem

    pb = synth.make_problem(name="all", contexts=[900, 300, 1024], q_per_req=2, num_kv_heads=2, topk=8, seed=21)
    dp = DeviceProblem(pb)
    dp.decode_step()
    sparse = dp.results()
    dp.dense_decode()
    dense = dp.results()
    assert msa.msa_check_device_status(dp.cache_ws) == msa.MSA_OK
    _, _, S, V = ref.dense_decode(pb, pb.q)
    # two results, each within the bound of the definition; the sparse decode's own is 4e-3, 1e-4
    assert np.abs(dense["out"] - sparse["out"]).max() <= 4e-3 + (2.0 ** -8 + 2.0 ** -11 + 2 * logit_error(S, S) + 2.0 ** -12) * V
    assert np.abs(dense["lse"] - sparse["lse"]).max() <= 1e-4 * np.abs(sparse["lse"]).max() + logit_error(S, S) + 2.0 ** -13


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", [1, 3, 20])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_any_softmax_scale(torch_cuda, kv, nq, scale):
    c = Cache([700, 200], nq, 1, 16, kv, seed=33)
    c.pb.softmax_scale = scale
    c.upload()
    c.decode()
    c.check_decode()
    w = c.torch.zeros((2, 1, c.pb.max_blocks * 128), device="cuda")
    c.accumulate(c.lse, None, w)
    check_weights(c, w, c.lse, None, 1.0, None, after=w)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", [1, 3, 20])
@pytest.mark.parametrize("e", [-100, -60, 60, 100])
def test_queries_far_outside_f16(torch_cuda, kv, nq, e):
    c = Cache([700, 200], nq, 1, 16, kv, seed=35)
    c.q = synth.f32_to_bf16_bits(np.ldexp(synth.bf16_bits_to_f32(c.q), e).astype(np.float32))
    c.pb.softmax_scale = float(np.ldexp(np.float32(0.0625), -e))
    c.upload()
    c.decode()
    c.check_decode()
    w = c.torch.zeros((2, 1, c.pb.max_blocks * 128), device="cuda")
    c.accumulate(c.lse, None, w)
    check_weights(c, w, c.lse, None, 1.0, None, after=w)


def test_many_requests_most_of_them_idle(torch_cuda):
    rng = np.random.default_rng(3)
    contexts = [int(x) for x in rng.integers(1, 300, 3000)]
    idle = tuple(int(x) for x in np.flatnonzero(rng.random(3000) < 0.9))
    c = Cache(contexts, 1, 1, 4, "fp8", seed=37, idle=idle)
    c.decode()
    c.check_decode()


def test_two_streams_at_once(torch_cuda):
    torch = torch_cuda
    a, b = Cache([9000, 3000], 4, 2, 16, seed=38), Cache([20000, 150], 1, 2, 16, "fp8", seed=39)
    for c in (a, b):
        c.w = torch.zeros((2, 2, c.pb.max_blocks * 128), device="cuda")
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.decode()
                c.accumulate(c.lse, None, c.w)
    torch.cuda.synchronize()
    for c in (a, b):
        c.check_decode()
        check_weights(c, c.w, c.lse, None, 1.0, None, after=c.w)


def test_two_host_threads_at_once(torch_cuda):
    # shapes with different shared-memory needs of one kernel instance
    import threading

    torch = torch_cuda
    a, b = Cache([3000, 500], 1, 1, 16, seed=44), Cache([3000, 500], 20, 1, 16, seed=45)
    want, failed = [], []
    for c in (a, b):
        c.decode()
        c.w = torch.zeros((2, 1, c.pb.max_blocks * 128), device="cuda")
        c.accumulate(c.lse, None, c.w)
        want.append(c.w.clone())
    torch.cuda.synchronize()

    def work(c, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    c.accumulate(c.lse, None, c.w)
                    c.decode()
            torch.cuda.synchronize()
            assert torch.equal(c.w, w)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip((a, b), want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for c in (a, b):
        c.check_decode()


def test_same_bits_each_time_and_on_another_stream(torch_cuda):
    c = Cache([5000, 70, 2222], 4, 2, 16, "fp8", seed=23)
    c.decode()
    first = c.out.clone(), c.lse.clone()
    c.torch.cuda.synchronize()
    s = c.torch.cuda.Stream()
    c.out.fill_(0)
    s.wait_stream(c.torch.cuda.current_stream())
    c.decode(stream=s)
    s.synchronize()
    assert c.torch.equal(first[0], c.out) and c.torch.equal(first[1], c.lse)


def test_captured_steps_follow_new_lengths(torch_cuda):
    # two graphs on one workspace, replayed in turn, after lengths and queries changed
    a, b = Cache([700, 1300], 1, 2, 16, seed=25), Cache([3000, 12], 4, 2, 16, seed=26)
    if b.nbytes < a.nbytes:
        a, b = b, a
    a.ws, a.nbytes = b.ws, b.nbytes
    wa = a.torch.zeros((2, 2, a.pb.max_blocks * 128), device="cuda")
    for c in (a, b):
        c.decode()
    a.torch.cuda.synchronize()
    graphs = []
    for c in (a, b):
        g = a.torch.cuda.CUDAGraph()
        with a.torch.cuda.graph(g):
            c.decode()
            if c is a:
                c.accumulate(c.lse, None, wa)
        graphs.append(g)
    for n in (0, 1):
        for c in (a, b):
            c.pb.seq_lens[0] -= n * 5
            c.lens.copy_(a.torch.from_numpy(c.pb.seq_lens))
            c.q = np.roll(c.q, 1, axis=1)
            c.dq.copy_(a.torch.from_numpy(c.q.view(np.int16)))
        for g in graphs + graphs[::-1]:
            g.replay()
        a.check_decode()
        b.check_decode()
        check_weights(a, wa, a.lse, None, 1.0, None, after=wa)


@pytest.mark.parametrize("kv", KV)
def test_bad_pages_and_lengths_are_reported(torch_cuda, kv):
    c = Cache([300, 400], 1, 1, 16, kv, seed=27)
    c.pb.block_table[0, 1] = c.pb.num_pages
    c.upload()
    w = c.torch.zeros((2, 1, c.pb.max_blocks * 128), device="cuda")
    for call in (c.decode, lambda: c.accumulate(c.lse, None, w)):
        call()
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK
        assert c.status() == msa.MSA_OK
    c = Cache([300, 400], 1, 1, 16, kv, seed=27)
    for bad in (-1, c.pb.max_blocks * 128 + 1, 2 ** 31 - 1):
        c.lens[1] = bad
        for call in (c.decode, lambda: c.accumulate(c.lse, None, w)):
            call()
            assert c.status() == msa.MSA_ERR_DEVICE_CHECK
    c.lens[1] = 400
    c.decode()
    c.check_decode()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", [1, 4, 24])
def test_a_wait_that_runs_out_is_reported(torch_cuda, kv, nq):
    # four CTAs with far more pages than their rings hold: a producer or its consumers wait
    c = Cache([20000, 3000], nq, 2, 16, kv, seed=29, ctas=4)
    w = c.torch.zeros((2, 2, c.pb.max_blocks * 128), device="cuda")
    c.decode()
    c.check_decode()
    msa.msa_set_decode_wait_limit(1)
    try:
        c.decode()
        assert c.status() == msa.MSA_ERR_TIMEOUT
        c.accumulate(c.lse, None, w)
        assert c.status() == msa.MSA_ERR_TIMEOUT
    finally:
        msa.msa_set_decode_wait_limit(0)
    c.decode()
    c.check_decode()


def test_page_offsets_beyond_32_bits(torch_cuda):
    # 75000 pages of 64 KiB; the request's pages are the last ones
    torch = torch_cuda
    c = Cache([700], 1, 1, 16, seed=31)
    pages = 75000
    pool = torch.zeros((pages, 2, 1, 128, 128), dtype=torch.int16, device="cuda")
    n = c.pb.num_pages
    pool[pages - n:] = c.kv
    c.kv = pool
    c.table += pages - n
    c.shape.num_pages = pages
    c.decode()
    c.check_decode()
    w = torch.zeros((1, 1, c.pb.max_blocks * 128), device="cuda")
    c.accumulate(c.lse, None, w)
    check_weights(c, w, c.lse, None, 1.0, None)


# ---------------------------------------------------------------------------
# accumulated weights

def check_weights(c, got, lse, before, decay, selected, after=None, extra=0.0):
    lse = lse.double().cpu().numpy()
    got = got.double().cpu().numpy()
    host = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
    want = ref.weights(c.pb, c.q, lse, host(before), decay, host(selected), after=got)
    _, _, S, _ = ref.dense_decode(c.pb, c.q)
    top = np.abs(lse[np.isfinite(lse)]).max(initial=0)
    rel = logit_error(S, S) + extra + 2.0 ** -22 + 2.0 ** -22 * (1 + top) + c.nq * c.G * 2.0 ** -24 + 2.0 ** -23
    # below 2^-126 the hardware exponential gives 0
    assert np.all(np.abs(got - want) <= rel * np.abs(want) + c.nq * c.G * 2.0 ** -126), np.abs(got - want).max()
    assert c.status() == msa.MSA_OK


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("contexts,nq,Hkv,G,decay", [
    ([1], 1, 1, 16, 1.0), ([127, 1290, 128], 1, 2, 16, 0.5), ([640, 77], 2, 2, 8, 1.0), ([900, 5], 5, 1, 3, 0.96875),
    ([513, 64], 64, 1, 16, 1.0), ([300], 1, 1, 1, 1.0), ([400, 70], 64, 2, 5, 0.0), ([200], 9, 1, 64, 2.0),
])
def test_weights_after_a_dense_step(torch_cuda, kv, contexts, nq, Hkv, G, decay):
    c = Cache(contexts, nq, Hkv, G, kv, seed=sum(contexts) + 3)
    c.decode()
    torch = c.torch
    shape = (len(contexts), Hkv, c.pb.max_blocks * 128)
    before = torch.rand(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    for w_in in (None, before):
        got = torch.full(shape, -3.0, device="cuda")
        c.accumulate(c.lse, w_in, got, decay)
        check_weights(c, got, c.lse, w_in, decay, None)
        for r, n in enumerate(contexts):
            assert bool((got[r, :, n:] == -3.0).all())
    same = before.clone()
    c.accumulate(c.lse, same, same, decay)
    for r, n in enumerate(contexts):
        assert torch.equal(same[r, :, :n], got[r, :, :n]) and torch.equal(same[r, :, n:], before[r, :, n:])
    if decay == 1.0:  # with no history the weights of a step sum to one per query row
        c.accumulate(c.lse, None, got)
        total = sum(float(got[r, :, :n].double().sum()) for r, n in enumerate(contexts))
        assert abs(total / (len(contexts) * nq * G * Hkv) - 1) < 1e-4


@pytest.mark.parametrize("nq", [1, 9])
def test_weights_of_queries_with_a_large_element_that_meets_zeros(torch_cuda, nq):
    # E4M3 keys take each query as an E4M3 pair, off by at most 2^-21.8 of the row's largest
    # element: as much as Sum |k| of that more in a logit (the others' elements are 2^-12 of it)
    c = Cache([700, 129 + nq], nq, 2, 16, "fp8", seed=47)
    c.pb.kv_pool[:, 0, :, :, 5] = 0
    c.q[..., 5] = synth.f32_to_bf16_bits(np.full(c.q.shape[:2], 4096.0, np.float32))
    c.upload()
    c.decode()
    got = c.torch.full((2, 2, c.pb.max_blocks * 128), -3.0, device="cuda")
    c.accumulate(c.lse, None, got)
    _, _, S, _ = ref.dense_decode(c.pb, synth.f32_to_bf16_bits(np.full(c.q.shape, 4096.0, np.float32)))
    check_weights(c, got, c.lse, None, 1.0, None, extra=2.0 ** -21.8 * np.max(S))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq,Hkv,Hi,topk", [(1, 2, 1, 1), (3, 2, 2, 4), (4, 4, 4, 16), (33, 1, 1, 7), (64, 2, 2, 5)])
def test_weights_after_a_sparse_step(torch_cuda, kv, nq, Hkv, Hi, topk):
    torch = torch_cuda
    contexts = [2500, 300, 1024, 64]
    c = Cache(contexts, nq, Hkv, 16, kv, seed=41 + nq, Hi=Hi)
    c.shape.topk = topk
    rng = np.random.default_rng(nq)
    Hs = 1 if Hi == 1 else Hkv
    sel = np.full((c.pb.num_tokens, Hs, topk), -1, np.int32)
    lse = np.zeros((c.pb.num_tokens, Hkv * 16), np.float32)
    for t in range(c.pb.num_tokens):
        nb = -(-(int(c.pb.seq_lens[t // nq]) + t % nq) // 128)
        for h in range(Hs):
            some = np.sort(rng.permutation(nb)[: rng.integers(0, topk + 1)])
            sel[t, h, : len(some)] = some
    for r, n in enumerate(contexts):
        for g in range(Hkv):
            s, _ = ref._logits(c.pb, c.q, r, g, n, sel)
            with np.errstate(divide="ignore"):
                m = np.maximum(s.max(-1), -1e30)
                lse[r * nq:(r + 1) * nq, g * 16:(g + 1) * 16] = np.log(np.exp(s - m[..., None]).sum(-1)) + m
    dsel, dlse = torch.from_numpy(sel).cuda(), torch.from_numpy(lse).cuda()
    before = torch.rand((4, Hkv, c.pb.max_blocks * 128), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    got = torch.full_like(before, -3.0)
    c.accumulate(dlse, before, got, 0.75, dsel)
    check_weights(c, got, dlse, before, 0.75, dsel)
    c.accumulate(dlse, None, got, 1.0, dsel)
    check_weights(c, got, dlse, None, 1.0, dsel)


def test_a_selected_block_that_no_token_sees_is_reported(torch_cuda):
    c = Cache([300], 2, 1, 16, seed=43)
    c.decode()
    w = c.torch.zeros((1, 1, c.pb.max_blocks * 128), device="cuda")
    for bad in (3, -2, 2 ** 31 - 1):
        sel = c.torch.tensor([[[0, 2, bad, -1]], [[0, 1, -1, -1]]], dtype=c.torch.int32, device="cuda")
        c.accumulate(c.lse, None, w, 1.0, sel)
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK


# ---------------------------------------------------------------------------
# eviction

def run_evict(c, keep, first, last, w, with_index=True, seed=0):
    torch, pb = c.torch, c.pb
    R, Hs, newB = pb.num_requests, 1 if c.Hi == 1 else c.Hkv, -(-keep // 128)
    used = set(pb.block_table[pb.block_table >= 0].tolist())
    free = np.array([p for p in range(pb.num_pages) if p not in used], np.int32)
    assert len(free) >= R * newB
    new_table = np.random.default_rng(seed).permutation(free)[: R * newB].reshape(R, newB).astype(np.int32)
    out = {"kept": torch.full((R, Hs, keep), -7, dtype=torch.int32, device="cuda"),
           "lens": torch.full((R,), -7, dtype=torch.int32, device="cuda"),
           "w": torch.full((R, c.Hkv, newB * 128), -7.0, device="cuda")}
    dw, dt = torch.from_numpy(w).cuda(), torch.from_numpy(new_table).cuda()
    msa.msa_cache_evict(c.shape, keep, first, last, dw, c.table, c.lens, dt, c.kv, c.idxk if with_index else None,
                        c.scales if with_index else None, out["w"], out["kept"], out["lens"], c.ws, c.nbytes)
    assert c.status() == msa.MSA_OK
    kept, lens = ref.evict_lists(pb.seq_lens, c.nq, w, Hs, keep, first, last)
    assert np.array_equal(out["kept"].cpu().numpy(), kept)
    assert np.array_equal(out["lens"].cpu().numpy(), lens)
    kv, idxk, scales, new_w = ref.evict(pb, kept, new_table, w, np.full(out["w"].shape, -7.0, np.float32), c.Hi if with_index else 0)
    got = lambda t, like: t.cpu().numpy().view(like.dtype)  # noqa: E731
    assert np.array_equal(got(c.kv, kv), kv)
    assert np.array_equal(got(c.idxk, idxk), idxk)
    if scales is not None:
        assert np.array_equal(got(c.scales, scales), scales)
    assert np.array_equal(out["w"].cpu().numpy(), new_w, equal_nan=True)
    return new_table, kept, lens, out


@pytest.mark.parametrize("kv,index", [("bf16", "bf16"), ("fp8", "nvfp4"), ("nvfp4", "nvfp4"), ("nvfp4", "bf16")])
@pytest.mark.parametrize("Hkv,Hi", [(1, 1), (4, 1), (2, 2), (2, 6)])
@pytest.mark.parametrize("keep,first,last", [(200, 4, 64), (1, 0, 0), (129, 0, 129), (640, 640, 0)])
def test_evict(torch_cuda, kv, index, Hkv, Hi, keep, first, last):
    contexts = [1500, 199, 128, 2049, 1]
    c = Cache(contexts, 1, Hkv, 16, kv, seed=51 + keep, extra_pages=5 * -(-keep // 128), Hi=Hi, index=index)
    w = np.random.default_rng(keep).random((5, Hkv, c.pb.max_blocks * 128)).astype(np.float32)
    run_evict(c, keep, first, last, w)


@pytest.mark.parametrize("values", ["zeros", "few", "wide", "negative", "nonfinite"])
@pytest.mark.parametrize("keep", [1, 77, 1000, 5003, 6000])
def test_evict_ranks_ties_and_odd_weights(torch_cuda, values, keep):
    contexts = [6000, 5003, 900, 37]
    c = Cache(contexts, 1, 2, 16, "fp8", seed=53, extra_pages=4 * -(-keep // 128), idle=(3,), Hi=1)
    rng = np.random.default_rng(7)
    shape = (4, 2, c.pb.max_blocks * 128)
    w = {"zeros": np.zeros(shape), "few": rng.integers(0, 3, shape) / 4, "wide": np.exp(rng.normal(size=shape) * 20),
         "negative": rng.normal(size=shape), "nonfinite": rng.normal(size=shape)}[values].astype(np.float32)
    if values == "zeros":
        w[rng.random(shape) < 0.5] = -0.0
    if values == "nonfinite":
        w[rng.random(shape) < 0.05] = np.nan
        w[rng.random(shape) < 0.05] = -np.nan
        w[rng.random(shape) < 0.05] = np.inf
        w[rng.random(shape) < 0.05] = -np.inf
    run_evict(c, keep, 0, 0, w)
    if keep > 20:
        c.upload()
        run_evict(c, keep, 3, 17, w, with_index=False)


def test_evict_of_more_positions_than_fit_in_shared_memory(torch_cuda):
    # 2600 blocks: slices of 41600 positions, beyond the keys a CTA holds
    n = 2600 * 128 - 3
    c = Cache([n, 400000 - n], 1, 1, 16, "nvfp4", seed=55, extra_pages=2 * 8)
    w = np.random.default_rng(8).integers(0, 50, (2, 1, c.pb.max_blocks * 128)).astype(np.float32)
    run_evict(c, 1000, 10, 100, w, with_index=False)


def test_evict_with_draft_tokens(torch_cuda):
    c = Cache([700, 150, 90], 4, 2, 16, seed=57, extra_pages=6)
    w = np.random.default_rng(9).random((3, 2, c.pb.max_blocks * 128)).astype(np.float32)
    _, kept, lens, _ = run_evict(c, 140, 2, 3, w)
    assert lens.tolist() == [137, 137, 87]
    assert kept[0, 0, -3:].tolist() == [697, 698, 699]


def test_evict_reports_bad_pages_and_writes_no_others(torch_cuda):
    c = Cache([700], 1, 1, 16, seed=59, extra_pages=4)
    torch = c.torch
    before = c.kv.clone()
    w = torch.rand((1, 1, c.pb.max_blocks * 128), device="cuda")
    kept = torch.empty((1, 1, 100), dtype=torch.int32, device="cuda")
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    for bad in (-1, c.pb.num_pages):
        table = torch.full((1, 1), bad, dtype=torch.int32, device="cuda")
        msa.msa_cache_evict(c.shape, 100, 0, 10, w, c.table, c.lens, table, c.kv, c.idxk, None, None, kept, lens, c.ws, c.nbytes)
        assert c.status() == msa.MSA_ERR_DEVICE_CHECK
    assert torch.equal(before, c.kv)


@pytest.mark.parametrize("as_int", [False, True])
def test_problem_methods_on_a_stream_beside_a_busy_one(torch_cuda, as_int):
    # what the methods allocate and fill belongs to the stream that is asked for
    from sparse_attention_decode_msa_gb300.runner import DeviceProblem

    torch = torch_cuda
    pb = synth.make_problem(name="side", contexts=[600, 301], q_per_req=1, num_kv_heads=2, topk=4, seed=62, num_pages=16)
    dp = DeviceProblem(pb)
    free = [p for p in range(pb.num_pages) if p not in set(pb.block_table[pb.block_table >= 0].tolist())]
    table = torch.tensor(free[:4], dtype=torch.int32, device="cuda").reshape(2, 2)
    w = torch.rand((2, 2, pb.max_blocks * 128), device="cuda")
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms on the current stream
    dp.dense_decode(stream)
    dp.weight_accumulate(w, w, stream=stream)
    new = dp.evict(w, table, keep=200, last=1, stream=stream)
    torch.cuda.synchronize()
    out, lse, S, V = ref.dense_decode(pb, pb.q)
    res = dp.results()
    check_attention(res["out"], res["lse"], out, lse, S, V, 700)
    kept = new["kept"].cpu().numpy()
    assert np.array_equal(kept, ref.evict_lists(pb.seq_lens, 1, w.cpu().numpy(), 1, 200, 0, 1)[0])
    got = np.take_along_axis(w.cpu().numpy(), np.broadcast_to(kept, (2, 2, 200)).astype(np.int64), 2)
    assert np.array_equal(new["weights"].cpu().numpy()[:, :, :200], got)
    assert msa.msa_check_device_status(dp.cache_ws) == msa.MSA_OK


@pytest.mark.parametrize("kv", KV)
def test_a_run_of_steps_with_eviction(torch_cuda, kv):
    """A cache is weighed by a prompt's last tokens, cut, and decoded on: update, attention, weights, each step."""
    from sparse_attention_decode_msa_gb300.runner import DeviceProblem

    torch = torch_cuda
    pb = synth.make_problem(name="run", contexts=[600, 301, 900], q_per_req=1, num_kv_heads=2, topk=4, kv_dtype=kv, seed=61, num_pages=32)
    if kv == "nvfp4":
        pb.k_scale, pb.v_scale = 0.75, 0.5
    dp = DeviceProblem(pb)
    w = torch.zeros((3, 2, pb.max_blocks * 128), device="cuda")
    want = np.zeros(w.shape)
    for step in range(4):
        dp.kv_update(synth.make_update(pb, seed=step))
        for name, a in dp.pools().items():
            setattr(pb, name, a)
        dp.dense_decode()
        dp.weight_accumulate(w, w, decay=0.875)
        out, lse, S, V = ref.dense_decode(pb, pb.q)
        res = dp.results()
        check_attention(res["out"], res["lse"], out, lse, S, V, 1000)
        want = ref.weights(pb, pb.q, lse, want, 0.875, after=want)
        seen = np.zeros(want.shape, bool)
        for r in range(3):
            seen[r, :, : pb.seq_lens[r]] = True
        got = w.cpu().numpy()
        assert np.allclose(got[seen], want[seen], rtol=(step + 1) * 2 * (logit_error(S, S) + 2.0 ** -19), atol=1e-12)
        if step == 1:
            free = [p for p in range(pb.num_pages) if p not in set(pb.block_table[pb.block_table >= 0].tolist())]
            table = np.array(free[: 3 * 3], np.int32).reshape(3, 3)
            new = dp.evict(w, torch.from_numpy(table).cuda(), keep=300, first=4, last=32)
            kept, lens = ref.evict_lists(pb.seq_lens, 1, got, 1, 300, 4, 32)
            assert np.array_equal(new["kept"].cpu().numpy(), kept) and np.array_equal(new["seq_lens"].cpu().numpy(), lens)
            short = np.zeros_like(want)
            short[:, :, :300] = np.take_along_axis(want, np.broadcast_to(kept, (3, 2, 300)).astype(np.int64), 2)
            want = short
            # the serving loop goes on with the new pages, lengths and weights
            w[:, :, : 3 * 128] = new["weights"]
            dp.block_table[:, :3] = torch.from_numpy(table).cuda()
            dp.seq_lens.copy_(new["seq_lens"])
            pb.block_table[:, :3], pb.seq_lens[:] = table, lens
            for name, a in dp.pools().items():
                setattr(pb, name, a)
        pb.seq_lens += 1
        dp.seq_lens += 1
    assert msa.msa_check_device_status(dp.cache_ws) == msa.MSA_OK
    assert msa.msa_check_device_status(dp.ws) == msa.MSA_OK
