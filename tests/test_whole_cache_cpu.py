"""Host side of the whole-cache operators: shapes, workspace sizes and refusals
(in a child process that sees no GPU), and pins of their 64-bit definitions."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import whole_cache as ref
from sparse_attention_decode_msa_gb300 import build, synth
from test_abi_cpu import statuses_without_a_gpu


@pytest.fixture(scope="module")
def lib():
    build.build()
    return msa.load()


def shape(**kw):
    base = dict(num_requests=8, q_per_req=4, num_kv_heads=4, num_pages=4096, max_blocks_per_seq=256, topk=16)
    base.update(kw)
    return msa.make_shape(**base)


@pytest.mark.parametrize("kw", [dict(num_q_heads=4), dict(num_q_heads=20), dict(num_q_heads=256), dict(topk=0), dict(topk=5000),
                                dict(init_blocks=50), dict(index_dim=64), dict(index_dtype=7), dict(kv_dtype="nvfp4"),
                                dict(q_per_req=64, num_requests=128), dict(num_requests=0),
                                dict(num_kv_heads=8192, num_pages=1, num_requests=1, max_blocks_per_seq=1)])
def test_shapes_that_are_taken(lib, kw):
    assert msa.msa_cache_workspace_bytes(shape(**kw)) > 256


@pytest.mark.parametrize("kw", [dict(head_dim=64), dict(page_size=64), dict(num_q_heads=6), dict(num_q_heads=260), dict(num_q_heads=0),
                                dict(q_per_req=0), dict(q_per_req=65), dict(num_requests=-1), dict(num_requests=8193, q_per_req=1),
                                dict(num_requests=4097, q_per_req=2), dict(max_blocks_per_seq=0), dict(max_blocks_per_seq=16385),
                                dict(num_pages=0), dict(kv_dtype=3), dict(softmax_scale=float("inf")), dict(decode_ctas=-1),
                                dict(decode_ctas=8193), dict(num_index_heads=0), dict(num_index_heads=6), dict(num_index_heads=68),
                                dict(num_pages=2 ** 31 // (2 * 4 * 144) + 1),
                                dict(num_kv_heads=8193, num_pages=1, num_requests=1, max_blocks_per_seq=1),
                                dict(num_requests=8192, q_per_req=1, max_blocks_per_seq=16384, num_kv_heads=64)])
def test_shapes_that_are_refused(lib, kw):
    s = shape(**kw)
    assert msa.msa_cache_workspace_bytes(s) == 0
    for name, args in (("msa_dense_decode", [None] * 7 + [0, None]),
                       ("msa_weight_accumulate", [None] * 6 + [1.0] + [None] * 3 + [0, None]),
                       ("msa_cache_evict", [100, 0, 10] + [None] * 11 + [0, None])):
        assert getattr(lib, name)(msa.ctypes.byref(s), *args) in (msa.MSA_ERR_INVALID_ARGUMENT, msa.MSA_ERR_UNSUPPORTED)


def test_workspace_grows_with_rows_and_ctas(lib):
    one = msa.msa_cache_workspace_bytes(shape(q_per_req=1))
    four = msa.msa_cache_workspace_bytes(shape(q_per_req=4))
    assert one >= 2 * 160 * 16 * 130 * 4 and four >= 2 * 160 * 64 * 130 * 4  # two partial slots a CTA
    assert msa.msa_cache_workspace_bytes(shape(decode_ctas=8)) < four


def test_buffers_are_checked_on_the_host(lib):
    got = statuses_without_a_gpu("""
s = shape()
n = msa.msa_cache_workspace_bytes(s)
def decode(args=None, ws=fake, nb=n):
    out.append(lib.msa_dense_decode(ctypes.byref(s), *(args or [fake] * 6), ws, nb, None))
decode(ws=None); decode(nb=n - 1); decode(ws=fake + 8)
for i in range(6):
    decode([None if k == i else fake for k in range(6)])
    decode([fake + 8 if k == i else fake for k in range(6)])
def weigh(a=None, decay=1.0, b=(fake, fake), sh=s):
    out.append(lib.msa_weight_accumulate(ctypes.byref(sh), *(a or [fake] * 6), decay, *b, fake, n, None))
for i in (0, 1, 2, 3, 5):
    weigh([None if k == i else fake for k in range(6)])
for i in range(6):
    weigh([fake + 4 if k == i else fake for k in range(6)])
weigh(decay=float("nan")); weigh(decay=float("inf")); weigh(b=(fake, None)); weigh(b=(fake + 4, fake)); weigh(b=(fake, fake + 4))
weigh(sh=shape(topk=0))
""")
    assert got == [msa.MSA_ERR_INVALID_ARGUMENT] * len(got)


def test_eviction_arguments_are_checked_on_the_host(lib):
    got = statuses_without_a_gpu("""
s = shape()
n = msa.msa_cache_workspace_bytes(s)
ptrs = [fake + 4096 * i for i in range(1, 11)]
def evict(keep=100, first=4, last=10, sh=s, **at):
    p = list(ptrs)
    for k, v in at.items():
        p[int(k[1:])] = v
    out.append(lib.msa_cache_evict(ctypes.byref(sh), keep, first, last, *p, fake, n, None))
evict(keep=0); evict(keep=-5); evict(keep=3); evict(first=-1); evict(last=2); evict(first=50, last=51)
evict(first=2**31 - 1, last=2**31 - 1)
for i in (0, 1, 2, 3, 4, 8, 9):
    evict(**{"p%d" % i: None})
for i in range(10):
    evict(**{"p%d" % i: fake + 8})
evict(p3=ptrs[1]); evict(p7=ptrs[0]); evict(p9=ptrs[2])
evict(sh=shape(index_dtype=2), p6=None)
evict(keep=2097153); evict(sh=shape(index_dim=64)); evict(sh=shape(index_dtype=1))
""")
    assert got == [msa.MSA_ERR_INVALID_ARGUMENT] * (len(got) - 3) + [msa.MSA_ERR_UNSUPPORTED] * 3


def test_no_requests_is_a_validated_no_op(lib):
    got = statuses_without_a_gpu("""
s = shape(num_requests=0)
n = msa.msa_cache_workspace_bytes(s)
p = [fake + 4096 * i for i in range(1, 11)]
out.append(lib.msa_dense_decode(ctypes.byref(s), *p[:6], fake, n, None))
out.append(lib.msa_weight_accumulate(ctypes.byref(s), *p[:6], 1.0, *p[:2], fake, n, None))
out.append(lib.msa_cache_evict(ctypes.byref(s), 100, 0, 10, *p, fake, n, None))
""")
    assert got == [msa.MSA_OK] * 3


def test_python_buffers_must_be_dense_cuda_tensors(lib):
    import torch

    with pytest.raises(ValueError):
        msa.msa_dense_decode(shape(), torch.zeros(4), *[0x10000] * 6, 1 << 30, 0)


# ---- pins of the definitions -------------------------------------------------

def test_definition_of_weights_sums_to_one_per_row():
    pb = synth.make_problem(name="pin", contexts=[200, 77], q_per_req=2, num_kv_heads=2, topk=2, kv_dtype="fp8", seed=3)
    out, lse, _, _ = ref.dense_decode(pb, pb.q)
    w = ref.weights(pb, pb.q, lse)
    assert np.allclose(w.sum(-1), 2 * 16)
    assert np.all(w[1, :, 77:] == 0)
    # the output is the weighted mean of the values: all-equal values come back
    pb.kv_pool[:, 1] = 0x38
    out, _, _, _ = ref.dense_decode(pb, pb.q)
    assert np.allclose(out, float(np.float32(pb.v_scale)))


def test_definition_of_the_kept_positions():
    w = np.array([[[5, 1, 3, 3, 0, 2, 9, 9]], [[1, 1, 1, 1, 1, 1, 1, 1]]], np.float32)
    kept, lens = ref.evict_lists(np.array([7, 3]), 1, w, 1, 4, 1, 1)
    assert kept.tolist() == [[[0, 2, 3, 6]], [[0, 1, 2, -1]]] and lens.tolist() == [4, 3]
    kept, _ = ref.evict_lists(np.array([8, 8]), 1, w, 1, 3, 0, 0)
    assert kept.tolist() == [[[0, 6, 7]], [[0, 1, 2]]]
    w[0, 0, 4] = np.nan
    assert ref.evict_lists(np.array([8, 8]), 1, w, 1, 2, 0, 1)[0][0, 0].tolist() == [4, 7]
