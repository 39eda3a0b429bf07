"""Host side of the calls on ragged batches: shapes, workspace sizes and refusals (in a child
process that sees no GPU), the frequencies' table, what the bindings refuse, and pins of the
64-bit definitions."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import ragged as ref
from oracle.whole_cache import bf16, e4m3
from sparse_attention_decode_msa_gb300 import build, synth
from test_abi_cpu import statuses_without_a_gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return msa.load()


def shape(**kw):
    base = dict(num_requests=8, q_per_req=1, num_kv_heads=4, num_pages=4096, max_blocks_per_seq=256, topk=1)
    base.update(kw)
    return msa.make_shape(**base)


@pytest.mark.parametrize("kw", [dict(num_q_heads=4), dict(num_q_heads=20), dict(num_q_heads=256), dict(topk=0), dict(q_per_req=0), dict(q_per_req=999),
                                dict(init_blocks=50), dict(kv_dtype="nvfp4"), dict(num_requests=0), dict(num_requests=8192), dict(num_index_heads=3)])
def test_shapes_that_are_taken(kw):
    assert msa.msa_ragged_workspace_bytes(shape(**kw)) > 256


@pytest.mark.parametrize("kw", [dict(head_dim=64), dict(page_size=64), dict(num_q_heads=6), dict(num_q_heads=260), dict(num_q_heads=0), dict(num_requests=-1),
                                dict(num_requests=8193), dict(max_blocks_per_seq=0), dict(max_blocks_per_seq=16385), dict(num_pages=0), dict(kv_dtype=3),
                                dict(softmax_scale=float("inf")), dict(k_scale=float("nan")), dict(decode_ctas=-1), dict(decode_ctas=8193),
                                dict(num_index_heads=0), dict(num_index_heads=65), dict(num_pages=2 ** 31 // (2 * 4 * 144) + 1),
                                dict(num_kv_heads=8193, num_pages=1)])
def test_shapes_that_are_refused(lib, kw):
    s = shape(**kw)
    assert msa.msa_ragged_workspace_bytes(s) == 0
    r = msa.make_rope(rotary_dim=0)
    bad = (msa.MSA_ERR_INVALID_ARGUMENT, msa.MSA_ERR_UNSUPPORTED)
    assert lib.msa_kv_append(msa.ctypes.byref(s), msa.ctypes.byref(r), None, 1, *[None] * 18, 0, None) in bad
    assert lib.msa_ragged_attention(msa.ctypes.byref(s), 1, 0, *[None] * 8, 0, None) in bad


def test_workspace_has_two_slots_a_cta():
    slot = 256 * 130 * 4
    assert msa.msa_ragged_workspace_bytes(shape()) >= 2 * 160 * slot
    assert 2 * 3 * slot <= msa.msa_ragged_workspace_bytes(shape(decode_ctas=3)) < 2 * 4 * slot


def test_attention_arguments_are_checked_on_the_host():
    got = statuses_without_a_gpu("""
s = shape(q_per_req=1)
n = msa.msa_ragged_workspace_bytes(s)
def attend(tokens=4, p=None, ws=fake, nb=n, sh=s):
    out.append(lib.msa_ragged_attention(ctypes.byref(sh), tokens, 1, *(p or [fake] * 7), ws, nb, None))
attend(ws=None); attend(nb=n - 1); attend(ws=fake + 8); attend(tokens=-1)
for i in range(7):
    attend(p=[None if k == i else fake for k in range(7)])
    attend(p=[fake + 8 if k == i else fake for k in range(7)])
attend(tokens=4194305); attend(tokens=4194304, sh=shape(num_requests=8192, q_per_req=1, max_blocks_per_seq=16384, decode_ctas=1))
attend(tokens=0, p=[None] * 7, ws=None, nb=0); attend(sh=shape(num_requests=0, q_per_req=1), p=[None] * 7, ws=None, nb=0)
""")
    assert got == [msa.MSA_ERR_INVALID_ARGUMENT] * 18 + [msa.MSA_ERR_UNSUPPORTED] * 2 + [msa.MSA_OK] * 2


def test_append_arguments_are_checked_on_the_host():
    got = statuses_without_a_gpu("""
s, r = shape(q_per_req=1), msa.make_rope(rotary_dim=64)
names = "offsets k k_weight v idxk idxk_weight q q_weight q_out q_idx q_idx_weight q_idx_out table lens pool idx_pool idx_scales ws".split()
def append(tokens=4, sh=s, rope=r, freqs=fake, nb=256, **kw):
    p = {n: fake + 4096 * i for i, n in enumerate(names)} | kw
    out.append(lib.msa_kv_append(ctypes.byref(sh), ctypes.byref(rope), freqs, tokens, *p.values(), nb, None))
def split():
    out.append(-1)
for n in "offsets k v table lens pool ws".split():
    append(**{n: None})
for n in names:
    append(**{n: fake + 8})
append(nb=255); append(tokens=-1); append(freqs=None); append(freqs=fake + 4)
append(q_out=None); append(q=None); append(q_idx=None); append(q_idx_out=None); append(idx_pool=None); append(sh=shape(index_dtype=2), idx_scales=None)
append(rope=msa.make_rope(rotary_dim=64, k_stride=508)); append(rope=msa.make_rope(rotary_dim=64, k_stride=504)); append(rope=msa.make_rope(rotary_dim=64, v_stride=-512))
append(rope=msa.make_rope(rotary_dim=64, q_stride=9000), q_out=fake + 4096 * 6)
append(rope=msa.make_rope(rotary_dim=-16)); append(rope=msa.make_rope(scale=float("inf"))); append(rope=msa.make_rope(norm_eps=-1.0))
append(rope=msa.make_rope(norm_eps=float("nan"))); append(rope=msa.make_rope(norm_offset=float("inf")))
split()
append(rope=msa.make_rope(rotary_dim=144)); append(rope=msa.make_rope(rotary_dim=24)); append(tokens=4194305); append(sh=shape(index_dim=64))
append(sh=shape(index_dtype=1))
split()
append(tokens=0, k=None, v=None, ws=None); append(sh=shape(num_requests=0, q_per_req=1), offsets=None)
""")
    a, b = [i for i, x in enumerate(got) if x == -1]
    assert set(got[:a]) == {msa.MSA_ERR_INVALID_ARGUMENT} and set(got[a + 1:b]) == {msa.MSA_ERR_UNSUPPORTED} and set(got[b + 1:]) == {msa.MSA_OK}


def test_norm_and_rotation_arguments_are_checked_on_the_host():
    got = statuses_without_a_gpu("""
r = msa.make_rope()
def turn(tokens=4, pos=fake, Hq=8, q=fake, w=None, qo=fake + 65536, Hk=2, k=fake + 4096, kw=None, ko=fake + 131072, rope=r, freqs=fake):
    out.append(lib.msa_qk_norm_rope(ctypes.byref(rope), freqs, tokens, pos, Hq, q, w, qo, Hk, k, kw, ko, None))
turn(pos=None); turn(pos=fake + 4); turn(q=None); turn(q=fake + 2); turn(qo=None); turn(w=fake + 2); turn(k=None); turn(ko=None); turn(ko=fake + 131080)
turn(Hq=0); turn(Hk=-1); turn(Hk=0); turn(tokens=-1); turn(freqs=None); turn(rope=msa.make_rope(q_stride=512)); turn(rope=msa.make_rope(q_stride=2048), qo=fake)
out.append(-1)
turn(Hq=8193); turn(Hk=8193); turn(tokens=4194305); turn(rope=msa.make_rope(rotary_dim=129))
out.append(-1)
turn(tokens=0, pos=None, q=None, qo=None, k=None, ko=None); turn(tokens=0, Hk=0, k=None, ko=None)
""")
    a, b = [i for i, x in enumerate(got) if x == -1]
    assert set(got[:a]) == {msa.MSA_ERR_INVALID_ARGUMENT} and set(got[a + 1:b]) == {msa.MSA_ERR_UNSUPPORTED} and set(got[b + 1:]) == {msa.MSA_OK}


# ---- the frequencies' table ----------------------------------------------------

def test_frequencies_are_fractions_of_a_turn():
    two_pi = 2 * np.pi
    got = msa.rope_frequencies([0.0, two_pi / 4, two_pi / 2, two_pi, 3 * two_pi / 4, -two_pi / 4, 1.0, 1e-9, -1e-30]).numpy().astype(np.uint64)
    turns = got.astype(np.float64) / 2.0 ** 64
    want = np.array([0, 0.25, 0.5, 0, 0.75, 0.75, 1 / two_pi, 1e-9 / two_pi, 0])
    assert np.abs((turns - want + 0.5) % 1 - 0.5).max() <= 2.0 ** -53
    assert msa.rope_frequencies([]).numel() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf"), 2 * np.pi * 2.0 ** 31])
def test_frequencies_that_are_refused(bad):
    with pytest.raises(msa.MsaError):
        msa.rope_frequencies([1.0, bad])


def test_frequencies_need_arrays(lib):
    assert lib.msa_rope_frequencies(None, 1, None) == msa.MSA_ERR_INVALID_ARGUMENT
    assert lib.msa_rope_frequencies(None, -1, None) == msa.MSA_ERR_INVALID_ARGUMENT
    assert lib.msa_rope_frequencies(None, 0, None) == msa.MSA_OK


# ---- bindings --------------------------------------------------------------------

def test_bindings_refuse_rows_that_lie_otherwise():
    import torch

    from sparse_attention_decode_msa_gb300.buffers import check_rows

    x = torch.zeros((6, 9, 128), dtype=torch.bfloat16)
    check_rows(x, 0, 9)
    check_rows(x.reshape(6, -1), 0, 9)
    check_rows(x[:, 2:6], 9 * 128, 4)
    check_rows(x[:1, 2:6], 777, 4)  # one token: no stride to speak of
    for bad, stride, heads in ((x, 0, 8), (x[:, 2:6], 0, 4), (x[:, ::2], 9 * 128, 5), (x[..., :64], 9 * 128, 9), (x.transpose(0, 1), 0, 6), (x[::2], 9 * 128, 9)):
        with pytest.raises(ValueError):
            check_rows(bad, stride, heads)


def test_bindings_refuse_other_element_types():
    import torch

    r, fake = msa.make_rope(), 0x10000
    kinds = "giRhhRhh"
    wrong = {"g": ("float64", "int32"), "i": ("int64", "float32"), "R": ("float16", "float32", "uint8"), "h": ("float32", "float16")}
    for i, k in enumerate(kinds):
        for dtype in wrong[k]:
            args = [fake] * 8
            args[i] = torch.zeros((1, 4, 128), dtype=getattr(torch, dtype))
            f, pos, q, qw, qo, kk, kw, ko = args
            with pytest.raises(ValueError, match="the argument takes torch."):
                msa.msa_qk_norm_rope(r, f, 1, pos, 4, q, qw, qo, 4, kk, kw, ko, stream=0)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        msa.msa_qk_norm_rope(r, fake, 1, fake, 4, torch.zeros((1, 4, 128), dtype=torch.bfloat16), None, fake, stream=0)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        msa.msa_kv_append(shape(), r, fake, 1, fake, fake, None, torch.zeros((1, 4, 128), dtype=torch.bfloat16), *[None] * 8, fake, fake, fake, None, None,
                          fake, 256, stream=0)
    with pytest.raises(ValueError, match="contiguous|not on the current"):
        msa.msa_ragged_attention(shape(), 1, True, torch.zeros((1, 128, 64), dtype=torch.bfloat16)[:, ::2], *[fake] * 7, 1 << 30, stream=0)


# ---- pins of the definitions -------------------------------------------------------

def test_definition_of_the_rotation():
    x = np.zeros((1, 1, 128), np.uint16)
    x[0, 0, 0] = 0x3F80  # 1
    y, _ = ref.turned(x, None, [3], [np.pi / 6], 2)
    assert np.allclose(y[0, 0, :3], [0, 1, 0])  # a quarter turn: (1, 0) -> (0, 1), the pair (0, 1) of rotary_dim 2
    x[0, 0, 1] = 0x4000  # 2
    y, _ = ref.turned(x, None, [1], np.zeros(64), 128)
    assert np.allclose(y, bf16(x))
    y, _ = ref.turned(x, None, [1], [np.pi] + [0] * 63, 128, interleaved=True, scale=2.0)
    assert np.allclose(y[0, 0, :2], [-2, -4])
    w = np.full(128, 0x3F00, np.uint16)  # 1/2
    y, _ = ref.turned(x, w, [0], [], 0, eps=0.0, offset=1.0)
    assert np.allclose(y[0, 0, :2], np.array([1, 2]) * 1.5 / np.sqrt(5 / 128))


def test_definition_of_the_codes():
    x = np.array([0, 1, -1, 1.0625, 1.1875, 500, -500, 1e-9, -2.0 ** -10, 3 * 2.0 ** -10])
    assert e4m3(ref.to_codes(x, ref.E4M3_VALUES)).tolist() == [0, 1, -1, 1, 1.25, 448, -448, 0, 0, 2.0 ** -8]
    assert ref.to_codes(np.array([-1e-9]), ref.E4M3_VALUES)[0] == 0
    assert ref.to_codes(np.array([0.25, 0.75, 2.5, 5, 7, -0.3]), ref.E2M1_VALUES).tolist() == [0, 2, 4, 6, 7, 9]


def test_definition_of_the_places():
    req, pos = ref.places([0, 2, 2, 5], [10, 3, 1], 6)
    assert req.tolist() == [0, 0, 2, 2, 2, -1] and pos.tolist() == [9, 10, 0, 1, 2, -1]


def test_definition_of_ragged_attention():
    # a causal batch of one token a request is what the dense decode's definition says
    from oracle import whole_cache

    pb = synth.make_problem(name="pin", contexts=[200, 77], q_per_req=1, num_kv_heads=2, topk=2, kv_dtype="fp8", seed=3)
    a = whole_cache.dense_decode(pb, pb.q)
    for causal in (True, False):
        b = ref.attention(pb, pb.q, [0, 1, 2], pb.seq_lens, causal)
        assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    # causal: the second token sees one position more, and equal values come back as they are
    pb.kv_pool[:, 1] = 0x38
    q = np.concatenate([pb.q, pb.q])
    out, lse, far, _, _ = ref.attention(pb, q, [0, 3, 4], np.array([150, 0]), True)
    assert np.allclose(out[:3], float(np.float32(pb.v_scale))) and np.all(far[:3] < 1e-12)
    assert np.all(out[3] == 0) and np.all(np.isneginf(lse[3]))
