"""Sizes of the buffers of the calls on ragged batches: a tensor shorter than what the call reaches is
refused before the library sees its address.  (No GPU: the tensors are the host's, taken for device
ones, and the library is one that only counts its calls.)"""

import pytest
import torch

import sparse_attention_decode_msa_gb300 as msa
from sparse_attention_decode_msa_gb300 import buffers

T, R, HQ, HKV, HI, PAGES, BLOCKS, ROT = 6, 3, 8, 2, 2, 5, 4, 64


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append(name) or msa.MSA_OK

    monkeypatch.setattr(msa, "load", lambda: Library())
    monkeypatch.setattr(msa, "_bufs", buffers.bufs)
    monkeypatch.setattr(msa, "_check_rows", buffers.check_rows)
    monkeypatch.setattr(buffers, "_get_device", lambda x: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return seen


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def raw(n):
    return torch.zeros(n, dtype=torch.uint8)


def weight(heads, per_head):
    return bf16(heads, 128) if per_head else bf16(128)


def norm_rope(per_head=False, tokens=T, **kw):
    a = dict(freqs=torch.zeros(ROT // 2, dtype=torch.int64), positions=i32(T), q=bf16(T, HQ, 128), q_weight=weight(HQ, per_head), q_out=bf16(T, HQ, 128),
             k=bf16(T, HKV, 128), k_weight=weight(HKV, per_head), k_out=bf16(T, HKV, 128)) | kw
    rope = msa.make_rope(rotary_dim=ROT, per_head_weights=per_head)
    return a, lambda: msa.msa_qk_norm_rope(rope, a["freqs"], tokens, a["positions"], HQ, a["q"], a["q_weight"], a["q_out"], HKV, a["k"], a["k_weight"],
                                           a["k_out"], stream=0)


def append(per_head=False, kv="bf16", index="bf16", tokens=T, requests=R, **kw):
    page = 2 * HKV * {"bf16": 32768, "fp8": 16384, "nvfp4": 9216}[kv]
    a = dict(freqs=torch.zeros(ROT // 2, dtype=torch.int64), offsets=i32(R + 1), k=bf16(T, HKV, 128), k_weight=weight(HKV, per_head), v=bf16(T, HKV, 128),
             idxk=bf16(T, HI, 128), idxk_weight=weight(HI, per_head), q=bf16(T, HQ, 128), q_weight=weight(HQ, per_head), q_out=bf16(T, HQ, 128),
             q_idx=bf16(T, HI, 128), q_idx_weight=weight(HI, per_head), q_idx_out=bf16(T, HI, 128), block_table=i32(R, BLOCKS), seq_lens=i32(R),
             kv_pool=raw(PAGES * page), idxk_pool=raw(PAGES * HI * (32768 if index == "bf16" else 8192)), idxk_scales=raw(PAGES * HI * 1024), workspace=raw(512)) | kw
    if index == "bf16" and "idxk_scales" not in kw:
        a["idxk_scales"] = None
    shape = msa.make_shape(num_requests=requests, q_per_req=1, num_kv_heads=HKV, num_q_heads=HQ, num_pages=PAGES, max_blocks_per_seq=BLOCKS, topk=1, kv_dtype=kv,
                           index_dtype=index, num_index_heads=HI)
    rope = msa.make_rope(rotary_dim=ROT, per_head_weights=per_head)
    names = list(a)
    return a, lambda: msa.msa_kv_append(shape, rope, a["freqs"], tokens, *[a[n] for n in names[1:]], 512, stream=0)


def attention(kv="bf16", tokens=T, requests=R, **kw):
    page = 2 * HKV * {"bf16": 32768, "fp8": 16384, "nvfp4": 9216}[kv]
    a = dict(q=bf16(T, HQ, 128), offsets=i32(R + 1), kv_pool=raw(PAGES * page), block_table=i32(R, BLOCKS), seq_lens=i32(R), out=bf16(T, HQ, 128),
             lse=torch.zeros(T, HQ), workspace=raw(512)) | kw
    shape = msa.make_shape(num_requests=requests, q_per_req=1, num_kv_heads=HKV, num_q_heads=HQ, num_pages=PAGES, max_blocks_per_seq=BLOCKS, topk=1, kv_dtype=kv)
    return a, lambda: msa.msa_ragged_attention(shape, tokens, True, *a.values(), 512, stream=0)


CALLS = [(norm_rope, {}), (norm_rope, dict(per_head=True)), (append, {}), (append, dict(per_head=True, kv="fp8", index="nvfp4")), (append, dict(kv="nvfp4")),
         (attention, {}), (attention, dict(kv="fp8")), (attention, dict(kv="nvfp4"))]


@pytest.mark.parametrize("call,kw", CALLS)
def test_buffers_that_are_just_long_enough_are_taken(calls, call, kw):
    call(**kw)[1]()
    assert len(calls) == 1


@pytest.mark.parametrize("call,kw", CALLS)
def test_a_buffer_that_is_one_element_short_is_refused(calls, call, kw):
    whole = call(**kw)[0]
    rows = ("k", "v", "idxk", "q", "q_idx") if call is not attention else ()
    for name, x in whole.items():
        if x is None:
            continue
        short = x[:-1] if name in rows else x.reshape(-1)[:-1]
        with pytest.raises(ValueError, match="the call takes"):
            call(**kw, **{name: short})[1]()
    assert calls == []


def test_weights_for_all_heads_are_not_weights_a_head(calls):
    for call, name in ((norm_rope, "q_weight"), (norm_rope, "k_weight"), (append, "k_weight"), (append, "q_idx_weight")):
        with pytest.raises(ValueError, match="buffer of 256 bytes"):
            call(per_head=True, **{name: bf16(128)})[1]()


def test_more_tokens_than_the_tensors_have_are_refused(calls):
    for call in (norm_rope, append, attention):
        with pytest.raises(ValueError, match="the call takes"):
            call(tokens=T + 1)[1]()
    assert calls == []


def test_calls_that_look_at_nothing_take_anything(calls):
    none = bf16(0, 128, 128)
    norm_rope(tokens=0, q_out=none, positions=i32(0))[1]()
    append(tokens=0, q_out=none, kv_pool=raw(0))[1]()
    append(requests=0, block_table=i32(0), kv_pool=raw(0))[1]()
    attention(tokens=0, kv_pool=raw(0))[1]()
    attention(requests=0, block_table=i32(0))[1]()
    assert len(calls) == 5
    # index pools without index keys are not looked at
    append(idxk=None, idxk_weight=None, idxk_pool=raw(0))[1]()
    assert len(calls) == 6
