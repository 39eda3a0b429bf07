"""Element types of the whole-cache operators' tensors: what the bindings refuse, and what
DeviceProblem allocates (no GPU: nothing is launched)."""

import pytest

import sparse_attention_decode_msa_gb300 as msa
from sparse_attention_decode_msa_gb300 import build

CALLS = {  # argument kinds: h bf16 rows, i int32, f fp32, b bytes
    "msa_dense_decode": ((), "hbiihfb", ()),
    "msa_weight_accumulate": ((), "hbiiif1ffb", ()),
    "msa_cache_evict": ((4, 0, 0), "fiiibbbfiib", ()),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return msa.load()


def shape():
    return msa.make_shape(num_requests=8, q_per_req=1, num_kv_heads=4, num_pages=64, max_blocks_per_seq=4, topk=4)


def cases():
    wrong = {"h": ("float16", "float32", "uint8"), "i": ("int64", "int16", "float32"), "f": ("float64", "float16", "bfloat16", "int32")}
    for name, (_, kinds, _) in CALLS.items():
        for i, k in enumerate(kinds):
            for dtype in wrong.get(k, ()):
                yield name, i, dtype


@pytest.mark.parametrize("name,i,dtype", list(cases()))
def test_other_element_types_are_refused(name, i, dtype):
    import torch

    lead, kinds, _ = CALLS[name]
    args = [1.0 if k == "1" else 0x10000 for k in kinds]
    args[i] = torch.zeros(64, dtype=getattr(torch, dtype))
    with pytest.raises(ValueError, match=f"buffer of torch.{dtype}: the argument takes torch."):
        getattr(msa, name)(shape(), *lead, *args, 1 << 30, stream=0)


@pytest.mark.parametrize("name", list(CALLS))
def test_the_right_types_pass_on_to_the_check_of_the_device(name):
    import torch

    right = {"h": (torch.bfloat16, torch.int16), "i": (torch.int32,), "f": (torch.float32,), "b": (torch.uint8, torch.bfloat16)}
    lead, kinds, _ = CALLS[name]
    for i, k in enumerate(kinds):
        for dtype in right.get(k, ()):
            args = [1.0 if k == "1" else 0x10000 for k in kinds]
            args[i] = torch.zeros(64, dtype=dtype)
            with pytest.raises(ValueError, match="not on the current CUDA device"):
                getattr(msa, name)(shape(), *lead, *args, 1 << 30, stream=0)


def test_buffers_are_fp32_whatever_the_default_type_is(monkeypatch):
    # the kernels write fp32: a buffer of 16-bit elements would be half as long as what they write
    import torch

    from sparse_attention_decode_msa_gb300 import runner, synth

    monkeypatch.setattr(runner, "msa_workspace_init", lambda *a: None)
    monkeypatch.setattr(runner, "msa_cache_evict", lambda *a: None)
    monkeypatch.setattr(runner.DeviceProblem, "_cache_workspace", lambda self: (None, 0, 0))
    pb = synth.make_problem(name="types", contexts=[300], q_per_req=1, num_kv_heads=1, topk=2)
    before = torch.get_default_dtype()
    try:
        for dtype in (torch.float16, torch.float64):
            torch.set_default_dtype(dtype)
            dp = runner.DeviceProblem(pb, device="cpu")
            assert dp.lse.dtype == dp.block_scores.dtype == torch.float32 and dp.out.dtype == torch.bfloat16
            assert dp.evict(None, None, keep=5)["weights"].dtype == torch.float32
    finally:
        torch.set_default_dtype(before)
