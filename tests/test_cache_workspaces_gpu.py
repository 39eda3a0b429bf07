"""DeviceProblem's whole-cache methods on several streams and in graphs: their workspaces on the GPU."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import whole_cache as ref
from sparse_attention_decode_msa_gb300 import synth
from test_whole_cache_gpu import check_attention

pytestmark = pytest.mark.gpu


def a_problem(nq=1, seed=81):
    from sparse_attention_decode_msa_gb300.runner import DeviceProblem

    pb = synth.make_problem(name="ws", contexts=[3000, 700, 129 + nq], q_per_req=nq, num_kv_heads=2, topk=4, seed=seed, num_pages=48)
    return pb, DeviceProblem(pb)


def check(pb, dp):
    out, lse, S, V = ref.dense_decode(pb, pb.q)
    res = dp.results()
    check_attention(res["out"], res["lse"], out, lse, S, V, 3001)


def test_an_error_on_one_stream_while_another_makes_its_first_call(torch_cuda):
    torch = torch_cuda
    pb, dp = a_problem()
    w = torch.rand((3, 2, pb.max_blocks * 128), device="cuda")
    bad = torch.full((3, 1), pb.num_pages, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(200_000_000)  # a tenth of a second: what a clears lands after b's call
    dp.dense_decode(stream=a)
    of_a = dp.cache_ws
    dp.evict(w, bad, keep=100, stream=b)
    of_b = dp.cache_ws
    torch.cuda.synchronize()
    assert msa.msa_check_device_status(of_b) == msa.MSA_ERR_DEVICE_CHECK
    assert msa.msa_check_device_status(of_a) == msa.MSA_OK
    check(pb, dp)


@pytest.mark.parametrize("nq", [1, 5])
def test_two_streams_with_outputs_of_their_own(torch_cuda, nq):
    torch = torch_cuda
    pb, dp = a_problem(nq)
    first, second = (dp.out, dp.lse), (torch.full_like(dp.out, -1), torch.full_like(dp.lse, -1))
    q, other = dp.q, dp.q.flip(1).contiguous()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(50):
        dp.q, (dp.out, dp.lse) = q, first
        dp.dense_decode(stream=a)
        dp.q, (dp.out, dp.lse) = other, second
        dp.dense_decode(stream=b)
    torch.cuda.synchronize()
    for qq, (dp.out, dp.lse) in ((pb.q, first), (np.ascontiguousarray(pb.q[:, ::-1]), second)):
        out, lse, S, V = ref.dense_decode(pb, qq)
        res = dp.results()
        check_attention(res["out"], res["lse"], out, lse, S, V, 3001)


@pytest.mark.parametrize("before", [True, False])
def test_a_graph_outlives_a_larger_workspace(torch_cuda, before):
    torch = torch_cuda
    pb, dp = a_problem(3)
    if before:
        dp.dense_decode()
        torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dp.dense_decode()
    captured = dp.cache_ws
    dp.set_decode_ctas(700)
    dp.dense_decode()
    assert dp.cache_ws.data_ptr() != captured.data_ptr() and dp.cache_ws.numel() > captured.numel()
    torch.cuda.synchronize()
    size, held = captured.numel(), [t.data_ptr() for t in (captured, dp.cache_ws)]
    del captured
    others = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not {t.data_ptr() for t in others} & set(held)
    dp.out.fill_(float("nan"))
    g.replay()
    check(pb, dp)
    assert all(bool((t == 77).all()) for t in others)
    dp.dense_decode()
    check(pb, dp)
    assert msa.msa_check_device_status(dp.cache_ws) == msa.MSA_OK


def test_two_graphs_captured_before_any_call(torch_cuda):
    torch = torch_cuda
    pb, dp = a_problem(2)
    graphs, words = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dp.dense_decode()
        graphs.append(g)
        words.append(dp.cache_ws)
    for g, ws in list(zip(graphs, words))[::-1]:  # the later one first
        dp.out.fill_(float("nan"))
        g.replay()
        check(pb, dp)
        assert msa.msa_check_device_status(ws) == msa.MSA_OK
    assert words[0].data_ptr() != words[1].data_ptr()
