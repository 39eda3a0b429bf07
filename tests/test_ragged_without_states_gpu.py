"""Requests without states among a ragged batch's: outputs of 0 and lse -inf, for one of them with
many tokens or for many of them, in about the time that writing takes."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from test_ragged_attention_gpu import KV, Ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("ctas", [0, 1, 2, 9])
def test_a_long_request_without_states(torch_cuda, kv, ctas):
    c = Ragged([700, 3, 41], [0, 300, 0], False, 2, 5, kv, seed=2, ctas=ctas, behind=3)
    c.run().check()


@pytest.mark.parametrize("R", [70, 1500])
@pytest.mark.parametrize("ctas", [0, 1])
def test_many_requests_without_states(torch_cuda, R, ctas):
    rng = np.random.default_rng(R)
    counts, lens = rng.integers(0, 4, R), rng.integers(0, 3, R) * rng.integers(1, 90, R)
    assert np.any((lens == 0) & (counts > 0)) and np.any((lens > 0) & (counts > 0))
    Ragged(counts.tolist(), lens.tolist(), False, 1, 3, seed=R, ctas=ctas, behind=1).run().check()


def test_a_batch_of_one_short_request_without_states(torch_cuda):
    Ragged([5], [0], False, 1, 2, seed=1).run().check()


@pytest.mark.parametrize("kv", KV)
def test_the_table_need_not_hold_tokens_that_see_nothing(torch_cuda, kv):
    c = Ragged([300, 2], [0, 100], True, 1, 4, kv, seed=6)
    assert c.pb.max_blocks == 1
    c.run().check()


def test_writing_them_takes_the_time_of_writing(torch_cuda):
    # 4096 tokens of 64 heads (67 MB) beside a short request: one warp takes 50 times as long as a fill does
    torch = torch_cuda
    c = Ragged([4096, 7], [0, 200], False, 4, 16, seed=3)

    def us(f):
        for _ in range(3):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(20):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 50

    fill = us(lambda: c.out.zero_())
    assert us(c.run) < 10 * fill + 50
    assert c.status() == msa.MSA_OK
    out, lse = c.result()
    assert not np.any(out[:4096]) and np.all(np.isneginf(lse[:4096])) and np.all(np.isfinite(lse[4096:]))
