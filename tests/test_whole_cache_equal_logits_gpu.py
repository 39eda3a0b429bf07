"""Dense decode where many positions have (nearly) the same logit: what rounds does so the same way
for all of them, so no error may count on averaging out.

The oracle of tests/test_whole_cache_gpu.py; tolerances from the worst case of every rounding.  With values
that are all 1 the output is 1 but for P (a bf16 pair: 2^-16 of it; fp16: 2^-11), the exponentials (2 (d + 2^-22),
d the error of a logit) and the sums (n 2^-23), together far under the 2^-9 below 1 that still stores 1: it is 1.
"""

import numpy as np
import pytest

from oracle import whole_cache as ref
from sparse_attention_decode_msa_gb300 import synth
from test_whole_cache_gpu import Cache, logit_error

pytestmark = pytest.mark.gpu

KV = ["bf16", "fp8", "nvfp4"]
ONE = {"bf16": 0x3F80, "fp8": 0x38}
ROWS = [1, 3, 6, 20]  # tokens of 16 heads: 16, 48, 96 and 320 query rows


def a_cache(kv, nq, contexts=(3000, 700), ctas=1):
    """Queries that start with 1, keys of zeros, values of ones, in long shares (few CTAs)."""
    c = Cache(list(contexts), nq, 1, 16, kv, seed=71 + nq, ctas=ctas)
    c.pb.k_scale = c.pb.v_scale = 1.0
    c.q[..., 0] = ONE["bf16"]
    c.pb.kv_pool[:, 0] = 0
    if kv == "nvfp4":
        c.pb.kv_pool[:, 1, :, :8192] = 0x22
        c.pb.kv_pool[:, :, :, 8192:] = 0x38
    else:
        c.pb.kv_pool[:, 1] = ONE[kv]
    return c


def set_first_dim(c, kv, which, r, at, value):
    """Dimension 0 of positions `at` of request r: `value`, 0 or 1."""
    page, row = c.pb.block_table[r, at // 128], at % 128
    if kv == "nvfp4":
        byte = c.pb.kv_pool[page, which, 0, row * 64]
        c.pb.kv_pool[page, which, 0, row * 64] = (byte & 0xF0) | (2 if value else 0)
    else:
        c.pb.kv_pool[page, which, 0, row, 0] = ONE[kv] if value else 0


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", ROWS)
@pytest.mark.parametrize("behind", [64, 128, 700])
def test_repeated_keys_behind_lower_ones(torch_cuda, kv, nq, behind):
    # logits 0, then 127 2^-15: exp of it is 1.00388, just below the middle of the bf16 numbers 1 and 1 + 2^-7
    c = a_cache(kv, nq)
    c.pb.softmax_scale = 127 * 2.0 ** -15
    for r in range(2):
        n = int(c.pb.seq_lens[r]) + nq - 1
        set_first_dim(c, kv, 0, r, np.arange(behind, n), 1)
    c.upload()
    c.decode()
    out, _ = c.check_decode()
    assert np.all(out == 1.0)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq", ROWS)
@pytest.mark.parametrize("scale", [2.0 ** -18, 2.0 ** -14, 2.0 ** -10])
def test_attention_close_to_uniform(torch_cuda, kv, nq, scale):
    c = a_cache(kv, nq, ctas=3)
    keys = Cache([3000, 700], nq, 1, 16, kv, seed=71 + nq).pb.kv_pool[:, 0]  # of a problem with keys at random
    c.pb.kv_pool[:, 0] = keys
    c.pb.softmax_scale = scale
    c.upload()
    c.decode()
    out, _ = c.check_decode()
    assert np.all(out == 1.0)


@pytest.mark.parametrize("nq", ROWS)
@pytest.mark.parametrize("lower,higher", [(62.5, 65.0), (63.5, 64.0)])
def test_values_that_follow_the_rounding_of_their_probability(torch_cuda, nq, lower, higher):
    # probabilities either side of 1 + 2^-8, where bf16 rounds to 1 or to 1 + 2^-7, with values -1 and +1
    c = a_cache("bf16", nq)
    c.pb.softmax_scale = 2.0 ** -14
    for r in range(2):
        at = np.arange(64, int(c.pb.seq_lens[r]) + nq - 1)
        page, row = c.pb.block_table[r, at // 128], at % 128
        c.pb.kv_pool[page, 0, 0, row, 0] = synth.f32_to_bf16_bits(np.where(at % 2, lower, higher).astype(np.float32))
        c.pb.kv_pool[page, 1, 0, row] = np.where(at % 2, 0xBF80, 0x3F80)[:, None]
    c.upload()
    c.decode()
    out, _ = c.check_decode()
    want, _, S, V = ref.dense_decode(c.pb, c.q)
    tol = 2.0 ** -8 * np.abs(want) + V * (2.0 ** -16 + 2 * (logit_error(S, S) + 2.0 ** -22) + 3100 * 2.0 ** -23)
    assert np.all(np.abs(out - want) <= tol), np.abs(out - want).max()
