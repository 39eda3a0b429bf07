"""Rows whose first position takes nearly all of the weight and has values of 0, as a sink has: the
outputs are what thousands of light positions add up to.

Tolerance.  With w the weights: a p of 16 bits is off by 2^-8 (bf16) or 2^-11 (fp16) of itself, or by 2^-25 of
its fp16 scale where that is more; 2^7 of the scale is the heaviest position's p, so 2^-32 of a weight of 1.  A
logit is off by at most d = 36 * 2^-23 S (128 exact products in at most 32 roundings, the scale, the
subtraction), which is 2 d of a weight against another, exp2 by 2^-22.  fp32 sums of n terms are off by n 2^-24
of their size, numerator and divisor alike.  So |out - o| <= sum w |v| (p + 2 d + 2^-21 + 2 n 2^-24) + n 2^-32 max |v|,
and 2^-8 |o| for the storage."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import ragged as ref
from oracle.whole_cache import rows
from test_ragged_attention_gpu import KV, Ragged, place, rows_of, set_row

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("bits", [12, 20, 26, 30])  # how far the sink's logit is above the others', base 2
@pytest.mark.parametrize("ctas", [0, 1])
def test_a_sink_over_a_long_context(torch_cuda, kv, bits, ctas):
    n = 20000
    c = Ragged([3], [n], False, 1, 4, kv, seed=bits, ctas=ctas)
    size = 4.0 if kv != "fp8" else 3.0
    for which, code in ((0, 0), (1, 0)):  # keys all 0; the sink's key has `size` everywhere, its values are 0
        for page, row in rows_of(c, 0, 0, n if which == 0 else 1, which):
            set_row(c, page, which, row, code, 0x38)
    place(c, 0, 0, size)
    k = rows(c.pb, 0, 0, 0, 1)[0]
    c.pb.softmax_scale = float(np.float32(bits * np.log(2.0) / k.sum()))
    c.q[:] = 0x3F80
    c.upload()
    out, lse = c.run().result()
    assert c.status() == msa.MSA_OK
    want, want_lse, _, S, V = ref.attention(c.pb, c.q, c.offsets, c.seq_lens, False)
    w = np.r_[2.0 ** bits, np.ones(n - 1)]
    mass = (w / w.sum()) @ np.abs(rows(c.pb, 0, 1, 0, n))
    d = 36 * 2.0 ** -23 * S
    p = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(want) + mass * (p + 2 * d + 2.0 ** -21 + 2 * n * 2.0 ** -24) + n * 2.0 ** -32 * V
    assert np.all(np.abs(out - want) <= tol), (np.abs(out - want) / tol).max()
    assert np.all(np.abs(lse - want_lse) <= d + 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(want_lse)))
