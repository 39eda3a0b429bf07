"""The whole-cache operators at the end of the cache: V rows that are not finite and that only some draft
tokens see, in every format, and what lies behind the last position in a buffer of weights.

Tolerances: those of tests/test_whole_cache_gpu.py.
"""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import whole_cache as ref
from test_whole_cache_gpu import Cache, check_attention, logit_error

pytestmark = pytest.mark.gpu

KV = ["bf16", "fp8", "nvfp4"]


def spoil(pb, kv, r, pos, g=0):
    """Make V at `pos` not finite; the dimensions hit."""
    page, row = pb.block_table[r, pos // 128], pos % 128
    if kv == "nvfp4":
        pb.kv_pool[page, 1, g, 8192 + row * 8 + 2] = 0x7F  # the scale of dimensions 32 .. 47
        return np.arange(32, 48)
    pb.kv_pool[page, 1, g, row, 37] = 0x7F80 if kv == "bf16" else 0x7F
    return np.array([37])


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq,G", [(2, 8), (3, 5), (2, 16), (4, 16), (5, 16), (8, 16), (9, 16), (40, 16)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("ctas", [0, 1, 3])
def test_a_value_that_is_not_finite_reaches_only_the_tokens_that_see_it(torch_cuda, kv, nq, G, where, ctas):
    # the draft tokens lie in one page, or across the end of one
    contexts = [700, 256 + (nq + 1) // 2]
    c = Cache(contexts, nq, 2, G, kv, seed=91 + nq, ctas=ctas)
    m = {"first": 0, "middle": (nq - 1) // 2, "last": nq - 2}[where]  # seen by tokens m + 1 ..
    for r in range(2):
        dims = spoil(c.pb, kv, r, int(c.pb.seq_lens[r]) + m, g=r)
    c.upload()
    c.decode()
    out, lse = c.result()
    with np.errstate(invalid="ignore"):
        want, want_lse, S, V = ref.dense_decode(c.pb, c.q)
    hit = np.zeros(out.shape, bool)
    for r in range(2):
        hit[r * nq + m + 1:(r + 1) * nq, r * G:(r + 1) * G, dims] = True
    assert np.array_equal(np.isfinite(want), ~hit) and np.array_equal(np.isfinite(out), ~hit)
    check_attention(np.where(hit, 0, out), lse, np.where(hit, 0, want), want_lse, S, V, 701)
    assert c.status() == msa.MSA_OK


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq,G", [(3, 5), (3, 16), (8, 16), (20, 16)])
def test_many_short_requests_with_values_that_are_not_finite(torch_cuda, kv, nq, G):
    # more units a CTA than there are marks of units with such values
    rng = np.random.default_rng(nq)
    contexts = [int(x) for x in rng.integers(nq, 200, 60)]
    c = Cache(contexts, nq, 1, G, kv, seed=95, ctas=2)
    hit = np.zeros((60 * nq, G, 128), bool)
    for r in range(0, 60, 3):
        m = int(rng.integers(0, nq - 1))
        dims = spoil(c.pb, kv, r, int(c.pb.seq_lens[r]) + m)
        hit[r * nq + m + 1:(r + 1) * nq, :, dims] = True
    c.upload()
    c.decode()
    out, lse = c.result()
    with np.errstate(invalid="ignore"):
        want, want_lse, S, V = ref.dense_decode(c.pb, c.q)
    assert np.array_equal(np.isfinite(out), ~hit)
    check_attention(np.where(hit, 0, out), lse, np.where(hit, 0, want), want_lse, S, V, 200)
    assert c.status() == msa.MSA_OK


def check_all_weights(c, got, lse, before, decay, selected, held):
    """Against the definition, with what the buffer held (`held`) behind the cache and in idle slots, exactly.
    The history may have either sign: what the relative bound of one term is taken of is the sum of the terms'
    sizes, decay |history| + the step's weights (each term is off by that much of itself, and every rounding of
    a sum by 2^-24 of the sum, which is no larger)."""
    host = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
    lse, got, held = host(lse).astype(np.float64), host(got).astype(np.float64), host(held).astype(np.float64)
    want = ref.weights(c.pb, c.q, lse, host(before), decay, host(selected), after=held)
    _, _, S, _ = ref.dense_decode(c.pb, c.q)
    inside = np.zeros(want.shape, bool)
    for r, n in ref._requests(c.pb):
        inside[r, :, :n] = True
    assert np.array_equal(got[~inside], held[~inside])
    top = np.abs(lse[np.isfinite(lse)]).max(initial=0)
    rel = logit_error(S, S) + 2.0 ** -22 + 2.0 ** -22 * (1 + top) + c.nq * c.G * 2.0 ** -24 + 2.0 ** -23
    sizes = ref.weights(c.pb, c.q, lse, None if before is None else np.abs(host(before)), decay, host(selected))
    off = np.where(inside, np.abs(got - want), 0)
    assert np.all(off <= rel * sizes + c.nq * c.G * 2.0 ** -126), off.max()
    assert c.status() == msa.MSA_OK


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nq,G", [(1, 16), (3, 5), (5, 16), (33, 16), (64, 16)])
@pytest.mark.parametrize("which", ["dense", "first pages", "last pages", "no page"])
@pytest.mark.parametrize("history", [True, False])
def test_weights_behind_the_cache_stay_as_they_are(torch_cuda, kv, nq, G, which, history):
    torch = torch_cuda
    contexts = [1000, 513, 256 + nq, 128, 64, 900]
    c = Cache(contexts, nq, 2, G, kv, seed=97 + nq, idle=(3,))
    c.shape.topk = 4
    c.decode()
    lse, sel = c.lse, None
    if which != "dense":
        table = np.full((c.pb.num_tokens, 1, 4), -1, np.int32)
        for t in range(c.pb.num_tokens):
            seen = int(c.pb.seq_lens[t // nq]) + t % nq
            blocks = -(-seen // 128) if c.pb.seq_lens[t // nq] else 0
            if which == "first pages":  # none of the last page, but where it is the only one
                some = np.arange(blocks)[: 2 if blocks > 2 else 1]
            elif which == "last pages":
                some = np.arange(blocks)[-2:]
            else:
                some = np.arange(0)
            table[t, 0, : len(some)] = some
        sel = torch.from_numpy(table).cuda()
    shape = (len(contexts), 2, c.pb.max_blocks * 128)
    rand = lambda seed: torch.rand(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) - 0.5  # noqa: E731
    before, held = rand(5) if history else None, rand(6)
    got = held.clone()
    c.accumulate(lse, before, got, 0.75, sel)
    check_all_weights(c, got, lse, before, 0.75, sel, held)
    if history:  # in place
        got = before.clone()
        c.accumulate(lse, got, got, 0.75, sel)
        check_all_weights(c, got, lse, before, 0.75, sel, before)
