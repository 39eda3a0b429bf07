"""Ragged batches whose device inputs are malformed: what is reported, what stays as it was, and
that the requests beside are right."""

import numpy as np
import pytest

import sparse_attention_decode_msa_gb300 as msa
from oracle import ragged as ref
from test_ragged_attention_gpu import KV, Ragged, bad_codes, check
from test_ragged_rows_gpu import Batch, host, is_near

pytestmark = pytest.mark.gpu


def changed_rows(b):
    """(page, row) of every K or V row that the append has written (bf16 pools), of the index pool alike."""
    pool = (host(b.d_pool) != b.pool).reshape(b.pages, 2, b.Hkv, 128, 256).any((1, 2, 4))
    idx = (host(b.d_idx) != b.idx_pool).any((1, 3))
    return set(zip(*np.nonzero(pool))), set(zip(*np.nonzero(idx)))


def place(b, r, j):
    pos = int(b.seq_lens[r]) - 1 + j
    return b.table[r, pos // 128], pos % 128


def check_tokens(b, tokens):
    """tokens: {row of the inputs: (request, its token)}: all that they give is right."""
    pos = np.zeros(b.T, np.int64)
    for t, (r, j) in tokens.items():
        pos[t] = int(b.seq_lens[r]) - 1 + j
    pool, idx, t = host(b.d_pool), host(b.d_idx), np.array(sorted(tokens))
    at = [place(b, *tokens[i]) for i in t]
    for i, y in ((0, host(b.q_out)), (1, host(b.qi_out)), (2, None), (4, None)):
        want, size = ref.turned(b.host[i], b.w[i], pos, b.rad, b.rot, b.interleaved, eps=float(np.float32(1e-6)))
        if i == 2:
            y = np.stack([pool[p, 0].reshape(b.Hkv, 128, 256)[:, row] for p, row in at]).view(np.uint16)
        elif i == 4:
            y = np.stack([idx[p, :, row] for p, row in at]).view(np.uint16)
        else:
            y = y[t]
        assert np.all(is_near(y, want[t], size[t]))
    v = np.stack([pool[p, 1].reshape(b.Hkv, 128, 256)[:, row] for p, row in at]).view(np.uint16)
    assert np.array_equal(v, b.host[3][t])


def left(b, tokens):
    return np.all(host(b.q_out)[tokens] == 7) and np.all(host(b.qi_out)[tokens] == 7)


@pytest.mark.parametrize("R", [3, 300])  # (more requests than a block has threads)
def test_append_reports_offsets_that_go_down(torch_cuda, R):
    b = Batch([4, 4, 4] + [0] * (R - 3), [10] * R, seed=5)
    offsets = np.full(R + 1, 12, np.int32)
    offsets[:4] = 0, 9, 3, 12
    assert b.run(torch_cuda, offsets=offsets) == msa.MSA_ERR_DEVICE_CHECK
    # requests 0 (tokens 0 .. 8) and 2 (3 .. 11) have tokens; those of both go to either's pages or nowhere, and nothing else does
    mine = {place(b, 0, j) for j in range(9)} | {place(b, 2, j) for j in range(9)}
    for rows in changed_rows(b):
        assert rows <= mine
    check_tokens(b, {0: (0, 0), 1: (0, 1), 2: (0, 2), 9: (2, 6), 10: (2, 7), 11: (2, 8)})


def test_append_reports_offsets_past_the_tokens_and_skips_the_request(torch_cuda):
    for last in (13, 2 ** 31 - 1):
        b = Batch([4, 4, 4], [10, 10, 10], seed=5)
        offsets = b.offsets.copy()
        offsets[3] = last
        assert b.run(torch_cuda, offsets=offsets) == msa.MSA_ERR_DEVICE_CHECK
        good = {place(b, r, j) for r in (0, 1) for j in range(4)}
        for rows in changed_rows(b):
            assert rows == good
        check_tokens(b, {4 * r + j: (r, j) for r in (0, 1) for j in range(4)})
        assert left(b, np.arange(8, 12))
    # beyond the last request's tokens there may be more
    b = Batch([4, 4, 4], [10, 10, 10], seed=5, behind=2)
    assert b.run(torch_cuda) == msa.MSA_OK
    b.check()


def test_append_with_a_bad_length_leaves_the_others_right(torch_cuda):
    for bad in (0, -4, 257, 2 ** 31 - 1):
        b = Batch([2, 3, 130], [100, 10, 50], seed=9)
        lens = b.seq_lens.copy()
        lens[1] = bad
        assert b.run(torch_cuda, seq_lens=lens) == msa.MSA_ERR_DEVICE_CHECK
        tokens = {t: (0, t) for t in range(2)} | {5 + j: (2, j) for j in range(130)}
        for rows in changed_rows(b):
            assert rows == {place(b, r, j) for r, j in tokens.values()}
        check_tokens(b, tokens)
        assert left(b, np.arange(2, 5))


def test_append_with_a_bad_page_skips_its_tokens_whole(torch_cuda):
    # the queries and index queries of a token without a page are left too
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        b = Batch([2, 3, 130], [100, 10, 50], seed=9, behind=1)
        table = b.table.copy()
        table[2, 1] = bad  # positions 128 .. 179 of request 2
        assert b.run(torch_cuda, table=table) == msa.MSA_ERR_DEVICE_CHECK
        tokens = {t: (0, t) for t in range(2)} | {2 + j: (1, j) for j in range(3)} | {5 + j: (2, j) for j in range(78)}
        for rows in changed_rows(b):
            assert rows == {place(b, r, j) for r, j in tokens.values()}
        check_tokens(b, tokens)
        assert left(b, np.arange(5 + 78, 136))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("R", [4, 1300])  # (more requests than a block has threads)
def test_attention_over_offsets_that_go_down_writes_nothing(torch_cuda, kv, R):
    # every other request would have all the batch's tokens: together more rows than there are
    c = Ragged([40] + [0] * (R - 1), [200] + [0, 130] * ((R - 1) // 2) + [77], True, 1, 4, kv, seed=3)
    offsets = np.array([0, 40] * (R // 2) + [40], np.int32)
    c.d_offsets.copy_(torch_cuda.from_numpy(offsets))
    out, lse = c.run().result()
    assert c.status() == msa.MSA_ERR_DEVICE_CHECK
    assert np.all(out == 7) and np.all(lse == 7)
    c.d_offsets.copy_(torch_cuda.from_numpy(c.offsets))
    c.run().check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("counts,lens,G,pos", [([30, 4], [200, 77], 4, 211), ([300, 2], [1, 300], 1, 140), ([40, 3], [120, 9], 48, 127)])
def test_keys_that_are_not_finite_reach_the_rows_that_see_them_alone(torch_cuda, kv, counts, lens, G, pos):
    for ctas in (0, 2):
        c = Ragged(counts, lens, True, 1, G, kv, seed=8, ctas=ctas)
        want, want_lse, far, S, V = ref.attention(c.pb, c.q, c.offsets, c.seq_lens, True)
        page, row = c.pb.block_table[0, pos // 128], pos % 128
        if kv == "nvfp4":
            c.pb.kv_pool[page, 0, 0, 8192 + 8 * row:8192 + 8 * row + 8] = 0x7F
        else:
            c.pb.kv_pool[page, 0, 0, row, ::3] = bad_codes(kv)[-1]
        c.upload()
        out, lse = c.run().result()
        assert c.status() == msa.MSA_OK
        others = np.r_[0:pos - lens[0] + 1, counts[0]:sum(counts)]  # token j sees lens + j positions
        check(out[others], lse[others], want[others], want_lse[others], far[others], S, V, 1000, kv)
