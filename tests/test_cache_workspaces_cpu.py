"""Which workspace DeviceProblem's whole-cache methods hand to the library: one per stream, none freed
while the problem lives (with stand-ins for the streams and for the library's launches)."""

import contextlib
import weakref

import pytest

import sparse_attention_decode_msa_gb300 as msa
from sparse_attention_decode_msa_gb300 import buffers, build, runner


class Stand:
    """A problem on the CPU whose calls record (stream, workspace address, its size, cleared on)."""

    def __init__(self, monkeypatch):
        import torch

        build.build()
        self.stream, self.capturing, self.calls, self.cleared, self.synced = 7, False, [], {}, []

        @contextlib.contextmanager
        def on(stream):
            before, self.stream = self.stream, self.stream if stream is None else stream
            yield
            self.stream = before

        def call(shape, *args):
            ws, size, stream = args[-3:]
            assert stream == self.stream
            assert size >= msa.msa_cache_workspace_bytes(shape) and size == ws.numel()
            self.calls.append((self.stream, ws.data_ptr(), size))

        def init(ws, size, stream=None):
            assert size == ws.numel()
            self.cleared[ws.data_ptr()] = "graph" if self.capturing else self.stream

        monkeypatch.setattr(runner, "msa_workspace_init", init)
        monkeypatch.setattr(runner, "msa_dense_decode", call)
        monkeypatch.setattr(runner, "msa_cache_evict", call)
        monkeypatch.setattr(runner, "msa_weight_accumulate", call)
        monkeypatch.setattr(buffers, "current_stream", lambda device=None: self.stream)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self)
        self.dp = dp = runner.DeviceProblem.__new__(runner.DeviceProblem)
        monkeypatch.setattr(runner.DeviceProblem, "_on", staticmethod(on))
        dp.shape = msa.make_shape(num_requests=2, q_per_req=1, num_kv_heads=1, num_pages=8, max_blocks_per_seq=2, topk=2)
        dp.device = "cpu"
        for name in ("q_idx", "idxk", "idxk_scales", "q", "kv", "block_table", "seq_lens", "block_scores", "selected", "out", "lse"):
            setattr(dp, name, None)
        dp.ws_bytes, dp.ws = 1 << 30, None
        if hasattr(dp, "_new_cache_workspaces"):
            dp._new_cache_workspaces()

    def synchronize(self):
        self.synced.append(self.stream)


@pytest.fixture
def stand(monkeypatch):
    return Stand(monkeypatch)


def test_each_stream_has_its_own_cleared_on_it(stand):
    for stream in (None, 11, 12, 11, None):
        stand.dp.dense_decode(stream=stream)
        assert stand.dp.cache_ws.data_ptr() == stand.calls[-1][1]
    at = {stream: ws for stream, ws, _ in stand.calls}
    assert [s for s, _, _ in stand.calls] == [7, 11, 12, 11, 7] and len(set(at.values())) == 3
    assert all(ws == at[s] for s, ws, _ in stand.calls)
    assert all(stand.cleared[ws] == s for s, ws in at.items())
    assert len(stand.synced) <= 1  # once, for the workspace of captured calls


def test_other_methods_take_the_workspace_of_their_stream(stand):
    dp = stand.dp
    for stream in (11, 12):
        dp.dense_decode(stream=stream)
        dp.weight_accumulate(None, None, stream=stream)
        dp.evict(None, None, keep=5, stream=stream)
    ws = [w for _, w, _ in stand.calls]
    assert ws[0] == ws[1] == ws[2] and ws[3] == ws[4] == ws[5] and ws[0] != ws[3]


def test_a_larger_workspace_leaves_the_old_one_alive(stand):
    dp = stand.dp
    dp.dense_decode(stream=11)
    old = weakref.ref(dp.cache_ws)
    dp.shape.decode_ctas = 400
    dp.dense_decode(stream=11)
    assert stand.calls[1][2] > stand.calls[0][2] and stand.calls[1][1] != stand.calls[0][1]
    assert old() is not None and old().data_ptr() == stand.calls[0][1]
    dp.shape.decode_ctas = 8  # a smaller one is not made anew
    dp.dense_decode(stream=11)
    assert stand.calls[2][1] == stand.calls[1][1]


def test_captured_calls_never_share_with_calls_of_another_stream(stand):
    dp = stand.dp
    dp.dense_decode(stream=11)
    stand.capturing = True
    dp.dense_decode(stream=20)  # cleared before the capture: nothing of it is in the graph
    assert "graph" not in stand.cleared.values() and stand.calls[1][1] != stand.calls[0][1]
    dp.dense_decode(stream=11)  # a stream with calls of its own
    assert stand.calls[2][1] == stand.calls[0][1]
    stand.capturing = False
    dp.dense_decode(stream=20)
    assert stand.calls[3][1] not in (stand.calls[0][1], stand.calls[1][1])


def test_a_first_call_may_be_captured(stand):
    stand.capturing = True
    for stream in (20, 21, 20):
        stand.dp.dense_decode(stream=stream)
    at = [ws for _, ws, _ in stand.calls]
    assert len(set(at)) == 3 and all(stand.cleared[ws] == "graph" for ws in at)
    stand.capturing = False
    stand.dp.dense_decode(stream=20)
    assert stand.calls[3][1] not in at and stand.cleared[stand.calls[3][1]] == 20
    stand.capturing = True
    stand.dp.dense_decode(stream=21)
    assert stand.cleared[stand.calls[4][1]] == 20 and stand.synced


def test_a_replica_has_workspaces_of_its_own(stand, monkeypatch):
    stand.dp.dense_decode(stream=11)
    stand.dp.ws_bytes = 256
    twin = stand.dp.replicate()
    twin.dense_decode(stream=11)
    stand.dp.dense_decode(stream=11)
    assert stand.calls[0][1] == stand.calls[2][1] != stand.calls[1][1]
