"""Python binding of the block-sparse paged decode attention library.

Argument marshalling only: every function forwards to the C ABI of
``include/msa.h`` in ``libmsa_gb300.so`` (built in-tree by ``build.py``),
passing device pointers (``torch.Tensor.data_ptr()`` or plain ints) and the
CUDA stream handle.  Every step of the computation runs in the library's
CUDA kernels; there is no fallback.  If the library is missing, loading
raises.
"""

from __future__ import annotations

import ctypes
import os

from . import build as _build

MSA_OK = 0
MSA_ERR_INVALID_ARGUMENT = 1
MSA_ERR_UNSUPPORTED = 2
MSA_ERR_CUDA = 3
MSA_ERR_DEVICE_CHECK = 4
MSA_ERR_TIMEOUT = 5

MSA_BF16 = 0
MSA_FP8_E4M3 = 1
MSA_NVFP4 = 2

DTYPE_CODES = {"bf16": MSA_BF16, "fp8": MSA_FP8_E4M3, "nvfp4": MSA_NVFP4}

# C entry points and their argument / return types (see include/msa.h).
_p = ctypes.c_void_p


class MsaShape(ctypes.Structure):
    _fields_ = [
        ("num_requests", ctypes.c_int32),
        ("q_per_req", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("num_index_heads", ctypes.c_int32),
        ("index_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("index_dtype", ctypes.c_int32),
        ("decode_ctas", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("init_blocks", ctypes.c_int32),
        ("local_blocks", ctypes.c_int32),
    ]


class MsaRope(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("per_head_weights", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("norm_eps", ctypes.c_float),
        ("norm_offset", ctypes.c_float),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("q_idx_stride", ctypes.c_int64),
        ("idxk_stride", ctypes.c_int64),
    ]


_SIGNATURES = {
    "msa_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MsaShape)]),
    "msa_workspace_init": (ctypes.c_int, [_p, ctypes.c_size_t, _p]),
    "msa_index_score": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, _p, _p, _p,
                                       ctypes.c_size_t, _p]),
    "msa_select_topk": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, ctypes.c_size_t,
                                       _p]),
    "msa_sparse_decode": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, _p, _p, _p, _p,
                                         ctypes.c_size_t, _p]),
    "msa_decode_step": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, _p, _p, _p, _p, _p,
                                       _p, _p, _p, ctypes.c_size_t, _p]),
    "msa_kv_update": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, _p, _p, _p, _p, _p,
                                     ctypes.c_size_t, _p]),
    "msa_select_rows": (ctypes.c_int, [ctypes.POINTER(MsaShape), _p, _p, _p, _p, ctypes.c_size_t,
                                       _p]),
    "msa_cache_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MsaShape)]),
    "msa_dense_decode": (ctypes.c_int, [ctypes.POINTER(MsaShape)] + [_p] * 7 + [ctypes.c_size_t, _p]),
    "msa_weight_accumulate": (ctypes.c_int, [ctypes.POINTER(MsaShape)] + [_p] * 6 + [
        ctypes.c_float, _p, _p, _p, ctypes.c_size_t, _p]),
    "msa_cache_evict": (ctypes.c_int, [ctypes.POINTER(MsaShape)] + [ctypes.c_int32] * 3 + [_p] * 11 + [
        ctypes.c_size_t, _p]),
    "msa_rope_frequencies": (ctypes.c_int, [_p, ctypes.c_int32, _p]),
    "msa_qk_norm_rope": (ctypes.c_int, [ctypes.POINTER(MsaRope), _p, ctypes.c_int32, _p] + [
        ctypes.c_int32, _p, _p, _p] * 2 + [_p]),
    "msa_ragged_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MsaShape)]),
    "msa_kv_append": (ctypes.c_int, [ctypes.POINTER(MsaShape), ctypes.POINTER(MsaRope), _p, ctypes.c_int32] + [
        _p] * 18 + [ctypes.c_size_t, _p]),
    "msa_ragged_attention": (ctypes.c_int, [ctypes.POINTER(MsaShape), ctypes.c_int32, ctypes.c_int32] + [_p] * 8 + [
        ctypes.c_size_t, _p]),
    "msa_set_decode_wait_limit": (ctypes.c_int, [ctypes.c_int64]),
    "msa_check_device_status": (ctypes.c_int, [_p, _p]),
    "msa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}

_lib = None


class MsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load (once) the in-tree library; raises OSError if it has not been built."""
    global _lib
    if _lib is None:
        path = path or _build.LIB_PATH
        if not os.path.exists(path):
            raise OSError(f"{path} is missing: run __graft_entry__.build() (nvcc, sm_103a) first")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().msa_status_string(int(status)).decode()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _bufs(stream, kinds, *xs, **needs):
    """buffers.bufs, which takes this name at the first call (torch is imported by then)."""
    global _bufs
    from .buffers import bufs as _bufs

    return _bufs(stream, kinds, *xs, **needs)


def _check_rows(x, stride, heads, tokens):
    """buffers.check_rows, in the same way."""
    global _check_rows
    from .buffers import check_rows as _check_rows

    _check_rows(x, stride, heads, tokens)


# bytes of the 128 rows that a page has of one head, by element type, and of index keys without their scales
_TILE_BYTES = {MSA_BF16: 32768, MSA_FP8_E4M3: 16384, MSA_NVFP4: 9216}
_INDEX_TILE_BYTES = {MSA_BF16: 32768, MSA_NVFP4: 8192}
_NO_NEEDS = (0,) * 32  # a call without tokens looks at nothing


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != MSA_OK:
        raise MsaError(status, where)


def make_shape(*, num_requests, q_per_req, num_kv_heads, num_pages, max_blocks_per_seq, topk,
               kv_dtype="bf16", index_dtype="bf16", softmax_scale=128 ** -0.5, k_scale=1.0,
               v_scale=1.0, decode_ctas=0, head_dim=128, index_dim=128, page_size=128,
               num_index_heads=1, num_q_heads=None, init_blocks=0, local_blocks=0) -> MsaShape:
    if isinstance(kv_dtype, str):
        kv_dtype = DTYPE_CODES[kv_dtype]
    if isinstance(index_dtype, str):
        index_dtype = DTYPE_CODES[index_dtype]
    return MsaShape(
        num_requests=num_requests, q_per_req=q_per_req,
        num_q_heads=16 * num_kv_heads if num_q_heads is None else num_q_heads,
        num_kv_heads=num_kv_heads, head_dim=head_dim, num_index_heads=num_index_heads,
        index_dim=index_dim, page_size=page_size, num_pages=num_pages,
        max_blocks_per_seq=max_blocks_per_seq, topk=topk, kv_dtype=kv_dtype,
        index_dtype=index_dtype, decode_ctas=decode_ctas, softmax_scale=softmax_scale,
        k_scale=k_scale, v_scale=v_scale, init_blocks=init_blocks, local_blocks=local_blocks)


def msa_workspace_bytes(shape: MsaShape) -> int:
    return int(load().msa_workspace_bytes(ctypes.byref(shape)))


def msa_workspace_init(workspace, nbytes: int, stream=None):
    _check(load().msa_workspace_init(_ptr(workspace), int(nbytes), _stream(stream)),
           "msa_workspace_init")


def msa_index_score(shape, q_idx, idxk_pool, idxk_scales, block_table, seq_lens, block_scores,
                    workspace, workspace_bytes, stream=None):
    _check(load().msa_index_score(ctypes.byref(shape), _ptr(q_idx), _ptr(idxk_pool),
                                  _ptr(idxk_scales), _ptr(block_table), _ptr(seq_lens),
                                  _ptr(block_scores), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)), "msa_index_score")


def msa_select_topk(shape, block_scores, seq_lens, selected, workspace, workspace_bytes,
                    stream=None):
    _check(load().msa_select_topk(ctypes.byref(shape), _ptr(block_scores), _ptr(seq_lens),
                                  _ptr(selected), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)), "msa_select_topk")


def msa_sparse_decode(shape, q, kv_pool, block_table, seq_lens, selected, out, lse, workspace,
                      workspace_bytes, stream=None):
    _check(load().msa_sparse_decode(ctypes.byref(shape), _ptr(q), _ptr(kv_pool),
                                    _ptr(block_table), _ptr(seq_lens), _ptr(selected), _ptr(out),
                                    _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream)), "msa_sparse_decode")


def msa_decode_step(shape, q_idx, idxk_pool, idxk_scales, q, kv_pool, block_table, seq_lens,
                    block_scores, selected, out, lse, workspace, workspace_bytes, stream=None):
    _check(load().msa_decode_step(ctypes.byref(shape), _ptr(q_idx), _ptr(idxk_pool),
                                  _ptr(idxk_scales), _ptr(q), _ptr(kv_pool), _ptr(block_table),
                                  _ptr(seq_lens), _ptr(block_scores), _ptr(selected), _ptr(out),
                                  _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)), "msa_decode_step")


def msa_kv_update(shape, k_new, v_new, idxk_new, block_table, seq_lens, kv_pool, idxk_pool,
                  idxk_scales, workspace, workspace_bytes, stream=None):
    _check(load().msa_kv_update(ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(idxk_new),
                                _ptr(block_table), _ptr(seq_lens), _ptr(kv_pool), _ptr(idxk_pool),
                                _ptr(idxk_scales), _ptr(workspace), int(workspace_bytes),
                                _stream(stream)), "msa_kv_update")


def msa_select_rows(shape, scores_hbt, seq_lens, selected, workspace, workspace_bytes,
                    stream=None):
    _check(load().msa_select_rows(ctypes.byref(shape), _ptr(scores_hbt), _ptr(seq_lens),
                                  _ptr(selected), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)), "msa_select_rows")


def msa_cache_workspace_bytes(shape: MsaShape) -> int:
    """Workspace of the whole-cache operators below (0: shape not taken)."""
    return int(load().msa_cache_workspace_bytes(ctypes.byref(shape)))


def msa_dense_decode(shape, q, kv_pool, block_table, seq_lens, out, lse, workspace, workspace_bytes,
                     stream=None):
    """Attention over every cached position a token sees."""
    st, bufs = _bufs(stream, "hbiihfb", q, kv_pool, block_table, seq_lens, out, lse, workspace)
    _check(load().msa_dense_decode(ctypes.byref(shape), *bufs, int(workspace_bytes), st),
           "msa_dense_decode")


def msa_weight_accumulate(shape, q, kv_pool, block_table, seq_lens, selected, lse, decay, weights_in,
                          weights_out, workspace, workspace_bytes, stream=None):
    """Add this step's attention weights to every cached position's sum (selected: None after a
    dense step, the block tables after a sparse one)."""
    st, (*bufs, w_in, w_out, ws) = _bufs(stream, "hbiiifffb", q, kv_pool, block_table, seq_lens, selected, lse,
                                         weights_in, weights_out, workspace)
    _check(load().msa_weight_accumulate(ctypes.byref(shape), *bufs, float(decay), w_in, w_out, ws,
                                        int(workspace_bytes), st), "msa_weight_accumulate")


def msa_cache_evict(shape, keep, first, last, weights, block_table, seq_lens, new_table, kv_pool, idxk_pool,
                    idxk_scales, new_weights, kept, new_lens, workspace, workspace_bytes, stream=None):
    """Keep the heaviest positions of every request, copied in order to the pages of new_table."""
    st, bufs = _bufs(stream, "fiiibbbfiib", weights, block_table, seq_lens, new_table, kv_pool, idxk_pool,
                     idxk_scales, new_weights, kept, new_lens, workspace)
    _check(load().msa_cache_evict(ctypes.byref(shape), int(keep), int(first), int(last), *bufs,
                                  int(workspace_bytes), st), "msa_cache_evict")


def make_rope(*, rotary_dim=128, interleaved=False, per_head_weights=False, scale=1.0, norm_eps=1e-6, norm_offset=0.0,
              q_stride=0, k_stride=0, v_stride=0, q_idx_stride=0, idxk_stride=0) -> MsaRope:
    """Norm and rotation of head rows; strides in elements between tokens (0: dense)."""
    return MsaRope(rotary_dim=rotary_dim, interleaved=int(interleaved), per_head_weights=int(per_head_weights), scale=scale,
                   norm_eps=norm_eps, norm_offset=norm_offset, q_stride=q_stride, k_stride=k_stride, v_stride=v_stride,
                   q_idx_stride=q_idx_stride, idxk_stride=idxk_stride)


def rope_frequencies(radians, device=None):
    """The rotation's table (int64 bits) from angles in radians a position, one for each pair: a tensor of 64 or 32
    bits, or a sequence of floats; on `device`, else where the tensor lies."""
    import torch

    x = torch.as_tensor(radians, dtype=torch.float64)
    device = x.device if device is None else device
    x = x.detach().cpu().contiguous()
    turns = torch.empty(x.numel(), dtype=torch.int64)
    _check(load().msa_rope_frequencies(x.data_ptr(), x.numel(), turns.data_ptr()), "msa_rope_frequencies")
    return turns.to(device)


def msa_qk_norm_rope(rope: MsaRope, freqs, num_tokens: int, positions, num_q_heads: int, q, q_weight, q_out,
                     num_k_heads: int = 0, k=None, k_weight=None, k_out=None, stream=None):
    """Norm and rotation of query heads, and of key heads in the same pass."""
    needs, row = _NO_NEEDS, 256 * num_tokens
    if num_tokens > 0:
        qw, kw = (256 * num_q_heads, 256 * num_k_heads) if rope.per_head_weights else (256, 256)
        needs = (4 * rope.rotary_dim, 4 * num_tokens, 0, qw, row * num_q_heads, 0, kw, row * num_k_heads)
    st, (f, at, a, b, c, d, e, g) = _bufs(stream, "giRhhRhh", freqs, positions, q, q_weight, q_out, k, k_weight, k_out, needs=needs)
    if q is not a:
        _check_rows(q, rope.q_stride, num_q_heads, num_tokens)
    if k is not d:
        _check_rows(k, rope.k_stride, num_k_heads, num_tokens)
    _check(load().msa_qk_norm_rope(rope, f, num_tokens, at, num_q_heads, a, b, c, num_k_heads, d, e, g,
                                   st), "msa_qk_norm_rope")


def msa_ragged_workspace_bytes(shape: MsaShape) -> int:
    """Workspace of the calls on ragged batches below (0: shape not taken)."""
    return int(load().msa_ragged_workspace_bytes(ctypes.byref(shape)))


def msa_kv_append(shape, rope, freqs, num_tokens, offsets, k, k_weight, v, idxk, idxk_weight, q, q_weight, q_out, q_idx,
                  q_idx_weight, q_idx_out, block_table, seq_lens, kv_pool, idxk_pool, idxk_scales, workspace,
                  workspace_bytes, stream=None):
    """A ragged batch's keys, values and index keys into their pages, with norm and rotation on the way, and its
    queries and index queries in the same pass."""
    Hq, Hkv, Hi, R = shape.num_q_heads, shape.num_kv_heads, shape.num_index_heads, shape.num_requests
    needs = _NO_NEEDS
    if num_tokens > 0 and R > 0:
        qw, kw, iw = (256 * Hq, 256 * Hkv, 256 * Hi) if rope.per_head_weights else (256, 256, 256)
        row, pages, idx_dtype = 256 * num_tokens, shape.num_pages, shape.index_dtype
        idx_rows = 0 if idxk is None else pages * Hi
        needs = (4 * rope.rotary_dim, 4 * R + 4, 0, kw, 0, 0, iw, 0, qw, row * Hq, 0, iw, row * Hi, 4 * R * shape.max_blocks_per_seq, 4 * R,
                 2 * pages * Hkv * _TILE_BYTES.get(shape.kv_dtype, 0), idx_rows * _INDEX_TILE_BYTES.get(idx_dtype, 0),
                 1024 * idx_rows if idx_dtype == MSA_NVFP4 else 0, workspace_bytes)
    st, out = _bufs(stream, "giRhRRhRhhRhhiibbbb", freqs, offsets, k, k_weight, v, idxk, idxk_weight, q, q_weight, q_out,
                    q_idx, q_idx_weight, q_idx_out, block_table, seq_lens, kv_pool, idxk_pool, idxk_scales, workspace, needs=needs)
    if k is not out[2]:
        _check_rows(k, rope.k_stride, Hkv, num_tokens)
    if v is not out[4]:
        _check_rows(v, rope.v_stride, Hkv, num_tokens)
    if idxk is not out[5]:
        _check_rows(idxk, rope.idxk_stride, Hi, num_tokens)
    if q is not out[7]:
        _check_rows(q, rope.q_stride, Hq, num_tokens)
    if q_idx is not out[10]:
        _check_rows(q_idx, rope.q_idx_stride, Hi, num_tokens)
    _check(load().msa_kv_append(shape, rope, out[0], num_tokens, *out[1:], workspace_bytes, st),
           "msa_kv_append")


def msa_ragged_attention(shape, num_tokens, causal, q, offsets, kv_pool, block_table, seq_lens, out, lse, workspace,
                         workspace_bytes, stream=None):
    """Attention of a ragged batch's query rows: causal (prompts, chunks, steps), or over all states of
    another length (cross attention)."""
    R, needs = shape.num_requests, _NO_NEEDS
    if num_tokens > 0 and R > 0:
        rows = num_tokens * shape.num_q_heads
        needs = (256 * rows, 4 * R + 4, 2 * shape.num_pages * shape.num_kv_heads * _TILE_BYTES.get(shape.kv_dtype, 0),
                 4 * R * shape.max_blocks_per_seq, 4 * R, 256 * rows, 4 * rows, workspace_bytes)
    st, bufs = _bufs(stream, "hibiihfb", q, offsets, kv_pool, block_table, seq_lens, out, lse, workspace, needs=needs)
    _check(load().msa_ragged_attention(shape, num_tokens, int(causal), *bufs, int(workspace_bytes), st),
           "msa_ragged_attention")


def msa_check_device_status(workspace, stream=None) -> int:
    """Synchronise, read and clear the workspace error word; returns the status code."""
    return int(load().msa_check_device_status(_ptr(workspace), _stream(stream)))


def msa_set_decode_wait_limit(clocks: int):
    """Test hook: the clock limit of the decode's bounded waits (<= 0: the default)."""
    _check(load().msa_set_decode_wait_limit(int(clocks)), "msa_set_decode_wait_limit")
