"""Device buffers of the whole-cache and ragged operators as the library takes them: addresses and a stream handle.

A step of a small cache takes about 10 us on the GPU, so every call counts here: what torch has to be
asked is asked once (7 tensors: 1.9 us without the element types, 2.2 with them).
"""

from __future__ import annotations

import torch

_TYPES = {
    "h": frozenset((torch.bfloat16, torch.int16, torch.uint16)),  # bf16, or its bits
    "i": frozenset((torch.int32, torch.uint32)),
    "f": frozenset((torch.float32,)),
    "g": frozenset((torch.int64, torch.uint64)),
    "R": frozenset((torch.bfloat16, torch.int16, torch.uint16)),  # rows of tokens, which check_rows has seen
    "b": None,  # pools and workspaces are bytes
}
_KINDS = {kinds: tuple(_TYPES[k] for k in kinds)
          for kinds in ("hbiihfb", "hbiiifffb", "fiiibbbfiib", "giRhhRhh", "giRhRRhRhhRhhiibbbb",
                        "hibiihfb")}
_ROWS = _TYPES["R"]
_ANY = (0,) * 32
_Tensor, _get_device, _is_contiguous, _data_ptr = (torch.Tensor, torch.Tensor.get_device, torch.Tensor.is_contiguous,
                                                   torch.Tensor.data_ptr)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def current_stream(device: int | None = None) -> int:
    """The current stream's handle, without building a Stream object (3 us) where torch has a way."""
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(torch.cuda.current_device() if device is None else device)


def bufs(stream, kinds: str, *xs, needs=_ANY):
    """The stream handle (None: the current stream) and the device pointers of a call's buffers, one
    letter of `kinds` each: tensors must be dense, on the current device, of the letter's element
    type and of the bytes in `needs` at least (the library sees only addresses); ints and None are taken as they are."""
    device, out = None, []
    for x, types, need in zip(xs, _KINDS[kinds], needs):
        if x.__class__ is not _Tensor and (x is None or isinstance(x, int)):
            out.append(x)
            continue
        if types is not None and x.dtype not in types:
            raise ValueError(f"buffer of {x.dtype}: the argument takes {' or '.join(sorted(map(str, types)))}")
        d = _get_device(x)
        if d != device:
            if device is None and d >= 0:
                device = torch.cuda.current_device()
            if d != device:
                raise ValueError(f"buffer on {x.device}: not on the current CUDA device")
        if types is not _ROWS and not _is_contiguous(x):
            raise ValueError("buffers must be contiguous")
        if need and x.nbytes < need:
            raise ValueError(f"buffer of {x.nbytes} bytes: the call takes {need}")
        out.append(_data_ptr(x))
    if stream is None:
        stream = current_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return stream, out


def check_rows(x, stride: int, heads: int, tokens: int = 0):
    """Rows of `tokens` tokens: a tensor [tokens, heads, 128] (or [tokens, heads * 128]) that may be part of a wider one,
    `stride` elements (0: dense) from a token's rows to the next token's, as the library will be told."""
    step, shape = x.stride(), x.shape
    if shape == (tokens, heads, 128) and step == (stride or heads * 128, 128, 1):
        return
    if tuple(shape[1:]) not in ((heads, 128), (heads * 128,)) or step[-1] != 1 or (len(shape) == 3 and heads > 1 and step[1] != 128):
        raise ValueError(f"rows of shape {tuple(shape)} and strides {step}: a token's {heads} heads of 128 lie one after another")
    if shape[0] < tokens:
        raise ValueError(f"rows of {shape[0]} tokens: the call takes {tokens}")
    if shape[0] > 1 and step[0] != (stride or heads * 128):
        raise ValueError(f"rows {step[0]} elements apart: the call says {stride or heads * 128}")
