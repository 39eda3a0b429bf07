"""Device buffers of the whole-cache operators as the library takes them: addresses and a stream handle.

A step of a small cache takes about 10 us on the GPU, so every call counts here: what torch has to be
asked is asked once (7 tensors: 1.9 us without the element types, 2.2 with them).
"""

from __future__ import annotations

import torch

_TYPES = {
    "h": frozenset((torch.bfloat16, torch.int16, torch.uint16)),  # bf16, or its bits
    "i": frozenset((torch.int32, torch.uint32)),
    "f": frozenset((torch.float32,)),
    "b": None,  # pools and workspaces are bytes
}
_KINDS = {kinds: tuple(_TYPES[k] for k in kinds) for kinds in ("hbiihfb", "hbiiifffb", "fiiibbbfiib")}
_Tensor, _get_device, _is_contiguous, _data_ptr = (torch.Tensor, torch.Tensor.get_device, torch.Tensor.is_contiguous,
                                                   torch.Tensor.data_ptr)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def current_stream(device: int | None = None) -> int:
    """The current stream's handle, without building a Stream object (3 us) where torch has a way."""
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(torch.cuda.current_device() if device is None else device)


def bufs(stream, kinds: str, *xs):
    """The stream handle (None: the current stream) and the device pointers of a call's buffers, one
    letter of `kinds` each: tensors must be dense, on the current device and of the letter's element
    type (the library sees only addresses); ints and None are taken as they are."""
    device, out = None, []
    for x, types in zip(xs, _KINDS[kinds]):
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
        if not _is_contiguous(x):
            raise ValueError("buffers must be contiguous")
        out.append(_data_ptr(x))
    if stream is None:
        stream = current_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return stream, out
