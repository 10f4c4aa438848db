"""Which stream a call runs on, and how the memory it touches there is kept.

torch's allocator hands a freed block out again in the order of the stream that
it was allocated on. A call that runs on another stream than the current one
therefore allocates on that other stream, lends it the caller's tensors, and
gives its results to the current stream. A stream given as a raw cudaStream_t has
to exist, as torch.cuda.ExternalStream asks, until the tensors of its calls are
dropped: torch records an event on it then.
"""
from __future__ import annotations

import contextlib

import torch

_HERE = contextlib.nullcontext()


def run_on(stream, dev):
    """(cudaStream_t, side) of a call with `stream=`: None, a torch stream or a
    cudaStream_t. side is the torch stream if it is not dev's current one, else None."""
    here = torch._C._cuda_getCurrentRawStream(dev.index)
    if stream is None:
        return here, None
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)  # 0 and 1 are CUDA's names of the default stream, not pointers
        stream = (torch.cuda.ExternalStream(raw, device=dev) if raw > 1
                  else torch.cuda.default_stream(dev))
    if stream.device != dev:
        raise RuntimeError(f"stream must be on {dev}, got {stream.device}")
    return stream.cuda_stream, None if stream.cuda_stream == here else stream


def on(dev, side):
    """A context with `dev` current (the library launches on the current device),
    and `side` its current stream if there is one: what is allocated inside is
    ordered with the call's own work."""
    if side is not None:
        return torch.cuda.stream(side)
    return _HERE if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)


def lend(side, *tensors) -> None:
    """The caller's tensors are used on `side`: their memory is not handed out
    before that work is over, even if the caller drops them at once."""
    if side is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(side)


def give(side, dev, *tensors) -> None:
    """Results allocated on `side` go to the caller, who uses them on the current
    stream (behind a wait of its own for `side`)."""
    if side is not None:
        lend(torch.cuda.current_stream(dev), *tensors)
