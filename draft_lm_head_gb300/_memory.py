"""Device memory of the calls: results and workspaces."""
from __future__ import annotations

import torch

# the current stream's handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_handle(stream, device) -> int:
    """The cudaStream_t of a call: that of `stream`, or the device's current one."""
    if stream is not None:
        return stream.cuda_stream
    index = getattr(device, "index", None)
    if _raw_stream is not None and index is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(device).cuda_stream


def _allocate(nbytes: int, device, stream) -> torch.Tensor:
    """Bytes of the pool of the call's stream: what that stream did with them
    before comes before the call, and what frees them may give them to it at once."""
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def result(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor for a call's result. One of a call on an explicit stream is
    of that stream's pool too (one of the current stream's may be memory that the
    current stream is not done with), and the current stream, where the
    caller goes on with it, is named to the allocator."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


class Workspace:
    """A reusable device workspace (grows on demand; 256-byte aligned). Calls in
    flight at once need one each. A captured graph keeps the address of the
    buffer that it was captured with: run the largest call before the capture."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._streams = set()  # handles of the streams that buf is known to be used on

    def get(self, nbytes: int, device, stream=None) -> torch.Tensor:
        """The buffer, for a call on `stream` (None: the current one). Streams other
        than the one it was allocated on are named to the allocator, so that a
        buffer that is outgrown is not handed out before they are done with it."""
        at = stream_handle(stream, device)
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
            self.buf = _allocate(nbytes, device, stream)
            self._streams = {at}
        elif at not in self._streams:
            self.buf.record_stream(stream if stream is not None else torch.cuda.current_stream(device))
            self._streams.add(at)
        return self.buf


def scratch(workspace, nbytes: int, device, stream) -> torch.Tensor:
    """The workspace of one call: a new one, a Workspace's, or the caller's tensor."""
    if workspace is None:
        return _allocate(nbytes, device, stream)
    if isinstance(workspace, torch.Tensor):
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on {device}, got one on "
                             f"{workspace.device} (contiguous={workspace.is_contiguous()})")
        if workspace.dtype is not torch.uint8:
            workspace = workspace.view(torch.uint8)  # callers count bytes
        if stream is not None:
            workspace.record_stream(stream)
        return workspace
    return workspace.get(nbytes, device, stream)
