"""A default stream that is busy while a test works beside it."""
import contextlib
import time

import torch


@contextlib.contextmanager
def busy_default_stream():
    """Copies from the host fill the default stream and outlast the block; they
    leave the SMs to it.  Memory that a new handle may get holds no zeros."""
    src = torch.empty(1 << 30, dtype=torch.uint8, pin_memory=True)
    dst = torch.empty_like(src, device="cuda")
    dirt = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirt
    torch.cuda.empty_cache()
    t = time.perf_counter()
    dst.copy_(src, non_blocking=True)
    torch.cuda.synchronize()
    for _ in range(max(4, int(0.4 / (time.perf_counter() - t)))):
        dst.copy_(src, non_blocking=True)
    end = torch.cuda.Event()
    end.record()
    yield
    assert not end.query(), "the default stream ended first: nothing was shown"
    torch.cuda.synchronize()
