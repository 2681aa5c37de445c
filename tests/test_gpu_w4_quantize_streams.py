"""Weights quantised on another stream than the current one."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests.test_gpu_lowbit import U8, _n

pytestmark = pytest.mark.gpu


def test_memory_that_the_current_stream_still_writes_is_not_taken(cuda):
    """A freed block goes back to its stream's allocations while that stream's work on it is still queued: the result
    of a call on another stream has to come from elsewhere."""
    N, K = 1024, 4096
    w = _n((N, K), 96, 1)
    d = hb.w4_desc(0, N, K)
    want = hb.w4_quantize(d, w)
    sizes = [(t.numel() * t.element_size()) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    big = torch.ones(8192, 8192, device=cuda)
    blocks = [torch.empty(n, dtype=U8, device=cuda) for n in sizes]
    torch.cuda.synchronize()
    for _ in range(8):
        big = big @ big * 1e-4
    for b in blocks:
        b.fill_(0xFF)
    old = {b.data_ptr() for b in blocks}
    del blocks, b
    got = hb.w4_quantize(d, w, stream=side)
    assert not old & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
