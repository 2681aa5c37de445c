"""Attention over 4-bit records with the sequence counts near which clusters of 8, 4 and 2 CTAs no longer fit the GPU at
once, lists and ragged positions, with and without a CTA budget."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests.test_gpu_lowbit import _attn_call, _attn_case, _attn_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [14, 15, 16, 18, 19, 35, 36, 37, 38, 73, 74, 75])
def test_sequence_counts_around_whole_waves(cuda, B):
    s = _attn_case(B, 16, 128, 64, 128, 4, [4000 - 3 * i for i in range(B)], k=512, page=16, seed=101)
    o = _attn_call(s)
    assert hb.device_status() == hb.HCA_OK
    _attn_check(s, o)
    for n in (B, 2 * B, 8 * B):
        _attn_check(s, _attn_call(s, max_ctas=n))
    r = _attn_case(B, 64, 256, 64, 128, 16, [(997 * i) % 5000 - 1 for i in range(B)], seed=102)
    _attn_check(r, _attn_call(r))
