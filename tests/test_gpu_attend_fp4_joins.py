"""Attention over 4-bit records where sequences are cut into many parts: several groups of 16 heads, more parts than one
batch of the join, many and few sequences, ragged and with empty ones between."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests.test_gpu_lowbit import _attn_call, _attn_case, _attn_check

pytestmark = pytest.mark.gpu

JOINS = [
    # B, n_h, c, rd, w, m, positions, k, page
    (12, 64, 512, 64, 128, 4, [30000] + [100 + 1500 * i for i in range(11)], 0, 24),     # many sequences, 1 to many parts
    (40, 64, 256, 64, 5, 8, [(9001 * i) % 40000 - 1 for i in range(40)], 0, 0),
    (200, 33, 128, 64, 0, 16, [(7919 * i) % 50000 if i % 7 else -1 for i in range(200)], 0, 64),
    (9, 17, 512, 0, 64, 1, [9000 if i == 4 else 5 for i in range(9)], 0, 0),
    (5, 64, 512, 64, 128, 4, [30000, -1, 29999, 2, 65535], 0, 16),                         # few: four warps to a column group
    (60, 48, 256, 64, 16, 4, [20000 + i for i in range(60)], 700, 48),                     # lists, cut into equal runs
]


@pytest.mark.parametrize("B,n_h,c,rd,w,m,positions,k,page", JOINS)
def test_cut_sequences(cuda, B, n_h, c, rd, w, m, positions, k, page):
    s = _attn_case(B, n_h, c, rd, w, m, positions, k=k, page=page, seed=81)
    o = _attn_call(s)
    assert hb.device_status() == hb.HCA_OK
    _attn_check(s, o)
    assert torch.equal(_attn_call(s), o)
    for n in (7, 100):
        _attn_check(s, _attn_call(s, max_ctas=n))
