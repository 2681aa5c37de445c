"""Residual + RMSNorm with the residual updated in place, where rows share the sectors and lines that other blocks write
at the same time, against a buffer of its own."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests.test_gpu_lowbit import BF16, F32, _n

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,t,rt", [(6000, 4104, BF16, BF16), (6000, 999, BF16, F32), (3000, 8200, F32, F32),
                                         (50000, 8, BF16, BF16), (40000, 17, F32, F32)])
def test_in_place_gives_what_a_separate_buffer_gives(cuda, rows, d, t, rt):
    x, res, g = _n((rows, d), 97, 1, t), _n((rows, d), 97, 2, rt), 1 + _n((d,), 97, 3, std=0.1)
    sep, o1, o2 = torch.empty_like(res), torch.empty(rows, d, dtype=BF16, device=cuda), torch.empty(rows, d, dtype=BF16, device=cuda)
    desc = hb.norm_desc(rows, d, hb.DTYPE_CODE[t], hb.DTYPE_CODE[rt])
    hb.add_rms_norm(desc, x, res, g, sep, o1)
    hb.add_rms_norm(desc, x, res, g, res, o2)
    assert torch.equal(sep, res) and torch.equal(o1, o2)
