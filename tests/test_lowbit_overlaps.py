"""The low-bit decode calls refuse buffers that share bytes with what they write (no GPU needed: refused before any
launch)."""
import pytest

from long_context_compressed_hca_b200 import binding as hb
from long_context_compressed_hca_b200 import build as hbuild

P = [(1 << 24) * (i + 1) for i in range(5)]      # made-up device addresses, never read


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return hb.lib()


def _bad(rc, text):
    assert rc == hb.HCA_ERR_INVALID
    assert text in hb.last_error(), hb.last_error()


def test_slots_inside_what_is_written(L):
    rows, rec = 4, 368
    _bad(L.hca_kv_quant_fp4(P[0], hb.HCA_BF16, rows, 512, 64, P[1], rows, P[1] + 16, None), "overlap slots")
    _bad(L.hca_kv_quant_fp4(P[0], hb.HCA_BF16, rows, 512, 64, P[1], rows, P[1] + rows * rec - 8, None), "overlap slots")
    _bad(L.hca_kv_dequant_fp4(P[0], rows, P[1] + 8, rows, 512, 64, P[1], None), "overlaps slots")


@pytest.mark.parametrize("i,j", [(i, j) for i in range(4) for j in range(i)])
def test_quantised_weights_share_no_bytes(L, i, j):
    p = list(P[:4])
    p[i] = p[j]
    _bad(L.hca_w4_quantize(hb.w4_desc(0, 64, 256), p[0], hb.HCA_F32, p[1], p[2], p[3], None), "overlap")
