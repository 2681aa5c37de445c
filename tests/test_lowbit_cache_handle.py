"""The handle of a cache of 4-bit records describes what its tensors hold."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb


def test_a_page_table_without_columns_is_a_cache_of_no_entries():
    """Its address is null, like a contiguous cache's; with the store's page size as capacity, sequence b's entries
    would be read at b * cap, past a store of fewer pages than sequences."""
    rows, pages = torch.zeros(2, 16, 240, dtype=torch.uint8), torch.zeros(5, 0, dtype=torch.int32)
    s = hb.fp4_cache(rows, 16, pages).struct
    assert not s.pages and s.cap == 0 and s.max_pages == 0
    assert hb.fp4_cache(rows, 16).struct.cap == 16
    assert hb.fp4_cache(rows, 16, torch.zeros(5, 3, dtype=torch.int32)).struct.cap == 16


@pytest.mark.gpu
def test_a_page_table_without_columns_leaves_the_window(cuda):
    from tests.test_gpu_lowbit import _attn_call, _attn_case, _attn_check
    s = _attn_case(5, 16, 128, 64, 8, 4, [300, 5, 90, -1, 2000], page=16, seed=91)
    s["store"], s["pages"] = s["store"][:2].contiguous(), torch.zeros(5, 0, dtype=torch.int32, device=cuda)
    s["dense"] = s["dense"][:, :0]
    _attn_check(s, _attn_call(s))


@pytest.mark.gpu
def test_a_handle_whose_tensor_has_fewer_records_is_refused(cuda):
    """The same address, but less behind it than the handle's sizes say."""
    from tests.test_gpu_lowbit import _attn_case
    s = _attn_case(2, 16, 128, 64, 8, 4, [300, 200], page=16, seed=92)
    d, o = hb.attn_desc(2, 16, 128, 64, 8, 4, dtype=hb.HCA_BF16), torch.empty_like(s["q"])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=cuda)
    cache = hb.fp4_cache(s["store"], s["cap"], s["pages"])
    call = lambda: hb.attend_fp4(d, s["q"], cache, None, s["win"], s["sink"], s["positions"], 300, o, ws)
    call()
    cache.rows = s["store"][:-1]
    with pytest.raises(hb.HcaError, match="records"):
        call()
