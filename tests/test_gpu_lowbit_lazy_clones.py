"""What the low-bit calls write goes to the tensor that was given, not through a lazy clone to the tensor that it was
cloned from."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests import lowbit_reference as R
from tests.test_gpu_lowbit import BF16, E4M3, F32, U8, _attn_case, _n, _w4_weights

pytestmark = pytest.mark.gpu


def _check(call, *outs):
    """call with lazy clones of outs: they get what plain tensors get, and the originals keep their bytes."""
    plain = [t.clone() for t in outs]
    call(*plain)
    before = [t.clone() for t in outs]
    lazy = [torch._lazy_clone(t) for t in outs]
    call(*lazy)
    torch.cuda.synchronize()
    for base, kept, want, got in zip(outs, before, plain, lazy):
        assert torch.equal(base.view(U8), kept.view(U8))
        assert torch.equal(got.view(U8), want.view(U8))


def test_outputs_that_are_lazy_clones(cuda):
    x = _n((4, 512), 95, 1, BF16)
    E = lambda *sh, t=BF16: torch.zeros(*sh, dtype=t, device=cuda)
    d = hb.norm_desc(4, 512, out_dtype=hb.HCA_FP8E4M3)
    _check(lambda ro, o, s: hb.add_rms_norm(d, x, x, None, ro, o, s), E(4, 512), E(4, 512, t=E4M3), E(4, 1, t=F32))
    _check(lambda r, o, s: hb.add_rms_norm(d, x, r, None, r, o, s), x.clone(), E(4, 512, t=E4M3), E(4, 1, t=F32))   # in place
    _, wts = _w4_weights(1, 40, 512, 32, "e2m1", 1)
    w = hb.w4_desc(4, 40, 512)
    ws = E(max(16, hb.w4_linear_workspace_size(w)), t=U8)
    _check(lambda o: hb.w4_linear(w, x, None, *wts, o, ws), E(4, 40))
    base = E(max(16, hb.w4_linear_workspace_size(w)), t=U8)
    hb.w4_linear(w, x, None, *wts, E(4, 40), torch._lazy_clone(base))
    assert (base == 0).all()
    _check(lambda r: hb.kv_quant_fp4(x, 512, 64, r), E(6, 368, t=U8))
    rec = R.encode_records(x, 64)
    _check(lambda o: hb.kv_dequant_fp4(rec, 512, 64, o), E(4, 512))
    s = _attn_case(2, 16, 128, 64, 8, 4, [300, 20])
    da = hb.attn_desc(2, 16, 128, 64, 8, 4, dtype=hb.HCA_BF16)
    wa, cache = E(max(16, hb.attend_fp4_workspace_size(da, 300)), t=U8), hb.fp4_cache(s["store"], s["cap"])
    _check(lambda o: hb.attend_fp4(da, s["q"], cache, None, s["win"], s["sink"], s["positions"], 300, o, wa), E(2, 16, 128))
