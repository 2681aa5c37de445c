"""The low-bit decode calls refuse what they do not take, before anything is
launched (no GPU needed), and the float64 references of their GPU tests hold
on hand-computed values."""
import ctypes

import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from long_context_compressed_hca_b200 import build as hbuild
from tests import lowbit_reference as R

X = 1 << 20          # made-up device addresses, never read: every call here is refused or empty
P = [16 * X * (i + 1) for i in range(9)]


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return hb.lib()


def _bad(rc, text):
    assert rc == hb.HCA_ERR_INVALID
    assert text in hb.last_error(), hb.last_error()


def test_norm_refusals(L):
    def call(x=P[0], res=P[1], g=P[2], ro=P[3], out=P[4], sc=P[5], **kw):
        return L.hca_add_rms_norm(hb.norm_desc(kw.pop("rows", 4), kw.pop("d", 256), **kw), x, res, g, ro, out, sc, None)
    _bad(L.hca_add_rms_norm(None, *P[:6], None), "null descriptor")
    _bad(call(rows=-1), "rows must")
    _bad(call(d=0), "d must be")
    _bad(call(d=32769), "d must be")
    _bad(call(x_dtype=hb.HCA_FP8E4M3), "x_dtype")
    _bad(call(x_dtype=hb.HCA_F32, res_dtype=hb.HCA_BF16), "res_dtype")
    _bad(call(out_dtype=hb.HCA_FP4), "out_dtype")
    _bad(call(scale_group=64), "scale_group")                                     # bf16 output
    _bad(call(out_dtype=hb.HCA_FP8E4M3, scale_group=32), "scale_group")
    _bad(call(out_dtype=hb.HCA_FP8E4M3, scale_group=128, d=192), "scale_group")
    _bad(call(out_dtype=hb.HCA_FP8E4M3, sc=None), "out_scale")
    _bad(call(ldx=255), "strides")
    _bad(call(x=None), "non-null")
    _bad(call(out=None), "non-null")
    _bad(call(x=P[0] + 8), "aligned")
    _bad(call(out=P[0]), "overlaps an input")
    _bad(call(ro=P[0] + 512), "overlaps an input")
    _bad(call(ro=P[1] + 512), "overlaps an input")       # in place only at the same address
    _bad(call(ro=P[4] + 16), "two outputs overlap")
    _bad(call(out_dtype=hb.HCA_FP8E4M3, sc=P[4]), "two outputs overlap")
    assert L.hca_add_rms_norm(hb.norm_desc(0, 256), *[None] * 6, None) == hb.HCA_OK


def test_w4_refusals(L):
    def call(x=P[0], xs=None, c=P[1], s=P[2], r=P[3], o=P[4], ws=P[5], nws=1 << 19, **kw):
        d = hb.w4_desc(kw.pop("T", 4), kw.pop("N", 64), kw.pop("K", 256), **kw)
        return L.hca_w4_linear(d, x, xs, c, s, r, o, ws, nws, None)
    _bad(L.hca_w4_linear(None, *P[:7], 0, None), "null descriptor")
    _bad(call(N=0), "N, K and groups")
    _bad(call(groups=0), "N, K and groups")
    _bad(call(T=-1), "T must")
    _bad(call(scale_group=16), "scale_group")
    _bad(call(K=48), "multiple of 32")
    _bad(call(K=96, scale_group=64), "multiple of 32 and of scale_group")
    _bad(call(K=32768 + 32), "K must be <= 32768")
    _bad(call(code=2), "code must")
    _bad(call(N=1 << 30, groups=4), "31 bits")
    _bad(call(x_dtype=hb.HCA_F32), "x_dtype")
    _bad(call(out_dtype=hb.HCA_FP8E4M3), "out_dtype")
    _bad(call(ldx=255), "strides")
    _bad(call(ldx=260), "multiples of 16")
    _bad(call(ldo=63), "strides")
    _bad(call(c=None), "non-null")
    _bad(call(xs=P[6]), "x_scale")
    _bad(call(x_dtype=hb.HCA_FP8E4M3), "x_scale")
    _bad(call(o=P[4] + 4), "aligned")
    _bad(call(o=P[0]), "out overlaps")
    big = dict(T=64, N=256, K=8192)
    need = L.hca_w4_linear_workspace_size(hb.w4_desc(**big))
    assert 0 < need <= 1 << 22
    _bad(call(nws=need - 1, **big), "workspace too small")
    _bad(call(ws=None, nws=1 << 30, **big), "workspace too small")
    _bad(call(ws=P[1], nws=need, **big), "workspace overlaps")
    _bad(call(o=P[5] + 256, nws=need, **big), "out overlaps")
    assert L.hca_w4_linear_workspace_size(hb.w4_desc(4, 64, 48)) == 0
    assert call(T=0, x=None, c=None, s=None, r=None, o=None, ws=None, nws=0) == hb.HCA_OK
    d = hb.w4_desc(0, 64, 256)
    _bad(L.hca_w4_quantize(d, P[0], hb.HCA_FP8E4M3, P[1], P[2], P[3], None), "w_dtype")
    _bad(L.hca_w4_quantize(d, None, hb.HCA_F32, P[1], P[2], P[3], None), "non-null")
    _bad(L.hca_w4_quantize(d, P[0] + 4, hb.HCA_F32, P[1], P[2], P[3], None), "aligned")


def test_kv_fp4_sizes_and_refusals(L):
    for c, rd in ((512, 64), (256, 64), (128, 64), (64, 0), (512, 0), (80, 16), (64, 64)):
        assert L.hca_kv_fp4_row_bytes(c, rd) == R.row_bytes(c, rd), (c, rd)
    assert L.hca_kv_fp4_row_bytes(512, 64) == 368          # 224 + 128 + 14 = 366, padded to 16
    for c, rd in ((512, 60), (640, 64), (512, 32), (64, 80), (0, 0), (128, -64)):
        assert L.hca_kv_fp4_row_bytes(c, rd) == 0, (c, rd)
    q, dq = L.hca_kv_quant_fp4, L.hca_kv_dequant_fp4
    _bad(q(P[0], hb.HCA_BF16, 4, 512, 32, P[1], 4, None, None), "unsupported")
    _bad(q(P[0], hb.HCA_FP8E4M3, 4, 512, 64, P[1], 4, None, None), "x_dtype")
    _bad(q(P[0], hb.HCA_BF16, -1, 512, 64, P[1], 4, None, None), "rows")
    _bad(q(P[0], hb.HCA_BF16, 4, 512, 64, P[1], -1, None, None), "records")
    _bad(q(P[0] + 8, hb.HCA_BF16, 4, 512, 64, P[1], 4, None, None), "aligned")
    _bad(q(None, hb.HCA_BF16, 4, 512, 64, P[1], 4, None, None), "non-null")
    _bad(q(P[0], hb.HCA_BF16, 4, 512, 64, P[1], 4, P[2] + 4, None), "8-byte")
    _bad(q(P[0], hb.HCA_BF16, 4, 512, 64, P[0] + 1024, 4, None, None), "overlap")
    _bad(dq(P[0], 4, None, 4, 512, 64, P[1] + 8, None), "aligned")
    _bad(dq(P[0], 4, None, 4, 512, 64, None, None), "non-null")
    _bad(dq(P[0], 4, None, 4, 512, 64, P[0], None), "overlap")
    assert q(None, hb.HCA_BF16, 0, 512, 64, None, 4, None, None) == hb.HCA_OK
    assert dq(None, 4, None, 0, 512, 64, None, None) == hb.HCA_OK


def test_attend_fp4_refusals(L):
    def call(q=P[0], idx=None, win=P[2], sink=P[3], pos=P[4], o=P[5], ws=P[6], nws=1 << 40, max_pos=1000, cap=256, rows=P[1],
             pages=None, max_pages=0, n_pages=0, **kw):
        a = dict(B=2, n_h=16, c=128, rd=64, w=32, m=4, dtype=hb.HCA_BF16)
        a.update(kw)
        d = hb.attn_desc(a.pop("B"), a.pop("n_h"), a.pop("c"), a.pop("rd"), a.pop("w"), a.pop("m"), **a)
        cache = hb.Fp4Cache(rows, cap, pages, max_pages, n_pages)
        return L.hca_attend_fp4(ctypes.byref(d), q, cache, idx, win, sink, pos, max_pos, o, ws, nws, None)
    _bad(call(B=0), "B must")
    _bad(call(n_h=65), "n_h must")
    _bad(call(c=192), "c must")
    _bad(call(rd=60), "rd must")
    _bad(call(m=0), "m >= 1")
    _bad(call(dtype=hb.HCA_F32), "dtype")
    _bad(call(kv_mixed=1), "kv_mixed")
    _bad(call(max_ctas=-1), "max_ctas")
    _bad(call(max_pos=-1), "max_pos")
    _bad(call(max_pos=2**31 - 1), "max_pos")
    _bad(call(q=None), "non-null")
    _bad(call(pos=None), "non-null")
    _bad(call(q=P[0] + 8), "aligned")
    _bad(call(win=None), "kv_win")
    _bad(call(idx=P[7]), "k >= 1")
    _bad(call(rows=None), "cache rows")
    _bad(call(cap=-1), "cache rows")
    _bad(call(pages=P[7], cap=0), "paged")
    _bad(call(pages=P[7], max_pages=-1), "paged")
    _bad(call(o=P[0]), "o overlaps")
    d = hb.attn_desc(2, 16, 128, 64, 32, 4, dtype=hb.HCA_BF16)
    need = L.hca_attend_fp4_workspace_size(ctypes.byref(d), 1000)
    if need:
        _bad(call(nws=need - 1), "workspace too small")
        _bad(call(ws=None), "workspace too small")
        _bad(call(ws=P[0]), "workspace overlaps")


def test_binding_refuses_host_tensors_and_wrong_shapes(L):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for f in (lambda: hb.add_rms_norm(hb.norm_desc(4, 256), x, None, None, None, x),
              lambda: hb.kv_quant_fp4(x, 256, 64, torch.zeros(4, 240, dtype=torch.uint8)),
              lambda: hb.w4_quantize(hb.w4_desc(0, 4, 256), x)):
        with pytest.raises(hb.HcaError) as e:
            f()
        assert "CUDA device" in str(e.value)
    with pytest.raises(hb.HcaError):
        hb.kv_quant_fp4(x, 250, 64, x)
    with pytest.raises(hb.HcaError):
        hb.fp4_cache(torch.zeros(4, 3, 368, dtype=torch.uint8), 4)


def test_reference_codes_by_hand():
    v = torch.tensor([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 9.0, -0.25, -0.3, -5.0], dtype=torch.float64)
    # ties (0.25, 0.75, 1.25, ...) go to the even code: 0, 1.0 (code 2), 1.0, 2.0 (4), 2.0, 4.0 (6), 4.0
    assert R.nearest_e2m1(v).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 0, 9, 14]
    assert R.nearest_e4m3(torch.tensor([447.0, 500.0, 2.0 ** -10, 1.0625], dtype=torch.float64)).tolist() == [448.0, 448.0, 0.0, 1.0]
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1], x[0, 40] = 6.0, -3.0, 6.5
    rec = R.encode_records(x, 0)
    # block 0: e = 0 (6 <= 6), codes 7 and 8 + 5; block 1: e = 1, 6.5 / 2 = 3.25 -> 3 (code 5)
    assert rec[0, 0] == 7 | 13 << 4 and rec[0, 20] == 5 and rec[0, 32] == 127 and rec[0, 33] == 128
    assert R.decode_records(rec, 64, 0)[0, [0, 1, 40]].tolist() == [6.0, -3.0, 6.0]
    # two keys with equal logits and no sink average their rows
    o, a = R.attend(torch.zeros(1, 4).double(), torch.tensor([[1.0, 2, 3, 4], [3, 2, 1, 0]]).double(), None, 1.0, 0, 0)
    assert o.tolist() == [[2.0, 2.0, 2.0, 2.0]] and a.tolist() == o.tolist()
