"""The low-bit decode calls at the edges of what they accept: refusals of device tensors, infinite sinks, the sequence
counts where the attention's runs are found another way, token counts beyond one launch, calls on two streams at once."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests import lowbit_reference as R
from tests.test_gpu_lowbit import BF16, E4M3, F32, U8, _attn_call, _attn_case, _attn_check, _close, _n, _w4_weights

pytestmark = pytest.mark.gpu


def _refused(text, f):
    with pytest.raises(hb.HcaError) as e:
        f()
    assert text in str(e.value)


def test_device_tensors_of_a_wrong_kind_are_refused(cuda):
    x, out, g = _n((4, 512), 1, 1, BF16), torch.empty(4, 512, device=cuda, dtype=BF16), torch.ones(512, device=cuda)
    d = hb.norm_desc(4, 512)
    _refused("res must be on the current CUDA device", lambda: hb.add_rms_norm(d, x, x.cpu(), g, None, out))
    _refused("out has dtype torch.float32, expected torch.bfloat16", lambda: hb.add_rms_norm(d, x, None, g, None, out.float()))
    _refused("x has shape (3, 512), expected (4, 512)", lambda: hb.add_rms_norm(d, x[:3], None, g, None, out))
    _refused("x must be contiguous", lambda: hb.add_rms_norm(d, _n((512, 4), 1, 1, BF16).t(), None, g, None, out))
    _refused("520 elements apart", lambda: hb.add_rms_norm(hb.norm_desc(4, 512, ldx=520), x, None, g, None, out))
    _refused("overlaps", lambda: hb.add_rms_norm(d, x, None, g, None, x))
    _refused("out must be a tensor", lambda: hb.add_rms_norm(d, x, None, g, None, None))
    _refused("needs out_scale", lambda: hb.add_rms_norm(hb.norm_desc(4, 512, out_dtype=hb.HCA_FP8E4M3), x, None, g, None,
                                                        torch.empty(4, 512, device=cuda, dtype=E4M3)))
    _refused("another type", lambda: hb.add_rms_norm(hb.w4_desc(4, 512, 32), x, None, g, None, out))
    _, (codes, scales, rs) = _w4_weights(1, 40, 512, 32, "e2m1", 1)
    w = hb.w4_desc(4, 40, 512)
    y, ws = torch.empty(4, 40, device=cuda, dtype=BF16), torch.empty(1 << 20, device=cuda, dtype=U8)
    _refused("codes has shape", lambda: hb.w4_linear(w, x, None, codes[:39], scales, rs, y, ws))
    _refused("x_scale goes with e4m3", lambda: hb.w4_linear(w, x, torch.ones(4, device=cuda), codes, scales, rs, y, ws))
    _refused("x_scale has shape", lambda: hb.w4_linear(w, x, torch.ones(4, 2, device=cuda), codes, scales, rs, y, ws))
    _refused("records of 368 bytes", lambda: hb.kv_quant_fp4(x, 512, 64, torch.empty(4, 360, device=cuda, dtype=U8)))
    rec = torch.empty(4, 368, device=cuda, dtype=U8)
    _refused("slots has dtype torch.int32", lambda: hb.kv_quant_fp4(x, 512, 64, rec, slots=torch.arange(4, device=cuda).int()))
    _refused("out has dtype", lambda: hb.kv_dequant_fp4(rec, 512, 64, out.float()))
    s = _attn_case(2, 16, 128, 64, 8, 4, [30, 20])
    s["sink"] = s["sink"][:15]
    _refused("sink has shape", lambda: _attn_call(s))
    s = _attn_case(2, 16, 128, 64, 8, 4, [30, 20])
    s["store"] = s["store"][:1]
    _refused("1 sequences, expected 2", lambda: _attn_call(s))
    s = _attn_case(2, 16, 128, 64, 8, 4, [30, 20])
    cache = hb.fp4_cache(s["store"], s["cap"])
    cache.rows = s["store"].clone()              # the handle's addresses are the old tensor's
    da, o = hb.attn_desc(2, 16, 128, 64, 8, 4, dtype=hb.HCA_BF16), torch.empty_like(s["q"])
    _refused("have moved", lambda: hb.attend_fp4(da, s["q"], cache, None, s["win"], s["sink"], s["positions"], 30, o, ws))
    assert torch.equal(x, _n((4, 512), 1, 1, BF16)) and hb.device_status() == hb.HCA_OK


@pytest.mark.parametrize("ctas", [1, 0])      # every sequence finished by its CTA, and joined from parts
def test_attend_fp4_infinite_sinks(cuda, ctas):
    s = _attn_case(1, 8, 128, 64, 8, 1, [3000], seed=61)
    s["sink"][1], s["sink"][2], s["sink"][3] = float("inf"), float("-inf"), 1e30
    o = _attn_call(s, max_ctas=ctas)
    assert (o[0, 1] == 0).all() and (o[0, 3].abs() < 1e-30).all()
    s["sink"][1] = s["sink"][3] = 0.0
    t = dict(s, sink=None)
    none = _attn_call(t, max_ctas=ctas)
    assert torch.equal(o[0, 2], none[0, 2])   # a sink of weight 0
    _attn_check(t, none)


@pytest.mark.parametrize("B", [127, 128, 129, 1000])
def test_attend_fp4_sequence_counts(cuda, B):
    s = _attn_case(B, 8, 128, 64, 5, 4, [(37 * i) % 150 - 1 for i in range(B)], seed=62, page=8)
    o = _attn_call(s)
    assert hb.device_status() == hb.HCA_OK
    _attn_check(s, o)


@pytest.mark.parametrize("T", [4096, 4100])
def test_w4_linear_more_tokens_than_one_launch(cuda, T):
    N, K = 130, 96
    _, (codes, scales, rs) = _w4_weights(1, N, K, 32, "int4", 63)
    x = _n((T, K), 63, 1, BF16)
    d = hb.w4_desc(T, N, K, 1, 32, hb.HCA_W4_INT4, out_dtype=hb.HCA_F32)
    ws = torch.full((max(16, hb.w4_linear_workspace_size(d)),), 0xFF, dtype=U8, device=cuda)
    out = torch.full((T + 1, N), 7.0, device=cuda)
    hb.w4_linear(d, x, None, codes, scales, rs, out[:T], ws)
    w = R.weights(codes, scales, rs, 1, N, K, 32, True)[0]
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    # K / 16 accumulations, up to 160 joined parts, scalings; f16 x at 2^-22 of a row's largest
    _close(out[:T], want, (K / 16 + 168) * 2.0 ** -23 * mag + 2.0 ** -24 * want.abs() + 1e-30)
    assert (out[T] == 7.0).all()


def test_two_streams_at_once(cuda):
    """The same calls on two streams, each with a workspace of its own, give what each gives alone."""
    cases = [_attn_case(3, 64, 512, 64, 128, 4, [9000, 50, 4000], page=24, seed=64 + i) for i in range(2)]
    alone = [_attn_call(s) for s in cases]
    _, wts = _w4_weights(1, 2000, 1024, 64, "e2m1", 66)
    d = hb.w4_desc(9, 2000, 1024, 1, 64)
    xs = [_n((9, 1024), 67 + i, 1, BF16) for i in range(2)]
    ys, outs = [torch.empty(9, 2000, device=cuda, dtype=BF16) for _ in range(4)], [torch.empty_like(s["q"]) for s in cases]
    nws = max(16, hb.w4_linear_workspace_size(d))
    wss = [torch.empty(nws, device=cuda, dtype=U8) for _ in range(2)]
    for i in range(2):
        hb.w4_linear(d, xs[i], None, *wts, ys[i], wss[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            _attn_call(cases[i], outs[i], stream=st, ws=cases[i].setdefault("ws", torch.empty(64 << 20, device=cuda, dtype=U8)))
            hb.w4_linear(d, xs[i], None, *wts, ys[2 + i], wss[i], stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], alone[i]) and torch.equal(ys[2 + i], ys[i])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_of_another_device_are_refused(cuda):
    other = torch.device("cuda:1")
    x, out = torch.zeros(4, 512, dtype=BF16, device=other), torch.zeros(4, 512, dtype=BF16, device=other)
    _refused("current CUDA device", lambda: hb.add_rms_norm(hb.norm_desc(4, 512), x, None, None, None, out))
    _refused("current CUDA device", lambda: hb.w4_quantize(hb.w4_desc(0, 4, 512), x))
    _refused("current CUDA device", lambda: hb.kv_quant_fp4(x, 512, 64, torch.zeros(4, 368, dtype=U8, device=cuda)))
