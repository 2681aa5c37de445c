"""The low-bit decode operators on the GPU against float64 references
(lowbit_reference.py): residual + RMSNorm, 4-bit-weight products, 4-bit KV
records, attention over them, and a decode step made of all four.

Tolerances count roundings: half a step of a type is eps/2 of its finfo
relative to the value (bf16 2^-8, e4m3 2^-4), fp32 operations 2^-24 each, and
a tensor-core accumulation of 16 products one truncation, 2^-23 of the sum of
magnitudes."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from long_context_compressed_hca_b200 import synth
from tests import lowbit_reference as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3, U8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _n(shape, seed, stream, dtype=F32, std=1.0):
    return synth.normal(shape, seed, stream, std=std, dtype=dtype).to("cuda")


def _close(got, want, tol):
    err = (got.double() - want).abs() - tol
    assert not torch.isnan(got.double()).any()
    assert (err <= 0).all(), f"worst excess {err.max().item():.3e} at {err.argmax().item()}"


# ------------------------------------------------------------------ residual + norm
NORM = [
    # rows, d, x, res, out, group, pad (extra elements of a row's stride)
    (1, 1, F32, F32, F32, 0, 0),
    (1, 4096, BF16, BF16, E4M3, 0, 0),
    (3, 4104, BF16, F32, BF16, 0, 0),
    (5, 257, BF16, BF16, E4M3, 0, 0),          # odd width: element accesses
    (7, 1000, F32, F32, BF16, 0, 24),          # strided rows, 16-byte accesses
    (7, 999, BF16, BF16, F32, 0, 4),           # strided rows, element accesses
    (33, 4096, BF16, BF16, E4M3, 128, 0),
    (33, 192, F32, F32, E4M3, 64, 8),
    (2, 8192, BF16, F32, E4M3, 64, 0),
    (2, 8448, F32, F32, E4M3, 128, 0),         # four units of 8 channels per thread, the last partly empty
    (2, 32768, F32, F32, F32, 0, 0),
    (70000, 16, BF16, BF16, BF16, 0, 0),       # more rows than a 16-bit grid dimension
]


@pytest.mark.parametrize("rows,d,xt,rt,ot,group,pad", NORM)
def test_add_rms_norm(cuda, rows, d, xt, rt, ot, group, pad):
    def strided(t):
        if not pad:
            return t
        b = torch.full((rows, d + pad), 7.0, device=cuda).to(t.dtype)
        b[:, :d] = t
        return b[:, :d]
    x, res = strided(_n((rows, d), 1, 1, xt)), strided(_n((rows, d), 1, 2, rt, std=4.0))
    gamma = 1.0 + _n((d,), 1, 3, std=0.1)
    fp8 = ot == E4M3
    ro, out = strided(torch.zeros_like(res)), strided(torch.zeros(rows, d, device=cuda).to(ot))
    sc = torch.full((rows, d // group if group else 1), -1.0, device=cuda) if fp8 else None
    desc = hb.norm_desc(rows, d, hb.DTYPE_CODE[xt], hb.DTYPE_CODE[rt], hb.DTYPE_CODE[ot], group,
                        ldx=d + pad if pad else 0, ldr=d + pad if pad else 0, ldo=d + pad if pad else 0)
    hb.add_rms_norm(desc, x, res, gamma, ro, out, sc)
    z, y = R.rms_norm(x, res, gamma, 1e-6)
    # z: one fp32 addition, then res_dtype; y: z's rounding, a sum of d squares (partial sums of at most 32 per
    # thread, 10 tree levels), square root, division, two products: below 32 + 10 + 8 roundings of 2^-24, half of
    # those of the sum (a square root); the sum's cancellation in z is relative to |x| + |res|
    _close(ro, z, (2.0 ** -24 + HALF[rt]) * z.abs() + 2.0 ** -24 * (x.double().abs() + res.double().abs()))
    rel = 40 * 2.0 ** -24
    y_err = rel * y.abs() + 2.0 ** -24 * (x.double().abs() + res.double().abs()) * (y / z.where(z != 0, 1)).abs()
    if not fp8:
        _close(out, y, y_err + HALF[ot] * y.abs() + 1e-30)
    else:
        g = group or d
        want_sc = y.abs().unflatten(1, (-1, g)).amax(2) / 448.0
        assert (sc.double() - want_sc).abs().le(2 * rel * want_sc).all()
        s = sc.double().repeat_interleave(g, 1)
        q = out.double()
        # half a step of e4m3: 2^-4 of the value, at least half of the subnormal step 2^-9
        _close(q * s, y, y_err + (2.0 ** -4 * y.abs()).clamp_min(2.0 ** -10 * s.max().item()) * (1 + 2.0 ** -8))
        # and the code is the nearest one wherever y / scale is not within the computation's error of a tie
        v = y / s
        lo, hi = R.nearest_e4m3(v * (1 - 3 * rel)), R.nearest_e4m3(v * (1 + 3 * rel))
        assert ((q == lo) | (q == hi)).all()
        assert (q.abs().unflatten(1, (-1, g)).amax(2) == 448.0).all()
    if pad:   # the gap between rows is untouched
        for t, fill in ((ro, 7.0), (out, 7.0)):
            full = t.as_strided((rows, pad), (d + pad, 1), d)[: rows - 1]
            assert (full.float() == fill).all()


def test_add_rms_norm_optional_inputs_in_place_and_zero_rows(cuda):
    rows, d = 4, 512
    x = _n((rows, d), 2, 1, BF16)
    x[1] = 0
    out, sc = torch.zeros(rows, d, device=cuda, dtype=E4M3), torch.full((rows, 1), -1.0, device=cuda)
    hb.add_rms_norm(hb.norm_desc(rows, d, out_dtype=hb.HCA_FP8E4M3), x, None, None, None, out, sc)
    assert sc[1] == 0 and (out[1].view(U8) == 0).all()       # an all-zero row: scale 0, codes 0
    z, y = R.rms_norm(x, None, None, 1e-6)
    _close(out.double() * sc.double(), y, 2.0 ** -4 * y.abs() * (1 + 2.0 ** -8) + 2.0 ** -10 * sc.double())
    # res_out = res in place gives what a separate buffer gives
    res, sep, o1, o2 = _n((rows, d), 2, 2, BF16), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    hb.add_rms_norm(hb.norm_desc(rows, d), x, res, None, sep, o1)
    hb.add_rms_norm(hb.norm_desc(rows, d), x, res, None, res, o2)
    assert torch.equal(sep, res) and torch.equal(o1, o2)
    # eps: <= 0 selects 1e-6
    x0 = torch.full((1, 8), 1e-3, device=cuda)
    o = torch.empty_like(x0)
    hb.add_rms_norm(hb.norm_desc(1, 8, hb.HCA_F32, out_dtype=hb.HCA_F32, eps=0.0), x0, None, None, None, o)
    _close(o, R.rms_norm(x0, None, None, 1e-6)[1], 1e-6)


# ------------------------------------------------------------------ 4-bit weights
W4 = [
    # T, N, K, groups, code, G, x, out, pad
    (1, 1, 32, 1, "e2m1", 32, BF16, F32, 0),
    (1, 512, 4096, 1, "e2m1", 32, BF16, BF16, 0),
    (2, 130, 96, 1, "int4", 32, BF16, F32, 0),          # N beyond one tile, K no multiple of a stage
    (7, 1024, 4096, 8, "int4", 128, BF16, BF16, 0),
    (8, 77, 224, 3, "e2m1", 32, E4M3, F32, 0),           # odd N, ragged K, several groups
    (9, 300, 320, 2, "int4", 64, E4M3, BF16, 16),
    (16, 129, 8192, 1, "e2m1", 128, BF16, F32, 0),
    (17, 256, 512, 1, "e2m1", 64, BF16, F32, 8),
    (32, 2048, 1024, 1, "e2m1", 64, E4M3, BF16, 0),
    (33, 513, 640, 1, "int4", 128, BF16, BF16, 0),
    (64, 1000, 2048, 1, "e2m1", 32, BF16, F32, 0),
    (65, 200, 256, 1, "e2m1", 32, BF16, F32, 0),         # beyond one token tile
    (150, 136, 32, 2, "int4", 32, E4M3, F32, 0),
    (3, 40, 32768, 1, "e2m1", 128, BF16, F32, 0),        # the longest K
    (4, 20000, 128, 1, "int4", 32, BF16, BF16, 0),
]


def _w4_weights(groups, N, K, G, code, seed):
    desc = hb.w4_desc(0, N, K, groups, G, hb.HCA_W4_INT4 if code == "int4" else hb.HCA_W4_E2M1)
    w = _n((groups * N, K), seed, 9, std=K ** -0.5)
    return w, hb.w4_quantize(desc, w)


@pytest.mark.parametrize("T,N,K,groups,code,G,xt,ot,pad", W4)
def test_w4_linear(cuda, T, N, K, groups, code, G, xt, ot, pad):
    _, (codes, scales, rs) = _w4_weights(groups, N, K, G, code, 5)
    xf = _n((T, groups * K), 5, 1)
    x, xs = xf.to(BF16), None
    if xt == E4M3:
        xs = xf.abs().amax(1) / 448.0
        x = (xf / xs[:, None]).to(E4M3)
    if pad:
        b = torch.full((T, groups * K + pad), 3.0, device=cuda).to(xt)
        b[:, : groups * K] = x
        x = b[:, : groups * K]
    out = torch.full((T, groups * N + pad), 7.0, device=cuda).to(ot)
    desc = hb.w4_desc(T, N, K, groups, G, hb.HCA_W4_INT4 if code == "int4" else hb.HCA_W4_E2M1, hb.DTYPE_CODE[xt],
                      hb.DTYPE_CODE[ot], ldx=groups * K + pad if pad else 0, ldo=groups * N + pad if pad else 0)
    ws = torch.full((max(16, hb.w4_linear_workspace_size(desc)),), 0xFF, dtype=U8, device=cuda)   # NaN patterns
    hb.w4_linear(desc, x, xs, codes, scales, rs, out[:, : groups * N] if pad else out, ws)
    w = R.weights(codes, scales, rs, groups, N, K, G, code == "int4")
    xd = x.double().view(T, groups, K) if not pad else x.double().reshape(T, groups, K)
    if xs is not None:
        xd = xd * xs.double()[:, None, None]
    want = torch.einsum("tgk,gnk->tgn", xd, w).reshape(T, -1)
    mag = torch.einsum("tgk,gnk->tgn", xd.abs(), w.abs()).reshape(T, -1)
    # K / 16 accumulations, at most 160 partial sums joined, 4 scalings, 2^-22 of the largest |x| for x in f16
    _close(out[:, : groups * N], want, (K / 16 + 160 + 8) * 2.0 ** -23 * mag + HALF[ot] * want.abs() + 1e-30)
    if pad:
        assert (out[:, groups * N:].float() == 7.0).all()
    again = torch.zeros_like(out)
    hb.w4_linear(desc, x, xs, codes, scales, rs, again[:, : groups * N] if pad else again, ws)
    assert torch.equal(again[:, : groups * N], out[:, : groups * N])          # the same sums in the same order


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e30])
def test_w4_linear_keeps_any_activation_range(cuda, scale):
    """bf16 activations far outside f16's range, token by token; a token of zeros; one large value among small."""
    T, N, K = 5, 200, 512
    _, (codes, scales, rs) = _w4_weights(1, N, K, 32, "e2m1", 6)
    x = _n((T, K), 6, 1)
    x[1] *= scale
    x[2] = 0
    x[3] *= 1e-3
    x[3, 17] = 30000.0 * min(scale, 1e20)
    x = x.to(BF16)
    desc = hb.w4_desc(T, N, K, out_dtype=hb.HCA_F32)
    out = torch.empty(T, N, device=cuda)
    ws = torch.empty(max(16, hb.w4_linear_workspace_size(desc)), dtype=U8, device=cuda)
    hb.w4_linear(desc, x, None, codes, scales, rs, out, ws)
    w = R.weights(codes, scales, rs, 1, N, K, 32, False)[0]
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    # an element far below its token's largest keeps 2^-24 of that largest at least
    low = (x.double().abs().amax(1)[:, None] * w.abs().sum(1)) * 2.0 ** -24
    _close(out, want, (K / 16 + 168) * 2.0 ** -23 * mag + low + 2.0 ** -24 * want.abs() + 1e-36)
    assert (out[2] == 0).all()


@pytest.mark.parametrize("code", ["e2m1", "int4"])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_w4_quantize_follows_its_formula(cuda, code, wt):
    groups, N, K, G = 2, 37, 192, 64
    # divisors as device tensors: torch divides by a host scalar through its rounded reciprocal
    top = torch.tensor(6.0 if code == "e2m1" else 7.0, device=cuda)
    w = _n((groups * N, K), 7, 1)
    w[3] = 0
    w[5, :64] = 0
    w[7] *= 1e-20
    w[9, 64:128] *= 1e-5                       # a group far below its row's maximum
    w = w.to(wt)
    desc = hb.w4_desc(0, N, K, groups, G, hb.HCA_W4_INT4 if code == "int4" else hb.HCA_W4_E2M1)
    codes, scales, rs = hb.w4_quantize(desc, w)
    f = w.float()
    want_rs = f.abs().amax(1) / (top * 448.0)
    assert torch.equal(rs, want_rs)
    assert (scales[:, :, N:] == 0).all() and scales.shape == (groups, K // G, 48)
    am = f.unflatten(1, (-1, G)).abs().amax(2)
    ratio = torch.where(want_rs[:, None] > 0, am / top / want_rs[:, None].clamp_min(1e-38), 0.0)
    want_s = R.nearest_e4m3(ratio.double())
    got_s = scales[:, :, :N].view(E4M3).double().transpose(1, 2).reshape(groups * N, -1)
    assert torch.equal(got_s, want_s)
    step = (want_rs[:, None] * got_s.float()).repeat_interleave(G, 1)
    v = torch.where(step > 0, f / step.clamp_min(1e-38), 0.0).double()
    q = R.unpack(codes)
    if code == "e2m1":
        assert torch.equal(q, R.nearest_e2m1(v.clamp(-6.0, 6.0)))
    else:
        assert torch.equal(q.to(torch.int64), torch.round(v).clamp(-7, 7).to(torch.int64) & 15)


# ------------------------------------------------------------------ 4-bit KV records
KV = [(1, 512, 64, BF16), (1003, 512, 64, BF16), (37, 256, 64, F32), (5, 128, 64, BF16), (4, 64, 0, BF16), (9, 64, 64, F32),
      (11, 80, 16, F32), (3, 512, 0, BF16), (0, 512, 64, BF16)]


def _kv_rows(rows, c, dtype, seed):
    x = _n((max(rows, 1), c), seed, 1) * torch.exp2(_n((max(rows, 1), 1), seed, 2, std=12.0).round())
    if rows >= 4:
        x[1, 32:64] = 0.0                       # an all-zero block
        x[2, 5] = -0.0
        x[3] = 0.0
        x[0, 7] = 1e-30                         # rounds to zero within its block
        x[0, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")   # ties
    return x[:rows].to(dtype)


@pytest.mark.parametrize("rows,c,rd,dtype", KV)
def test_kv_fp4_records(cuda, rows, c, rd, dtype):
    x = _kv_rows(rows, c, dtype, 40 + c + rd)
    n = rows + 3
    rec = torch.full((n, hb.kv_fp4_row_bytes(c, rd)), 0xA5, dtype=U8, device=cuda)
    hb.kv_quant_fp4(x, c, rd, rec)
    back = torch.full((rows, c), float("nan"), dtype=BF16, device=cuda)
    hb.kv_dequant_fp4(rec, c, rd, back)
    assert (rec[rows:] == 0xA5).all()           # records behind the last row
    if rows:
        assert torch.equal(rec[:rows], R.encode_records(x, rd))
        assert torch.equal(back.double(), R.decode_records(rec[:rows], c, rd))
        # the format's error: half a step of E2M1 is at most 2^e and 1/6 of the block's largest value
        z = x[:, : c - rd].double().unflatten(1, (-1, 32)) if c > rd else None
        if z is not None:
            err = (back[:, : c - rd].double().unflatten(1, (-1, 32)) - z).abs()
            assert (err <= z.abs().amax(2, keepdim=True) / 3.0).all()


def test_kv_fp4_slots(cuda):
    rows, c, rd, n = 50, 512, 64, 64
    x = _kv_rows(rows, c, BF16, 3)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:rows].cuda()
    slots[4], slots[9], slots[10], slots[11] = -1, n, 1 << 40, -(1 << 40)
    rec = torch.full((n, 368), 0xA5, dtype=U8, device=cuda)
    hb.kv_quant_fp4(x, c, rd, rec, slots=slots)
    want = torch.full_like(rec, 0xA5)
    ok = (slots >= 0) & (slots < n)
    want[slots[ok]] = R.encode_records(x[ok], rd)
    assert torch.equal(rec, want)
    back = torch.full((rows, c), 9.0, dtype=BF16, device=cuda)
    hb.kv_dequant_fp4(rec, c, rd, back, slots=slots)
    assert (back[~ok] == 0).all()
    assert torch.equal(back[ok].double(), R.decode_records(rec[slots[ok]], c, rd))


@pytest.mark.parametrize("amax", [3e38, 6.0 * 2.0 ** -126, 2.0 ** -127, 1e-44])
def test_kv_fp4_ends_of_the_exponent_range(cuda, amax):
    x = torch.zeros(1, 64, device=cuda)
    x[0, 0], x[0, 33] = amax, -amax / 2
    rec = torch.zeros(1, 48, dtype=U8, device=cuda)
    hb.kv_quant_fp4(x, 64, 0, rec)
    assert torch.equal(rec, R.encode_records(x, 0))


# ------------------------------------------------------------------ attention over 4-bit records
def _attn_case(B, n_h, c, rd, w, m, positions, k=0, page=0, sink=True, cap=None, seed=11, extra_cap=0):
    max_pos = max(positions)
    E = max((max_pos + 1) // m, 1) if cap is None else cap
    E += extra_cap
    s = dict(B=B, n_h=n_h, c=c, rd=rd, w=w, m=m, k=k, max_pos=max(max_pos, 0))
    s["positions"] = torch.tensor(positions, dtype=torch.int32, device="cuda")
    s["q"] = _n((B, n_h, c), seed, 1, BF16)
    s["sink"] = _n((n_h,), seed, 2) if sink else None
    s["win"] = _n((B, max(w, 1), c), seed, 3, BF16) if w else None
    rows = R.encode_records(_n((B * E, c), seed, 4, BF16), rd).view(B, E, -1)
    s["dense"] = rows
    if page:
        per = -(-E // page)
        perm = torch.randperm(B * per + 2, generator=torch.Generator().manual_seed(seed))[: B * per].view(B, per)
        store = torch.full((B * per + 2, page, rows.shape[2]), 0xFF, dtype=U8, device="cuda")   # bf16 NaN where unused
        padded = torch.nn.functional.pad(rows, (0, 0, 0, per * page - E), value=0xFF).view(B, per, page, -1)
        store[perm.cuda()] = padded
        s["pages"], s["store"], s["cap"] = perm.int().cuda(), store, page
    else:
        s["pages"], s["store"], s["cap"] = None, rows, E
    s["idx"] = None
    if k:
        idx = torch.full((B, k), -1, dtype=torch.int32)
        g = torch.Generator().manual_seed(seed + 1)
        for b, p in enumerate(positions):
            V = min((p + 1) // m, E) if p >= 0 else 0
            pick = torch.randperm(V, generator=g)[:k].sort().values
            idx[b, : len(pick)] = pick.int()
        s["idx"] = idx.cuda()
    return s


def _attn_call(s, o=None, ws=None, max_ctas=0, stream=None, scale=0.0):
    d = hb.attn_desc(s["B"], s["n_h"], s["c"], s["rd"], s["w"], s["m"], k=s["k"], dtype=hb.HCA_BF16, max_ctas=max_ctas,
                     scale=scale)
    o = torch.full_like(s["q"], float("nan")) if o is None else o
    if ws is None:
        ws = torch.full((max(16, hb.attend_fp4_workspace_size(d, s["max_pos"])),), 0xFF, dtype=U8, device="cuda")
    hb.attend_fp4(d, s["q"], hb.fp4_cache(s["store"], s["cap"], s["pages"]), s["idx"], s["win"], s["sink"],
                  s["positions"], s["max_pos"], o, ws, stream=stream)
    return o


def _attn_check(s, o, scale=None, dead_pages=()):
    c, rd, w, m = s["c"], s["rd"], s["w"], s["m"]
    scale = c ** -0.5 if scale is None else scale
    for b, pos in enumerate(s["positions"].tolist()):
        pos = min(pos, s["max_pos"])
        E = s["dense"].shape[1]
        V = min((pos + 1) // m, E) if pos >= 0 else 0
        at = s["idx"][b][(s["idx"][b] >= 0) & (s["idx"][b] < V)].long() if s["idx"] is not None else torch.arange(V, device="cuda")
        if dead_pages:
            at = at[[i for i, e in enumerate(at.tolist()) if (b, e // s["cap"]) not in dead_pages]]
        rows = R.decode_records(s["dense"][b, at], c, rd)
        if w and pos >= 0:
            t = torch.arange(max(0, pos - w + 1), pos + 1, device="cuda")
            rows = torch.cat((s["win"][b, t % w].double(), rows))
        q = s["q"][b].double()
        ref, a = R.attend(q, rows, s["sink"].double() if s["sink"] is not None else None, scale, max(pos, 0), rd)
        # p in bf16 (2^-8 of its value at most) and fp32 logits: c / 16 + 16 accumulations of 2^-23 of sum |q k| move p
        # by that much relative, counted twice (its own and the normalisation's); the rotation, the exponential and
        # the joining of parts stay below 2^-18; then the output's rounding
        dz = (c / 16 + 16) * 2.0 ** -23 * scale * (q.abs() @ rows.abs().t()).amax().item() if rows.shape[0] else 0.0
        _close(o[b], ref, (2.0 ** -8 + 2 * dz + 2.0 ** -18) * a + 2.0 ** -8 * ref.abs() + 1e-30)
        if rows.shape[0] == 0:
            assert (o[b] == 0).all()


ATTN = [
    # B, n_h, c, rd, w, m, positions, k, page
    (1, 16, 128, 64, 128, 1, [500], 0, 0),
    (1, 1, 128, 64, 0, 1, [0], 0, 0),                                # one key
    (3, 8, 256, 64, 16, 4, [0, 3, 2], 0, 0),                         # a window of one to four tokens, 0 or 1 entries
    (4, 64, 512, 64, 128, 4, [131, 4099, 70, -1], 0, 16),            # a sequence without keys
    (2, 64, 512, 64, 40, 4, [2047, 1023], 64, 24),
    (2, 24, 512, 64, 0, 128, [127, 8000], 0, 24),                    # no window
    (2, 64, 512, 64, 128, 4, [100, 9000], 512, 64),                  # an index list longer than what is visible
    (5, 17, 256, 64, 7, 2, [1, 64, 65, 127, 129], 0, 8),             # odd head count, tiles cut by one
    (2, 33, 128, 0, 5, 1, [63, 64], 0, 0),                           # no RoPE channels
    (2, 16, 128, 128, 5, 1, [63, 200], 0, 0),                        # only RoPE channels
    (1, 64, 512, 64, 128, 128, [1048575], 0, 24),                    # the long end
    (40, 16, 256, 64, 20, 1, list(range(0, 400, 10)), 0, 0),         # more sequences than split CTAs, ragged
    (300, 8, 128, 64, 3, 4, [(7 * i) % 90 for i in range(300)], 0, 4),
    (1, 64, 512, 64, 1, 1, [20000], 0, 0),                           # more parts than one merge pass
]


@pytest.mark.parametrize("B,n_h,c,rd,w,m,positions,k,page", ATTN)
def test_attend_fp4(cuda, B, n_h, c, rd, w, m, positions, k, page):
    s = _attn_case(B, n_h, c, rd, w, m, positions, k=k, page=page)
    o = _attn_call(s)
    assert hb.device_status() == hb.HCA_OK
    _attn_check(s, o)
    assert torch.equal(_attn_call(s), o)                             # a fixed order of sums
    if B <= 5:                                                       # any CTA budget
        for n in (1, 3):
            _attn_check(s, _attn_call(s, max_ctas=n))


def test_attend_fp4_without_sink_and_with_a_scale(cuda):
    s = _attn_case(3, 16, 128, 64, 8, 4, [300, -5, 2], sink=False)
    o = _attn_call(s, scale=0.3)
    _attn_check(s, o, scale=0.3)
    assert (o[1] == 0).all()


def test_attend_fp4_bad_entries_are_skipped(cuda):
    """Pages outside the store, entries beyond the visible ones, negative ones, capacity below what is visible, a
    position above max_pos, a duplicate that counts twice: nothing outside the tensors is read."""
    s = _attn_case(3, 16, 256, 64, 16, 4, [400, 399, 200], page=16, seed=21)
    s["pages"][0, 1], s["pages"][1, 3], s["pages"][2, 0] = -1, 1 << 30, -(1 << 31)
    _attn_check(s, _attn_call(s), dead_pages={(0, 1), (1, 3), (2, 0)})
    s = _attn_case(2, 16, 256, 64, 16, 4, [400, 90], k=64, seed=22)
    s["idx"][0, 3], s["idx"][0, 5], s["idx"][0, 7] = 100, 1 << 30, -(1 << 31)
    s["idx"][1] = -1                                                # a list that leaves the window alone
    _attn_check(s, _attn_call(s))
    s["idx"][0, 10] = s["idx"][0, 11]                                # twice the same entry
    _attn_check(s, _attn_call(s))
    s = _attn_case(2, 16, 256, 64, 16, 4, [400, 90], cap=30, seed=23)
    _attn_check(s, _attn_call(s))
    s = _attn_case(2, 16, 256, 64, 16, 4, [400, 500], cap=126, seed=24)
    s["max_pos"] = 450
    _attn_check(s, _attn_call(s))
    s = _attn_case(2, 16, 128, 64, 0, 4, [2, 400], seed=25)          # the first sequence sees nothing
    s["pages"] = torch.full((2, 7), -1, dtype=torch.int32, device="cuda")
    s["cap"], s["store"] = 16, s["store"].reshape(-1, s["store"].shape[2])[: 16 * 5].view(5, 16, -1).contiguous()
    assert (_attn_call(s) == 0).all()


def test_attend_fp4_large_logits_and_masked_nan(cuda):
    """Logits up to +-300 (the running maximum moves), NaN in records and ring rows that no query sees."""
    s = _attn_case(2, 16, 256, 64, 32, 1, [700, 20], seed=31, extra_cap=50)
    s["q"] = (s["q"].float() * 12.0).to(BF16)
    q = 192 // 2
    for b, pos in enumerate((700, 20)):
        s["store"][b, pos + 1:, q: q + 128] = 0xFF                   # bf16 NaN in the RoPE channels
    s["win"][1, 21:] = float("nan")
    o = _attn_call(s)
    s["win"][1, 21:] = 0
    _attn_check(s, o)


def test_attend_fp4_streams_graphs_and_shared_workspaces(cuda):
    """Captured and replayed with positions changed in between; two captured graphs with one workspace, replayed in
    turn; another stream; both against the eager call."""
    s = _attn_case(4, 32, 512, 64, 64, 4, [3000, 1000, 2, 1999], page=16, seed=41)
    t = _attn_case(2, 64, 512, 64, 64, 4, [2500, 3000], k=64, page=16, seed=42)
    d = [hb.attn_desc(u["B"], u["n_h"], 512, 64, 64, 4, k=u["k"], dtype=hb.HCA_BF16) for u in (s, t)]
    ws = torch.empty(max(16, *(hb.attend_fp4_workspace_size(x, 3000) for x in d)), dtype=U8, device=cuda)
    os, ot = torch.zeros_like(s["q"]), torch.zeros_like(t["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gs, gt = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        _attn_call(s, os, ws)
        _attn_call(t, ot, ws)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(gs):
        _attn_call(s, os, ws)
    with torch.cuda.graph(gt):
        _attn_call(t, ot, ws)
    for pos in ([3000, 1000, 2, 1999], [5, 3000, 2999, -1]):
        s["positions"].copy_(torch.tensor(pos, dtype=torch.int32))
        for _ in range(2):
            os.fill_(float("nan"))
            ot.fill_(float("nan"))
            gs.replay()
            gt.replay()
            _attn_check(s, os)
            _attn_check(t, ot)


# ------------------------------------------------------------------ together
def test_a_decode_step_of_the_operators(cuda):
    """One layer's token step: norm with 8-bit output -> 4-bit-weight q and KV projections -> KV rows into a paged
    4-bit cache -> attention -> grouped 4-bit-weight output projection -> norm; each stage against the float64 formula
    on the inputs that it got, and the whole step captured and replayed bit for bit."""
    B, d, n_h, c, rd, w, g, dg = 5, 512, 16, 128, 64, 16, 4, 64
    pos = [40, 63, 64, 0, 100]
    page, per = 8, 16
    mk = lambda groups, N, K, G, code, seed: _w4_weights(groups, N, K, G, code, seed)[1]
    wq, wkv = mk(1, n_h * c, d, 64, "e2m1", 51), mk(1, c, d, 32, "int4", 52)
    wa, wb = mk(g, dg, n_h // g * c, 128, "e2m1", 53), mk(1, d, g * dg, 32, "e2m1", 54)
    store = R.encode_records(_n((B * per * page, c), 50, 1, BF16), rd).view(B * per, page, -1)
    pages = torch.randperm(B * per, generator=torch.Generator().manual_seed(5)).int().view(B, per).cuda()
    positions = torch.tensor(pos, dtype=torch.int32, device=cuda)
    slots = pages.long()[torch.arange(B), positions.long() // page] * page + positions.long() % page
    ring, sink, gamma = _n((B, w, c), 50, 2, BF16), _n((n_h,), 50, 3), 1 + _n((d,), 50, 4, std=0.1)
    h, res = _n((B, d), 50, 5, BF16), _n((B, d), 50, 6, BF16)
    E = lambda *sh, t=BF16: torch.empty(*sh, dtype=t, device=cuda)
    res1, res2, x8, xs, x8b, xsb = E(B, d), E(B, d), E(B, d, t=E4M3), E(B, 1, t=F32), E(B, d, t=E4M3), E(B, 1, t=F32)
    q, kv, o, low, y = E(B, n_h * c), E(B, c), E(B, n_h, c), E(B, g * dg), E(B, d)
    nd = hb.norm_desc(B, d, out_dtype=hb.HCA_FP8E4M3)
    dq = hb.w4_desc(B, n_h * c, d, 1, 64, x_dtype=hb.HCA_FP8E4M3)
    dkv = hb.w4_desc(B, c, d, 1, 32, hb.HCA_W4_INT4, x_dtype=hb.HCA_FP8E4M3)
    da, db = hb.w4_desc(B, dg, n_h // g * c, g, 128), hb.w4_desc(B, d, g * dg, 1, 32)
    at = hb.attn_desc(B, n_h, c, rd, w, 1, dtype=hb.HCA_BF16)
    nws = max([hb.w4_linear_workspace_size(x) for x in (dq, dkv, da, db)] + [hb.attend_fp4_workspace_size(at, 127)])
    ws = E(max(16, nws), t=U8)
    cache = hb.fp4_cache(store, page, pages)

    def step():
        hb.add_rms_norm(nd, h, res, gamma, res1, x8, xs)
        hb.w4_linear(dq, x8, xs, *wq, q, ws)
        hb.w4_linear(dkv, x8, xs, *wkv, kv, ws)
        hb.kv_quant_fp4(kv, c, rd, store, slots=slots)
        ring[torch.arange(B, device=cuda), positions.long() % w] = kv
        hb.attend_fp4(at, q.view(B, n_h, c), cache, None, ring, sink, positions, 127, o, ws)
        hb.w4_linear(da, o.view(B, -1), None, *wa, low, ws)
        hb.w4_linear(db, low, None, *wb, y, ws)
        hb.add_rms_norm(nd, y, res1, gamma, res2, x8b, xsb)

    step()
    torch.cuda.synchronize()

    def lin(x, wts, groups, N, K, G, int4):
        wd = R.weights(*wts, groups, N, K, G, int4)
        xd = x.reshape(B, groups, K)
        return (torch.einsum("bgk,gnk->bgn", xd, wd).reshape(B, -1), torch.einsum("bgk,gnk->bgn", xd.abs(), wd.abs()).reshape(B, -1))

    def check_lin(got, ref, K):
        _close(got, ref[0], (K / 16 + 168) * 2.0 ** -23 * ref[1] + 2.0 ** -8 * ref[0].abs())
    z, yn = R.rms_norm(h, res, gamma, 1e-6)
    _close(res1, z, (2.0 ** -8 + 2.0 ** -23) * z.abs() + 2.0 ** -24 * (h.double().abs() + res.double().abs()))
    x = x8.double() * xs.double()
    _close(x, yn, 2.0 ** -4 * 1.01 * yn.abs() + 2.0 ** -10 * xs.double())
    check_lin(q, lin(x, wq, 1, n_h * c, d, 64, False), d)
    check_lin(kv, lin(x, wkv, 1, c, d, 32, True), d)
    assert torch.equal(store.view(-1, store.shape[2])[slots], R.encode_records(kv, rd))
    dense = store[pages.long()].view(B, per * page, -1)
    s = dict(B=B, n_h=n_h, c=c, rd=rd, w=w, m=1, k=0, max_pos=127, positions=positions, q=q.view(B, n_h, c), sink=sink, win=ring,
             dense=dense, idx=None)
    _attn_check(s, o)
    check_lin(low, lin(o.double().view(B, -1), wa, g, dg, n_h // g * c, 128, False), n_h // g * c)
    check_lin(y, lin(low.double(), wb, 1, d, g * dg, 32, False), g * dg)
    z2, yn2 = R.rms_norm(y, res1, gamma, 1e-6)
    _close(x8b.double() * xsb.double(), yn2, 2.0 ** -4 * 1.01 * yn2.abs() + 2.0 ** -10 * xsb.double())

    eager = [t.clone() for t in (res1, x8.view(U8), q, kv, o, low, y, res2, x8b.view(U8), store)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q, kv, o, low, y, res2):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert hb.device_status() == hb.HCA_OK
    for a, b in zip(eager, (res1, x8.view(U8), q, kv, o, low, y, res2, x8b.view(U8), store)):
        assert torch.equal(a, b)


def test_another_current_device_is_refused_and_streams_are_used(cuda):
    """The calls run on the stream they are given: work queued there before them is seen."""
    rows, d = 64, 4096
    side = torch.cuda.Stream()
    x, out = torch.zeros(rows, d, device=cuda), torch.empty(rows, d, device=cuda)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.ones(4096, 4096, device=cuda)
        for _ in range(4):
            big = big @ big * 1e-4
        x.copy_(big[:rows])
    hb.add_rms_norm(hb.norm_desc(rows, d, hb.HCA_F32, out_dtype=hb.HCA_F32), x, None, None, None, out, stream=side)
    side.synchronize()
    _close(out, R.rms_norm(x, None, None, 1e-6)[1], 1e-5)
