"""Float64 references of the low-bit decode operators, written from their
formulas on torch tensors of any device: code tables, record and weight
decoding, nearest-value rounding by search, attention by a softmax over the
gathered rows."""
import math

import torch

E2M1_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e2m1_values(codes):
    t = torch.tensor(E2M1_MAG, dtype=torch.float64, device=codes.device)
    v = t[(codes & 7).long()]
    return torch.where(codes >= 8, -v, v)


def nearest_e2m1(v):
    """Codes of the E2M1 values nearest to v (float64), ties to the even code, zero as +0."""
    t = torch.tensor(E2M1_MAG, dtype=torch.float64, device=v.device)
    d = (v.abs()[..., None] - t).abs()
    best = d.amin(-1, keepdim=True)
    hit = d == best
    k = torch.arange(8, device=v.device)
    even = torch.where(hit & (k % 2 == 0), k, -1).amax(-1)
    code = torch.where(even >= 0, even, torch.where(hit, k, -1).amax(-1))
    return torch.where((v < 0) & (code > 0), code + 8, code).to(torch.uint8)


def unpack(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def row_bytes(c, rd):
    return -(-((c - rd) // 2 + 2 * rd + (c - rd) // 32) // 16) * 16


def encode_records(x, rd):
    """Rows x [n, c] (bf16 / f32) -> records [n, bytes]."""
    n, c = x.shape
    q = c - rd
    z = x[:, :q].double().unflatten(1, (-1, 32))
    amax = z.abs().amax(-1)
    safe = amax.clamp_min(1e-300)
    e = torch.floor(torch.log2(safe / 6.0))
    e = torch.where(safe > 6.0 * torch.exp2(e), e + 1, e)          # smallest e with amax <= 6 * 2^e
    e = torch.where(safe <= 6.0 * torch.exp2(e - 1), e - 1, e).clamp_min(-126)
    codes = nearest_e2m1(z / torch.exp2(e)[..., None]).flatten(1)
    rec = torch.zeros(n, row_bytes(c, rd), dtype=torch.uint8, device=x.device)
    rec[:, : q // 2] = pack(codes)
    rec[:, q // 2 : q // 2 + 2 * rd] = x[:, q:].to(torch.bfloat16).contiguous().view(torch.uint8)
    rec[:, q // 2 + 2 * rd : q // 2 + 2 * rd + q // 32] = torch.where(amax > 0, e + 127, 0.0).to(torch.uint8)
    return rec


def decode_records(rec, c, rd):
    q = c - rd
    v = e2m1_values(unpack(rec[..., : q // 2])).unflatten(-1, (-1, 32))
    e = rec[..., q // 2 + 2 * rd : q // 2 + 2 * rd + q // 32].double() - 127.0
    rope = rec[..., q // 2 : q // 2 + 2 * rd].contiguous().view(torch.bfloat16).double()
    return torch.cat(((v * torch.exp2(e)[..., None]).flatten(-2), rope), -1)


def nearest_e4m3(v):
    """The e4m3 values nearest to v (float64), ties to even, saturating at 448."""
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent.clamp_min(-5) - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def weights(codes, scales, row_scale, groups, N, K, G, int4):
    """Float64 weights [groups, N, K]."""
    q = unpack(codes).view(groups, N, K)
    v = torch.where(q >= 8, q.double() - 16.0, q.double()) if int4 else e2m1_values(q)
    s = scales.view(torch.float8_e4m3fn)[:, :, :N].double().transpose(1, 2).repeat_interleave(G, 2)
    return v * s * row_scale.double().view(groups, N, 1)


def rms_norm(x, res, gamma, eps):
    z = x.double() + (res.double() if res is not None else 0.0)
    y = z / torch.sqrt(z.square().mean(1, keepdim=True) + eps)
    return z, y * (gamma.double() if gamma is not None else 1.0)


def attend(q, rows, sink, scale, pos, rd, theta=10000.0):
    """One query token: q [n_h, c], rows [keys, c] -> (o, a): a bounds sum p |v| / (sum p + sink), pairs added
    where the rotation mixes them."""
    n_h, c = q.shape
    if rows.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    z = q @ rows.t() * scale
    s = sink if sink is not None else torch.full((n_h,), -math.inf, dtype=torch.float64, device=q.device)
    top = torch.maximum(z.amax(1), s)
    p = torch.exp(z - top[:, None])
    den = (p.sum(1) + torch.exp(s - top))[:, None]
    o, a = p @ rows / den, p @ rows.abs() / den
    if rd:
        f = theta ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=q.device) / rd)
        co, si = torch.cos(pos * f), torch.sin(pos * f)
        u, v = o[:, c - rd :: 2].clone(), o[:, c - rd + 1 :: 2].clone()
        o[:, c - rd :: 2], o[:, c - rd + 1 :: 2] = u * co + v * si, v * co - u * si
        both = a[:, c - rd :: 2] + a[:, c - rd + 1 :: 2]
        a[:, c - rd :: 2] = both
        a[:, c - rd + 1 :: 2] = both
    return o, a
