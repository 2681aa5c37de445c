"""The low-bit decode operators: what they are measured on, and their plain forms.

Four operators of one decode step between two attention layers: residual addition + RMSNorm with an 8-bit output
(`norm`), products of a few tokens with 4-bit weights (`w4`), KV rows written to and read from 4-bit records (`kv`), and
single-token attention over a cache of such records (`attend`).  `run` computes them with elementary torch operations in
32 bits, or, where `own` is true, with the framework's kernels.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
INT4 = (0.0, 1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0, -8.0, -7.0, -6.0, -5.0, -4.0, -3.0, -2.0, -1.0)


# ------------------------------------------------------------------------------------------------------------- cases
def _norm(name, rows, d, x="bf16", out="e4m3", group=0):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "x": x, "out": out, "group": group}


def _w4(name, T, N, K, groups=1, code="e2m1", G=32, x="bf16", out="bf16"):
    return {"name": name, "op": "w4", "T": T, "N": N, "K": K, "groups": groups, "code": code, "G": G, "x": x, "out": out}


def _kv(name, rows, c, rd, x="bf16"):
    return {"name": name, "op": "kv", "rows": rows, "c": c, "rd": rd, "x": x}


def _attend(name, B, n_h, c, rd, w, m, pos, k=0, page=0, spread=0.0):
    return {"name": name, "op": "attend", "B": B, "n_h": n_h, "c": c, "rd": rd, "w": w, "m": m, "pos": pos, "k": k,
            "page": page, "spread": spread}


def listed():
    return [
        # one decode token's hidden state between two layers (d_model 4096): latency
        _norm("norm_one_token", 1, 4096),
        # a decode batch, 8-bit groups of 128 for the next projection
        _norm("norm_decode_b32", 32, 4096, group=128),
        # a prompt's hidden states in a model of an odd width, bf16 out
        _norm("norm_prompt_16k", 16411, 4104, out="bf16"),
        # the window KV projection of one token (d 4096 -> c 512): the smallest product
        _w4("w4_kv_one_token", 1, 512, 4096),
        # the query up-projection of a decode batch (d_c 1024 -> 64 heads x 512) on 8-bit activations
        _w4("w4_uq_b32", 32, 32768, 1024, x="e4m3", G=64),
        # the grouped first stage of the output projection (8 groups of 8 heads x 512 -> 1024 each)
        _w4("w4_oproj_b7", 7, 1024, 4096, groups=8, code="int4", G=128),
        # a wide layer at the largest decode batch of one tile, an odd number of outputs, fp32 out
        _w4("w4_wide_b64", 64, 28677, 8192, out="f32"),
        # a decode batch's new entries stored in the cache and read back
        _kv("kv_decode_b32", 32, 512, 64),
        # a prompt's entries stored (65536 tokens at ratio 4, 8 sequences) and read back
        _kv("kv_prompt", 131075, 512, 64),
        # one short sequence, few heads, one entry per token (no compression): latency
        _attend("attend_short", 1, 16, 128, 64, 128, 1, 500),
        # a CSA layer's decode step at 131072 tokens: top-512 entries of a paged cache + window
        _attend("attend_csa_b32", 32, 64, 512, 64, 128, 4, 131072, k=512, page=64),
        # an HCA layer's decode step over ragged sequences of up to a million tokens, paged
        _attend("attend_hca_ragged", 32, 64, 512, 64, 128, 128, 1048576, page=24, spread=0.9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "w4", "kv", "attend"))
    if op == "norm":
        out, group = rng.choice((("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 64), ("e4m3", 128)))
        d = 128 * _log(rng, 2, 64) if group else _log(rng, 256, 8192)
        return {"op": op, "rows": _log(rng, 1, 30_000_000 // d), "d": d, "x": rng.choice(("bf16", "bf16", "f32")), "out": out,
                "group": group}
    if op == "w4":
        G = rng.choice((32, 64, 128))
        groups = rng.choice((1, 1, 1, 8))
        K, N = 128 * _log(rng, 2, 64), _log(rng, 256, 28000 // groups)
        return {"op": op, "T": _log(rng, 1, 64), "N": N, "K": K, "groups": groups, "code": rng.choice(("e2m1", "int4")), "G": G,
                "x": rng.choice(("bf16", "e4m3")), "out": rng.choice(("bf16", "f32"))}
    if op == "kv":
        c, rd = rng.choice(((512, 64), (256, 64), (128, 64)))
        return {"op": op, "rows": _log(rng, 8, 130_000), "c": c, "rd": rd, "x": rng.choice(("bf16", "f32"))}
    c = rng.choice((128, 256, 512))
    m = rng.choice((1, 4, 128))
    k = rng.choice((0, 0, 64, 512)) if m == 4 else 0
    B = _log(rng, 1, 32)
    entries = _log(rng, 16, min(8192, 130_000 // B))
    return {"op": op, "B": B, "n_h": rng.choice((8, 16, 24, 64)), "c": c, "rd": 64, "w": rng.choice((0, 40, 128)), "m": m,
            "pos": entries * m + rng.randrange(m), "k": k, "page": rng.choice((0, 16, 24, 64)), "spread": rng.choice((0.0, 0.9))}


# ------------------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _encode_e2m1(v):
    """Codes of the E2M1 values nearest to v, ties to the even mantissa, saturating at 6; zero as +0."""
    a = v.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return mag + 8 * ((v < 0) & (mag > 0)).to(torch.uint8)


def _pack(codes):
    """[..., n] codes -> [..., n / 2] bytes, the even channel in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _record_bytes(c, rd):
    return -(-((c - rd) // 2 + 2 * rd + (c - rd) // 32) // 16) * 16


def _records(x, rd):
    """bf16 rows [n, c] as 4-bit records: codes, RoPE channels, one exponent byte per 32 codes, padding."""
    n, c = x.shape
    nq = c - rd
    z = x[:, :nq].float().unflatten(1, (-1, 32))
    f, e = torch.frexp(z.abs().amax(-1))                   # amax = f * 2^e, f in [0.5, 1)
    e = torch.where(f > 0.75, e - 2, e - 3).clamp(-126, 126)   # the smallest e with amax <= 6 * 2^e
    e = torch.where(f == 0, torch.full_like(e, -127), e)
    codes = _encode_e2m1(torch.ldexp(z, -e.unsqueeze(-1))).flatten(1)
    rec = torch.zeros(n, _record_bytes(c, rd), dtype=torch.uint8, device=x.device)
    rec[:, : nq // 2] = _pack(codes)
    rec[:, nq // 2 : nq // 2 + 2 * rd] = x[:, nq:].contiguous().view(torch.uint8)
    rec[:, nq // 2 + 2 * rd : nq // 2 + 2 * rd + nq // 32] = (e + 127).to(torch.uint8)
    return rec


def prepare(case, seed):
    g = _gen(seed)

    def normal(*shape, dtype=F32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        rows, d, dt = case["rows"], case["d"], DTYPES[case["x"]]
        s["x_"], s["res"] = normal(rows, d, dtype=dt), normal(rows, d, dtype=dt, std=4.0)
        s["gamma"] = 1.0 + normal(d, std=0.1)
        s["res_out"], s["out_"] = torch.empty_like(s["res"]), torch.empty(rows, d, dtype=DTYPES[case["out"]], device="cuda")
        s["scale"] = torch.empty(rows, d // case["group"] if case["group"] else 1, device="cuda") if case["out"] == "e4m3" else None
    elif case["op"] == "w4":
        T, N, K, G, n = case["T"], case["N"], case["K"], case["G"], case["groups"]
        top = 6.0 if case["code"] == "e2m1" else 7.0
        codes, scales, rows = [], [], []
        for _ in range(n):
            w = normal(N, K, std=K ** -0.5).unflatten(1, (-1, G))
            amax = w.abs().amax(-1)
            rs = (amax.amax(-1) / (top * 448.0)).clamp_min(1e-30)
            sc = (amax / top / rs[:, None]).to(E4M3)
            v = w / (rs[:, None] * sc.float()).clamp_min(1e-30)[..., None]
            q = _encode_e2m1(v) if case["code"] == "e2m1" else v.round().clamp(-7, 7).to(torch.int8).view(torch.uint8) & 15
            codes.append(_pack(q.flatten(1)))
            pad = torch.zeros(K // G, -(-N // 16) * 16, dtype=torch.uint8, device="cuda")
            pad[:, :N] = sc.view(torch.uint8).t()
            scales.append(pad)
            rows.append(rs)
        s["codes"], s["scales"], s["row_scale"] = torch.cat(codes), torch.stack(scales), torch.cat(rows)
        x = normal(T, n * K)
        s["x_scale"] = None
        if case["x"] == "e4m3":
            s["x_scale"] = x.abs().amax(1) / 448.0
            s["x_"] = (x / s["x_scale"][:, None]).to(E4M3)
        else:
            s["x_"] = x.to(BF16)
        s["out_"] = torch.empty(T, n * N, dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] == "kv":
        rows, c, rd = case["rows"], case["c"], case["rd"]
        s["x_"] = normal(rows, c, dtype=DTYPES[case["x"]])
        # the cache slots that the rows go to (a paged cache hands them out in any order)
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")
        s["cache"] = torch.zeros(rows, _record_bytes(c, rd), dtype=torch.uint8, device="cuda")
        s["out_"] = torch.empty(rows, c, dtype=BF16, device="cuda")
    else:
        B, c, rd, m, k = case["B"], case["c"], case["rd"], case["m"], case["k"]
        pos = (case["pos"] * (1.0 - case["spread"] * torch.rand(B, generator=g, device="cuda", dtype=torch.float64))).long()
        pos[0] = case["pos"]
        cap = (case["pos"] + 1) // m
        s["positions"] = pos.int()
        s["q"], s["sink"] = normal(B, case["n_h"], c, dtype=BF16), normal(case["n_h"])
        s["win"] = normal(B, max(case["w"], 1), c, dtype=BF16)
        if case["page"]:
            per = -(-cap // case["page"])
            n = B * per * case["page"]
            s["pages"] = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
        else:
            n, s["pages"] = B * cap, None
        rec = torch.empty(n, _record_bytes(c, rd), dtype=torch.uint8, device="cuda")
        for i in range(0, n, 65536):
            rec[i : i + 65536] = _records(normal(min(65536, n - i), c, dtype=BF16), rd)
        s["rows_"] = rec.view(-1, case["page"] or cap, rec.shape[1])
        s["cap"] = case["page"] or cap
        s["idx"] = None
        if k:
            V = ((pos + 1) // m)[:, None]
            at = torch.sort(torch.rand(B, cap, generator=g, device="cuda").masked_fill(torch.arange(cap, device="cuda") >= V, 2.0), 1)
            at = torch.where(at.values < 2.0, at.indices, cap)[:, :k].sort(1).values
            s["idx"] = torch.nn.functional.pad(torch.where(at < cap, at, -1), (0, k - at.shape[1]), value=-1).int()
        s["out_"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def _codes(b):
    """Bytes [..., n / 2] -> their codes [..., n], as indices."""
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).int()


def _values(rec, c, rd):
    """Records [..., bytes] -> fp32 rows [..., c]."""
    nq = c - rd
    table = torch.tensor(E2M1, device=rec.device)
    e = rec[..., nq // 2 + 2 * rd : nq // 2 + 2 * rd + nq // 32].int() - 127
    v = torch.ldexp(table[_codes(rec[..., : nq // 2])].unflatten(-1, (-1, 32)), e.unsqueeze(-1)).flatten(-2)
    return torch.cat((v, rec[..., nq // 2 : nq // 2 + 2 * rd].contiguous().view(BF16).float()), -1)


def _plain_norm(s):
    z = s["x_"].float() + s["res"].float()
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + 1e-6) * s["gamma"]
    if s["out"] != "e4m3":
        return {"res": z.to(s["res"].dtype), "out": y.to(DTYPES[s["out"]])}
    y = y.unflatten(1, (-1, s["group"] or s["d"]))
    scale = y.abs().amax(-1) / 448.0
    q = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0).flatten(1)
    return {"res": z.to(s["res"].dtype), "out": q.clamp(-448.0, 448.0).to(E4M3), "scale": scale}


def _plain_w4(s):
    T, N, K, G, n = s["T"], s["N"], s["K"], s["G"], s["groups"]
    table = torch.tensor(E2M1 if s["code"] == "e2m1" else INT4, device="cuda")
    w = table[_codes(s["codes"])].view(n, N, K // G, G)
    w = w * s["scales"].view(E4M3)[:, :, :N].float().transpose(1, 2).unsqueeze(-1)
    y = torch.matmul(s["x_"].float().view(T, n, K).transpose(0, 1), w.view(n, N, K).transpose(1, 2))   # [n, T, N]
    y = y.transpose(0, 1).reshape(T, n * N) * s["row_scale"]
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    return y.to(DTYPES[s["out"]])


def _plain_kv(s):
    nq = s["c"] - s["rd"]
    z = s["x_"][:, :nq].float().unflatten(1, (-1, 32))
    f, e = torch.frexp(z.abs().amax(-1, keepdim=True))
    e = torch.where(f > 0.75, e - 2, e - 3).clamp(-126, 126)
    v = torch.tensor(E2M1, device="cuda")[_encode_e2m1(torch.ldexp(z, -e)).int()]
    v = torch.cat((torch.ldexp(v, e).flatten(1), s["x_"][:, nq:].to(BF16).float()), 1)
    return v.to(BF16)


def _plain_attend(s):
    B, c, rd, w, m = s["B"], s["c"], s["rd"], s["w"], s["m"]
    pos = s["positions"].long()[:, None]
    V = (pos + 1) // m
    at = s["idx"].long() if s["idx"] is not None else torch.arange((s["pos"] + 1) // m, device="cuda").expand(B, -1)
    live = (at >= 0) & (at < V)
    at = at.clamp_min(0)
    if s["pages"] is not None:
        rows = s["rows_"][s["pages"].long().gather(1, at // s["page"]), at % s["page"]]
    else:
        rows = s["rows_"][torch.arange(B, device="cuda")[:, None], at]
    keys = _values(rows, c, rd)
    if w:
        t = pos - torch.arange(w, device="cuda")
        live = torch.cat((t >= 0, live), 1)
        win = s["win"][torch.arange(B, device="cuda")[:, None], t.clamp_min(0) % w].float()
        keys = torch.cat((win, keys), 1)
    z = torch.matmul(s["q"].float(), keys.transpose(1, 2)) * c ** -0.5
    z = torch.cat((z.masked_fill(~live[:, None], -math.inf), s["sink"].expand(B, -1).unsqueeze(-1)), 2)
    p = torch.exp(z - z.amax(2, keepdim=True))
    o = torch.matmul(p[..., :-1] / p.sum(2, keepdim=True), keys)
    ang = pos.double() * 10000.0 ** (-torch.arange(0, rd, 2, device="cuda", dtype=torch.float64) / rd)
    co, si = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = o[..., c - rd :: 2], o[..., c - rd + 1 :: 2]
    return torch.cat((o[..., : c - rd], torch.stack((a * co + b * si, b * co - a * si), -1).flatten(2)), 2).to(BF16)


# ------------------------------------------------------------------------------------------------- framework's calls
def _own(s):
    from long_context_compressed_hca_b200 import binding as hb

    if s["op"] == "norm":
        if "desc" not in s:
            s["desc"] = hb.norm_desc(s["rows"], s["d"], x_dtype=hb.DTYPE_CODE[s["x_"].dtype], res_dtype=hb.DTYPE_CODE[s["res"].dtype],
                                     out_dtype=hb.DTYPE_CODE[s["out_"].dtype], scale_group=s["group"])
        hb.add_rms_norm(s["desc"], s["x_"], s["res"], s["gamma"], s["res_out"], s["out_"], s["scale"])
        out = {"res": s["res_out"], "out": s["out_"]}
        return out if s["scale"] is None else out | {"scale": s["scale"]}
    if s["op"] == "w4":
        if "desc" not in s:
            s["desc"] = hb.w4_desc(s["T"], s["N"], s["K"], groups=s["groups"], scale_group=s["G"],
                                   code=hb.HCA_W4_E2M1 if s["code"] == "e2m1" else hb.HCA_W4_INT4,
                                   x_dtype=hb.DTYPE_CODE[s["x_"].dtype], out_dtype=hb.DTYPE_CODE[s["out_"].dtype])
            s["ws"] = torch.empty(max(16, hb.w4_linear_workspace_size(s["desc"])), dtype=torch.uint8, device="cuda")
        hb.w4_linear(s["desc"], s["x_"], s["x_scale"], s["codes"], s["scales"], s["row_scale"], s["out_"], s["ws"])
        return s["out_"]
    if s["op"] == "kv":
        hb.kv_quant_fp4(s["x_"], s["c"], s["rd"], s["cache"], slots=s["slots"])
        hb.kv_dequant_fp4(s["cache"], s["c"], s["rd"], s["out_"], slots=s["slots"])
        return s["out_"]
    if "desc" not in s:
        s["desc"] = hb.attn_desc(s["B"], s["n_h"], s["c"], s["rd"], s["w"], s["m"], k=s["k"], dtype=hb.HCA_BF16)
        s["store"] = hb.fp4_cache(s["rows_"], s["cap"], s["pages"])
        s["ws"] = torch.empty(max(16, hb.attend_fp4_workspace_size(s["desc"], s["pos"])), dtype=torch.uint8, device="cuda")
    hb.attend_fp4(s["desc"], s["q"], s["store"], s["idx"], s["win"] if s["w"] else None, s["sink"], s["positions"], s["pos"],
                  s["out_"], s["ws"])
    return s["out_"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "w4": _plain_w4, "kv": _plain_kv, "attend": _plain_attend}[state["op"]](state)


# -------------------------------------------------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] == "norm":
        n = case["rows"] * case["d"]
        per_row = case["d"] // case["group"] if case["group"] else 1
        return {"bytes": n * (3 * size[case["x"]] + size[case["out"]]) + 4 * case["d"] + (4 * case["rows"] * per_row if case["out"] == "e4m3" else 0),
                "flops": 6 * n}
    if case["op"] == "w4":
        T, N, K, n = case["T"], case["N"], case["K"], case["groups"]
        w = n * N * K
        return {"bytes": w / 2 + w // case["G"] + 4 * n * N + T * n * K * size[case["x"]] + T * n * N * size[case["out"]],
                "flops": 2 * T * w}
    if case["op"] == "kv":
        # each row is read, its record written, the record read and the row written; slots are read twice
        return {"bytes": case["rows"] * (case["c"] * (size[case["x"]] + 2) + 2 * _record_bytes(case["c"], case["rd"]) + 16),
                "flops": 4 * case["rows"] * case["c"]}
    # every sequence's visible entries (their mean where positions spread), its window, its queries and output
    mean = (case["pos"] + 1) // case["m"] * (1.0 - case["spread"] / 2 * (case["B"] - 1) / case["B"])
    keys = min(case["k"], mean) if case["k"] else mean
    win = min(case["w"], case["pos"] + 1)
    return {"bytes": case["B"] * (keys * _record_bytes(case["c"], case["rd"]) + win * 2 * case["c"] + 4 * case["n_h"] * case["c"]
                                  + 4 * case["k"]),
            "flops": 4 * case["B"] * case["n_h"] * case["c"] * (keys + win)}


# ------------------------------------------------------------------------------------------------------------- exact
def _e4m3(v):
    """The e4m3 value nearest to v (float64), ties to even, saturating at 448."""
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent.clamp_min(-5) - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _e2m1_of(code):
    mag, neg = code % 8, code >= 8
    e, f = mag // 2, mag % 2
    v = torch.where(e == 0, 0.5 * f, (1.0 + 0.5 * f) * 2.0 ** (e - 1.0)).double()
    return torch.where(neg, -v, v)


def _row_codes(words):
    """int32 words (little-endian) -> codes in channel order, by shifts: channel j of eight at bit 4j."""
    w = words.long() & 0xFFFFFFFF
    return torch.stack([(w >> (4 * j)) & 15 for j in range(8)], -1).flatten(-2)


def _exact_rows(rec, c, rd):
    nq = c - rd
    v = _e2m1_of(_row_codes(rec[:, : nq // 2].contiguous().view(torch.int32)))
    e = rec[:, nq // 2 + 2 * rd :][:, : nq // 32].double() - 127.0
    return torch.cat((v * torch.exp2(e).repeat_interleave(32, 1), rec[:, nq // 2 : nq // 2 + 2 * rd].contiguous().view(BF16).double()), 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        z = s["x_"].double() + s["res"].double()
        y = z / (z.square().sum(1, keepdim=True) / case["d"] + 1e-6).sqrt() * s["gamma"].double()
        if case["out"] != "e4m3":
            return {"res": z, "out": y}
        group = case["group"] or case["d"]
        scale = y.abs().view(case["rows"], -1, group).amax(2) / 448.0
        return {"res": z, "out": _e4m3(y / scale.repeat_interleave(group, 1)), "scale": scale}
    if case["op"] == "w4":
        N, K, G, out = case["N"], case["K"], case["G"], []
        x = s["x_"].double() * (s["x_scale"].double()[:, None] if s["x_scale"] is not None else 1.0)
        for i in range(case["groups"]):
            parts = []
            for n in range(0, N, 4096):
                q = _row_codes(s["codes"][i * N + n : i * N + min(N, n + 4096)].view(torch.int32))
                w = _e2m1_of(q) if case["code"] == "e2m1" else torch.where(q >= 8, q - 16, q).double()
                sc = s["scales"][i, :, n : min(N, n + 4096)].contiguous().view(E4M3).double().t().repeat_interleave(G, 1)
                parts.append(x[:, i * K : (i + 1) * K] @ (w * sc).t() * s["row_scale"][i * N + n : i * N + min(N, n + 4096)].double())
            out += parts
        return torch.cat(out, 1)
    if case["op"] == "kv":
        nq = case["c"] - case["rd"]
        x = s["x_"].double()
        z = x[:, :nq].reshape(-1, 32)
        amax = z.abs().amax(1, keepdim=True)
        step = torch.exp2(torch.ceil(torch.log2(amax / 6.0) - 1e-12).clamp(-126, 126))
        grid = torch.tensor([-6.0, -4.0, -3.0, -2.0, -1.5, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda", dtype=torch.float64)
        even = torch.tensor([0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0], device="cuda", dtype=torch.float64)   # 1: an even mantissa
        out = []
        for i in range(0, z.shape[0], 1 << 18):
            far = (z[i : i + (1 << 18), :, None] / step[i : i + (1 << 18), :, None] - grid).abs() - 1e-9 * even
            out.append(grid[far.argmin(-1)] * step[i : i + (1 << 18)])
        return torch.cat((torch.cat(out).view(-1, nq), x[:, nq:]), 1)
    c, rd, w, m = case["c"], case["rd"], case["w"], case["m"]
    out = []
    for b, pos in enumerate(s["positions"].tolist()):
        V = (pos + 1) // m
        at = s["idx"][b][s["idx"][b] >= 0].long() if s["idx"] is not None else torch.arange(V, device="cuda")
        rows = s["rows_"][s["pages"][b].long()[at // case["page"]], at % case["page"]] if s["pages"] is not None else s["rows_"][b, at]
        keys = _exact_rows(rows, c, rd)
        keys = torch.cat([keys] + [s["win"][b, t % w].double()[None] for t in range(max(0, pos - w + 1), pos + 1)])
        z = s["q"][b].double() @ keys.t() / math.sqrt(c)
        top = torch.maximum(z.amax(1), s["sink"].double()) if keys.shape[0] else s["sink"].double()
        p = (z - top[:, None]).exp()
        o = p @ keys / (p.sum(1) + (s["sink"].double() - top).exp())[:, None]
        turn = torch.polar(torch.ones(rd // 2, device="cuda", dtype=torch.float64),
                           -pos * torch.pow(10000.0, -torch.arange(rd // 2, device="cuda", dtype=torch.float64) * 2.0 / rd))
        rot = torch.view_as_real(torch.view_as_complex(o[:, c - rd :].reshape(-1, rd // 2, 2).contiguous()) * turn).flatten(1)
        out.append(torch.cat((o[:, : c - rd], rot), 1))
    return torch.stack(out)
