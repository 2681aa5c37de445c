"""Products with 4-bit weights on each way that x takes to the tensor cores (staged per run of units, staged whole,
streamed through rings), against the float64 formula: activations of a wide range within a token, groups of different
size, runs longer than the rings, tiles cut between long runs.

Tolerance: K / 16 accumulations and a joined part per 256 channels, each a truncation of 2^-23 of the sum of
magnitudes, and 8 for the scalings and the output; x itself enters exactly wherever its element is at least 2^-31 of
the token's largest in its group (bf16 has 8 bits, f16 keeps them down to 2^-17, the largest stands at 2^14).  Elements
below that are off by half of f16's smallest step, 2^-25 where the largest is at least 2^14, so 2^-39 of the largest,
times their weight."""
import pytest
import torch

from long_context_compressed_hca_b200 import binding as hb
from tests import lowbit_reference as R
from tests.test_gpu_lowbit import BF16, E4M3, F32, HALF, U8, _close, _n

pytestmark = pytest.mark.gpu

CODE = {"e2m1": hb.HCA_W4_E2M1, "int4": hb.HCA_W4_INT4}


def _run(x, xs, w, T, N, K, groups, code, G, ot, refs=slice(None)):
    """Product of x with the quantised w, checked on the outputs refs of every group."""
    d = hb.w4_desc(T, N, K, groups, G, CODE[code], hb.HCA_BF16 if xs is None else hb.HCA_FP8E4M3, hb.DTYPE_CODE[ot])
    codes, scales, rs = hb.w4_quantize(d, w)
    ws = torch.full((max(16, hb.w4_linear_workspace_size(d)),), 0xFF, dtype=U8, device="cuda")
    out = torch.full((T, groups * N), float("nan"), dtype=ot, device="cuda")
    hb.w4_linear(d, x, xs, codes, scales, rs, out, ws)
    assert hb.device_status() == hb.HCA_OK
    wd = R.weights(codes, scales, rs, groups, N, K, G, code == "int4")[:, refs]
    xd = x.double().view(T, groups, K) * (1.0 if xs is None else xs.double().view(T, 1, 1))
    want, mag = torch.einsum("tgk,gnk->tgn", xd, wd), torch.einsum("tgk,gnk->tgn", xd.abs(), wd.abs())
    top = xd.abs().amax(2, keepdim=True)
    low = torch.einsum("tgk,gnk->tgn", (xd.abs() < 2.0 ** -31 * top).double() * 2.0 ** -39 * top, wd.abs())
    got = out.view(T, groups, N)[:, :, refs]
    _close(got, want, (K / 16 + -(-K // 256) + 8) * 2.0 ** -23 * mag + low + HALF[ot] * want.abs() + 1e-36)
    assert not torch.isnan(out.double()).any()


# T, N, K, groups: runs that pass from group to group, units of one group, all of x, rings
RANGE = [(7, 1024, 4096, 8), (3, 8, 32, 300), (40, 130, 256, 200), (1, 512, 4096, 1), (5, 200, 512, 1), (17, 40, 1024, 1),
         (4, 10240, 4096, 1), (65, 200, 512, 2)]


@pytest.mark.parametrize("code", ["e2m1", "int4"])
@pytest.mark.parametrize("T,N,K,groups", RANGE)
def test_small_activations_beside_a_large_one(cuda, T, N, K, groups, code):
    """A large activation whose weights are zero leaves the sum of the small ones, which fp32 sums would keep."""
    w = _n((groups * N, K), 71, 1, std=K ** -0.5)
    w[:, 0] = 0.0
    x = _n((T, groups, K), 71, 2)
    for t in range(T):
        big, rest = [(1.0, 1e-6), (1.9, 2.0 ** -26), (200.0, 1e-4), (60000.0, 1e-3), (2.0 ** -20, 2.0 ** -45),
                     (1e30, 1e22)][t % 6]
        x[t] *= rest
        x[t, :, 0] = big
    _run(x.to(BF16).view(T, -1), None, w, T, N, K, groups, code, 32, F32)


@pytest.mark.parametrize("T,N,K,groups", [r for r in RANGE if r[3] > 1])
def test_groups_of_different_size(cuda, T, N, K, groups):
    """A group's outputs do not depend on how large another group's activations are."""
    w = _n((groups * N, K), 72, 1, std=K ** -0.5)
    x = _n((T, groups, K), 72, 2)
    x *= torch.exp2((torch.arange(groups, device=cuda) * 17 % 60 - 40).double()).float()[None, :, None]
    x[:, :: 3] = 0.0
    _run(x.to(BF16).view(T, -1), None, w, T, N, K, groups, "e2m1", 32, F32)


# T, N, K, groups, code, G, x: rings with more units a CTA than stages, tiles cut between runs, several token tiles
LONG = [(16, 20000, 8192, 1, "e2m1", 32, BF16), (16, 5000, 8192, 2, "int4", 128, E4M3), (32, 20000, 4096, 1, "e2m1", 64, E4M3),
        (31, 3000, 8160, 3, "int4", 32, BF16), (64, 20000, 8192, 1, "int4", 128, BF16), (61, 2311, 8224, 2, "e2m1", 32, E4M3),
        (65, 9000, 2048, 1, "e2m1", 64, BF16), (200, 4000, 4096, 1, "int4", 64, E4M3), (130, 1000, 1056, 4, "e2m1", 32, BF16)]


@pytest.mark.parametrize("T,N,K,groups,code,G,xt", LONG)
def test_long_runs(cuda, T, N, K, groups, code, G, xt):
    w = _n((groups * N, K), 73, 1, std=K ** -0.5)
    x, xs = _n((T, groups * K), 73, 2), None
    if xt == E4M3:
        xs = x.abs().amax(1) / 448.0
        x = x / xs[:, None]
    refs = torch.cat((torch.arange(0, N, 97), torch.arange(max(0, N - 140), N))).unique().cuda()
    _run(x.to(xt), xs, w, T, N, K, groups, code, G, F32, refs)
