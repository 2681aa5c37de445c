// w4.cu -- products of a few tokens with 4-bit weights, and the quantiser that
// makes the weights.
//
//   out[t, g N + n] = xs[t] rs[g, n] sum_k x[t, g K + k] s[g, k / G, n] code[g, n, k]
//
// A code (E2M1: 2 significant bits, INT4: 3) times an e4m3 scale (4 bits) is
// exact in f16, so the weights enter the tensor cores as f16 without a
// rounding.  x enters as f16 too: e4m3 values are f16 values; a bf16 row (a
// token's channels of one group) is multiplied by a power of two that leaves
// its elements exact down to 2^-31 of its largest, and smaller ones to 2^-39
// of that, and the sum is multiplied back.  The power of two comes from the
// row or from those of its channels that a block has, never from another
// group's.  The sums are fp32 (tensor memory).
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

constexpr int kBlk = 256;        // channels of one work unit (one pipeline stage)
constexpr int kTileN = 128;      // outputs of one tile: the MMA's M

// ---------------------------------------------------------------- codes
// Eight codes as f16 pairs, times the scale.  E2M1 pairs are neighbouring
// channels.  INT4 pairs are channels (i, i + 4), which the masks leave in
// place, and x is laid out alike: with u = code + 8 in the low bits under the
// exponent of 1024 the f16 value is 1024 + u, four bits higher 1024 + 16 u, so
// that one shift serves four pairs (the integer pipe bounds the decoding);
// (1024 + u) s - 1032 s and (1024 + 16 u) s / 16 - 72 s by one fused
// multiply-add are (u - 8) s, exact since 1032 s and 72 s have at most 11
// significant bits.  s is the scale times 2^-9 there so that 1032 s stays in
// range, and s / 16 is a multiple of 2^-22; the 2^9 is in the epilogue's factor.
template <int CODE>
struct W4Scale {
  uint32_t s, t, s16, t16;       // INT4: t = -1032 s, s / 16, t16 = -72 s
  __device__ __forceinline__ explicit W4Scale(uint32_t byte) : s(e4m3_f16x2_dup(byte)), t(0u), s16(0u), t16(0u) {
    if constexpr (CODE == HCA_W4_INT4) {
      s = hmul2_u32(s, 0x18001800u);          // 2^-9
      t = hmul2_u32(s, 0xE408E408u);          // -1032
      s16 = hmul2_u32(s, 0x2C002C00u);        // 1/16
      t16 = hmul2_u32(s, 0xD480D480u);        // -72
    }
  }
};
template <int CODE>
__device__ __forceinline__ void w4_decode8(uint32_t w, const W4Scale<CODE> &sc, uint32_t *r) {
  if constexpr (CODE == HCA_W4_E2M1) {
    uint32_t f[4];
    e2m1x8_f16(w, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = hmul2_u32(f[j], sc.s);
  } else {
    const uint32_t h = w >> 8;
    r[0] = hfma2_u32((w & 0x000F000Fu) ^ 0x64086408u, sc.s, sc.t);
    r[1] = hfma2_u32((w & 0x00F000F0u) ^ 0x64806480u, sc.s16, sc.t16);
    r[2] = hfma2_u32((h & 0x000F000Fu) ^ 0x64086408u, sc.s, sc.t);
    r[3] = hfma2_u32((h & 0x00F000F0u) ^ 0x64806480u, sc.s16, sc.t16);
  }
}
// Eight values of x in the order of the pairs.
template <int CODE>
__device__ __forceinline__ uint4 w4_x8(const float (&v)[8]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = CODE == HCA_W4_INT4 ? __floats2half2_rn(v[i], v[i + 4]) : __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  return *reinterpret_cast<const uint4 *>(h);
}
template <int CODE>
__device__ __forceinline__ uint4 w4_x8(const uint2 &u) {   // e4m3
  if constexpr (CODE == HCA_W4_INT4)
    return make_uint4(e4m3x2_f16x2(__byte_perm(u.x, u.y, 0x40)), e4m3x2_f16x2(__byte_perm(u.x, u.y, 0x51)),
                      e4m3x2_f16x2(__byte_perm(u.x, u.y, 0x62)), e4m3x2_f16x2(__byte_perm(u.x, u.y, 0x73)));
  else
    return make_uint4(e4m3x2_f16x2(u.x), e4m3x2_f16x2(u.x >> 16), e4m3x2_f16x2(u.y), e4m3x2_f16x2(u.y >> 16));
}
// The 32 of a 16-byte chunk.
template <int CODE>
__device__ __forceinline__ void w4_decode(const uint4 &q, const W4Scale<CODE> &sc, uint32_t (&r)[16]) {
  w4_decode8<CODE>(q.x, sc, r);
  w4_decode8<CODE>(q.y, sc, r + 4);
  w4_decode8<CODE>(q.z, sc, r + 8);
  w4_decode8<CODE>(q.w, sc, r + 12);
}

// ---------------------------------------------------------------- x in f16
// Row (g, t) of the workspace: K f16 values, zeros up to Kp, and the factor
// that the sum over them is multiplied by.
// One block per row, up to 1024 threads, each with up to 4 times 8 values, so
// that a row is read once.
constexpr int kXChunks = 4;
template <int CODE, typename XT>
__global__ void __launch_bounds__(1024) w4_x_kernel(W4Params p, __half *xh, float *xd, int Kp) {
  __shared__ float part[32];
  pdl_trigger();   // the product kernel may start on its weights
  const int r = blockIdx.x, g = r / p.T, t = r - g * p.T, tid = threadIdx.x, nthr = blockDim.x;
  const XT *x = static_cast<const XT *>(p.x) + (long long)t * p.ldx + (long long)g * p.K;
  uint4 *o = reinterpret_cast<uint4 *>(xh + (long long)r * Kp);
  if constexpr (sizeof(XT) == 1) {
    for (int k = tid; k < Kp / 8; k += nthr)
      o[k] = w4_x8<CODE>(8 * k < p.K ? __ldg(reinterpret_cast<const uint2 *>(x) + k) : make_uint2(0, 0));
    if (tid == 0) xd[r] = p.x_scale[t];
  } else {
    uint4 u[kXChunks];
    uint32_t am = 0u;    // |x| as bits, in the order of the values
#pragma unroll
    for (int i = 0; i < kXChunks; ++i) {
      const int k = tid + i * nthr;
      u[i] = 8 * k < p.K ? __ldg(reinterpret_cast<const uint4 *>(x) + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kXChunks; ++i)
      am = __vmaxu2(am, __vmaxu2(__vmaxu2(u[i].x & 0x7FFF7FFFu, u[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(u[i].z & 0x7FFF7FFFu, u[i].w & 0x7FFF7FFFu)));
    am = __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
    uint32_t *top = reinterpret_cast<uint32_t *>(part);
    if ((tid & 31) == 0) top[tid >> 5] = am;
    __syncthreads();
    am = __reduce_max_sync(0xffffffffu, (tid & 31) < (nthr >> 5) ? top[tid & 31] : 0u);
    // 2^e <= the largest value < 2^(e + 1), e at least -110 so that 2^(14 - e) and its inverse are normal
    const int e = max((int)(am >> 7) - 127, -110);
    const float up = pow2f(14 - e);
#pragma unroll
    for (int i = 0; i < kXChunks; ++i) {
      const int k = tid + i * nthr;
      if (8 * k >= Kp) break;
      const float v[8] = {bf16_lo(u[i].x) * up, bf16_hi(u[i].x) * up, bf16_lo(u[i].y) * up, bf16_hi(u[i].y) * up,
                          bf16_lo(u[i].z) * up, bf16_hi(u[i].z) * up, bf16_lo(u[i].w) * up, bf16_hi(u[i].w) * up};
      o[k] = w4_x8<CODE>(v);
    }
    if (tid == 0) xd[r] = pow2f(e - 14);
  }
}

// ---------------------------------------------------------------- the product
// Outputs are the MMA's M (128 per tile), tokens its N (TN <= 64).  The work
// is the list of (tile, 256-channel unit) pairs; every CTA takes an equal run
// of it, so that HBM is read evenly whatever the tile count, and a tile cut
// between CTAs is joined from fp32 parts in a fixed order by w4_join_kernel.
// Roles: warp 0 streams codes and scales by TMA, another warp x; 16 warps turn
// codes into f16 weights, a thread per output row and quarter of a unit, and
// write them to tensor memory as the A operand (no shared-memory round trip);
// two warps issue the MMAs, each of one half of every unit's channels into an
// accumulator of its own; four warps add the two and store.  A unit is a chain
// of waits, MMAs and commits in its issuing warp (about 1000 cycles for 16
// MMAs, of which the tensor pipe works 512 at 64 tokens), hence the two: 64
// tokens x 28677 x 8192 took 56 us with one.
//
// x reaches shared memory in one of two ways.  Where a block needs few units
// of it (kByUnit: its run has at most NX; kByBlock: one group whose rows have
// at most NX) the weight warps stage it themselves at the start, while the
// first codes are on their way, and it stays (no kernel before this one, no
// ring).  Otherwise w4_x_kernel writes it to the workspace and a warp streams
// it by TMA.
enum W4X { kRing = 0, kByUnit = 1, kByBlock = 2 };
struct W4Work {
  int nk, nb, ntt, G;      // units per tile, output blocks, token tiles, CTAs
  int gran, x;             // a run is a multiple of gran units; W4X
  int U, base, rem;        // units; CTA c's run: base * gran units, gran more for c < rem
  __host__ __device__ int lo(int c) const { return (c * base + (c < rem ? c : rem)) * gran; }
  // For gran = 1: the CTA of a unit, and the part of tile i that CTA c
  // computes, as a slot of the workspace: a CTA has at most two parts, the one
  // its run begins with and the one it ends with.
  __host__ __device__ int cta_of(int u) const {
    const int cut = rem * (base + 1);
    return u < cut ? u / (base + 1) : rem + (u - cut) / base;
  }
  __host__ __device__ int slot(int c, int i) const { return 2 * c + (lo(c) >= i * nk ? 0 : 1); }
};
W4Work w4_work(const W4Params &p, int tn) {
  W4Work w;
  const int NX = tn == 64 ? 4 : 8;
  w.nk = (p.K + kBlk - 1) / kBlk;
  w.nb = (p.N + kTileN - 1) / kTileN;
  w.ntt = (p.T + tn - 1) / tn;
  const int tiles = p.groups * w.nb * w.ntt;
  w.U = tiles * w.nk;
  w.G = std::min(num_sms(), w.U);
  w.gran = 1;
  // whole tiles per CTA where the longest run gets at most 6 units longer by
  // it: joining parts costs a launch, 2 to 3 us, and a unit about 0.4.  5 longer:
  // 64 tokens x 12800 x 4096 13.2 us, cut 15.7; 6 longer: 64 x 9600 x 3328 11.8,
  // cut 13.5; 7 longer: 16 x 19200 x 2048 13.1, cut 12.2; 9 longer: 16 x 20480 x
  // 2560 12.8, cut 11.7
  const int wt = (tiles + num_sms() - 1) / num_sms();
  if (wt * w.nk <= (w.U + w.G - 1) / w.G + 6) {
    w.gran = w.nk;
    w.G = (tiles + wt - 1) / wt;
  }
  w.base = w.U / w.gran / w.G;
  w.rem = w.U / w.gran - w.base * w.G;
  const int run = (w.base + (w.rem > 0)) * w.gran;   // the longest
  const bool block = p.groups == 1 && w.nk <= NX;
  w.x = w.ntt > 1 ? kRing : block && w.nk <= run ? kByBlock : run <= NX ? kByUnit : kRing;
  return w;
}
constexpr int kMaxT = 4096;               // tokens of one launch
int w4_tn(const W4Params &p) { return p.T <= 16 ? 16 : p.T <= 32 ? 32 : 64; }

// Workspace: x in f16 and its factors (kRing), the parts of cut tiles.
struct W4Ws {
  size_t x, d, part, bytes;
  int Kp;
};
W4Ws w4_ws(const W4Params &p) {
  const int tn = w4_tn(p);
  const W4Work w = w4_work(p, tn);
  W4Ws l;
  l.Kp = w.nk * kBlk;
  const size_t rows = w.x == kRing ? (size_t)p.groups * p.T : 0;
  l.x = 0;
  l.d = (rows * l.Kp * 2 + 255) & ~(size_t)255;
  l.part = l.d + ((rows * 4 + 255) & ~(size_t)255);
  l.bytes = l.part + (w.gran == 1 ? (size_t)2 * w.G * std::min(tn, p.T) * kTileN * 4 : 0);
  return l;
}

// Tensor memory: 128 columns of accumulators -- up to 32 tokens two pairs, so
// that one is stored while the other fills; at 64 tokens one pair -- then the
// buffers of decoded weights, 128 columns each.
constexpr int kNA = 3;
constexpr uint32_t kACol = 128;

template <int TN>
struct W4Layout {
  // Codes and x have rings of their own: a stage of codes is free once it has
  // been decoded, x stays until its MMAs have run.  Both sizes cover the time
  // from a load's issue to its use: 64 tokens x 28677 x 8192 takes 38.1 us with
  // 5 stages of codes and 4 of x, 38.3 with 7 and 3 or with 4 and 4, 39.3 with 3
  // and 5, 40.1 with 3 and 2.
  static constexpr uint32_t kCodes = kTileN * 128, kX = 4 * TN * 128, kScales = 8 * 128;
  static constexpr uint32_t kStage = kCodes + kScales;
  static constexpr int NC = TN == 64 ? 5 : TN == 32 ? 5 : 9, NX = TN == 64 ? 4 : 8;
  static constexpr int ND = TN == 64 ? 1 : 2;
  static constexpr uint32_t kSecond = TN == 64 ? 64 : 32;   // column of the second accumulator in its pair
  static constexpr uint32_t x_off = NC * kStage;
  // factors of x; staged bf16: and maxima
  static constexpr uint32_t xd_off = x_off + NX * kX, bar_off = xd_off + 2 * NX * TN * 4;
  static constexpr uint32_t bytes = bar_off + 512 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory");
};
constexpr int kDecWarps = 16, kEpi0 = 2 + kDecWarps;     // first epilogue warp
constexpr int kXWarp = kEpi0 + 4, kMma1 = kEpi0 + 5;    // x loads; MMAs of the second half (warp 1: of the first)
constexpr int kW4Threads = (kMma1 + 1) * 32;

// Barrier of the weight warps.
__device__ __forceinline__ void w4_dec_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kDecWarps * 32) : "memory"); }

// The weight warps' staging of x: `units` units of TN tokens as f16 in the
// layout that the MMAs read, and the factor per group of the run and token,
// xd[NX][TN].  A warp takes a token of a unit at a time, a lane 8 channels.
// bf16 values are scaled as w4_x_kernel scales them, by the largest of the
// token's values of the group that are staged here; they wait in registers for
// it, a first batch of two is read again.
template <int TN, int CODE, typename XT>
__device__ __forceinline__ void w4_stage_x(const W4Params &p, const W4Work &wk, int u0, int units, uint8_t *xs, float *xd) {
  constexpr int kBatch = 8;                // loads on their way before the first is used
  constexpr int kPer = TN / kDecWarps, kUnits = kBatch / kPer;   // a warp's tokens of a unit, units of a batch
  constexpr int kRows = W4Layout<TN>::NX * TN;
  using V = std::conditional_t<sizeof(XT) == 1, uint2, uint4>;
  const int w = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31, tid = threadIdx.x - 64;
  int first = 0, g0 = 0, t0 = 0;           // first unit's channels, group and tile of the group
  if (wk.x == kByUnit) {
    const int tile = u0 / wk.nk;
    first = u0 - tile * wk.nk;
    g0 = tile / wk.nb;
    t0 = tile - g0 * wk.nb;
  }
  V v[kBatch];
  uint32_t sets;                           // group of the run of each unit of the batch, 4 bits each
  auto load = [&](int b) {
    int kb = first, t = t0, set = 0;
    auto next = [&]() {
      if (++kb < wk.nk) return;
      kb = 0;
      if (++t < wk.nb) return;
      t = 0;
      ++set;
    };
    for (int i = 0; i < b * kUnits; ++i) next();
    sets = 0u;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (j > 0 && j % kPer == 0) next();
      if (j % kPer == 0) sets |= (uint32_t)set << (4 * (j / kPer));
      const int row = w + kDecWarps * (j % kPer), k = kb * kBlk + 8 * lane;
      v[j] = V{};
      if (b * kUnits + j / kPer < units && row < p.T && k < p.K)
        v[j] = __ldg(reinterpret_cast<const V *>(static_cast<const XT *>(p.x) + row * p.ldx + (long long)(g0 + set) * p.K + k));
    }
  };
  // f(load j, unit, token, row of the factors) of a batch
  auto each = [&](int b, auto f) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int un = b * kUnits + j / kPer, row = w + kDecWarps * (j % kPer);
      if (un < units) f(v[j], un, row, (int)((sets >> (4 * (j / kPer))) & 15u) * TN + row);
    }
  };
  auto store = [&](int un, int row, const uint4 &h) {
    *reinterpret_cast<uint4 *>(xs + un * W4Layout<TN>::kX + (lane / 8) * (TN * 128) + sw128_off(row, lane % 8)) = h;
  };
  const int batches = (units + kUnits - 1) / kUnits;
  if constexpr (sizeof(XT) == 1) {
#pragma unroll 1
    for (int b = 0; b < batches; ++b) {
      load(b);
      each(b, [&](const V &u, int un, int row, int) { store(un, row, w4_x8<CODE>(u)); });
    }
    if (tid < kRows && tid % TN < p.T) xd[tid] = p.x_scale[tid % TN];
  } else {
    auto top = [](const V &u) {              // largest |x| of the warp's 256 as bits, in the order of the values
      const uint32_t am = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
      return __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
    };
    // 2^e <= the largest value < 2^(e + 1), e at least -110 so that 2^(14 - e) and its inverse are normal
    auto expo = [](uint32_t am) { return max((int)(am >> 7) - 127, -110); };
    auto f16 = [](const V &u, float up) {
      const float f[8] = {bf16_lo(u.x) * up, bf16_hi(u.x) * up, bf16_lo(u.y) * up, bf16_hi(u.y) * up,
                          bf16_lo(u.z) * up, bf16_hi(u.z) * up, bf16_lo(u.w) * up, bf16_hi(u.w) * up};
      return w4_x8<CODE>(f);
    };
    if (units == 1) {
      // a warp has its tokens' whole rows: no exchange (1 token x 512 x 4096: 8.1 us with it, 6.8 without)
      load(0);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int row = w + kDecWarps * j, e = expo(top(v[j]));
        store(0, row, f16(v[j], pow2f(14 - e)));
        if (lane == 0) xd[row] = pow2f(e - 14);
      }
      return;
    }
    uint32_t *amax = reinterpret_cast<uint32_t *>(xd + kRows);
    if (tid < kRows) amax[tid] = 0u;
    load(0);
    w4_dec_sync();
#pragma unroll 1
    for (int b = 0;;) {
      each(b, [&](const V &u, int, int, int i) {
        const uint32_t am = top(u);
        if (lane == 0 && am) atomicMax(&amax[i], am);
      });
      if (++b == batches) break;
      load(b);
    }
    w4_dec_sync();
#pragma unroll 1
    for (int b = batches - 1;;) {
      each(b, [&](const V &u, int un, int row, int i) { store(un, row, f16(u, pow2f(14 - expo(amax[i])))); });
      if (--b < 0) break;
      load(b);
    }
    if (tid < kRows) xd[tid] = pow2f(expo(amax[tid]) - 14);
  }
}

template <int TN, int CODE, typename XT, typename OT>
__global__ void __launch_bounds__(kW4Threads, 1)
    w4_linear_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                     const __grid_constant__ CUtensorMap tmX, W4Params p, W4Work wk, const float *xd, float *part) {
  using L = W4Layout<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  struct Bars {
    uint64_t c_full[L::NC], c_empty[L::NC], x_full[L::NX], x_empty[L::NX], a_full[2][kNA], a_empty[2][kNA], d_full[2],
        d_empty[2], done[2];
    uint32_t tmem, ran_out;
  };
  static_assert(sizeof(Bars) <= 512, "barriers");
  Bars *bars = reinterpret_cast<Bars *>(smem + L::bar_off);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  const Waits wait{p.status, &bars->ran_out};
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NC; ++i) {
      mbar_init(bar(bars->c_full[i]), 1);
      mbar_init(bar(bars->c_empty[i]), kDecWarps);
    }
    for (int i = 0; i < L::NX; ++i) {
      mbar_init(bar(bars->x_full[i]), wk.x == kRing ? 1 : kDecWarps);
      mbar_init(bar(bars->x_empty[i]), 2);
    }
    for (int i = 0; i < 2 * kNA; ++i) {
      mbar_init(bar(bars->a_full[i / kNA][i % kNA]), kDecWarps / 2);
      mbar_init(bar(bars->a_empty[i / kNA][i % kNA]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars->d_full[i]), 2);
      mbar_init(bar(bars->d_empty[i]), 4);
      mbar_init(bar(bars->done[i]), 1);
    }
    bars->ran_out = 0u;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
  float *xds = reinterpret_cast<float *>(smem + L::xd_off);   // [TN]; staged x: [NX][TN]
  const int u0 = wk.lo(blockIdx.x), u1 = wk.lo(blockIdx.x + 1), n = u1 - u0;
  pdl_trigger();

  if (warp == 0 || warp == kXWarp) {
    if (lane == 0) {
      // walks the units; the tile's place is worked out once per tile
      int tile = u0 / wk.nk, kb = u0 - tile * wk.nk, n0, g, row;
      auto place = [&]() {   // token tiles innermost: the CTAs of one weight block run together
        const int blk = tile / wk.ntt;
        g = blk / wk.nb;
        n0 = (blk - g * wk.nb) * kTileN;
        row = g * p.T + (tile - blk * wk.ntt) * TN;
      };
      auto next = [&]() {
        if (++kb == wk.nk) {
          kb = 0;
          ++tile;
          place();
        }
      };
      place();
      if (warp == 0) {
        // the weights do not depend on the kernel that writes x
        tma_prefetch_desc(&tmC);
        tma_prefetch_desc(&tmS);
        const uint32_t bytes = L::kCodes + (uint32_t)(kBlk / p.G) * 128u;
        const int sshift = p.G == 32 ? 3 : p.G == 64 ? 2 : 1;   // scale rows of a unit: 2^sshift
        for (int i = 0; i < n; ++i, next()) {
          const int st = i % L::NC;
          if (!wait.until(bar(bars->c_empty[st]), ((i / L::NC) & 1) ^ 1)) break;
          const uint32_t b = bar(bars->c_full[st]), a = sbase + st * L::kStage;
          mbar_arrive_expect_tx(b, bytes);
          tma_load_3d(a, &tmC, kb * (kBlk / 2), n0, g, b);
          tma_load_3d(a + L::kCodes, &tmS, n0, kb << sshift, g, b);
        }
      } else if (wk.x == kRing) {
        tma_prefetch_desc(&tmX);
        pdl_wait();
        for (int i = 0; i < n; ++i, next()) {
          const int st = i % L::NX;
          if (!wait.until(bar(bars->x_empty[st]), ((i / L::NX) & 1) ^ 1)) break;
          const uint32_t b = bar(bars->x_full[st]), a = sbase + L::x_off + st * L::kX;
          mbar_arrive_expect_tx(b, L::kX);
#pragma unroll
          for (int j = 0; j < 4; ++j) tma_load_2d(a + j * TN * 128, &tmX, kb * kBlk + 64 * j, row, b);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == kMma1) {
    constexpr uint32_t IDESC = idesc_f16(128, TN);
    const int half = warp == 1 ? 0 : 1;
    const uint64_t xdesc0 = sdesc_sw128(sbase + L::x_off, 16, 1024) + ((half * 2 * TN * 128) >> 4);
    int ab = 0, xs = 0, left = wk.nk - u0 % wk.nk;   // left: units of the tile
    if (wk.x == kByBlock) xs = wk.nk - left;
    uint32_t aph = 0, xph = 0;
    for (int i = 0, piece = 0; i < n; ++piece) {
      const int end = min(n, i + left), d = piece % L::ND;   // units [i, end) of one tile
      left = wk.nk;
      wait(bar(bars->d_empty[d]), ((piece / L::ND) & 1) ^ 1);
      const uint32_t td = tmem + d * 64 + half * L::kSecond;
      for (uint32_t acc = 0; i < end; ++i, acc = 1) {
        wait(bar(bars->x_full[xs]), xph);
        wait(bar(bars->a_full[half][ab]), aph);
        tc_fence_after();
        if (elect_one()) {
          const uint64_t xdesc = xdesc0 + xs * (L::kX >> 4);
          const uint32_t ta = tmem + kACol + ab * 128 + half * 64;
#pragma unroll
          for (int kk = 0; kk < kBlk / 32; ++kk)
            umma_bf16_ts(td, ta + 8 * kk, xdesc + (((kk / 4) * TN * 128 + (kk % 4) * 32) >> 4), IDESC,
                         kk > 0 ? 1u : acc);
          umma_commit(bar(bars->a_empty[half][ab]));
          umma_commit(bar(bars->x_empty[xs]));
          if (i + 1 == end) umma_commit(bar(bars->d_full[d]));
        }
        __syncwarp();
        if (++ab == kNA) {
          ab = 0;
          aph ^= 1;
        }
        // staged x stays in phase 0
        if (++xs == (wk.x == kByBlock ? wk.nk : L::NX)) {
          xs = 0;
          xph ^= wk.x == kRing;
        }
      }
    }
    wait.settle(bar(bars->done[half]));
  } else if (warp < kEpi0) {
    if (wk.x != kRing) {
      pdl_wait();   // x of the kernel before
      const int units = wk.x == kByUnit ? n : wk.nk;
      w4_stage_x<TN, CODE, XT>(p, wk, u0, units, smem + L::x_off, xds);
      fence_proxy_async();     // the tensor cores read it through the async proxy
      __syncwarp();
      if (lane == 0)
        for (int i = 0; i < units; ++i) mbar_arrive(bar(bars->x_full[i]));
    }
    // weights: row r of the tile, 16-byte chunks 2 kq and 2 kq + 1 of the stage's 8
    const int q = warp & 3, kq = (warp - 2) >> 2, r = q * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + kACol + kq * 32;
    const int gsh = p.G == 32 ? 0 : p.G == 64 ? 1 : 2;
    const uint32_t o0 = r * 128 + (((2 * kq) ^ (r & 7)) << 4), o1 = r * 128 + (((2 * kq + 1) ^ (r & 7)) << 4);
    const uint32_t s0 = L::kCodes + ((2 * kq) >> gsh) * 128 + r, s1 = L::kCodes + ((2 * kq + 1) >> gsh) * 128 + r;
    int st = 0, ab = 0;
    uint32_t cph = 0, aph = 1;
    for (int i = 0; i < n; ++i) {
      wait(bar(bars->c_full[st]), cph);
      const uint8_t *stage = smem + st * L::kStage;
      const uint4 v0 = *reinterpret_cast<const uint4 *>(stage + o0), v1 = *reinterpret_cast<const uint4 *>(stage + o1);
      const uint32_t ba = stage[s0], bb = stage[s1];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->c_empty[st]));
      uint32_t f0[16], f1[16];
      w4_decode<CODE>(v0, W4Scale<CODE>(ba), f0);
      w4_decode<CODE>(v1, W4Scale<CODE>(bb), f1);
      wait(bar(bars->a_empty[kq >> 1][ab]), aph);
      tc_fence_after();
      tmem_st_32x32b_x16(ta + ab * 128, f0);
      tmem_st_32x32b_x16(ta + ab * 128 + 16, f1);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->a_full[kq >> 1][ab]));
      if (++st == L::NC) {
        st = 0;
        cph ^= 1;
      }
      if (++ab == kNA) {
        ab = 0;
        aph ^= 1;
      }
    }
  } else {
    // finished accumulators: thread = output row.  Short code, 8 tokens a step:
    // a block runs it two or three times, so that fetching instructions is
    // most of its cost (64 tokens unrolled by 16 with two 64-bit products per
    // store: 9000 cycles per tile).
    pdl_wait();   // xd of the kernel before; out may still be read by it
    const int q = warp & 3, f = q * 32 + lane;
    const uint32_t td = tmem + ((uint32_t)(q * 32) << 16);
    if (wk.x != kRing) wait(bar(bars->x_full[0]), 0);   // xds is written
    int piece = 0;
    const int g0 = u0 / wk.nk / wk.ntt / wk.nb;
    for (int u = u0; u < u1; ++piece) {
      const int d = piece % L::ND;
      const int tile = u / wk.nk, end = min((tile + 1) * wk.nk, u1);
      const bool whole = u == tile * wk.nk && end == (tile + 1) * wk.nk;
      const int blk = tile / wk.ntt, g = blk / wk.nb, o = (blk - g * wk.nb) * kTileN + f;
      const int t0 = (tile - blk * wk.ntt) * TN, nt = min(TN, p.T - t0);
      const float *xt = xds + (wk.x == kRing ? 0 : g - g0) * TN;
      if (wk.x == kRing) {
        if (f < nt) xds[f] = xd[g * p.T + t0 + f];
        asm volatile("bar.sync 2, 128;" ::: "memory");
      }
      float rs = 1.f;
      if (whole && o < p.N) rs = p.row_scale[(long long)g * p.N + o] * (CODE == HCA_W4_INT4 ? 512.f : 1.f);
      float *pp = part + (long long)wk.slot(blockIdx.x, tile) * min(TN, p.T) * kTileN + f;
      OT *po = static_cast<OT *>(p.out) + (long long)t0 * p.ldo + (long long)g * p.N + o;
      wait(bar(bars->d_full[d]), (piece / L::ND) & 1);
      tc_fence_after();
#pragma unroll 1
      for (int j0 = 0; j0 < nt; j0 += 8) {
        uint32_t v[8], v1[8];
        tmem_ld_32x32b_x8(td + d * 64 + j0, v);
        tmem_ld_32x32b_x8(td + d * 64 + L::kSecond + j0, v1);
        float x[8], a[8];                   // read before the first store, which might be to the same memory for all
        load8(xt + j0, x);                  // that the compiler knows
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = (__uint_as_float(v[j]) + __uint_as_float(v1[j])) * x[j] * rs;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j < nt) {
            if (!whole) *pp = a[j];
            else if (o < p.N) Elt<OT>::store(po, a[j]);
          }
          pp += kTileN;
          po += p.ldo;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->d_empty[d]));
      if (wk.x == kRing) asm volatile("bar.sync 2, 128;" ::: "memory");   // xds has been read
      u = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Tiles that were cut: their parts summed in the order of their channels.
// Block = (tile, 4 tokens), thread = output.
template <int TN, typename OT>
__global__ void __launch_bounds__(kTileN) w4_join_kernel(W4Params p, W4Work wk, const float *part) {
  const int tile = blockIdx.x;
  const int c0 = wk.cta_of(tile * wk.nk), c1 = wk.cta_of((tile + 1) * wk.nk - 1);
  if (c0 == c1) {
    pdl_wait();   // this grid may not end before the one that it depends on
    return;
  }
  const int blk = tile / wk.ntt, g = blk / wk.nb, o = (blk - g * wk.nb) * kTileN + threadIdx.x;
  const int t0 = (tile - blk * wk.ntt) * TN, tl = 4 * blockIdx.y, nt = min(4, min(TN, p.T - t0) - tl);
  const int per = min(TN, p.T) * kTileN;
  float rs = 0.f;
  if (o < p.N) rs = p.row_scale[(long long)g * p.N + o] * (p.code == HCA_W4_INT4 ? 512.f : 1.f);
  pdl_wait();
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float *pp = part + (long long)wk.slot(c, tile) * per + tl * kTileN + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < nt) acc[j] += pp[j * kTileN];
  }
  if (o >= p.N) return;   // nt may be <= 0 in the last token tile
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nt)
      Elt<OT>::store(static_cast<OT *>(p.out) + (long long)(t0 + tl + j) * p.ldo + (long long)g * p.N + o,
                     acc[j] * rs);
}

template <typename... KArgs, typename... Args>
int w4_launch(const char *name, dim3 grid, int threads, size_t smem, cudaStream_t s, bool dependent,
              void (*kernel)(KArgs...), Args... args) {
  LaunchScope ls(name, s);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(HCA_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  }
  return ls.done();
}

template <int TN, int CODE, typename XT, typename OT>
int launch_w4_t(const W4Params &p, cudaStream_t s) {
  using L = W4Layout<TN>;
  static std::atomic<bool> attr_dev[kMaxDevices];
  std::atomic<bool> &attr = attr_dev[device_slot()];
  if (!attr) {
    const cudaError_t e = cudaFuncSetAttribute(w4_linear_kernel<TN, CODE, XT, OT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes);
    if (e != cudaSuccess) return fail(HCA_ERR_CUDA, "w4_linear smem attribute: %s", cudaGetErrorString(e));
    attr = true;
  }
  const W4Work wk = w4_work(p, TN);
  const W4Ws l = w4_ws(p);
  char *ws = static_cast<char *>(p.ws);
  float *xd = reinterpret_cast<float *>(ws + l.d), *part = reinterpret_cast<float *>(ws + l.part);
  __half *xh = reinterpret_cast<__half *>(ws + l.x);
  CUtensorMap tmC, tmS, tmX;
  int rc = encode_tmap_3d(&tmC, p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)p.K / 2, (uint64_t)p.N,
                          (uint64_t)p.groups, (uint64_t)p.K / 2, (uint64_t)p.N * (p.K / 2), 128, kTileN,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  if (!rc)
    rc = encode_tmap_3d(&tmS, p.scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)p.ldn, (uint64_t)(p.K / p.G),
                        (uint64_t)p.groups, (uint64_t)p.ldn, (uint64_t)p.ldn * (p.K / p.G), kTileN, kBlk / p.G,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!rc && wk.x == kRing)
    rc = encode_tmap_2d(&tmX, xh, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)l.Kp, (uint64_t)p.groups * p.T,
                        (uint64_t)l.Kp * 2, 64, TN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  if (wk.x == kRing) {
    const int thr = std::min(1024, l.Kp / 8);   // Kp is a multiple of 256, at most 32768
    rc = HCA_LAUNCH("w4_x", s, w4_x_kernel<CODE, XT><<<(unsigned)p.groups * p.T, thr, 0, s>>>(p, xh, xd, l.Kp));
    if (rc) return rc;
  } else {
    tmX = tmC;      // not used
  }
  // dependent on w4_x only; without it an ordinary launch, since the weights are read before any wait
  rc = w4_launch("w4_linear", dim3(wk.G), kW4Threads, L::bytes, s, wk.x == kRing, w4_linear_kernel<TN, CODE, XT, OT>,
                 tmC, tmS, tmX, p, wk, (const float *)xd, part);
  if (rc || wk.gran > 1) return rc;
  return w4_launch("w4_join", dim3((unsigned)(wk.U / wk.nk), (std::min(TN, p.T) + 3) / 4), kTileN, 0, s, true,
                   w4_join_kernel<TN, OT>, p, wk, (const float *)part);
}
template <int TN, int CODE>
int launch_w4_o(const W4Params &p, hca_dtype xd, hca_dtype od, cudaStream_t s) {
  if (xd == HCA_BF16)
    return od == HCA_F32 ? launch_w4_t<TN, CODE, __nv_bfloat16, float>(p, s)
                         : launch_w4_t<TN, CODE, __nv_bfloat16, __nv_bfloat16>(p, s);
  return od == HCA_F32 ? launch_w4_t<TN, CODE, unsigned char, float>(p, s)
                       : launch_w4_t<TN, CODE, unsigned char, __nv_bfloat16>(p, s);
}
template <int TN>
int launch_w4_c(const W4Params &p, hca_dtype xd, hca_dtype od, cudaStream_t s) {
  return p.code == HCA_W4_E2M1 ? launch_w4_o<TN, HCA_W4_E2M1>(p, xd, od, s) : launch_w4_o<TN, HCA_W4_INT4>(p, xd, od, s);
}

__device__ __forceinline__ float load_w(const float *p) { return *p; }
__device__ __forceinline__ float load_w(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// A warp per row of weights, a lane per pair of channels of a group.
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T *__restrict__ w, W4Params p, unsigned char *codes,
                                                           unsigned char *scales, float *row_scale) {
  const int lane = threadIdx.x & 31;
  const long long o = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= (long long)p.groups * p.ldn) return;
  const int g = (int)(o / p.ldn), n = (int)(o - (long long)g * p.ldn);
  unsigned char *sc = scales + (long long)g * (p.K / p.G) * p.ldn + n;
  if (n >= p.N) {   // the padding columns
    for (int k = lane; k < p.K / p.G; k += 32) sc[(long long)k * p.ldn] = 0;
    return;
  }
  const long long row = (long long)g * p.N + n;
  const T *x = w + row * p.K;
  const float top = p.code == HCA_W4_E2M1 ? 6.0f : 7.0f;
  float am = 0.f;
  for (int k = lane; k < p.K; k += 32) am = fmaxf(am, fabsf(load_w(x + k)));
  const float rs = __fdiv_rn(warp_max(am), top * 448.0f);
  if (lane == 0) row_scale[row] = rs;
  unsigned char *cp = codes + row * (p.K / 2);
  for (int b = 0; b < p.K / p.G; ++b) {
    float m = 0.f;
    for (int k = lane; k < p.G; k += 32) m = fmaxf(m, fabsf(load_w(x + b * p.G + k)));
    m = warp_max(m);
    const uint32_t sb = rs > 0.f ? f32_e4m3(__fdiv_rn(__fdiv_rn(m, top), rs)) : 0u;
    const float step = __fmul_rn(rs, e4m3_f32(sb));
    if (lane == 0) sc[(long long)b * p.ldn] = (unsigned char)sb;
    for (int k = 2 * lane; k < p.G; k += 64) {
      uint32_t q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = step > 0.f ? __fdiv_rn(load_w(x + b * p.G + k + i), step) : 0.f;
        q[i] = p.code == HCA_W4_E2M1 ? e2m1_code(v) : (uint32_t)__float2int_rn(fminf(fmaxf(v, -7.f), 7.f)) & 15u;
      }
      cp[(b * p.G + k) / 2] = (unsigned char)(q[0] | (q[1] << 4));
    }
  }
}

}  // namespace

size_t w4_workspace_bytes(const W4Params &p) {
  if (p.T <= 0) return 0;
  W4Params c = p;
  c.T = std::min(p.T, kMaxT);
  const size_t most = w4_ws(c).bytes;
  c.T = p.T % kMaxT;                        // a last, shorter run may be laid out otherwise
  return c.T && p.T > kMaxT ? std::max(most, w4_ws(c).bytes) : most;
}

int launch_w4_linear(const W4Params &p, hca_dtype xd, hca_dtype od, cudaStream_t s) {
  if (p.T == 0) return HCA_OK;
  // many tokens: runs of at most kMaxT, so that unit numbers stay within 31 bits
  W4Params c = p;
  for (int t0 = 0; t0 < p.T; t0 += kMaxT) {
    c.T = std::min(kMaxT, p.T - t0);
    c.x = static_cast<const char *>(p.x) + (long long)t0 * p.ldx * (xd == HCA_BF16 ? 2 : 1);
    if (p.x_scale) c.x_scale = p.x_scale + t0;
    c.out = static_cast<char *>(p.out) + (long long)t0 * p.ldo * (od == HCA_BF16 ? 2 : 4);
    const int tn = w4_tn(c);
    const int rc = tn == 16 ? launch_w4_c<16>(c, xd, od, s)
                   : tn == 32 ? launch_w4_c<32>(c, xd, od, s) : launch_w4_c<64>(c, xd, od, s);
    if (rc) return rc;
  }
  return HCA_OK;
}

int launch_w4_quantize(const void *w, hca_dtype wd, const W4Params &p, void *codes, void *scales, float *row_scale,
                       cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.groups * p.ldn + 7) / 8);
  unsigned char *c = static_cast<unsigned char *>(codes), *sc = static_cast<unsigned char *>(scales);
  if (wd == HCA_F32)
    return HCA_LAUNCH("w4_quantize", s,
                      w4_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float *>(w), p, c, sc, row_scale));
  return HCA_LAUNCH("w4_quantize", s,
                    w4_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(w), p, c, sc, row_scale));
}

}  // namespace hca
