// w4.cu -- products of a few tokens with 4-bit weights, and the quantiser that
// makes the weights.
//
//   out[t, g N + n] = xs[t] rs[g, n] sum_k x[t, g K + k] s[g, k / G, n] code[g, n, k]
//
// A code (E2M1: 2 significant bits, INT4: 3) times an e4m3 scale (4 bits) is
// exact in f16, so the weights enter the tensor cores as f16 without a
// rounding.  x enters as f16 too: e4m3 values are f16 values; a bf16 row is
// first multiplied by the power of two that puts its largest value into
// [2^14, 2^15), which keeps every element to 2^-39 of that largest one, and
// the sum is multiplied back.  The sums are fp32 (tensor memory).
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

constexpr int kBlk = 256;        // channels of one work unit (one pipeline stage)
constexpr int kTileN = 128;      // outputs of one tile: the MMA's M

// ---------------------------------------------------------------- x in f16
// Row (g, t) of the workspace: K f16 values, zeros up to Kp, and the factor
// that the sum over them is multiplied by.
template <typename XT>
__global__ void __launch_bounds__(256) w4_x_kernel(W4Params p, __half *xh, float *xd, int Kp) {
  __shared__ float part[8];
  pdl_trigger();   // the product kernel may start on its weights
  const int r = blockIdx.x, g = r / p.T, t = r - g * p.T, tid = threadIdx.x;
  const XT *x = static_cast<const XT *>(p.x) + (long long)t * p.ldx + (long long)g * p.K;
  __half *o = xh + (long long)r * Kp;
  if constexpr (sizeof(XT) == 1) {
    for (int k = 16 * tid; k < Kp; k += 16 * 256) {
      uint32_t h[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      if (k < p.K) {
        const uint4 v = *reinterpret_cast<const uint4 *>(x + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = e4m3x2_f16x2(w[i >> 1] >> (16 * (i & 1)));
      }
      reinterpret_cast<uint4 *>(o + k)[0] = make_uint4(h[0], h[1], h[2], h[3]);
      reinterpret_cast<uint4 *>(o + k)[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
    if (tid == 0) xd[r] = p.x_scale[t];
  } else {
    float am = 0.f;
    for (int k = 8 * tid; k < p.K; k += 8 * 256) {
      float v[8];
      load8(x + k, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[i]));
    }
    am = warp_max(am);
    if ((tid & 31) == 0) part[tid >> 5] = am;
    __syncthreads();
    am = part[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) am = fmaxf(am, part[i]);
    // e: am = f * 2^e, 1 <= f < 2, not below -110 so that 2^(14 - e) and its inverse are normal
    const int e = max((int)((__float_as_uint(am) >> 23) & 0xFFu) - 127, -110);
    const float up = pow2f(14 - e);
    for (int k = 8 * tid; k < Kp; k += 8 * 256) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (k < p.K) load8(x + k, v);
      __half2 h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i] * up, v[2 * i + 1] * up);
      *reinterpret_cast<uint4 *>(o + k) = *reinterpret_cast<const uint4 *>(h);
    }
    if (tid == 0) xd[r] = pow2f(e - 14);
  }
}

// ---------------------------------------------------------------- the product
// Outputs are the MMA's M (128 per tile), tokens its N (TN <= 64).  The work
// is the list of (tile, 256-channel unit) pairs; every CTA takes an equal run
// of it, so that HBM is read evenly whatever the tile count, and a tile cut
// between CTAs is joined from fp32 parts in a fixed order by w4_join_kernel.
// Roles: warp 0 streams codes, scales and x by TMA; warps 2-9 turn codes into
// f16 weights, a thread per output row, and write them to tensor memory as
// the A operand (no shared-memory round trip); warp 1 issues the MMAs; warps
// 10-13 read finished accumulators while the next tile's run.
struct W4Work {
  int nk, nb, ntt, G;      // units per tile, output blocks, token tiles, CTAs
  long long U;             // units of all tiles
  __host__ __device__ long long lo(int c) const { return U * c / G; }
  __host__ __device__ int cta_of(long long u) const { return (int)(((u + 1) * G - 1) / U); }
  // Part of tile i that CTA c computes, as a slot of the workspace: a CTA has
  // at most two parts, the one its run begins with and the one it ends with.
  __host__ __device__ int slot(int c, long long i) const { return 2 * c + (lo(c) >= i * nk ? 0 : 1); }
};
W4Work w4_work(const W4Params &p, int tn) {
  W4Work w;
  w.nk = (p.K + kBlk - 1) / kBlk;
  w.nb = (p.N + kTileN - 1) / kTileN;
  w.ntt = (p.T + tn - 1) / tn;
  w.U = (long long)p.groups * w.nb * w.ntt * w.nk;
  w.G = (int)std::min<long long>(num_sms(), w.U);
  return w;
}
int w4_tn(const W4Params &p) { return p.T <= 16 ? 16 : p.T <= 32 ? 32 : 64; }

// Workspace: x in f16, its factors, the parts.
struct W4Ws {
  size_t x, d, part, bytes;
  int Kp;
};
W4Ws w4_ws(const W4Params &p) {
  const int tn = w4_tn(p);
  const W4Work w = w4_work(p, tn);
  W4Ws l;
  l.Kp = w.nk * kBlk;
  const size_t rows = (size_t)p.groups * p.T;
  l.x = 0;
  l.d = (rows * l.Kp * 2 + 255) & ~(size_t)255;
  l.part = l.d + ((rows * 4 + 255) & ~(size_t)255);
  l.bytes = l.part + (size_t)2 * w.G * std::min(tn, p.T) * kTileN * 4;
  return l;
}

template <int TN>
struct W4Layout {
  static constexpr uint32_t kCodes = kTileN * 128, kX = 4 * TN * 128, kScales = 8 * 128;
  static constexpr uint32_t kStage = kCodes + kX + kScales;
  static constexpr int NST = TN == 64 ? 4 : TN == 32 ? 6 : 8;
  static constexpr uint32_t bar_off = NST * kStage;
  static constexpr uint32_t bytes = bar_off + 256 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory");
};
constexpr int kNA = 3;                   // A buffers in tensor memory, 128 columns each, behind two accumulators of 64
constexpr uint32_t kACol = 128;
constexpr int kW4Threads = 14 * 32;

// 32 codes of a 16-byte chunk as 16 f16 pairs, times the scale s2 (t2: INT4's offset).
template <int CODE>
__device__ __forceinline__ void w4_decode(const uint4 &q, uint32_t s2, uint32_t t2, uint32_t (&r)[16]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (CODE == HCA_W4_E2M1) {
      uint32_t f[4];
      e2m1x8_f16(w[i], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[4 * i + j] = hmul2_u32(f[j], s2);
    } else {
      // u = code + 8 in 0..15 read as an e4m3 byte is u 2^-9 (subnormals, then exponent 1): the value
      // (u - 8) 2^-9 s by one fused multiply-add, exact; the 2^9 is in the epilogue's factor
      const uint32_t u = w[i] ^ 0x88888888u, a = u & 0x0F0F0F0Fu, d = (u >> 4) & 0x0F0F0F0Fu;
      const uint32_t lo = __byte_perm(a, d, 0x5140), hi = __byte_perm(a, d, 0x7362);
      r[4 * i] = hfma2_u32(e4m3x2_f16x2(lo), s2, t2);
      r[4 * i + 1] = hfma2_u32(e4m3x2_f16x2(lo >> 16), s2, t2);
      r[4 * i + 2] = hfma2_u32(e4m3x2_f16x2(hi), s2, t2);
      r[4 * i + 3] = hfma2_u32(e4m3x2_f16x2(hi >> 16), s2, t2);
    }
  }
}

template <int TN, int CODE, typename OT>
__global__ void __launch_bounds__(kW4Threads, 1)
    w4_linear_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                     const __grid_constant__ CUtensorMap tmX, W4Params p, W4Work wk, const float *xd, float *part) {
  using L = W4Layout<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  struct Bars {
    uint64_t full[L::NST], empty[L::NST], a_full[kNA], a_empty[kNA], d_full[2], d_empty[2];
    uint32_t tmem;
  };
  static_assert(sizeof(Bars) <= 256, "barriers");
  Bars *bars = reinterpret_cast<Bars *>(smem + L::bar_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NST; ++i) {
      mbar_init(bar(bars->full[i]), 1);
      mbar_init(bar(bars->empty[i]), 9);       // 8 weight warps and the MMAs' commit
    }
    for (int i = 0; i < kNA; ++i) {
      mbar_init(bar(bars->a_full[i]), 8);
      mbar_init(bar(bars->a_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars->d_full[i]), 1);
      mbar_init(bar(bars->d_empty[i]), 4);
    }
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const long long u0 = wk.lo(blockIdx.x), u1 = wk.lo(blockIdx.x + 1);
  const int n = (int)(u1 - u0);
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmC);
      tma_prefetch_desc(&tmS);
      tma_prefetch_desc(&tmX);
      const uint32_t bytes = L::kCodes + L::kX + (uint32_t)(kBlk / p.G) * 128u;
      auto where = [&](int i, int &k, int &n0, int &g, int &row) {
        const long long u = u0 + i, tile = u / wk.nk;
        k = (int)(u - tile * wk.nk) * kBlk;
        // token tiles innermost: the CTAs of one weight block run together
        const long long blk = tile / wk.ntt;
        g = (int)(blk / wk.nb);
        n0 = (int)(blk - (long long)g * wk.nb) * kTileN;
        row = g * p.T + (int)(tile - blk * wk.ntt) * TN;
      };
      auto load_w = [&](int i, int st) {
        int k, n0, g, row;
        where(i, k, n0, g, row);
        const uint32_t b = bar(bars->full[st]), a = sbase + st * L::kStage;
        mbar_arrive_expect_tx(b, bytes);
        tma_load_3d(a, &tmC, k / 2, n0, g, b);
        tma_load_3d(a + L::kCodes + L::kX, &tmS, n0, k / p.G, g, b);
      };
      auto load_x = [&](int i, int st) {
        int k, n0, g, row;
        where(i, k, n0, g, row);
        const uint32_t b = bar(bars->full[st]), a = sbase + st * L::kStage + L::kCodes;
#pragma unroll
        for (int j = 0; j < 4; ++j) tma_load_2d(a + j * TN * 128, &tmX, k + 64 * j, row, b);
      };
      // the weights of the first stages do not depend on the kernel that writes x
      const int pre = min(n, L::NST);
      for (int i = 0; i < pre; ++i) load_w(i, i);
      pdl_wait();
      for (int i = 0; i < pre; ++i) load_x(i, i);
      for (int i = pre; i < n; ++i) {
        const int st = i % L::NST;
        if (!mbar_wait_sleep(bar(bars->empty[st]), ((i / L::NST) & 1) ^ 1, p.status)) break;
        load_w(i, st);
        load_x(i, st);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_f16(128, TN);
      int d = 0, dph = 0;                       // accumulator and its phase
      int kb = (int)(u0 % wk.nk);
      bool first = true;
      for (int i = 0; i < n; ++i) {
        const int st = i % L::NST, ab = i % kNA;
        if (!mbar_wait(bar(bars->full[st]), (i / L::NST) & 1, p.status)) break;
        if (!mbar_wait(bar(bars->a_full[ab]), (i / kNA) & 1, p.status)) break;
        if (first && !mbar_wait(bar(bars->d_empty[d]), dph ^ 1, p.status)) break;
        tc_fence_after();
        const uint64_t xdesc = sdesc_sw128(sbase + st * L::kStage + L::kCodes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk)
          umma_bf16_ts(tmem + d * 64, tmem + kACol + ab * 128 + 8 * kk,
                       xdesc + (((kk / 4) * TN * 128 + (kk % 4) * 32) >> 4), IDESC, first && kk == 0 ? 0u : 1u);
        umma_commit(bar(bars->a_empty[ab]));
        umma_commit(bar(bars->empty[st]));
        first = false;
        if (++kb == wk.nk || i == n - 1) {
          umma_commit(bar(bars->d_full[d]));
          kb = 0;
          first = true;
          d ^= 1;
          dph ^= d == 0;
        }
      }
    }
    __syncwarp();
  } else if (warp < 10) {
    // weights: row r of the tile, 16-byte chunks [4 half, 4 half + 4) of the stage's 8
    const int q = warp & 3, half = (warp - 2) >> 2, r = q * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + kACol;
    const int gsh = p.G == 32 ? 0 : p.G == 64 ? 1 : 2;
    for (int i = 0; i < n; ++i) {
      const int st = i % L::NST, ab = i % kNA;
      if (!mbar_wait(bar(bars->full[st]), (i / L::NST) & 1, p.status)) break;
      const uint8_t *codes = smem + st * L::kStage + r * 128;
      const uint8_t *sc = smem + st * L::kStage + L::kCodes + L::kX + r;
      uint4 v[4];
      uint32_t s2[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = *reinterpret_cast<const uint4 *>(codes + (((4 * half + c) ^ (r & 7)) << 4));
        s2[c] = sc[((4 * half + c) >> gsh) * 128];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->empty[st]));
      if (!mbar_wait(bar(bars->a_empty[ab]), ((i / kNA) & 1) ^ 1, p.status)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t s = e4m3_f16x2_dup(s2[c]);
        uint32_t t = 0;
        if constexpr (CODE == HCA_W4_INT4) t = hmul2_u32(s, 0xA400A400u);   // -2^-6: -8 of the byte's units
        uint32_t f[16];
        w4_decode<CODE>(v[c], s, t, f);
        tmem_st_32x32b_x16(ta + ab * 128 + (4 * half + c) * 16, f);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->a_full[ab]));
    }
  } else {
    pdl_wait();   // xd of the kernel before
    const int q = warp & 3, f = q * 32 + lane;
    const uint32_t td = tmem + ((uint32_t)(q * 32) << 16);
    int d = 0, dph = 0;
    for (long long u = u0; u < u1;) {
      const long long tile = u / wk.nk, end = min((tile + 1) * wk.nk, u1);
      const bool whole = u == tile * wk.nk && end == (tile + 1) * wk.nk;
      const long long blk = tile / wk.ntt;
      const int g = (int)(blk / wk.nb), o = (int)(blk - (long long)g * wk.nb) * kTileN + f;
      const int t0 = (int)(tile - blk * wk.ntt) * TN, nt = min(TN, p.T - t0);
      float rs = 0.f;
      if (whole && o < p.N) rs = p.row_scale[(long long)g * p.N + o] * (CODE == HCA_W4_INT4 ? 512.f : 1.f);
      if (!mbar_wait(bar(bars->d_full[d]), dph, p.status)) break;
      tc_fence_after();
      float *pp = part + (long long)wk.slot(blockIdx.x, tile) * min(TN, p.T) * kTileN + f;
#pragma unroll 1
      for (int j0 = 0; j0 < nt; j0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(td + d * 64 + j0, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = j0 + j;
          if (t < nt) {
            if (!whole) pp[t * kTileN] = __uint_as_float(v[j]);
            else if (o < p.N)
              Elt<OT>::store(static_cast<OT *>(p.out) + (long long)(t0 + t) * p.ldo + (long long)g * p.N + o,
                             __uint_as_float(v[j]) * rs * xd[g * p.T + t0 + t]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->d_empty[d]));
      d ^= 1;
      dph ^= d == 0;
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
__global__ void __launch_bounds__(kTileN) w4_join_kernel(W4Params p, W4Work wk, const float *xd, const float *part) {
  const long long tile = blockIdx.x;
  const int c0 = wk.cta_of(tile * wk.nk), c1 = wk.cta_of((tile + 1) * wk.nk - 1);
  if (c0 == c1) {
    pdl_wait();   // this grid may not end before the one that it depends on
    return;
  }
  const long long blk = tile / wk.ntt;
  const int g = (int)(blk / wk.nb), o = (int)(blk - (long long)g * wk.nb) * kTileN + threadIdx.x;
  const int t0 = (int)(tile - blk * wk.ntt) * TN, tl = 4 * blockIdx.y, nt = min(4, min(TN, p.T - t0) - tl);
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
                     acc[j] * rs * xd[g * p.T + t0 + tl + j]);
}

template <typename... KArgs, typename... Args>
int w4_launch(const char *name, dim3 grid, int threads, size_t smem, cudaStream_t s, void (*kernel)(KArgs...),
              Args... args) {
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
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(HCA_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  }
  return ls.done();
}

template <int TN, int CODE, typename OT>
int launch_w4_t(const W4Params &p, cudaStream_t s) {
  using L = W4Layout<TN>;
  static std::atomic<bool> attr_dev[kMaxDevices];
  std::atomic<bool> &attr = attr_dev[device_slot()];
  if (!attr) {
    const cudaError_t e = cudaFuncSetAttribute(w4_linear_kernel<TN, CODE, OT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes);
    if (e != cudaSuccess) return fail(HCA_ERR_CUDA, "w4_linear smem attribute: %s", cudaGetErrorString(e));
    attr = true;
  }
  const W4Work wk = w4_work(p, TN);
  const W4Ws l = w4_ws(p);
  char *ws = static_cast<char *>(p.ws);
  float *xd = reinterpret_cast<float *>(ws + l.d), *part = reinterpret_cast<float *>(ws + l.part);
  CUtensorMap tmC, tmS, tmX;
  int rc = encode_tmap_3d(&tmC, p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)p.K / 2, (uint64_t)p.N,
                          (uint64_t)p.groups, (uint64_t)p.K / 2, (uint64_t)p.N * (p.K / 2), 128, kTileN,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  if (!rc)
    rc = encode_tmap_3d(&tmS, p.scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)p.ldn, (uint64_t)(p.K / p.G),
                        (uint64_t)p.groups, (uint64_t)p.ldn, (uint64_t)p.ldn * (p.K / p.G), kTileN, kBlk / p.G,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!rc)
    rc = encode_tmap_2d(&tmX, ws + l.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)l.Kp, (uint64_t)p.groups * p.T,
                        (uint64_t)l.Kp * 2, 64, TN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  rc = w4_launch("w4_linear", dim3(wk.G), kW4Threads, L::bytes, s, w4_linear_kernel<TN, CODE, OT>, tmC, tmS, tmX, p, wk,
                 (const float *)xd, part);
  if (rc || wk.U % wk.G == 0 && (wk.U / wk.G) % wk.nk == 0) return rc;   // every run is made of whole tiles
  return w4_launch("w4_join", dim3((unsigned)(wk.U / wk.nk), (std::min(TN, p.T) + 3) / 4), kTileN, 0, s,
                   w4_join_kernel<TN, OT>, p, wk, (const float *)xd, (const float *)part);
}
template <int TN, int CODE>
int launch_w4_o(const W4Params &p, hca_dtype od, cudaStream_t s) {
  return od == HCA_F32 ? launch_w4_t<TN, CODE, float>(p, s) : launch_w4_t<TN, CODE, __nv_bfloat16>(p, s);
}
template <int TN>
int launch_w4_c(const W4Params &p, hca_dtype od, cudaStream_t s) {
  return p.code == HCA_W4_E2M1 ? launch_w4_o<TN, HCA_W4_E2M1>(p, od, s) : launch_w4_o<TN, HCA_W4_INT4>(p, od, s);
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

size_t w4_workspace_bytes(const W4Params &p) { return p.T > 0 ? w4_ws(p).bytes : 0; }

int launch_w4_linear(const W4Params &p, hca_dtype xd, hca_dtype od, cudaStream_t s) {
  if (p.T == 0) return HCA_OK;
  const W4Ws l = w4_ws(p);
  char *ws = static_cast<char *>(p.ws);
  __half *xh = reinterpret_cast<__half *>(ws + l.x);
  float *f = reinterpret_cast<float *>(ws + l.d);
  const unsigned rows = (unsigned)p.groups * p.T;
  const int rc =
      xd == HCA_BF16
          ? HCA_LAUNCH("w4_x", s, w4_x_kernel<__nv_bfloat16><<<rows, 256, 0, s>>>(p, xh, f, l.Kp))
          : HCA_LAUNCH("w4_x", s, w4_x_kernel<unsigned char><<<rows, 256, 0, s>>>(p, xh, f, l.Kp));
  if (rc) return rc;
  const int tn = w4_tn(p);
  return tn == 16 ? launch_w4_c<16>(p, od, s) : tn == 32 ? launch_w4_c<32>(p, od, s) : launch_w4_c<64>(p, od, s);
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
