// norm.cu -- residual addition + RMSNorm of rows, with an f32, bf16 or e4m3
// output.
//
//   z = x + res,  y = z * gamma / sqrt(mean z^2 + eps),
//   e4m3: scale = amax|y| / 448 over a row or a group, code = e4m3(y / scale).
//
// A block holds a row in registers (8 C channels per thread), so every input
// is read once and every output written once.  A row-wide e4m3 scale needs
// amax|y| = max|z gamma| / sqrt(..), which is reduced together with the sum of
// squares: one block reduction either way.  Group scales are maxima over 8 or
// 16 neighbouring lanes.  Bound: HBM.  With many rows a block takes several:
// gamma stays in registers (read again for every row it is as many bytes as x
// and res in bf16) and the next row's loads are on their way while this one is
// reduced and written (16411 x 4104 bf16: 83 us, 6.5 TB/s; 127 with a block per
// row).
// Rows beyond 8192 channels take 4 times 8 channels per thread, for which the
// registers hold neither gamma nor another row.
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

// 8 channels from p (element offset a multiple of 8 when vec), the first n of
// them valid.
template <typename T>
__device__ __forceinline__ void load_row8(const T *p, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    load8(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? Elt<T>::load(p + i) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_row8(T *p, int n, bool vec, const float (&v)[8]) {
  if (vec && n >= 8) {
    store8(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) Elt<T>::store(p + i, v[i]);
}

struct E4M3 {
  unsigned char b;
};

// Eight channels as they lie in memory: 16 bytes of bf16 or 32 of f32.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
// kWritten: memory that the kernel may write, so not through the read-only path
// and read once, where it stands.  A plain load keeps its place among all stores
// (16411 x 4104 bf16: 99 us), which it need not: an element is written by the
// thread that reads it, with a value made from it.
template <bool kWritten, typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p, int n, bool vec) {
  Raw8<T> r;
  if (vec && n >= 8) {
    const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      if constexpr (kWritten)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[i].x), "=r"(r.w[i].y), "=r"(r.w[i].z), "=r"(r.w[i].w) : "l"(q + i));
      else
        r.w[i] = __ldg(q + i);
    }
    return r;
  }
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : T(0.f);
  memcpy(&r, t, sizeof r);
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&v)[8]) { memcpy(v, &r, sizeof v); }
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <typename XT, typename RT, typename OT, int C>
__global__ void __launch_bounds__(C <= 2 ? 512 : 1024) add_rms_norm_kernel(NormParams p) {
  constexpr bool kFp8 = sizeof(OT) == 1, kAhead = C <= 2;
  __shared__ float2 parts[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  // res may be res_out: a row of it is read before any thread of its block writes it, and by no other block
  Raw8<XT> xr[C];
  Raw8<RT> rr[C];
  auto load = [&](long long r) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int e = 8 * (tid + j * nthr), n = p.d - e;
      xr[j] = load_raw8<false>(static_cast<const XT *>(p.x) + r * p.ldx + e, n, p.vec);
      if (p.res) rr[j] = load_raw8<true>(static_cast<const RT *>(p.res) + r * p.ldr + e, n, p.vec);
    }
  };
  auto load_g = [&](int j, float (&g)[8]) {
    const int e = 8 * (tid + j * nthr);
    if (p.gamma) load_row8(p.gamma + e, p.d - e, true, g);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
  };
  float g[kAhead ? C : 1][8];
  if constexpr (kAhead) {
    load(blockIdx.x);
#pragma unroll
    for (int j = 0; j < C; ++j) load_g(j, g[j]);
  }
  int it = 0;
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x, it ^= 1) {
    float z[C][8];
    float ss = 0.f, am = 0.f;
    RT *ro = static_cast<RT *>(p.res_out) + r * p.ldr;
    if constexpr (!kAhead) load(r);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      unpack8(xr[j], z[j]);
      if (p.res) {
        float a[8];
        unpack8(rr[j], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] += a[i];
      }
    }
    if constexpr (kAhead)
      if (r + gridDim.x < p.rows) load(r + gridDim.x);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int e = 8 * (tid + j * nthr), n = p.d - e;
      if (p.res_out) store_row8(ro + e, n, p.vec, z[j]);
      float(&gj)[8] = g[kAhead ? j : 0];
      if constexpr (!kAhead) load_g(j, gj);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += z[j][i] * z[j][i];
        z[j][i] *= gj[i];
        if (kFp8) am = fmaxf(am, fabsf(z[j][i]));
      }
    }
    ss = warp_sum(ss);
    if (kFp8) am = warp_max(am);
    float2 *part = parts[it];
    if (lane == 0) part[warp] = make_float2(ss, am);
    __syncthreads();
    const float2 q = lane < (nthr >> 5) ? part[lane] : make_float2(0.f, 0.f);
    ss = warp_sum(q.x);
    if (kFp8) am = warp_max(q.y);
    const float rstd = 1.0f / sqrtf(ss / (float)p.d + p.eps);

    float scale = 0.f;
    if (kFp8 && p.group == 0) {
      scale = __fdiv_rn(am * rstd, 448.0f);
      if (tid == 0) p.out_scale[r] = scale;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int e = 8 * (tid + j * nthr), n = p.d - e;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] *= rstd;
      if constexpr (kFp8) {
        if (p.group) {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(z[j][i]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          if (p.group == 128) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          scale = __fdiv_rn(m, 448.0f);
          if (n > 0 && e % p.group == 0) p.out_scale[r * (p.d / p.group) + e / p.group] = scale;
        }
        if (n <= 0) continue;
        uint32_t w[2] = {0u, 0u};
        if (scale > 0.f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i >> 2] |= f32_e4m3(__fdiv_rn(z[j][i], scale)) << (8 * (i & 3));
        }
        unsigned char *o = static_cast<unsigned char *>(p.out) + r * p.ldo + e;
        if (p.vec && n >= 8) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < n) o[i] = (unsigned char)(w[i >> 2] >> (8 * (i & 3)));
      } else {
        if (n > 0) store_row8(static_cast<OT *>(p.out) + r * p.ldo + e, n, p.vec, z[j]);
      }
    }
  }
}

// One wave of blocks, each with every gridDim-th row (2.3 waves: 97 us where
// this takes 83 at 16411 x 4104 bf16).
template <typename XT, typename RT, typename OT, int C>
int launch_norm_c(const NormParams &p, int thr, cudaStream_t s) {
  const unsigned grid = (unsigned)std::min<long long>(p.rows, resident_blocks<add_rms_norm_kernel<XT, RT, OT, C>>(thr));
  return HCA_LAUNCH("add_rms_norm", s, add_rms_norm_kernel<XT, RT, OT, C><<<grid, thr, 0, s>>>(p));
}

template <typename XT, typename RT, typename OT>
int launch_norm_t(const NormParams &p, cudaStream_t s) {
  // threads of 8 channels up to 512 of them, then of 16, then (up to 1024 threads) of 32
  const int units = (p.d + 7) / 8;
  const int C = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
  const int thr = ((units + C - 1) / C + 31) / 32 * 32;
  if (C == 1) return launch_norm_c<XT, RT, OT, 1>(p, thr, s);
  if (C == 2) return launch_norm_c<XT, RT, OT, 2>(p, thr, s);
  return launch_norm_c<XT, RT, OT, 4>(p, thr, s);
}
template <typename XT, typename RT>
int launch_norm_o(const NormParams &p, hca_dtype od, cudaStream_t s) {
  if (od == HCA_F32) return launch_norm_t<XT, RT, float>(p, s);
  if (od == HCA_BF16) return launch_norm_t<XT, RT, __nv_bfloat16>(p, s);
  return launch_norm_t<XT, RT, E4M3>(p, s);
}

}  // namespace

int launch_add_rms_norm(const NormParams &p, hca_dtype xd, hca_dtype rd, hca_dtype od, cudaStream_t s) {
  if (p.rows == 0) return HCA_OK;
  if (xd == HCA_F32) return launch_norm_o<float, float>(p, od, s);
  if (rd == HCA_F32) return launch_norm_o<__nv_bfloat16, float>(p, od, s);
  return launch_norm_o<__nv_bfloat16, __nv_bfloat16>(p, od, s);
}

}  // namespace hca
