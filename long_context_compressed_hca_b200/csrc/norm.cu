// norm.cu -- residual addition + RMSNorm of rows, with an f32, bf16 or e4m3
// output.
//
//   z = x + res,  y = z * gamma / sqrt(mean z^2 + eps),
//   e4m3: scale = amax|y| / 448 over a row or a group, code = e4m3(y / scale).
//
// One block per row holds the row in registers (8 C channels per thread), so
// every input is read once and every output written once.  A row-wide e4m3
// scale needs amax|y| = max|z gamma| / sqrt(..), which is reduced together
// with the sum of squares: one block reduction either way.  Group scales are
// maxima over 8 or 16 neighbouring lanes.
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

template <typename XT, typename RT, typename OT, int C>
__global__ void __launch_bounds__(1024)
    add_rms_norm_kernel(NormParams p) {
  constexpr bool kFp8 = sizeof(OT) == 1;
  __shared__ float2 part[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const long long r = blockIdx.x;
  const XT *x = static_cast<const XT *>(p.x) + r * p.ldx;
  const RT *res = static_cast<const RT *>(p.res) + r * p.ldr;
  RT *ro = static_cast<RT *>(p.res_out) + r * p.ldr;

  float z[C][8], g[C][8];
  float ss = 0.f, am = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int e = 8 * (tid + j * nthr), n = p.d - e;
    load_row8(x + e, n, p.vec, z[j]);
    if (p.res) {
      float a[8];
      load_row8(res + e, n, p.vec, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] += a[i];
    }
    if (p.gamma) load_row8(p.gamma + e, n, true, g[j]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) g[j][i] = 1.f;
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int e = 8 * (tid + j * nthr), n = p.d - e;
    if (p.res_out) store_row8(ro + e, n, p.vec, z[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss += z[j][i] * z[j][i];
      z[j][i] *= g[j][i];
      if (kFp8) am = fmaxf(am, fabsf(z[j][i]));
    }
  }
  ss = warp_sum(ss);
  if (kFp8) am = warp_max(am);
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

template <typename XT, typename RT, typename OT>
int launch_norm_t(const NormParams &p, cudaStream_t s) {
  // threads of 8 channels up to 512 of them, then more channels per thread
  const int units = (p.d + 7) / 8;
  const int C = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
  const int thr = ((units + C - 1) / C + 31) / 32 * 32;
  const unsigned grid = (unsigned)p.rows;
  if (C == 1) return HCA_LAUNCH("add_rms_norm", s, add_rms_norm_kernel<XT, RT, OT, 1><<<grid, thr, 0, s>>>(p));
  if (C == 2) return HCA_LAUNCH("add_rms_norm", s, add_rms_norm_kernel<XT, RT, OT, 2><<<grid, thr, 0, s>>>(p));
  return HCA_LAUNCH("add_rms_norm", s, add_rms_norm_kernel<XT, RT, OT, 4><<<grid, thr, 0, s>>>(p));
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
