// w4.cu -- products of a few tokens with 4-bit weights, and the quantiser that
// makes the weights.
//
//   out[t, g N + n] = xs[t] rs[g, n] sum_k x[t, g K + k] s[g, k / G, n] code[g, n, k]
//
// An E2M1 or INT4 code (at most 4 significant bits) times an e4m3 scale (4
// bits) is exact in f16 and in fp32, so the only roundings are the fp32 sums
// and the output's.
#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

// value of a code
__device__ __forceinline__ float w4_value(uint32_t q, int code) {
  q &= 15u;
  if (code == HCA_W4_INT4) return (float)((int)(q ^ 8u) - 8);
  const uint32_t m = q & 7u;
  const float a = m < 4u ? 0.5f * (float)m : m < 6u ? (float)m - 2.f : 2.f * (float)m - 8.f;
  return q & 8u ? -a : a;
}

// A warp per output, lanes over words of eight codes, eight tokens a pass.
template <typename XT, typename OT>
__global__ void __launch_bounds__(256) w4_simple_kernel(W4Params p) {
  const int lane = threadIdx.x & 31;
  const long long o = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= (long long)p.groups * p.N) return;
  const int g = (int)(o / p.N), n = (int)(o - (long long)g * p.N);
  const uint32_t *w = reinterpret_cast<const uint32_t *>(p.codes + o * (p.K / 2));
  const unsigned char *sc = p.scales + (long long)g * (p.K / p.G) * p.ldn + n;
  const float rs = p.row_scale[o];
  for (int t0 = 0; t0 < p.T; t0 += 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 8 * lane; k < p.K; k += 256) {
      const uint32_t q = w[k / 8];
      const float s = e4m3_f32(sc[(long long)(k / p.G) * p.ldn]);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s * w4_value(q >> (4 * i), p.code);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (t0 + t >= p.T) break;
        const XT *x = static_cast<const XT *>(p.x) + (t0 + t) * p.ldx + (long long)g * p.K + k;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float xv;
          if constexpr (sizeof(XT) == 1) xv = e4m3_f32(x[i]);
          else xv = Elt<XT>::load(x + i);
          acc[t] += v[i] * xv;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t0 + t >= p.T) break;
      const float a = warp_sum(acc[t]) * rs * (p.x_scale ? p.x_scale[t0 + t] : 1.f);
      if (lane == 0) Elt<OT>::store(static_cast<OT *>(p.out) + (t0 + t) * p.ldo + o, a);
    }
  }
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

size_t w4_workspace_bytes(const W4Params &) { return 0; }

int launch_w4_linear(const W4Params &p, hca_dtype xd, hca_dtype od, cudaStream_t s) {
  if (p.T == 0) return HCA_OK;
  const unsigned grid = (unsigned)(((long long)p.groups * p.N + 7) / 8);
  if (xd == HCA_BF16) {
    if (od == HCA_F32)
      return HCA_LAUNCH("w4_linear", s, w4_simple_kernel<__nv_bfloat16, float><<<grid, 256, 0, s>>>(p));
    return HCA_LAUNCH("w4_linear", s, w4_simple_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, s>>>(p));
  }
  if (od == HCA_F32) return HCA_LAUNCH("w4_linear", s, w4_simple_kernel<unsigned char, float><<<grid, 256, 0, s>>>(p));
  return HCA_LAUNCH("w4_linear", s, w4_simple_kernel<unsigned char, __nv_bfloat16><<<grid, 256, 0, s>>>(p));
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
