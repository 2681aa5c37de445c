// kv_fp4.cu -- KV rows in 4-bit records: written from f32 / bf16 rows, read
// back as bf16 rows.
//
// Record: E2M1 codes of the c - rd leading channels (two to a byte), the rd
// RoPE channels in bf16, one exponent byte per 32 code channels.  With a
// block's amax <= 6 * 2^e the smallest such e loses no value to saturation,
// and code * 2^e has two significant bits, so bf16 holds it exactly.
//
// Both kernels are HBM streams.  A lane holds 16 channels of a row, so a row
// takes c / 16 lanes and a warp 32 / (c / 16) rows; the two lanes of a block
// exchange their maxima with one shuffle.
#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

constexpr int kFp4KvWarps = 8;

__device__ __forceinline__ void load16(const float *p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p) + i);
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = bf16_lo(w[j]);
      v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Lane l of a warp holds channels 16 (l % L) .. +15 of row l / L (L = c / 16);
// lanes from per * L on have no row.
struct LaneRow {
  int u;          // 16-channel unit of the row
  int sub;        // row within the warp
  int partner;    // lane with the other half of the block
  bool on;
};
__device__ __forceinline__ LaneRow lane_row(int lane, int L) {
  LaneRow r;
  r.sub = lane / L;
  r.u = lane - r.sub * L;
  r.on = r.sub < 32 / L;
  r.partner = min(r.sub * L + (r.u ^ 1), 31);
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kFp4KvWarps * 32)
    kv_quant_fp4_kernel(const T *__restrict__ x, long long rows, int c, int rd, unsigned char *__restrict__ out, int rec,
                        long long records, const long long *__restrict__ slots) {
  const int lane = threadIdx.x & 31, L = c / 16, per = 32 / L;
  const LaneRow lr = lane_row(lane, L);
  const int nq = c - rd, ncl = nq / 16;
  const int soff = nq / 2 + 2 * rd, payload = soff + nq / 32;
  const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long r0 = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * per; r0 < rows; r0 += nwarps * per) {
    const long long r = r0 + lr.sub;
    const bool on = lr.on && r < rows;
    long long slot = -1;
    if (on) slot = slots ? __ldg(slots + r) : r;
    float v[16], amax = 0.f;
    if (on) {
      load16(x + r * c + 16 * lr.u, v);
      if (lr.u < ncl) {
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
      }
    }
    amax = fmaxf(amax, __shfl_sync(0xffffffffu, amax, lr.partner));
    if (!on || slot < 0 || slot >= records) continue;
    unsigned char *rp = out + slot * rec;
    if (lr.u < ncl) {
      uint32_t w[2] = {0u, 0u};
      uint32_t eb = 0u;
      if (amax > 0.f) {
        const int e = fp4_block_exp(amax);
        eb = (uint32_t)(e + 127);
        const float inv = pow2f(-e);     // -126 <= -e <= 126: exact products
        float q[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i >> 3][i & 7] = v[i] * inv;
        w[0] = e2m1x8_code(q[0]);
        w[1] = e2m1x8_code(q[1]);
      }
      *reinterpret_cast<uint2 *>(rp + 8 * lr.u) = make_uint2(w[0], w[1]);
      if ((lr.u & 1) == 0) rp[soff + (lr.u >> 1)] = (unsigned char)eb;
    } else {
      uint4 *d = reinterpret_cast<uint4 *>(rp + nq / 2 + 32 * (lr.u - ncl));
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    }
    for (int b = payload + lr.u; b < rec; b += L) rp[b] = 0;
  }
}

__global__ void __launch_bounds__(kFp4KvWarps * 32)
    kv_dequant_fp4_kernel(const unsigned char *__restrict__ in, long long records, const long long *__restrict__ slots,
                          long long rows, int c, int rd, __nv_bfloat16 *__restrict__ out, int rec) {
  const int lane = threadIdx.x & 31, L = c / 16, per = 32 / L;
  const LaneRow lr = lane_row(lane, L);
  const int nq = c - rd, ncl = nq / 16, soff = nq / 2 + 2 * rd;
  const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
  if (!lr.on) return;
  for (long long r0 = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * per; r0 < rows; r0 += nwarps * per) {
    const long long r = r0 + lr.sub;
    if (r >= rows) continue;
    const long long slot = slots ? __ldg(slots + r) : r;
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (slot >= 0 && slot < records) {
      const unsigned char *rp = in + slot * rec;
      if (lr.u < ncl) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(rp + 8 * lr.u));
        const uint32_t eb = __ldg(rp + soff + (lr.u >> 1));
        // byte 0 (an all-zero block): the codes are zero, any finite scale does
        const float sc = pow2f(max((int)eb, 1) - 127);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t f[4];
          e2m1x8_f16(h ? w.y : w.x, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&f[i]));
            o[4 * h + i] = pack_bf16x2(a.x * sc, a.y * sc);
          }
        }
      } else {
        const uint4 *s = reinterpret_cast<const uint4 *>(rp + nq / 2 + 32 * (lr.u - ncl));
        const uint4 a = __ldg(s), b = __ldg(s + 1);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
      }
    }
    uint4 *d = reinterpret_cast<uint4 *>(out + r * c + 16 * lr.u);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

int fp4_kv_grid(long long rows, int c) {
  const long long per = (long long)kFp4KvWarps * (32 / (c / 16));
  const long long blocks = (rows + per - 1) / per;
  const long long cap = (long long)num_sms() * 16;
  return (int)(blocks < cap ? blocks : cap);
}

}  // namespace

// Alignment inside a record: q / 2 is a multiple of 32 and the record of 16,
// so codes, RoPE channels and their 16-byte accesses stay aligned.
size_t kv_fp4_row_bytes(int c, int rd) {
  if (c < 16 || c > 512 || rd < 0 || rd > c || rd % 16 != 0 || (c - rd) % 64 != 0) return 0;
  const size_t q = (size_t)(c - rd);
  return (q / 2 + 2 * (size_t)rd + q / 32 + 15) & ~(size_t)15;
}

int launch_kv_quant_fp4(const void *x, hca_dtype dt, long long rows, int c, int rd, void *out, long long records,
                        const long long *slots, cudaStream_t s) {
  if (rows == 0) return HCA_OK;
  const int rec = (int)kv_fp4_row_bytes(c, rd), grid = fp4_kv_grid(rows, c);
  unsigned char *o = static_cast<unsigned char *>(out);
  if (dt == HCA_F32)
    return HCA_LAUNCH("kv_quant_fp4", s,
                      kv_quant_fp4_kernel<float><<<grid, kFp4KvWarps * 32, 0, s>>>(static_cast<const float *>(x), rows, c,
                                                                                   rd, o, rec, records, slots));
  return HCA_LAUNCH("kv_quant_fp4", s,
                    kv_quant_fp4_kernel<__nv_bfloat16><<<grid, kFp4KvWarps * 32, 0, s>>>(
                        static_cast<const __nv_bfloat16 *>(x), rows, c, rd, o, rec, records, slots));
}

int launch_kv_dequant_fp4(const void *in, long long records, const long long *slots, long long rows, int c, int rd,
                          void *out, cudaStream_t s) {
  if (rows == 0) return HCA_OK;
  const int rec = (int)kv_fp4_row_bytes(c, rd);
  return HCA_LAUNCH("kv_dequant_fp4", s,
                    kv_dequant_fp4_kernel<<<fp4_kv_grid(rows, c), kFp4KvWarps * 32, 0, s>>>(
                        static_cast<const unsigned char *>(in), records, slots, rows, c, rd,
                        static_cast<__nv_bfloat16 *>(out), rec));
}

}  // namespace hca
