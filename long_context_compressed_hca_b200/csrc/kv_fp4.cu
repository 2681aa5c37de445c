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
// exchange their maxima with one shuffle.  The loads of further rows are on
// their way while one is converted (131075 rows of 512, 184 MB each way: written
// in 38 us, 41 without; read in 33 us, 37 without), and a grid is one wave.
#include <algorithm>

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
  const int soff = nq / 2 + 2 * rd, pad = soff + 4 * ((L + 7) / 8);   // exponents, zeros after the lanes' words
  const long long step = (((long long)gridDim.x * blockDim.x) >> 5) * per;
  // the next row is on its way while this one is written
  long long slot = -1;
  float v[16];
  auto load = [&](long long r0) {
    const long long r = r0 + lr.sub;
    slot = -1;
    if (!lr.on || r >= rows) return;
    slot = slots ? __ldg(slots + r) : r;
    load16(x + r * c + 16 * lr.u, v);
  };
  const long long first = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * per;
  load(first);
  for (long long r0 = first; r0 < rows; r0 += step) {
    const bool on = slot >= 0 && slot < records;
    unsigned char *rp = out + (on ? slot * rec : 0);
    float amax = 0.f;
    if (lr.u < ncl) {
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    }
    amax = fmaxf(amax, __shfl_sync(0xffffffffu, amax, lr.partner));
    uint32_t eb = 0u, w[8];
    if (lr.u < ncl) {
      w[0] = w[1] = 0u;
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
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    load(r0 + step);
    // four exponent bytes to a word, in every eighth lane of a row
    uint32_t y = __shfl_down_sync(0xffffffffu, eb, 2);
    eb |= lr.u + 2 < ncl ? y << 8 : 0u;
    y = __shfl_down_sync(0xffffffffu, eb, 4);
    eb |= lr.u + 4 < ncl ? y << 16 : 0u;
    if (!on) continue;
    if ((lr.u & 7) == 0 && soff + lr.u / 2 < rec) *reinterpret_cast<uint32_t *>(rp + soff + lr.u / 2) = eb;
    if (lr.u < ncl) {
      *reinterpret_cast<uint2 *>(rp + 8 * lr.u) = make_uint2(w[0], w[1]);
    } else {
      uint4 *d = reinterpret_cast<uint4 *>(rp + nq / 2 + 32 * (lr.u - ncl));
      d[0] = make_uint4(w[0], w[1], w[2], w[3]);
      d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    for (int b = pad + 4 * lr.u; b < rec; b += 4 * L) *reinterpret_cast<uint32_t *>(rp + b) = 0u;
  }
}

// A warp's rows are read kAhead at a time: the slots of all, then the records
// of all, then the rows are written.
__global__ void __launch_bounds__(kFp4KvWarps * 32)
    kv_dequant_fp4_kernel(const unsigned char *__restrict__ in, long long records, const long long *__restrict__ slots,
                          long long rows, int c, int rd, __nv_bfloat16 *__restrict__ out, int rec) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31, L = c / 16, per = 32 / L;
  const LaneRow lr = lane_row(lane, L);
  const int nq = c - rd, ncl = nq / 16, soff = nq / 2 + 2 * rd;
  const long long step = (((long long)gridDim.x * blockDim.x) >> 5) * per;
  if (!lr.on) return;
  const bool codes = lr.u < ncl;
  const int off = codes ? 8 * lr.u : nq / 2 + 32 * (lr.u - ncl), eoff = soff + (lr.u >> 1);
  for (long long r0 = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * per + lr.sub; r0 < rows; r0 += kAhead * step) {
    long long slot[kAhead];
    uint4 a[kAhead], b[kAhead];            // codes in a.x, a.y and their exponent byte in a.z; or 16 bf16
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long r = r0 + k * step;
      slot[k] = r >= rows ? -1 : slots ? __ldg(slots + r) : r;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      if (slot[k] < 0 || slot[k] >= records) continue;
      const unsigned char *rp = in + slot[k] * rec;
      if (codes) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(rp + off));
        a[k] = make_uint4(w.x, w.y, __ldg(rp + eoff), 0);
      } else {
        a[k] = __ldg(reinterpret_cast<const uint4 *>(rp + off));
        b[k] = __ldg(reinterpret_cast<const uint4 *>(rp + off) + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long r = r0 + k * step;
      if (r >= rows) break;
      if (codes) {
        // byte 0 (an all-zero block): the codes are zero, any finite scale does
        const float sc = pow2f(max((int)a[k].z, 1) - 127);
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t f[4];
          e2m1x8_f16(h ? a[k].y : a[k].x, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f[i]));
            o[4 * h + i] = pack_bf16x2(v.x * sc, v.y * sc);
          }
        }
        a[k] = make_uint4(o[0], o[1], o[2], o[3]);
        b[k] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      uint4 *d = reinterpret_cast<uint4 *>(out + r * c + 16 * lr.u);
      d[0] = a[k];
      d[1] = b[k];
    }
  }
}

// Blocks for the rows, up to `most` of them.
int fp4_kv_grid(long long rows, int c, int most) {
  const long long per = (long long)kFp4KvWarps * (32 / (c / 16));
  return (int)std::min<long long>((rows + per - 1) / per, most);
}
template <typename T>
int launch_quant_t(const void *x, long long rows, int c, int rd, void *out, long long records, const long long *slots,
                   cudaStream_t s) {
  const int grid = fp4_kv_grid(rows, c, resident_blocks<kv_quant_fp4_kernel<T>>(kFp4KvWarps * 32));
  return HCA_LAUNCH("kv_quant_fp4", s,
                    kv_quant_fp4_kernel<T><<<grid, kFp4KvWarps * 32, 0, s>>>(
                        static_cast<const T *>(x), rows, c, rd, static_cast<unsigned char *>(out),
                        (int)kv_fp4_row_bytes(c, rd), records, slots));
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
  return dt == HCA_F32 ? launch_quant_t<float>(x, rows, c, rd, out, records, slots, s)
                       : launch_quant_t<__nv_bfloat16>(x, rows, c, rd, out, records, slots, s);
}

int launch_kv_dequant_fp4(const void *in, long long records, const long long *slots, long long rows, int c, int rd,
                          void *out, cudaStream_t s) {
  if (rows == 0) return HCA_OK;
  const int rec = (int)kv_fp4_row_bytes(c, rd);
  const int grid = fp4_kv_grid(rows, c, resident_blocks<kv_dequant_fp4_kernel>(kFp4KvWarps * 32));
  return HCA_LAUNCH("kv_dequant_fp4", s,
                    kv_dequant_fp4_kernel<<<grid, kFp4KvWarps * 32, 0, s>>>(
                        static_cast<const unsigned char *>(in), records, slots, rows, c, rd,
                        static_cast<__nv_bfloat16 *>(out), rec));
}

}  // namespace hca
