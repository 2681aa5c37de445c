// attend_fp4.cu -- decode attention (one query token per sequence) over a
// cache of 4-bit KV records, one position per sequence.
//
// The formula is attend.cu's: keys are the window rows of tokens
// max(0, pos - w + 1) .. pos and the compressed entries (listed, or all that
// are visible); z_j = scale q_h . row_j; o_h = sum_j e^{z_j} row_j /
// (sum_j e^{z_j} + e^{sink_h}); the last rd dims of o_h rotated by -pos.
#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

// The key set of sequence b.
struct Fp4Keys {
  int pos, nw, V, n;   // position, window rows, visible entries the cache can hold, key slots (idx slots included)
};
__device__ __forceinline__ Fp4Keys fp4_keys(const AttendFp4Params &p, int b) {
  Fp4Keys k;
  k.pos = min(__ldg(p.positions + b), p.max_pos);
  if (k.pos < 0) {
    k.pos = -1;
    k.nw = k.V = k.n = 0;
    return k;
  }
  k.nw = min(p.w, k.pos + 1);
  const long long room = p.pages ? (long long)p.max_pages * p.cap : (long long)p.cap;
  k.V = (int)min((long long)((k.pos + 1) / p.m), room);
  k.n = k.nw + (p.idx ? p.k : k.V);
  return k;
}
// Record of compressed key slot j (0 <= j < n - nw); NULL = skipped.
__device__ __forceinline__ const unsigned char *fp4_record(const AttendFp4Params &p, int b, const Fp4Keys &k, int j) {
  const int e = p.idx ? __ldg(p.idx + (long long)b * p.k + j) : j;
  if (e < 0 || e >= k.V) return nullptr;
  long long row;
  if (p.pages) {
    const int pg = __ldg(p.pages + (long long)b * p.max_pages + e / p.cap);
    if (pg < 0 || pg >= p.n_pages) return nullptr;
    row = (long long)pg * p.cap + e % p.cap;
  } else {
    row = (long long)b * p.cap + e;
  }
  return p.rows + row * p.rec;
}

constexpr int kSimpleTile = 16;

// One block per (head, sequence): 16 keys at a time in shared memory, a warp
// per two keys' logits, a thread per two channels' output.
__global__ void __launch_bounds__(256) attend_fp4_simple_kernel(AttendFp4Params p) {
  extern __shared__ float sm[];
  float *kv = sm, *q = sm + kSimpleTile * p.c, *z = q + p.c;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Fp4Keys ks = fp4_keys(p, b);
  const int nq = p.c - p.rd;
  const __nv_bfloat16 *qp = p.q + ((long long)b * p.n_h + h) * p.c;
  for (int i = tid; i < p.c; i += 256) q[i] = __bfloat162float(qp[i]);
  const float sink = p.sink ? p.sink[h] * 1.4426950408889634f : -INFINITY;
  float m = sink, l = p.sink ? 1.f : 0.f, o[2] = {0.f, 0.f};
  for (int j0 = 0; j0 < ks.n; j0 += kSimpleTile) {
    __syncthreads();
    for (int i = tid; i < kSimpleTile * p.c; i += 256) {
      const int jj = i / p.c, ch = i - jj * p.c, j = j0 + jj;
      float v = 0.f;
      if (j < ks.nw) {
        const int tok = ks.pos - ks.nw + 1 + j;
        v = __bfloat162float(p.kv_win[((long long)b * p.w + tok % p.w) * p.c + ch]);
      } else if (j < ks.n) {
        const unsigned char *r = fp4_record(p, b, ks, j - ks.nw);
        if (r) {
          if (ch < nq) {
            uint32_t f[4];
            e2m1x8_f16(reinterpret_cast<const uint32_t *>(r)[ch / 8], f);
            const uint32_t pr = ch & 4 ? (ch & 2 ? f[3] : f[2]) : (ch & 2 ? f[1] : f[0]);
            __half_raw h;
            h.x = (unsigned short)(ch & 1 ? pr >> 16 : pr & 0xFFFFu);
            v = __half2float(__half(h)) * pow2f(max((int)r[nq / 2 + 2 * p.rd + ch / 32], 1) - 127);
          } else {
            v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(r + nq / 2)[ch - nq]);
          }
        }
      }
      kv[i] = v;
    }
    __syncthreads();
    for (int jj = warp; jj < kSimpleTile; jj += 8) {
      const int j = j0 + jj;
      const bool live = j < ks.n && (j < ks.nw || fp4_record(p, b, ks, j - ks.nw));
      float a = 0.f;
      for (int i = lane; i < p.c; i += 32) a += q[i] * kv[jj * p.c + i];
      a = warp_sum(a);
      if (lane == 0) z[jj] = live ? a * p.scale * 1.4426950408889634f : -INFINITY;
    }
    __syncthreads();
    float mt = m;
    for (int jj = 0; jj < kSimpleTile; ++jj) mt = fmaxf(mt, z[jj]);
    if (mt == -INFINITY) continue;
    const float f = exp2f(m - mt);
    m = mt;
    l *= f;
    o[0] *= f;
    o[1] *= f;
    for (int jj = 0; jj < kSimpleTile; ++jj) {
      const float e = exp2f(z[jj] - m);
      l += e;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (2 * tid + i < p.c) o[i] += e * kv[jj * p.c + 2 * tid + i];
    }
  }
  if (2 * tid >= p.c) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  o[0] *= inv;
  o[1] *= inv;
  if (2 * tid >= nq && ks.pos >= 0) {
    float si, co;
    rope_sincos_tab(p.rope_freq, ks.pos, (2 * tid - nq) / 2, p.rd, p.theta, &si, &co);
    const float a = o[0] * co + o[1] * si, c = o[1] * co - o[0] * si;
    o[0] = a;
    o[1] = c;
  }
  reinterpret_cast<uint32_t *>(p.o + ((long long)b * p.n_h + h) * p.c)[tid] = pack_bf16x2(o[0], o[1]);
}

}  // namespace

size_t attend_fp4_workspace_bytes(const AttendFp4Params &) { return 0; }

int run_attend_fp4(const AttendFp4Params &p, void *, size_t, cudaStream_t s) {
  const size_t smem = ((kSimpleTile + 1) * (size_t)p.c + kSimpleTile) * 4;
  return HCA_LAUNCH("attend_fp4", s, attend_fp4_simple_kernel<<<dim3(p.n_h, p.B), 256, smem, s>>>(p));
}

}  // namespace hca
