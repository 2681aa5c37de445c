// attend_fp4.cu -- decode attention (one query token per sequence) over a
// cache of 4-bit KV records, one position per sequence.
//
// The formula is attend.cu's: keys are the window rows of tokens
// max(0, pos - w + 1) .. pos and the compressed entries (listed, or all that
// are visible); z_j = scale q_h . row_j; o_h = sum_j e^{z_j} row_j /
// (sum_j e^{z_j} + e^{sink_h}); the last rd dims of o_h rotated by -pos.
//
// Keys are taken 64 at a time, a sequence's window tiles last.  Two ways to
// spread the tiles (fp4_cluster chooses):
//   runs      the tiles of all sequences form one list, and every CTA takes an
//             equal run of it, so that ragged lengths cost nothing; the runs
//             follow from the positions on the device, which each CTA sums up
//             itself.  A sequence inside one run is finished there; one that
//             was cut leaves unnormalised fp32 parts in the workspace, which
//             fp4_combine_kernel joins in their order.
//   clusters  2, 4 or 8 CTAs share a sequence's tiles equally and join their
//             parts through distributed shared memory (fp4_cluster_join).
//
// Per tile (tcgen05, the sequence's n_h <= 64 heads as the MMA's M = 64):
//   8 loader warps   codes of the next tile on their way into shared memory
//                    (cp.async, every thread its own parts: no barrier; asked
//                    for before this tile's are converted) while this one's
//                    become bf16 (exact: two significant bits and a
//                    power of two) in a 128B-swizzled tile that serves as K
//                    (K-major) and V (MN-major); RoPE channels and window rows
//                    are copied into the tile, skipped keys are zero rows
//   1 MMA warp       S = Q K^T (Q in tensor memory, the A operand), O += P V;
//                    S of the next tile is issued before P V of this one
//   4 softmax warps  S from tensor memory, running maximum moved only when it
//                    grows by more than 2^8, P in bf16 (its rounding, 2^-8 of
//                    p, is that of the bf16 output; sums and statistics fp32)
// Bound: a tile takes 3250 cycles of a CTA at c = 512 (32 sequences of 16384
// entries: 122 us).  M = 64 uses half the tensor pipe, 2460 cycles of MMAs; the
// loader warps need 3100, about the same with the conversion by other
// instructions (byte lookups in the integer pipe, a mixture of both) or ordered
// otherwise, and wait for 300.  64 x 368 bytes of HBM are 1000 cycles of an
// SM's share.  With few tiles per CTA the fixed parts (entry, page and code
// loads one after another, Q, the join) are most of the time: 5 tiles a
// sequence and CTA pair took 24 us as runs, 2 or 3 a CTA 19 in clusters.
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace hca {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int KT = 64;
constexpr int kMmaWarp = 4, kLoad0 = 5, kLoadWarps = 8;
constexpr int kThreads = (kLoad0 + kLoadWarps) * 32;
constexpr uint32_t kTileBytes = 64 * 128;   // 64 rows x 128 B: one 64-channel block of a tile
constexpr int SP = 2;                        // S and P buffers

// Launch-time sizes beside the call's parameters.
struct Fp4Plan {
  int G;                   // CTAs
  int S;                   // CTAs of a cluster that has one sequence; 0: runs over all sequences
  FastDiv fd_m, fd_cap;
  float4 *part_o;          // [2 G] parts of fp4_part's layout
  float2 *part_ml;         // [2 G][n_h]
  int4 *meta;              // [B]: first and last CTA of a cut sequence and the first one's slot; x < 0: finished
};

// A part's O, in the workspace or in shared memory: for every 16 heads and 4 columns i, i + 1, .. of either half of
// the channels, the 32 threads (half, head) side by side.  float4 index of
// heads 16 q .. and columns 4 i of part `slot`, thread 0.
__device__ __forceinline__ long long fp4_part(const AttendFp4Params &p, long long slot, int q, int i) {
  return ((slot * ((p.n_h + 15) / 16) + q) * (p.c / 8) + i) * 32;
}

// The key set of sequence b.
struct Fp4Keys {
  int pos, nw, V, ne;   // position, window rows, visible entries the cache can hold, entry slots (listed or V)
  int nwt, nt;          // window tiles, all tiles
};
__device__ __forceinline__ Fp4Keys fp4_keys(const AttendFp4Params &p, const Fp4Plan &pl, int b) {
  Fp4Keys k;
  k.pos = min(__ldg(p.positions + b), p.max_pos);
  if (k.pos < 0) {
    k.pos = -1;
    k.nw = k.V = k.ne = k.nwt = k.nt = 0;
    return k;
  }
  k.nw = min(p.w, k.pos + 1);
  const long long room = p.pages ? (long long)p.max_pages * p.cap : (long long)p.cap;
  k.V = (int)min((long long)fdiv(k.pos + 1, pl.fd_m), room);
  k.ne = p.idx ? p.k : k.V;
  k.nwt = (k.nw + KT - 1) / KT;
  k.nt = k.nwt + (k.ne + KT - 1) / KT;
  return k;
}

template <int C>
struct Fp4Layout {
  static constexpr int NKB = C / 64;
  static constexpr int NS = C == 512 ? 3 : C == 256 ? 6 : 8;     // key-tile stages
  static constexpr uint32_t kRawBytes = 256 * (4 * 16 + 4);      // a tile's codes: 4 chunks and 4 exponents per thread
  static constexpr uint32_t p_off = NS * NKB * kTileBytes;
  static constexpr uint32_t raw_off = p_off + SP * kTileBytes;
  static constexpr uint32_t bar_off = raw_off + kRawBytes;
  static constexpr uint32_t mask_off = bar_off + 512;            // [NS][2] uint32: keys of a stage
  static constexpr uint32_t run_off = mask_off + 64;             // [8] int: this CTA's run
  static constexpr uint32_t sum_off = run_off + 64;              // [32] int: sums of the warps
  static constexpr uint32_t bytes = sum_off + 128 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory");
  // tensor memory: O in lane-half 0, columns [0, C); in lane-half 1 S buffers
  // at [0, 128) and Q (bf16, two per column) at [128, 128 + C / 2)
  static constexpr uint32_t q_col = SP * KT;
};

struct Fp4Bars {
  uint64_t q_full, q_empty, o_empty, all_done, settled, kv_full[8], kv_empty[8], s_full[SP], s_empty[SP], p_full[SP], pv_done[SP];
  uint32_t tmem, ran_out;
};

// This CTA's run of tiles: from tile `j0` of sequence `b0`, `n` tiles; `before`
// = tiles of all sequences before the run's first tile.
struct Fp4Run {
  int b0, j0;
  int n, before, base, rem;
};
// Runs are base or base + 1 tiles long, the first rem ones the longer.
__device__ __forceinline__ int fp4_cta_of(const Fp4Run &r, int tile) {
  const int cut = r.rem * (r.base + 1);
  return tile < cut ? tile / (r.base + 1) : r.rem + (tile - cut) / r.base;
}

// Walks the pieces of a run: tiles [j, j + cnt) of sequence b.
struct Fp4Walk {
  int b, j, cnt, left;
  Fp4Keys k;
};
__device__ __forceinline__ Fp4Walk fp4_walk(const Fp4Run &r) {
  Fp4Walk w;
  w.b = r.b0 - 1;
  w.j = r.j0;
  w.cnt = 0;
  w.left = r.n;
  return w;
}
// The next piece; false at the end of the run.
__device__ __forceinline__ bool fp4_next(const AttendFp4Params &p, const Fp4Plan &pl, const Fp4Run &r, Fp4Walk &w) {
  if (w.left <= 0) return false;
  do {
    if (++w.b >= p.B) return false;
    w.k = fp4_keys(p, pl, w.b);
  } while (w.k.nt == 0);
  w.j = w.b == r.b0 ? r.j0 : 0;
  w.cnt = min(w.k.nt - w.j, w.left);
  w.left -= w.cnt;
  return true;
}

// ---------------------------------------------------------------- loaders
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// A tile on its way through a loader thread (one of 4 for one of 64 keys).
struct Fp4Tile {
  int kind;                // 0: none, 1: entries, 2: window rows
  int b, e, win0;          // sequence; entry of this thread's key; first token of the rows
  int cnt;                 // visible entries, then whether the key has a record; rows of a window tile
};

template <int C>
__device__ __forceinline__ void fp4_load(const AttendFp4Params &p, const Fp4Plan &pl, const Fp4Run &run, uint8_t *smem,
                                         Fp4Bars *bars) {
  using L = Fp4Layout<C>;
  const int pt = threadIdx.x - kLoad0 * 32, lw = pt >> 5, lane = pt & 31;
  const int kk = (lw & 1) * 32 + lane, grp = lw >> 1;          // key of the tile, quarter of the record
  const int nq = C - p.rd, units = nq / 32, rch = p.rd / 8;     // 16-byte code units, 16-byte RoPE chunks
  const int per = units <= 4 ? 1 : units <= 8 ? 2 : 4;          // units of this thread: u0 .. u0 + nu - 1
  const int u0 = grp * per, nu = max(0, min(per, units - u0));
  const int eoff = nq / 2 + 2 * p.rd + (u0 & ~3), esh = 8 * (u0 & 3);
  // RoPE chunks go to the threads with fewer than `per` units, where there are any
  const int busy = units / per, rfirst = busy == 4 ? grp : grp < busy ? rch : grp - busy, rstep = busy == 4 ? 4 : 4 - busy;
  const uint32_t sbase = smem_u32(smem), rawc = sbase + L::raw_off + pt * 16, rawe = sbase + L::raw_off + 4 * 4096 + pt * 4;
  const unsigned char *none = reinterpret_cast<const unsigned char *>(p.q);   // an address for copies of nothing

  Fp4Walk w = fp4_walk(run);
  int t = 0;                                                     // next tile of the piece
  bool more = true;
  // The loads of a tile stand in three rounds of one loop -- its entries, their
  // pages, their codes -- so that none is waited for in the round that issues
  // it: t3 entry on its way, t2 page on its way, t1 codes asked for, t0 written
  // to its stage.
  Fp4Tile t0{}, t1{}, t2{}, t3{};
  const unsigned char *rp0 = none, *rp1 = none;
  int pg = 0, st = 0;
  uint32_t ph = 1;
  const Waits wait{p.status, &bars->ran_out};
  while (true) {
    // ---- codes' address of t1 from the page that the round before asked for
    rp1 = none;
    if (t1.kind == 1 && t1.cnt) {
      long long row = (long long)t1.b * p.cap + t1.e;
      if (p.pages) {
        t1.cnt = pg >= 0 && pg < p.n_pages;
        row = (long long)pg * p.cap + (t1.e - fdiv(t1.e, pl.fd_cap) * p.cap);
      }
      if (t1.cnt) rp1 = p.rows + row * p.rec;
    }
    // ---- page of t2
    if (t2.kind == 1) {
      t2.cnt = t2.e >= 0 && t2.e < t2.cnt;
      if (p.pages && t2.cnt) pg = __ldg(p.pages + (long long)t2.b * p.max_pages + fdiv(t2.e, pl.fd_cap));
    }
    // ---- the next tile
    t3.kind = 0;
    if (more && t == w.cnt) {
      more = fp4_next(p, pl, run, w);
      t = 0;
    }
    if (more) {
      const int j = w.j + t++, net = w.k.nt - w.k.nwt;
      t3.b = w.b;
      if (j < net) {
        t3.kind = 1;
        t3.cnt = w.k.V;
        t3.e = j * KT + kk;
        if (p.idx) t3.e = t3.e < w.k.ne ? __ldg(p.idx + (long long)w.b * p.k + t3.e) : -1;
      } else {
        t3.kind = 2;
        t3.win0 = w.k.pos - w.k.nw + 1 + (j - net) * KT;
        t3.cnt = min(KT, w.k.nw - (j - net) * KT);
      }
    }
    if (!(t0.kind | t1.kind | t2.kind | t3.kind)) break;
    // ---- t0 into its stage
    uint8_t *tile = smem + st * L::NKB * kTileBytes;
    const uint32_t full = smem_u32(&bars->kv_full[st]);
    uint32_t ex = 0u;
    if (t0.kind) {
      wait(smem_u32(&bars->kv_empty[st]), ph);
      uint32_t *mask = reinterpret_cast<uint32_t *>(smem + L::mask_off) + 2 * st;
      const uint32_t tdst = sbase + st * L::NKB * kTileBytes;
      if (t0.kind == 2) {
        // window rows, 16-byte chunks in the order of the row
        constexpr int CPR = C / 8, RPP = kLoadWarps * 32 / CPR;
        const int chunk = pt % CPR;
        const __nv_bfloat16 *ring = p.kv_win + (long long)t0.b * p.w * C + chunk * 8;
        int slot = (t0.win0 + pt / CPR) % p.w;
#pragma unroll 4
        for (int r = pt / CPR; r < KT; r += RPP) {
          const bool on = r < t0.cnt;
          cp_async16(tdst + (chunk / 8) * kTileBytes + sw128_off(r, chunk % 8), ring + (on ? (long long)slot * C : 0), on ? 16 : 0);
          slot += RPP;
          while (slot >= p.w) slot -= p.w;
        }
        if (pt == 0) {
          mask[0] = range_bits(0, 0, t0.cnt);
          mask[1] = range_bits(32, 0, t0.cnt);
        }
      } else {
        cp_async_wait_all();               // this thread's codes are here
        for (int ch = rfirst; ch < rch; ch += rstep)
          cp_async16(tdst + ((nq / 8 + ch) / 8) * kTileBytes + sw128_off(kk, (nq / 8 + ch) % 8),
                     rp0 + (t0.cnt ? nq / 2 + 16 * ch : 0), t0.cnt ? 16 : 0);
        const uint32_t m = __ballot_sync(0xffffffffu, t0.cnt);
        if (grp == 0 && lane == 0) mask[lw] = m;
        if (nu) ex = *reinterpret_cast<const uint32_t *>(smem + L::raw_off + 4 * 4096 + pt * 4) >> esh;
      }
      cp_async_arrive_noinc(full);         // before the next tile's copies
    }
    // ---- its codes, and in their place those of t1, asked for before this tile's are converted
    uint4 code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < nu && t0.kind == 1) code[i] = *reinterpret_cast<const uint4 *>(smem + L::raw_off + i * 4096 + pt * 16);
    if (t1.kind == 1) {
      if (nu) cp_async4(rawe, rp1 + (t1.cnt ? eoff : 0), t1.cnt ? 4 : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < nu) cp_async16(rawc + i * 4096, rp1 + (t1.cnt ? 16 * (u0 + i) : 0), t1.cnt ? 16 : 0);
    }
    if (t0.kind == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i, ex >>= 8) {
        if (i >= nu) break;
        const int u = u0 + i;                // channels 32 u .. 32 u + 31
        const float sc = pow2f(max((int)(ex & 255u), 1) - 127);   // byte 0: all codes are zero
        const uint32_t wd[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        uint8_t *dst = tile + (u / 2) * kTileBytes;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t f[4], o[4];
          e2m1x8_f16(wd[h], f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f[q]));
            o[q] = pack_bf16x2(v.x * sc, v.y * sc);
          }
          *reinterpret_cast<uint4 *>(dst + sw128_off(kk, (u & 1) * 4 + h)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    if (t0.kind) {
      fence_proxy_async();      // the tensor cores read the tile through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      if (++st == L::NS) {
        st = 0;
        ph ^= 1;
      }
    }
    t0 = t1;
    t1 = t2;
    t2 = t3;
    rp0 = rp1;
  }
  cp_async_wait_all();
}

// ---------------------------------------------------------------- MMA issue
template <int C>
__device__ __forceinline__ void fp4_mma(const AttendFp4Params &p, const Fp4Plan &pl, const Fp4Run &run, uint32_t sbase,
                                        Fp4Bars *bars, uint32_t tmem) {
  using L = Fp4Layout<C>;
  constexpr uint32_t IDESC_S = idesc_bf16(64, KT, 0, 0);
  constexpr int NPV = C < 256 ? C : 256;
  constexpr uint32_t IDESC_PV = idesc_bf16(64, NPV, 0, 1);
  const uint32_t tS = tmem + (16u << 16);
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  int ks = 0, vs = 0;                     // stage of the next S and of the next P V
  uint32_t kph = 0, gs = 0, gv = 0;       // tiles issued so far
  int npiece = 0;
  const Waits wait{p.status, &bars->ran_out};
  auto issue_pv = [&](bool first) {
    const int st = gv % SP;
    wait(bar(bars->p_full[st]), (gv / SP) & 1);
    if (first) wait(bar(bars->o_empty), (npiece & 1) ^ 1);
    tc_fence_after();
    if (elect_one()) {
      const uint64_t pd = sdesc_sw128(sbase + L::p_off + st * kTileBytes, 16, 1024);
      const uint64_t vd = sdesc_sw128(sbase + vs * L::NKB * kTileBytes, kTileBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
        for (int nh = 0; nh < C / NPV; ++nh)
          umma_bf16(tmem + nh * NPV, pd + ((kk * 32) >> 4), vd + ((nh * (NPV / 64) * kTileBytes + kk * 16 * 128) >> 4),
                    IDESC_PV, first && kk == 0 ? 0u : 1u);
      umma_commit(bar(bars->kv_empty[vs]));
      umma_commit(bar(bars->pv_done[st]));
    }
    __syncwarp();
    if (++vs == L::NS) vs = 0;
    ++gv;
  };
  for (Fp4Walk w = fp4_walk(run); fp4_next(p, pl, run, w); ++npiece) {
    wait(bar(bars->q_full), npiece & 1);
    for (int j = 0; j < w.cnt; ++j) {
      const int st = gs % SP;
      wait(bar(bars->kv_full[ks]), kph);
      wait(bar(bars->s_empty[st]), ((gs / SP) & 1) ^ 1);
      fence_proxy_async();                // window rows come by cp.async
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = sdesc_sw128(sbase + ks * L::NKB * kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          umma_bf16_ts(tS + st * KT, tS + L::q_col + 8 * kk, kd + (((kk / 4) * kTileBytes + (kk % 4) * 32) >> 4), IDESC_S,
                       kk > 0 ? 1u : 0u);
        umma_commit(bar(bars->s_full[st]));
        if (j == w.cnt - 1) umma_commit(bar(bars->q_empty));
      }
      __syncwarp();
      if (++ks == L::NS) {
        ks = 0;
        kph ^= 1;
      }
      ++gs;
      if (j > 0) issue_pv(j == 1);
    }
    issue_pv(w.cnt == 1);
  }
  if (pl.S && run.n > 0 && elect_one()) umma_commit(bar(bars->all_done));   // the loaders wait for it
  wait.settle(bar(bars->settled));
  __syncwarp();
}

// sin and cos of position pos for pair i; the angle is reduced in double to
// [-pi, pi], where the fast sine and cosine are within 2^-20.
__device__ __forceinline__ void fp4_rope(const AttendFp4Params &p, int pos, int i, float &sn, float &cs) {
  const double f = p.rd <= 64 ? p.rope_freq[i] : exp2(-2.0 * (double)i / (double)p.rd * log2((double)p.theta));
  double a = (double)pos * f;
  a -= 6.283185307179586476925286766559 * rint(a * 0.15915494309189533576888376337251);
  __sincosf((float)a, &sn, &cs);
}

// Part `slot`'s sums of heads 16 q .. from tensor memory, 32 columns of either
// half at a time, every step-th of these from the first-th on.  A warp reads
// the lanes 32 (warp % 4) .., so q is warp % 4.
template <int C>
__device__ __forceinline__ void fp4_part_store(const AttendFp4Params &p, float4 *part, long long slot, uint32_t tmem, int q,
                                               int first, int step) {
  if (16 * q >= p.n_h) return;
  float4 *dst = part + fp4_part(p, slot, q, 8 * first) + (threadIdx.x & 31);
#pragma unroll 1
  for (int c0 = 32 * first; c0 < C / 2; c0 += 32 * step, dst += 256 * step) {
    uint32_t ov[32];
    tmem_ld_16x32bx2_x16<C / 2>(tmem + ((uint32_t)(q * 32) << 16) + c0, *reinterpret_cast<uint32_t(*)[16]>(&ov[0]));
    tmem_ld_16x32bx2_x16<C / 2>(tmem + ((uint32_t)(q * 32) << 16) + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&ov[16]));
    tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 8; ++x)
      dst[32 * x] = make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]), __uint_as_float(ov[4 * x + 2]),
                                __uint_as_float(ov[4 * x + 3]));
  }
}

// ---------------------------------------------------------------- softmax + epilogue
template <int C>
__device__ __forceinline__ void fp4_softmax(const AttendFp4Params &p, const Fp4Plan &pl, const Fp4Run &run, uint8_t *smem,
                                            Fp4Bars *bars, uint32_t tmem) {
  using L = Fp4Layout<C>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = lane & 15, half = lane >> 4;
  const int r = warp * 16 + hl;           // head; the thread has keys [32 half, +32) of a tile, then half of O's columns
  const bool live = r < p.n_h;
  const float zs = p.scale * kLog2e;
  const uint32_t lane_S = (uint32_t)(warp * 32 + 16) << 16, lane_O = (uint32_t)(warp * 32) << 16;
  float2 *rope = reinterpret_cast<float2 *>(smem + L::p_off);   // [256], between pieces
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  uint32_t g = 0;                         // tiles so far
  int ks = 0, npiece = 0;
  uint32_t kph = 0;
  int before = run.before;
  const Waits wait{p.status, &bars->ran_out};

  // Q into tensor memory, 64 channels of either half at a time: read 8 lanes to
  // 128 contiguous bytes and turned through this warp's 4 KB of the P buffers
  // (a lane to a row of its own touches 32 lines per load: 64 x 512 took 9000
  // cycles).  No P V may be reading the buffers.
  auto write_q = [&](int b) {
    tc_fence_after();
    const int sg = lane >> 3, ch = lane & 7;        // of 4 segments (head, half) per load; 16-byte chunk
    uint8_t *turn = smem + L::p_off + warp * 4096;
    const __nv_bfloat16 *src = p.q + (long long)b * p.n_h * C + 8 * ch;
    const uint32_t tq = tmem + lane_S + L::q_col;
    auto load = [&](int c0, uint4 (&v)[8]) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int seg = 4 * x + sg, row = warp * 16 + (seg & 15);
        v[x] = row < p.n_h ? __ldg(reinterpret_cast<const uint4 *>(src + (long long)row * C + (seg >> 4) * (C / 2) + c0))
                           : make_uint4(0, 0, 0, 0);
      }
    };
    auto turned = [&](int c0, uint4 (&v)[8]) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int seg = 4 * x + sg;
        *reinterpret_cast<uint4 *>(turn + seg * 128 + ((ch ^ (seg & 7)) << 4)) = v[x];
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = *reinterpret_cast<const uint4 *>(turn + lane * 128 + ((x ^ (lane & 7)) << 4));
      __syncwarp();
      tmem_st_16x32bx2_x16<C / 4>(tq + c0 / 2, *reinterpret_cast<const uint32_t(*)[16]>(&v[0]));
      tmem_st_16x32bx2_x16<C / 4>(tq + c0 / 2 + 16, *reinterpret_cast<const uint32_t(*)[16]>(&v[4]));
    };
    uint4 v0[8];
#pragma unroll 1
    for (int c0 = 0; c0 < C / 2; c0 += 64) {
      load(c0, v0);
      turned(c0, v0);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bars->q_full));
  };
  Fp4Walk w = fp4_walk(run);
  bool more = fp4_next(p, pl, run, w);
  if (more) write_q(w.b);
  // in a cluster the rotation's table is worked out before it is needed
  float2 turns[2] = {};
  if (pl.S) {
    const int pos = min(__ldg(p.positions + run.b0), p.max_pos);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if ((int)threadIdx.x + 128 * x < p.rd / 2) fp4_rope(p, pos, threadIdx.x + 128 * x, turns[x].y, turns[x].x);
  }
  for (; more; ++npiece) {
    float m_used = -INFINITY, l = 0.f;    // running maximum (log2 units; -inf until a key is seen), sum of this half
    for (int j = 0; j < w.cnt; ++j, ++g) {
      const int st = g % SP;
      const uint32_t ph = (g / SP) & 1;
      // the loaders' mask of this stage
      wait(bar(bars->kv_full[ks]), kph);
      const uint32_t vmask = reinterpret_cast<const uint32_t *>(smem + L::mask_off)[2 * ks + half];
      if (++ks == L::NS) {
        ks = 0;
        kph ^= 1;
      }
      wait(bar(bars->s_full[st]), ph);
      tc_fence_after();
      uint32_t sv[32];
      tmem_ld_16x32bx2_x16<32>(tmem + lane_S + st * KT, *reinterpret_cast<uint32_t(*)[16]>(&sv[0]));
      tmem_ld_16x32bx2_x16<32>(tmem + lane_S + st * KT + 16, *reinterpret_cast<uint32_t(*)[16]>(&sv[16]));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->s_empty[st]));
      float z[32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        z[x] = ((vmask >> x) & 1u) ? __uint_as_float(sv[x]) * zs : -INFINITY;
        mx[x & 3] = fmaxf(mx[x & 3], z[x]);
      }
      float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 16));
      bool need = false;
      float alpha = 1.f;
      if (tmax != -INFINITY && (m_used == -INFINITY || tmax > m_used + 8.f)) {
        if (m_used != -INFINITY) {        // before the first key O and l are 0
          need = true;
          alpha = ex2_approx(m_used - tmax);
          l *= alpha;
        }
        m_used = tmax;
      }
      if (__any_sync(0xffffffffu, need)) {
        // rescale O once the previous tile's P V has landed
        wait(bar(bars->pv_done[(g - 1) % SP]), ((g - 1) / SP) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < C / 2; c0 += 16) {
          uint32_t ov[16];
          tmem_ld_16x32bx2_x16<C / 2>(tmem + lane_O + c0, ov);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * alpha);
          tmem_st_16x32bx2_x16<C / 2>(tmem + lane_O + c0, ov);
        }
        tmem_st_wait();
      }
      const float m_eff = m_used == -INFINITY ? 0.f : m_used;
      float ps[2] = {0.f, 0.f};
      uint32_t pk[16];
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float p0 = ex2_approx(z[x] - m_eff), p1 = ex2_approx(z[x + 1] - m_eff);
        ps[(x >> 1) & 1] += p0 + p1;
        pk[x / 2] = pack_bf16x2(p0, p1);
      }
      l += ps[0] + ps[1];
      // P buffer st is free once the P V of two tiles ago has completed
      wait(bar(bars->pv_done[st]), ph ^ 1);
      uint8_t *prow = smem + L::p_off + st * kTileBytes;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4 *>(prow + sw128_off(r, half * 4 + u)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->p_full[st]));
    }

    // the last P V, then the next piece's Q before this one's epilogue, so that its first S need not wait for that
    wait(bar(bars->pv_done[(g - 1) % SP]), ((g - 1) / SP) & 1);
    Fp4Walk wn = w;
    more = fp4_next(p, pl, run, wn);
    if (more) {
      wait(bar(bars->q_empty), npiece & 1);
      asm volatile("bar.sync 1, 128;" ::: "memory");   // all warps are past the P V that reads all of P
      write_q(wn.b);
    }
    // ---- epilogue
    const bool whole = w.cnt == w.k.nt && !pl.S;
    const float ltot = l + __shfl_xor_sync(0xffffffffu, l, 16);
    if (pl.meta && threadIdx.x == 0 && w.j == 0) {
      // the CTA that has a sequence's first tile says who else has some
      const int last = before + w.k.nt - 1;
      pl.meta[w.b] = whole ? make_int4(-1, 0, 0, 0)
                           : make_int4(blockIdx.x, fp4_cta_of(run, last), before == run.before ? 0 : 1, 0);
    }
    tc_fence_after();
    if (whole) {
      // the rotation's table, where P was (and other warps' Q on its way)
      if (more) asm volatile("bar.sync 1, 128;" ::: "memory");
      for (int i = threadIdx.x; i < p.rd / 2; i += 128) {
        float sn, cs;
        fp4_rope(p, w.k.pos, i, sn, cs);
        rope[i] = make_float2(cs, sn);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    const long long slot = 2 * (int)blockIdx.x + (before == run.before ? 0 : 1);
    float inv = 0.f;
    if (m_used != -INFINITY) inv = 1.f / (ltot + (p.sink && live ? exp2f(p.sink[r] * kLog2e - m_used) : 0.f));
    if (!whole) {
      // 16 rows of a warp side by side, so that a store is 512 contiguous bytes; in a cluster they go where the
      // key tiles were
      float2 *ml = pl.S ? reinterpret_cast<float2 *>(smem + L::p_off) : pl.part_ml + slot * p.n_h;
      if (live && half == 0) ml[r] = make_float2(m_used, ltot);
      if (pl.S) fp4_part_store<C>(p, reinterpret_cast<float4 *>(smem), 0, tmem, warp, 0, 3);   // the loaders store the rest
      else fp4_part_store<C>(p, pl.part_o, slot, tmem, warp, 0, 1);
    } else {
      uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((long long)w.b * p.n_h + r) * C + half * (C / 2));
#pragma unroll 1
      for (int c0 = 0; c0 < C / 2; c0 += 16, dst += 2) {
        uint32_t ov[16];
        tmem_ld_16x32bx2_x16<C / 2>(tmem + lane_O + c0, ov);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = __uint_as_float(ov[x]) * inv;
        const int col0 = half * (C / 2) + c0;
        if (col0 >= C - p.rd) {             // rd is a multiple of 64
          const float2 *t = rope + (col0 - (C - p.rd)) / 2;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float2 cs = t[x];
            const float a = v[2 * x], b = v[2 * x + 1];
            v[2 * x] = a * cs.x + b * cs.y;
            v[2 * x + 1] = b * cs.x - a * cs.y;
          }
        }
        uint32_t o[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
        if (live) {
          dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
          dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
    if (whole) asm volatile("bar.sync 1, 128;" ::: "memory");   // the table has been read
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bars->o_empty));
    before += w.cnt;
    w = wn;
  }
  if (pl.S) {
    if (run.n == 0 && threadIdx.x < 64)   // a part without keys
      reinterpret_cast<float2 *>(smem + L::p_off)[threadIdx.x] = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if ((int)threadIdx.x + 128 * x < p.rd / 2)
        reinterpret_cast<float2 *>(smem + L::p_off + 1024)[threadIdx.x + 128 * x] = turns[x];
  }
}

// Sums of parts: maximum (log2 units), denominator, 4 columns of O.
struct Fp4Sum {
  float M, den;
  float4 acc;
  __device__ __forceinline__ void add(float m, float l, const float4 &o) {   // l and o under the maximum m
    if (m == -INFINITY) return;                                              // nothing in it
    const float n = fmaxf(M, m), f = M == n ? 1.f : exp2f(M - n), e = m == n ? 1.f : exp2f(m - n);
    M = n;
    den = den * f + e * l;
    acc.x = acc.x * f + e * o.x; acc.y = acc.y * f + e * o.y; acc.z = acc.z * f + e * o.z; acc.w = acc.w * f + e * o.w;
  }
};
// The rotation of two pairs and the store.
__device__ __forceinline__ void fp4_rotate_store(const AttendFp4Params &p, int b, int h, int col, float4 v, float2 cs0, float2 cs1) {
  if (col >= p.c - p.rd)
    v = make_float4(v.x * cs0.x + v.y * cs0.y, v.y * cs0.x - v.x * cs0.y, v.z * cs1.x + v.w * cs1.y, v.w * cs1.x - v.z * cs1.y);
  *reinterpret_cast<uint2 *>(p.o + ((long long)b * p.n_h + h) * p.c + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// A cluster's sequence: its CTAs have their parts in shared memory, and each
// joins a share of the columns, first the heads' weights of the parts.
template <int C>
__device__ __forceinline__ void fp4_cluster_join(const AttendFp4Params &p, const Fp4Plan &pl, int b, uint8_t *smem) {
  using L = Fp4Layout<C>;
  const int lane = threadIdx.x & 31, per = C / 8 / pl.S, rank = blockIdx.x % pl.S;
  const float2 *rope = reinterpret_cast<const float2 *>(smem + L::p_off + 1024);
  float *wts = reinterpret_cast<float *>(smem + L::p_off + 4096);    // [64][8]
  const uint32_t sbase = smem_u32(smem);
  if ((int)threadIdx.x < p.n_h) {
    const int h = threadIdx.x;
    const float sink = p.sink ? p.sink[h] * kLog2e : -INFINITY;
    float2 ml[8];
    float M = sink;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      ml[s] = s < pl.S ? ld_dsmem_f32x2(cluster_map(sbase + L::p_off + 8 * h, s)) : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int s = 0; s < 8; ++s) M = fmaxf(M, ml[s].x);
    float den = sink == -INFINITY ? 0.f : sink == M ? 1.f : exp2f(sink - M);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      ml[s].x = ml[s].x == -INFINITY ? 0.f : exp2f(ml[s].x - M);     // 0: a part without keys
      den += ml[s].x * ml[s].y;
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) wts[8 * h + s] = ml[s].x * inv;
  }
  __syncthreads();
#pragma unroll 1
  for (int pair = threadIdx.x >> 5; pair < (p.n_h + 15) / 16 * per; pair += kThreads / 32) {
    const int q = pair / per, i = rank * per + pair % per, h = 16 * q + (lane & 15), col = (lane >> 4) * (C / 2) + 4 * i;
    if (h >= p.n_h) continue;
    const uint32_t off = (uint32_t)(fp4_part(p, 0, q, i) + lane) * 16u;
    float4 o[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < pl.S) o[s] = ld_dsmem_f32x4(cluster_map(sbase + off, s));
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float w = wts[8 * h + s];
      if (w == 0.f) continue;        // its sums may be anything
      v.x += w * o[s].x; v.y += w * o[s].y; v.z += w * o[s].z; v.w += w * o[s].w;
    }
    const int k = (col - (C - p.rd)) / 2;
    const bool rot = col >= C - p.rd;
    fp4_rotate_store(p, b, h, col, v, rot ? rope[k] : make_float2(1.f, 0.f), rot ? rope[k + 1] : make_float2(1.f, 0.f));
  }
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1) attend_fp4_kernel(AttendFp4Params p, Fp4Plan pl) {
  using L = Fp4Layout<C>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Fp4Bars *bars = reinterpret_cast<Fp4Bars *>(smem + L::bar_off);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](uint64_t &b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    mbar_init(bar(bars->q_full), 4);
    mbar_init(bar(bars->q_empty), 1);
    mbar_init(bar(bars->o_empty), 4);
    mbar_init(bar(bars->all_done), 1);
    mbar_init(bar(bars->settled), 1);
    bars->ran_out = 0u;
    for (int i = 0; i < L::NS; ++i) {
      mbar_init(bar(bars->kv_full[i]), kLoadWarps * 33);   // every thread's copies, every warp's stores
      mbar_init(bar(bars->kv_empty[i]), 1);
    }
    for (int i = 0; i < SP; ++i) {
      mbar_init(bar(bars->s_full[i]), 1);
      mbar_init(bar(bars->s_empty[i]), 4);
      mbar_init(bar(bars->p_full[i]), 4);
      mbar_init(bar(bars->pv_done[i]), 1);
    }
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem), 512);
    tmem_relinquish();
  }
  pdl_trigger();
  {
    // the lists and page tables, read by whoever needs them after two more
    // dependent loads: every CTA brings a part of them into L2
    const long long line = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (p.idx && line * 32 < (long long)p.B * p.k) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.idx + line * 32));
    if (p.pages && line * 32 < (long long)p.B * p.max_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pages + line * 32));
  }
  // ---- this CTA's run: tiles of all sequences summed up, then the sequence where the run begins
  Fp4Run run;
  auto cut = [&](int total) {
    run.base = total / pl.G;
    run.rem = total - run.base * pl.G;
    run.before = blockIdx.x * run.base + min((int)blockIdx.x, run.rem);
    run.n = run.base + ((int)blockIdx.x < run.rem ? 1 : 0);
    run.b0 = run.j0 = 0;
  };
  // inclusive sum over the warp's lanes
  auto scan = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  if (pl.S) {
    // the sequence's tiles in equal shares
    const int nt = fp4_keys(p, pl, blockIdx.x / pl.S).nt, r = blockIdx.x % pl.S;
    run.base = nt / pl.S;
    run.rem = nt - run.base * pl.S;
    run.before = 0;
    run.n = run.base + (r < run.rem ? 1 : 0);
    run.b0 = blockIdx.x / pl.S;
    run.j0 = r * run.base + min(r, run.rem);
  } else if (p.B <= 128) {
    // every warp for itself: 4 sequences per lane
    int nt[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 4 * lane + i;
      nt[i] = b < p.B ? fp4_keys(p, pl, b).nt : 0;
      mine += nt[i];
    }
    const int upto = scan(mine);
    cut(__shfl_sync(0xffffffffu, upto, 31));
    int first = upto - mine, b0 = -1, j0 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (nt[i] > 0 && run.before >= first && run.before < first + nt[i]) {
        b0 = 4 * lane + i;
        j0 = run.before - first;
      }
      first += nt[i];
    }
    const uint32_t has = __ballot_sync(0xffffffffu, b0 >= 0);
    const int src = has ? __ffs(has) - 1 : 0;
    run.b0 = __shfl_sync(0xffffffffu, b0, src);
    run.j0 = __shfl_sync(0xffffffffu, j0, src);
  } else {
    constexpr int NW = kThreads / 32;
    int *sums = reinterpret_cast<int *>(smem + L::sum_off), *at = reinterpret_cast<int *>(smem + L::run_off);
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) mine += fp4_keys(p, pl, b).nt;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    cut(__reduce_add_sync(0xffffffffu, lane < NW ? sums[lane] : 0));
    int done = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int nt = b < p.B ? fp4_keys(p, pl, b).nt : 0;
      const int x = scan(nt);
      __syncthreads();
      if (lane == 31) sums[warp] = x;
      __syncthreads();
      const int t = lane < NW ? sums[lane] : 0;
      const int first = done + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0) + x - nt;
      if (nt > 0 && run.before >= first && run.before < first + nt) {
        at[0] = b;
        at[1] = run.before - first;
      }
      done += __reduce_add_sync(0xffffffffu, t);
    }
    __syncthreads();
    if (run.n > 0) {
      run.b0 = at[0];
      run.j0 = at[1];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);

  if (warp >= kLoad0) {
    fp4_load<C>(p, pl, run, smem, bars);
    // a cluster's CTA has one piece; its sums are there once all MMAs have run (pv_done's phases are not followed here)
    if (pl.S && run.n > 0) {
      Waits{p.status, &bars->ran_out}(bar(bars->all_done), 0);
      tc_fence_after();
      __syncwarp();
      fp4_part_store<C>(p, reinterpret_cast<float4 *>(smem), 0, tmem, warp & 3, 1 + (warp - kLoad0) / 4, 3);
    }
  } else if (warp == kMmaWarp) {
    fp4_mma<C>(p, pl, run, smem_u32(smem), bars, tmem);
  } else {
    fp4_softmax<C>(p, pl, run, smem, bars, tmem);
    // sequences without keys: zeros
    for (int b = pl.S ? p.B : (int)blockIdx.x; b < p.B; b += pl.G) {
      if (fp4_keys(p, pl, b).nt) continue;
      for (int i = threadIdx.x; i < p.n_h * C / 8; i += 128)
        reinterpret_cast<uint4 *>(p.o + (long long)b * p.n_h * C)[i] = make_uint4(0, 0, 0, 0);
      if (pl.meta && threadIdx.x == 0) pl.meta[b] = make_int4(-1, 0, 0, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (pl.S) {
    // every thread of the cluster comes here, whatever its waits did
    __syncwarp();
    cluster_sync();
    fp4_cluster_join<C>(p, pl, run.b0, smem);
    __syncwarp();
    cluster_sync();          // the parts have been read
  }
}

// Cut sequences: o = sum_i 2^(m_i - M) O_i / (sum_i 2^(m_i - M) l_i + 2^(sink -
// M)) over their parts from the workspace.  A warp has 16 heads and 4 columns of
// either half (a thread 4 columns of a head).  F = 4: the four warps of a block
// have the same columns and every fourth part each, summed in the order of the
// warps; for few sequences, whose many parts one warp would read one batch
// after another (4 sequences of 7620 entries at 16 x 128, 37 parts: the call
// 25.3 us with one warp, 18.8 with four).
template <int F>
__global__ void __launch_bounds__(128) fp4_combine_kernel(AttendFp4Params p, Fp4Plan pl) {
  __shared__ float4 so[F][32];
  __shared__ float2 sm[F][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = F == 1 ? blockIdx.y * 4 + warp : blockIdx.y, q = blockIdx.z, b = blockIdx.x;
  const int h = 16 * q + (lane & 15), col = (lane >> 4) * (p.c / 2) + 4 * i;
  pdl_wait();
  const int4 meta = pl.meta[b];
  if (meta.x < 0) return;
  auto slot = [&](int c) { return (long long)(2 * c + (c == meta.x ? meta.z : 0)); };
  Fp4Sum r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (h < p.n_h) {
    for (int c0 = meta.x + (F == 1 ? 0 : warp); c0 <= meta.y; c0 += 4 * F) {
      float2 ml[4];
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (c0 + F * k <= meta.y) {
          ml[k] = pl.part_ml[slot(c0 + F * k) * p.n_h + h];
          o[k] = pl.part_o[fp4_part(p, slot(c0 + F * k), q, i) + lane];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) r.add(ml[k].x, ml[k].y, o[k]);
    }
  }
  if constexpr (F > 1) {
    so[warp][lane] = r.acc;
    sm[warp][lane] = make_float2(r.M, r.den);
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 1; k < F; ++k) r.add(sm[k][lane].x, sm[k][lane].y, so[k][lane]);
  }
  if (h >= p.n_h) return;
  if (p.sink) r.add(p.sink[h] * kLog2e, 1.f, make_float4(0.f, 0.f, 0.f, 0.f));   // an infinite one takes all the weight
  const float inv = r.den > 0.f ? 1.f / r.den : 0.f;
  const float4 v = make_float4(r.acc.x * inv, r.acc.y * inv, r.acc.z * inv, r.acc.w * inv);
  float2 cs0 = make_float2(1.f, 0.f), cs1 = cs0;
  if (col >= p.c - p.rd) {
    const int pos = min(__ldg(p.positions + b), p.max_pos), k = (col - (p.c - p.rd)) / 2;
    fp4_rope(p, pos, k, cs0.y, cs0.x);
    fp4_rope(p, pos, k + 1, cs1.y, cs1.x);
  }
  fp4_rotate_store(p, b, h, col, v, cs0, cs1);
}

// CTAs of a call: the budget, no more than there can be tiles.  A part costs
// its n_h x c sums written and read again, so a CTA gets at least as many tiles
// as keep that small beside them (64 x 512: 4), and listed entries, whose count
// is known here, are cut into equal parts of each sequence: 32 sequences of 10
// tiles at 64 x 512, as runs, took 27.5 us on 64 CTAs, 31 on 32 (whole
// sequences), 96 and 148.
int fp4_ctas(const AttendFp4Params &p, int ne, bool listed) {
  const int sms = num_sms(), budget = p.max_ctas > 0 && p.max_ctas < sms ? p.max_ctas : sms;
  const int nw = std::min(p.w, p.max_pos + 1), tiles = (nw + KT - 1) / KT + (ne + KT - 1) / KT;
  const int least = std::max(1, p.n_h * p.c / 8192);
  if (listed && p.B <= budget) return p.B * std::max(1, std::min(budget / p.B, tiles / least));
  return (int)std::max<long long>(1, std::min<long long>(budget, std::max<long long>(std::min(p.B, budget), (long long)p.B * tiles / least)));
}
template <int C>
int fp4_attr() {
  static std::atomic<bool> attr_dev[kMaxDevices];
  std::atomic<bool> &attr = attr_dev[device_slot()];
  if (!attr) {
    const cudaError_t e = cudaFuncSetAttribute(attend_fp4_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Fp4Layout<C>::bytes);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return fail(HCA_ERR_CUDA, "attend_fp4 smem attribute: %s", cudaGetErrorString(e));
    }
    attr = true;
  }
  return HCA_OK;
}
template <int C>
cudaLaunchConfig_t fp4_config(int G, int S, cudaLaunchAttribute *at) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(G, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Fp4Layout<C>::bytes;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = S;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S ? 1 : 0;
  return cfg;
}
// Clusters of S CTAs, one to an SM, that the GPU holds at once: fewer than its
// SMs over S, since a cluster stays within a group of SMs (of 8: 15, not 18).
template <int C>
int fp4_resident(int S) {
  static std::atomic<int> n_dev[kMaxDevices][9];
  std::atomic<int> &n = n_dev[device_slot()][S];
  if (!n) {
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = fp4_config<C>(S, S, &at);
    int v = 0;
    if (fp4_attr<C>() || cudaOccupancyMaxActiveClusters(&v, attend_fp4_kernel<C>, &cfg) != cudaSuccess || v <= 0) {
      (void)cudaGetLastError();
      v = std::max(1, num_sms() / S);   // the launch reports what is wrong
    }
    n = v;
  }
  return n;
}
int fp4_resident(const AttendFp4Params &p, int S) {
  return p.c == 128 ? fp4_resident<128>(S) : p.c == 256 ? fp4_resident<256>(S) : fp4_resident<512>(S);
}
// CTAs per sequence where a cluster takes each sequence and joins it through
// shared memory: no parts in the workspace and no second launch, which cost as
// much as about 4 tiles, but at most 8 CTAs, and a ragged batch waits for its
// longest sequence (half of the most tiles is taken as the mean where only the
// positions tell).  0 where runs over all sequences have that much less.  32
// sequences of 10 tiles at 64 x 512: 19.6 us in clusters of 4, 23.9 as runs;
// one of 10 tiles at 16 x 128: 9.5 us in a cluster of 8, 9.9 as runs; 64 x 512
// with positions spread over 0.4 to 1 of the most entries: 30 sequences of 1000
// 21.9 us in clusters, 27.3 as runs, 8 of 7500 38.4 and 31.0.  Clusters
// that the GPU does not hold at once wait for others to end: 16 sequences of 10
// tiles at 64 x 512 took 31.7 us in clusters of 8, 18.5 in clusters of 4; 36 of
// them 36.0 in clusters of 4, 24.8 in clusters of 2.
int fp4_cluster(const AttendFp4Params &p, int ne, bool listed) {
  const int sms = num_sms(), budget = p.max_ctas > 0 && p.max_ctas < sms ? p.max_ctas : sms;
  const int nw = std::min(p.w, p.max_pos + 1), tiles = (nw + KT - 1) / KT + (ne + KT - 1) / KT;
  int S = 1;
  while (S < 8 && 2 * S <= tiles && (long long)p.B * 2 * S <= budget && p.B <= fp4_resident(p, 2 * S)) S *= 2;
  if (S == 1) return 0;
  const int runs = (int)(((long long)p.B * tiles + fp4_ctas(p, ne, listed) - 1) / fp4_ctas(p, ne, listed));
  return (tiles + S - 1) / S <= (listed ? runs : runs / 2) + 4 ? S : 0;
}
size_t fp4_align(size_t n) { return (n + 255) & ~(size_t)255; }
size_t fp4_part_bytes(const AttendFp4Params &p, size_t G) { return fp4_align(2 * G * ((p.n_h + 15) / 16 * 16) * p.c * 4); }

template <int C>
int launch_fp4(const AttendFp4Params &p, const Fp4Plan &pl, cudaStream_t s) {
  if (const int rc = fp4_attr<C>()) return rc;
  LaunchScope ls("attend_fp4", s);
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = fp4_config<C>(pl.G, pl.S, &at);
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attend_fp4_kernel<C>, p, pl);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(HCA_ERR_CUDA, "attend_fp4 launch: %s", cudaGetErrorString(e));
  }
  return ls.done();
}

}  // namespace

// A cluster per sequence and one CTA for all need no workspace.
size_t attend_fp4_workspace_bytes(const AttendFp4Params &p) {
  size_t most = 0;
  for (const bool listed : {true, false}) {
    const int ne = listed ? p.k : (p.max_pos + 1) / p.m;
    const size_t G = (size_t)fp4_ctas(p, ne, listed);
    if (G == 1 || fp4_cluster(p, ne, listed)) continue;
    most = std::max(most, fp4_part_bytes(p, G) + fp4_align(2 * G * p.n_h * 8) + fp4_align((size_t)p.B * 16));
  }
  return most;
}

int run_attend_fp4(const AttendFp4Params &p, void *ws, size_t, cudaStream_t s) {
  Fp4Plan pl{};
  const bool listed = p.idx != nullptr;
  const int ne = listed ? p.k : (p.max_pos + 1) / p.m;
  pl.S = fp4_cluster(p, ne, listed);
  pl.G = pl.S ? p.B * pl.S : fp4_ctas(p, ne, listed);
  pl.fd_m = make_fastdiv((uint32_t)p.m);
  pl.fd_cap = make_fastdiv((uint32_t)std::max(p.cap, 1));
  if (pl.G > 1 && !pl.S) {
    char *w = static_cast<char *>(ws);
    pl.part_o = reinterpret_cast<float4 *>(w);
    w += fp4_part_bytes(p, pl.G);
    pl.part_ml = reinterpret_cast<float2 *>(w);
    w += fp4_align((size_t)2 * pl.G * p.n_h * 8);
    pl.meta = reinterpret_cast<int4 *>(w);
  }
  const int rc = p.c == 128 ? launch_fp4<128>(p, pl, s) : p.c == 256 ? launch_fp4<256>(p, pl, s) : launch_fp4<512>(p, pl, s);
  if (rc || pl.G == 1 || pl.S) return rc;
  LaunchScope ls("attend_fp4_combine", s);
  cudaLaunchConfig_t cfg{};
  // a part-parallel block per column group where that is at most a wave of blocks
  // (ragged, 12000 entries: 8 sequences at 16 x 128 20.2 us, 27.1 with a warp per
  // group; 20 at 64 x 512 57.7, with a warp 54.2)
  const bool few = (long long)p.B * (p.c / 8) * ((p.n_h + 15) / 16) <= 16LL * num_sms();
  cfg.gridDim = dim3(p.B, few ? p.c / 8 : p.c / 32, (p.n_h + 15) / 16);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, fp4_combine_kernel<4>, p, pl)
                            : cudaLaunchKernelEx(&cfg, fp4_combine_kernel<1>, p, pl);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(HCA_ERR_CUDA, "attend_fp4_combine launch: %s", cudaGetErrorString(e));
  }
  return ls.done();
}

}  // namespace hca
