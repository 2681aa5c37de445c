// lowbit_api.cu -- the extern "C" entry points of the low-bit decode step:
// host-side validation and dispatch.  See include/hca.h.
#include <algorithm>
#include <climits>

#include "internal.h"

using namespace hca;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t esize(hca_dtype t) { return t == HCA_F32 ? 4 : t == HCA_BF16 ? 2 : 1; }
// Whether two buffers (NULL = none) share a byte.
bool overlap(const void *a, size_t an, const void *b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}

#define REQUIRE(cond, ...)                                   \
  do {                                                       \
    if (!(cond)) return fail(HCA_ERR_INVALID, __VA_ARGS__);  \
  } while (0)

int w4_params(const hca_w4_desc *d, W4Params *p) {
  REQUIRE(d != nullptr, "null descriptor");
  REQUIRE(d->N >= 1 && d->K >= 1 && d->groups >= 1, "N, K and groups must be >= 1");
  REQUIRE(d->scale_group == 32 || d->scale_group == 64 || d->scale_group == 128,
          "scale_group must be 32, 64 or 128 (got %d)", d->scale_group);
  REQUIRE(d->K % 32 == 0 && d->K % d->scale_group == 0, "K (%d) must be a multiple of 32 and of scale_group", d->K);
  REQUIRE(d->K <= 32768, "K must be <= 32768 (got %d)", d->K);
  REQUIRE(d->code == HCA_W4_E2M1 || d->code == HCA_W4_INT4, "code must be HCA_W4_E2M1 or HCA_W4_INT4");
  REQUIRE((long long)d->groups * d->N <= INT_MAX - 1024 && (long long)d->groups * d->K <= INT_MAX - 1024,
          "groups * N and groups * K must fit 31 bits");
  REQUIRE((long long)d->groups * ((d->N + 127) / 128) * ((d->K + 255) / 256) <= INT_MAX / 64,
          "groups * N * K is too large");
  *p = W4Params{};
  p->N = d->N; p->K = d->K; p->groups = d->groups; p->G = d->scale_group; p->code = d->code;
  p->ldn = (d->N + 15) / 16 * 16;
  return HCA_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- residual + norm
int hca_add_rms_norm(const hca_norm_desc *d, const void *x, const void *res, const float *gamma, void *res_out,
                     void *out, float *out_scale, hca_stream_t stream) {
  REQUIRE(d != nullptr, "null descriptor");
  REQUIRE(d->rows >= 0 && d->rows <= INT_MAX, "rows must be in [0, 2^31)");
  REQUIRE(d->d >= 1 && d->d <= 32768, "d must be in [1, 32768] (got %d)", d->d);
  REQUIRE(d->x_dtype == HCA_F32 || d->x_dtype == HCA_BF16, "x_dtype must be f32 or bf16");
  REQUIRE(d->res_dtype == d->x_dtype || d->res_dtype == HCA_F32, "res_dtype must be x_dtype or f32");
  REQUIRE(d->out_dtype == HCA_F32 || d->out_dtype == HCA_BF16 || d->out_dtype == HCA_FP8E4M3,
          "out_dtype must be f32, bf16 or e4m3");
  const bool fp8 = d->out_dtype == HCA_FP8E4M3;
  REQUIRE(d->scale_group == 0 || (fp8 && (d->scale_group == 64 || d->scale_group == 128) && d->d % d->scale_group == 0),
          "scale_group must be 0, or 64 or 128 with an e4m3 output and d a multiple of it");
  const long long ldx = d->ldx ? d->ldx : d->d, ldr = d->ldr ? d->ldr : d->d, ldo = d->ldo ? d->ldo : d->d;
  REQUIRE(ldx >= d->d && ldr >= d->d && ldo >= d->d, "row strides must be 0 or >= d");
  if (d->rows == 0) return HCA_OK;
  REQUIRE(x && out, "x and out must be non-null");
  REQUIRE(!fp8 || out_scale, "an e4m3 output needs out_scale");
  REQUIRE(aligned16(x) && aligned16(res) && aligned16(gamma) && aligned16(res_out) && aligned16(out) &&
              aligned16(out_scale), "pointers must be 16-byte aligned");
  const size_t nx = (size_t)((d->rows - 1) * ldx + d->d) * esize(d->x_dtype);
  const size_t nr = (size_t)((d->rows - 1) * ldr + d->d) * esize(d->res_dtype);
  const size_t no = (size_t)((d->rows - 1) * ldo + d->d) * esize(d->out_dtype);
  const size_t ng = (size_t)d->d * 4;
  const size_t ns = fp8 ? (size_t)d->rows * (d->scale_group ? d->d / d->scale_group : 1) * 4 : 0;
  const struct { const void *p; size_t n; } in[3] = {{x, nx}, {res, nr}, {gamma, ng}},
                                            outs[3] = {{res_out, nr}, {out, no}, {out_scale, ns}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool in_place = i == 0 && j == 1 && res_out == res;
      REQUIRE(in_place || !overlap(outs[i].p, outs[i].n, in[j].p, in[j].n), "an output overlaps an input");
    }
    for (int j = 0; j < i; ++j)
      REQUIRE(!overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n), "two outputs overlap");
  }
  NormParams p{};
  p.rows = d->rows; p.d = d->d; p.ldx = ldx; p.ldr = ldr; p.ldo = ldo; p.group = d->scale_group;
  p.vec = ldx % 8 == 0 && ldr % 8 == 0 && ldo % 8 == 0;
  p.eps = d->eps > 0.f ? d->eps : 1e-6f;
  p.x = x; p.res = res; p.gamma = gamma; p.res_out = res_out; p.out = out; p.out_scale = out_scale;
  return launch_add_rms_norm(p, d->x_dtype, d->res_dtype, d->out_dtype, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------- 4-bit weights
size_t hca_w4_linear_workspace_size(const hca_w4_desc *d) {
  W4Params p;
  if (w4_params(d, &p) || d->T < 0 || (long long)d->groups * d->T > INT_MAX - 1024) return 0;
  p.T = d->T;
  return w4_workspace_bytes(p);
}

int hca_w4_linear(const hca_w4_desc *d, const void *x, const float *x_scale, const void *codes, const void *scales,
                  const float *row_scale, void *out, void *ws, size_t ws_bytes, hca_stream_t stream) {
  W4Params p;
  const int rc = w4_params(d, &p);
  if (rc) return rc;
  REQUIRE(d->T >= 0 && (long long)d->groups * d->T <= INT_MAX - 1024, "T must be >= 0 and groups * T fit 31 bits");
  REQUIRE(d->x_dtype == HCA_BF16 || d->x_dtype == HCA_FP8E4M3, "x_dtype must be bf16 or e4m3");
  REQUIRE(d->out_dtype == HCA_F32 || d->out_dtype == HCA_BF16, "out_dtype must be f32 or bf16");
  p.T = d->T;
  p.ldx = d->ldx ? d->ldx : (long long)d->groups * d->K;
  p.ldo = d->ldo ? d->ldo : (long long)d->groups * d->N;
  REQUIRE(p.ldx >= (long long)d->groups * d->K && p.ldo >= (long long)d->groups * d->N,
          "row strides must be 0 or cover a row");
  REQUIRE((p.ldx * (long long)esize(d->x_dtype)) % 16 == 0, "rows of x must start at multiples of 16 bytes");
  if (d->T == 0) return HCA_OK;
  REQUIRE(x && codes && scales && row_scale && out, "x, codes, scales, row_scale and out must be non-null");
  REQUIRE((d->x_dtype == HCA_FP8E4M3) == (x_scale != nullptr), "x_scale goes with e4m3 x, and only with it");
  REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales) && aligned16(row_scale) && aligned16(out) &&
              aligned16(ws) && aligned4(x_scale), "pointers must be 16-byte aligned");
  const size_t need = w4_workspace_bytes(p);
  REQUIRE(need == 0 || (ws && ws_bytes >= need), "workspace too small (%zu of %zu bytes)", ws_bytes, need);
  {
    const size_t gn = (size_t)d->groups * d->N, nx = (size_t)((d->T - 1) * p.ldx + (long long)d->groups * d->K) * esize(d->x_dtype);
    const size_t no = (size_t)((d->T - 1) * p.ldo + (long long)gn) * esize(d->out_dtype);
    const size_t nsc = (size_t)d->groups * (d->K / p.G) * p.ldn;
    const struct { const void *p; size_t n; } in[6] = {{x, nx}, {x_scale, (size_t)d->T * 4}, {codes, gn * (d->K / 2)},
                                                       {scales, nsc}, {row_scale, gn * 4}, {ws, need}};
    for (const auto &b : in) REQUIRE(!overlap(out, no, b.p, b.n), "out overlaps an input or the workspace");
    for (int i = 0; i < 5; ++i) REQUIRE(!overlap(ws, need, in[i].p, in[i].n), "the workspace overlaps an input");
  }
  p.ws = ws;
  p.x = x; p.x_scale = x_scale; p.codes = static_cast<const unsigned char *>(codes);
  p.scales = static_cast<const unsigned char *>(scales); p.row_scale = row_scale; p.out = out;
  p.status = device_status_ptr();
  return launch_w4_linear(p, d->x_dtype, d->out_dtype, static_cast<cudaStream_t>(stream));
}

int hca_w4_quantize(const hca_w4_desc *d, const void *w, hca_dtype w_dtype, void *codes, void *scales,
                    float *row_scale, hca_stream_t stream) {
  W4Params p;
  const int rc = w4_params(d, &p);
  if (rc) return rc;
  REQUIRE(w_dtype == HCA_F32 || w_dtype == HCA_BF16, "w_dtype must be f32 or bf16");
  REQUIRE(w && codes && scales && row_scale, "w, codes, scales and row_scale must be non-null");
  REQUIRE(aligned16(w) && aligned16(codes) && aligned16(scales) && aligned16(row_scale),
          "pointers must be 16-byte aligned");
  {
    const size_t gn = (size_t)d->groups * d->N;
    const struct { const void *p; size_t n; } b[4] = {{w, gn * d->K * esize(w_dtype)}, {codes, gn * (d->K / 2)},
                                                      {scales, (size_t)d->groups * (d->K / p.G) * p.ldn}, {row_scale, gn * 4}};
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < i; ++j) REQUIRE(!overlap(b[i].p, b[i].n, b[j].p, b[j].n), "w, codes, scales and row_scale overlap");
  }
  return launch_w4_quantize(w, w_dtype, p, codes, scales, row_scale, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------- 4-bit KV records
size_t hca_kv_fp4_row_bytes(int c, int rd) { return kv_fp4_row_bytes(c, rd); }

int hca_kv_quant_fp4(const void *x, hca_dtype x_dtype, long long rows, int c, int rd, void *out, long long records,
                     const long long *slots, hca_stream_t stream) {
  REQUIRE(kv_fp4_row_bytes(c, rd) > 0, "unsupported (c, rd) = (%d, %d): need c <= 512, rd %% 16 == 0, "
          "(c - rd) %% 64 == 0", c, rd);
  REQUIRE(rows >= 0 && records >= 0, "rows and records must be >= 0");
  REQUIRE(x_dtype == HCA_F32 || x_dtype == HCA_BF16, "x_dtype must be HCA_F32 or HCA_BF16");
  if (rows == 0) return HCA_OK;
  REQUIRE(x && out, "x and out must be non-null");
  REQUIRE(aligned16(x) && aligned16(out), "x and out must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(slots) & 7u) == 0, "slots must be 8-byte aligned");
  REQUIRE(!overlap(out, (size_t)records * kv_fp4_row_bytes(c, rd), x, (size_t)rows * c * esize(x_dtype)),
          "the records overlap x");
  REQUIRE(!overlap(out, (size_t)records * kv_fp4_row_bytes(c, rd), slots, (size_t)rows * 8), "the records overlap slots");
  return launch_kv_quant_fp4(x, x_dtype, rows, c, rd, out, records, slots, static_cast<cudaStream_t>(stream));
}

int hca_kv_dequant_fp4(const void *in, long long records, const long long *slots, long long rows, int c, int rd,
                       void *out, hca_stream_t stream) {
  REQUIRE(kv_fp4_row_bytes(c, rd) > 0, "unsupported (c, rd) = (%d, %d): need c <= 512, rd %% 16 == 0, "
          "(c - rd) %% 64 == 0", c, rd);
  REQUIRE(rows >= 0 && records >= 0, "rows and records must be >= 0");
  if (rows == 0) return HCA_OK;
  REQUIRE(in && out, "in and out must be non-null");
  REQUIRE(aligned16(in) && aligned16(out), "in and out must be 16-byte aligned");
  REQUIRE((reinterpret_cast<uintptr_t>(slots) & 7u) == 0, "slots must be 8-byte aligned");
  REQUIRE(!overlap(in, (size_t)records * kv_fp4_row_bytes(c, rd), out, (size_t)rows * c * 2),
          "out overlaps the records");
  REQUIRE(!overlap(out, (size_t)rows * c * 2, slots, (size_t)rows * 8), "out overlaps slots");
  return launch_kv_dequant_fp4(in, records, slots, rows, c, rd, out, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------- attention over 4-bit records
static int attend_fp4_params(const hca_attn_desc *d, int max_pos, AttendFp4Params *p) {
  REQUIRE(d != nullptr, "null descriptor");
  REQUIRE(d->B >= 1 && d->B <= 65535, "B must be in [1, 65535] (got %d)", d->B);
  REQUIRE(d->n_h >= 1 && d->n_h <= 64, "n_h must be in [1, 64] (got %d)", d->n_h);
  REQUIRE(d->c == 128 || d->c == 256 || d->c == 512, "c must be 128, 256 or 512 (got %d)", d->c);
  REQUIRE(kv_fp4_row_bytes(d->c, d->rd) > 0, "rd must be a multiple of 16 with c - rd a multiple of 64 (got %d)", d->rd);
  REQUIRE(d->w >= 0 && d->m >= 1 && d->k >= 0, "w and k must be >= 0 and m >= 1");
  REQUIRE(d->dtype == HCA_BF16, "dtype must be HCA_BF16");
  REQUIRE(d->kv_mixed == 0, "kv_mixed must be 0");
  REQUIRE(d->max_ctas >= 0, "max_ctas must be >= 0 (0 = every SM)");
  REQUIRE(max_pos >= 0 && max_pos <= INT_MAX - 4096, "max_pos must be in [0, 2^31 - 4096)");
  REQUIRE(d->w <= (1 << 20) && d->k <= (1 << 28), "w must be <= 2^20 and k <= 2^28");
  const long long most = std::max<long long>(d->k, ((long long)max_pos + 1) / d->m);
  REQUIRE((long long)d->B * (d->w / 64 + most / 64 + 2) <= INT_MAX, "B times the keys of a sequence must be below 2^37");
  *p = AttendFp4Params{};
  p->B = d->B; p->n_h = d->n_h; p->c = d->c; p->rd = d->rd; p->w = d->w; p->m = d->m; p->k = d->k;
  p->rec = (int)kv_fp4_row_bytes(d->c, d->rd);
  p->max_pos = max_pos; p->max_ctas = d->max_ctas;
  p->scale = d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)d->c);
  p->theta = d->rope_theta > 0.f ? d->rope_theta : 10000.f;
  fill_rope_freq(p->rope_freq, d->rd, p->theta);
  return HCA_OK;
}

size_t hca_attend_fp4_workspace_size(const hca_attn_desc *d, int max_pos) {
  AttendFp4Params p;
  if (attend_fp4_params(d, max_pos, &p)) return 0;
  return attend_fp4_workspace_bytes(p);
}

int hca_attend_fp4(const hca_attn_desc *d, const void *q, const hca_fp4_cache *cache, const int32_t *idx,
                   const void *kv_win, const float *sink, const int32_t *positions, int max_pos, void *o, void *ws,
                   size_t ws_bytes, hca_stream_t stream) {
  AttendFp4Params p;
  const int rc = attend_fp4_params(d, max_pos, &p);
  if (rc) return rc;
  REQUIRE(q && o && positions && cache, "q, o, positions and cache must be non-null");
  REQUIRE(aligned16(q) && aligned16(o) && aligned16(ws), "q, o and ws must be 16-byte aligned");
  REQUIRE(aligned4(idx) && aligned4(positions) && aligned4(sink) && aligned4(cache->pages),
          "idx, positions, sink and pages must be 4-byte aligned");
  REQUIRE(d->w == 0 || (kv_win && aligned16(kv_win)), "kv_win must be non-null and 16-byte aligned when w > 0");
  REQUIRE(!idx || d->k >= 1, "idx needs k >= 1");
  REQUIRE(cache->cap >= 0 && (cache->cap == 0 || (cache->rows && aligned16(cache->rows))),
          "cache rows must be non-null and 16-byte aligned");
  REQUIRE(!cache->pages || (cache->cap >= 1 && cache->max_pages >= 0 && cache->n_pages >= 0),
          "a paged cache needs cap >= 1, max_pages >= 0 and n_pages >= 0");
  p.q = static_cast<const __nv_bfloat16 *>(q); p.o = static_cast<__nv_bfloat16 *>(o);
  p.kv_win = static_cast<const __nv_bfloat16 *>(kv_win); p.rows = static_cast<const unsigned char *>(cache->rows);
  p.cap = cache->cap; p.pages = cache->pages; p.max_pages = cache->max_pages; p.n_pages = cache->n_pages;
  p.idx = idx; p.sink = sink; p.positions = positions;
  p.status = device_status_ptr();
  const size_t need = attend_fp4_workspace_bytes(p);
  REQUIRE(need == 0 || (ws && ws_bytes >= need), "workspace too small (%zu of %zu bytes)", ws_bytes, need);
  {
    const size_t no = (size_t)p.B * p.n_h * p.c * 2;
    const size_t nrec = (size_t)(cache->pages ? cache->n_pages : p.B) * p.cap * p.rec;
    const struct { const void *p; size_t n; } in[7] = {{q, no}, {cache->rows, nrec}, {kv_win, (size_t)p.B * p.w * p.c * 2},
                                                       {positions, (size_t)p.B * 4}, {idx, (size_t)p.B * p.k * 4},
                                                       {sink, (size_t)p.n_h * 4}, {cache->pages, (size_t)p.B * p.max_pages * 4}};
    for (const auto &b : in) {
      REQUIRE(!overlap(o, no, b.p, b.n), "o overlaps an input");
      REQUIRE(!overlap(ws, need, b.p, b.n), "the workspace overlaps an input");
    }
    REQUIRE(!overlap(o, no, ws, need), "o overlaps the workspace");
  }
  return run_attend_fp4(p, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
