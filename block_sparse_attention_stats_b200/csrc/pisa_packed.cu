// libpisa C ABI, second translation unit: attention over packed sequences and
// over a paged key/value cache, with the cache's bookkeeping.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "packed_host.cuh"
#include "packed_schedule.cuh"
#include "k9_pages.cuh"
#include "k10_attend_rows.cuh"
#include "k11_attend_tc.cuh"

namespace pisa {

pisa_status take_packed_status(unsigned *bits) { return take_status_word(&g_device_status, bits); }

// ---- scratch ---------------------------------------------------------------------
// Two partial slots and one cut a CTA (rows: of a unit).
struct PackedScratch {
  size_t cuts, part, total;
};
static PackedScratch packed_scratch(int d, int rows) {
  PackedScratch s;
  s.cuts = 0;
  s.part = align_up(kPackedCtas * sizeof(PackedCut), 256);
  s.total = s.part + align_up((size_t)kPackedCtas * 2 * rows * (d + 3) * sizeof(float), 256);
  return s;
}

// ---- launches ----------------------------------------------------------------------
template <typename T, int D, int V>
static pisa_status launch_combine(const PackedProblem &p, const PackedCut *cuts, const float *part, int R,
                                  const PackedOut &o, int clear, cudaStream_t st) {
  const int y = std::max(1, R * (D / (4 * V)) / 128);
  return launch_after(packed_combine_kernel<T, D, V>, dim3(kPackedCtas, y), 128, 0, st, p, cuts, part, R, o, clear);
}

template <typename T, int D, KeySource KEYS, bool ROUNDED>
static pisa_status launch_tc(PackedProblem p, const PagedKV &cache, const pisa_rows &q, const CUtensorMap &mk,
                             const CUtensorMap &mv, float scale, const PackedOut &o, int clear,
                             unsigned char *ws, cudaStream_t st) {
  using C = AttendCfg<D>;
  const int tq1 = 128 / p.G;
  p.tq = 2 * tq1;
  // what a unit's start and end take, in tiles (measured at 1.5 / 2 / 2.5 / 3 / 4: 858 / 864 / 868 / 875 / 883
  // us on 12000 + 700 + 4608 tokens, 98 / 99 / 100 / 99 / 102 us on 16 x 1000; with the float32 output 2317 /
  // 2272 / 2252 / - / 2253 us a training step on 8192 + 4608 + 1500).  Cutting a unit of four tiles costs more
  // than it balances: 13.8 against 11.5 us on seven prompts of up to 200 tokens
  p.unit_cost = ROUNDED ? 3 * kKeyTile : 3 * kKeyTile / 2;
  p.min_range = 3 * kKeyTile / 2;   // at most a unit a CTA where there are few
  p.whole = 4 * kKeyTile;
  CUtensorMap mq;
  PISA_TRY(map_query(&mq, q, Half16<T>::kBf16, D, p.G, p.T, p.Hkv, tq1));
  const PackedScratch s = packed_scratch(D, C::kRows);
  PackedCut *cuts = (PackedCut *)(ws + s.cuts);
  float *part = (float *)(ws + s.part);
  PISA_CUDA(cudaFuncSetAttribute(attend_tc_kernel<T, D, KEYS, ROUNDED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem));
  PISA_TRY(launch_after(attend_tc_kernel<T, D, KEYS, ROUNDED>, dim3(kPackedCtas), C::kThreads, C::kSmem, st, mq, mk,
                        mv, p, cache, scale, o, cuts, part));
  return launch_combine<T, D, 4>(p, cuts, part, C::kRows, o, clear, st);
}

template <typename T, int D, int R>
static pisa_status launch_rows(PackedProblem p, const PagedKV &cache, const pisa_rows &q, const CUtensorMap &mk,
                               const CUtensorMap &mv, float scale, const PackedOut &o, unsigned char *ws,
                               cudaStream_t st) {
  using C = RowsCfg<D, R>;
  p.tq = R / p.G;
  // (at 1.5 / 2 / 3 / 5 tiles a unit: 167 / 162 / 168 / 178 us on 300 requests of 1 to 1500 keys, 72 / 66 /
  // 68 / 71 us on 300 of 1 to 300, 154 / 152 / 154 / 154 us on 48 of 1 to 8000)
  p.unit_cost = 2 * kKeyTile;
  p.min_range = kKeyTile;
  p.whole = 0;
  CUtensorMap mq;
  PISA_TRY(map_query(&mq, q, Half16<T>::kBf16, D, p.G, p.T, p.Hkv, p.tq));
  const PackedScratch s = packed_scratch(D, R);
  PackedCut *cuts = (PackedCut *)(ws + s.cuts);
  float *part = (float *)(ws + s.part);
  PISA_CUDA(cudaFuncSetAttribute(attend_rows_kernel<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem));
  PISA_TRY(launch_after(attend_rows_kernel<T, D, R>, dim3(kPackedCtas), C::kThreads, C::kSmem, st,
      mq, mk, mv, p, cache, scale, o, cuts, part));
  return launch_combine<T, D, 2>(p, cuts, part, R, o, 0, st);
}

template <typename T, int D>
static pisa_status run_varlen(const PackedProblem &p, const pisa_rows &q, const pisa_rows &k,
                              const pisa_rows &v, float scale, const PackedOut &o, int clear,
                              unsigned char *ws, cudaStream_t st) {
  CUtensorMap mk, mv;
  PISA_TRY(map_rows(&mk, k, Half16<T>::kBf16, D, p.T, p.Hkv, kKeyTile));
  PISA_TRY(map_rows(&mv, v, Half16<T>::kBf16, D, p.T, p.Hkv, kKeyTile));
  if (o.f32) return launch_tc<T, D, kPackedKeys, true>(p, PagedKV{}, q, mk, mv, scale, o, clear, ws, st);
  return launch_tc<T, D, kPackedKeys, false>(p, PagedKV{}, q, mk, mv, scale, o, clear, ws, st);
}

template <typename T, int D>
static pisa_status run_paged(const PackedProblem &p, const PagedKV &cache, const pisa_rows &q,
                             const pisa_pages &k, const pisa_pages &v, float scale, const PackedOut &o,
                             unsigned char *ws, cudaStream_t st) {
  // Requests of up to 16 rows (tokens times the heads of a group) are for the kernel of few rows: single
  // tokens of 3 to 16 heads a key head, or drafts of 2 to 5, take 0.76 to 0.88 of the time of 128-row
  // products there (48 single tokens over 4000 keys: 127 against 145 us; 100 over 300: 15.6 and 20.6;
  // 64 drafts of 4: 165 and 191).  Of more rows it gains nothing: a form with 32 took 0.95 to 1.07 of the
  // time for single tokens of 17 to 32 heads and 1.06 to 1.23 for drafts.
  // The lengths are on the device, and either kernel serves any of them, but this one reads a request's
  // keys once for every 16 rows.  So it is taken only where what T allows beyond one token a request,
  // were it all one request's, is 64 rows: beside 48 single tokens over 4000 keys, a chunk over 60000
  // takes 1.05 / 1.11 / 1.18 / 1.5 / 2.1 / 3.1 times as long here at 24 / 64 / 64 / 96 / 192 / 384 rows, and
  // 330 single tokens beside a chunk of 2980 took 3222 us here, 613 there.  T says no more than that: a batch
  // of T = k B rows may be k tokens each, or one chunk and padding, so drafts of large batches forgo the
  // seventh that they would gain (64 of 4: 191 us).
  const long long r = std::max<long long>(((long long)p.T * p.G + p.B - 1) / p.B, p.G);
  const bool few = r <= 16 && (long long)std::max(p.T - p.B, 0) * p.G <= 64;
  CUtensorMap mk, mv;
  const bool spread = D == 128 && cache.page_size == 16;
  const int halves = few || spread ? D / 64 : 1;   // 64-column boxes in a copy
  PISA_TRY(map_pages(&mk, k, Half16<T>::kBf16, D, cache.page_size, p.Hkv, cache.num_pages, halves));
  PISA_TRY(map_pages(&mv, v, Half16<T>::kBf16, D, cache.page_size, p.Hkv, cache.num_pages, halves));
  if (!few) {
    // (pages of 16 whole / box by box: 185 / 220 us on 2048 tokens after 6952, 24 / 8 heads)
    if constexpr (D == 128)
      if (spread) return launch_tc<T, D, kSpreadPages, false>(p, cache, q, mk, mv, scale, o, 0, ws, st);
    return launch_tc<T, D, kPages, false>(p, cache, q, mk, mv, scale, o, 0, ws, st);
  }
  return launch_rows<T, D, 16>(p, cache, q, mk, mv, scale, o, ws, st);
}

// ---- argument checks --------------------------------------------------------------------
static pisa_status check_heads(int B, int T, int Hq, int Hkv, int d, pisa_dtype dtype) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv) return PISA_ERR_INVALID_ARG;
  if (dtype != PISA_BF16 && dtype != PISA_F16 && dtype != PISA_F32) return PISA_ERR_INVALID_ARG;
  if (dtype == PISA_F32) return PISA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return PISA_ERR_UNSUPPORTED;
  // (a warp steps over empty sequences one by one: 65536 of them take a few milliseconds)
  if (Hq > 65535 || Hq / Hkv > 128 || T > (1 << 24) || B > (1 << 16)) return PISA_ERR_UNSUPPORTED;
  return PISA_OK;
}

static PackedProblem problem(const int32_t *cu, const int32_t *kv_lens, int B, int T, int Hq, int Hkv,
                             int causal, long long max_kv) {
  PackedProblem p{};
  p.cu = cu;
  p.kv_lens = kv_lens;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.causal = causal != 0;
  p.max_kv = (int)std::min<long long>(max_kv, 1 << 30);
  return p;
}

static bool is_int32(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }

// (rows of a cache that is written must not share memory)
static pisa_status check_pages(const pisa_pages &c, int H, int ps, int pages, int d, bool written) {
  if (!aligned16(c.data)) return PISA_ERR_INVALID_ARG;
  const int64_t s[3] = {c.page_stride, c.head_stride, c.row_stride};
  const int n[3] = {pages, H, ps};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < d || s[i] % 8 || s[i] >= (1ll << 38))) return PISA_ERR_INVALID_ARG;
  if (written && !area(c, pages, H, ps, d).nested) return PISA_ERR_INVALID_ARG;
  return PISA_OK;
}

static bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

// What a plan writes, and what every CTA of it reads while others write.
struct StepWritten {
  Area a[5];
};
struct StepRead {
  Area a[4];
};
static StepWritten step_written(const pisa_page_step &s) {
  return {{area(s.block_table, 4ll * s.B * s.width), area(s.slots, 8ll * s.T), area(s.cu_seqlens, 4ll * (s.B + 1)),
           area(s.kv_lens, 4ll * s.B), area(s.num_free_out, 4)}};
}
static StepRead step_read(const pisa_page_step &s) {
  return {{area(s.past_lens, 4ll * s.B), area(s.new_lens, 4ll * s.B), area(s.num_free, 4),
           area(s.free_pages, 4ll * s.free_cap)}};
}

static pisa_status check_step(const pisa_page_step *s) {
  if (!s || s->B < 1 || s->T < 0 || s->width < 1 || s->page_size < 1 || s->free_cap < 0)
    return PISA_ERR_INVALID_ARG;
  if (!page_size_ok(s->page_size) || s->B > kPlanMaxB || s->T > (1 << 24)) return PISA_ERR_UNSUPPORTED;
  if ((long long)s->width * s->page_size > 0x7fffffffll) return PISA_ERR_UNSUPPORTED;
  if (!is_int32(s->past_lens) || !is_int32(s->new_lens) || !is_int32(s->block_table) ||
      !is_int32(s->num_free) || !is_int32(s->cu_seqlens) || !is_int32(s->kv_lens) ||
      !is_int32(s->num_free_out))
    return PISA_ERR_INVALID_ARG;
  if (s->free_cap && !is_int32(s->free_pages)) return PISA_ERR_INVALID_ARG;
  if (s->T && (!s->slots || ((uintptr_t)s->slots & 7u))) return PISA_ERR_INVALID_ARG;
  return check_apart(step_written(*s).a, 5, step_read(*s).a, 4);
}

}  // namespace pisa

using namespace pisa;

extern "C" {

size_t pisa_varlen_attention_workspace_bytes(int Hq, int Hkv, int d) {
  if (check_heads(1, 1, Hq, Hkv, d, PISA_BF16) != PISA_OK) return 0;
  return packed_scratch(d, 256).total;
}

pisa_status pisa_varlen_attention(pisa_rows q, pisa_rows k, pisa_rows v, pisa_dtype dtype,
                                  const int32_t *cu_seqlens, int B, int T, int Hq, int Hkv, int d,
                                  float scale, int flags, pisa_rows out, float *lse, float *out_f32,
                                  void *workspace, size_t ws_bytes, pisa_stream_t stream) {
  PISA_TRY(check_heads(B, T, Hq, Hkv, d, dtype));
  if (!(scale >= 0.f) || !std::isfinite(scale) || !is_int32(cu_seqlens)) return PISA_ERR_INVALID_ARG;
  if (flags & ~(PISA_CAUSAL | PISA_ZERO_TAIL)) return PISA_ERR_INVALID_ARG;
  if (T == 0) return PISA_OK;
  PISA_TRY(check_rows(q, Hq, T, d, false));
  PISA_TRY(check_rows(k, Hkv, T, d, false));
  PISA_TRY(check_rows(v, Hkv, T, d, false));
  PISA_TRY(check_rows(out, Hq, T, d, true));
  if (lse && !is_int32(lse)) return PISA_ERR_INVALID_ARG;
  if (out_f32 && !aligned16(out_f32)) return PISA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return PISA_ERR_INVALID_ARG;
  const size_t need = packed_scratch(d, 256).total;
  const Area read[] = {area(q, Hq, T, d), area(k, Hkv, T, d), area(v, Hkv, T, d), area(cu_seqlens, 4ll * (B + 1))};
  const Area written[] = {area(out, Hq, T, d), area(lse, 4ll * Hq * T), area(out_f32, 4ll * Hq * T * d),
                          area(workspace, need)};
  PISA_TRY(check_apart(written, 3, read, 4));
  if (ws_bytes < need) return PISA_ERR_WORKSPACE;
  PISA_TRY(check_apart(written, 4, read, 4, 3));
  const PackedProblem p = problem(cu_seqlens, nullptr, B, T, Hq, Hkv, flags & PISA_CAUSAL, T);
  const PackedOut o{out.data, out.head_stride, out.row_stride, lse, out_f32};
  const int clear = flags & PISA_ZERO_TAIL;
  const float s = scale == 0.f ? 1.f / std::sqrt((float)d) : scale;
  unsigned char *ws = (unsigned char *)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PISA_BF16)
    return d == 128 ? run_varlen<__nv_bfloat16, 128>(p, q, k, v, s, o, clear, ws, st)
                    : run_varlen<__nv_bfloat16, 64>(p, q, k, v, s, o, clear, ws, st);
  return d == 128 ? run_varlen<__half, 128>(p, q, k, v, s, o, clear, ws, st)
                  : run_varlen<__half, 64>(p, q, k, v, s, o, clear, ws, st);
}

size_t pisa_paged_attention_workspace_bytes(int Hq, int Hkv, int d) {
  return pisa_varlen_attention_workspace_bytes(Hq, Hkv, d);
}

pisa_status pisa_paged_attention(pisa_rows q, pisa_pages k_cache, pisa_pages v_cache, pisa_dtype dtype,
                                 int num_pages, int page_size, const int32_t *block_table, int width,
                                 const int32_t *cu_seqlens, const int32_t *kv_lens, int B, int T, int Hq,
                                 int Hkv, int d, float scale, pisa_rows out, float *lse, void *workspace,
                                 size_t ws_bytes, pisa_stream_t stream) {
  PISA_TRY(check_heads(B, T, Hq, Hkv, d, dtype));
  if (num_pages < 1 || page_size < 1 || width < 1) return PISA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size)) return PISA_ERR_UNSUPPORTED;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return PISA_ERR_INVALID_ARG;
  if (!is_int32(block_table) || !is_int32(cu_seqlens) || !is_int32(kv_lens)) return PISA_ERR_INVALID_ARG;
  if (T == 0) return PISA_OK;
  PISA_TRY(check_rows(q, Hq, T, d, false));
  PISA_TRY(check_rows(out, Hq, T, d, true));
  PISA_TRY(check_pages(k_cache, Hkv, page_size, num_pages, d, false));
  PISA_TRY(check_pages(v_cache, Hkv, page_size, num_pages, d, false));
  if (lse && !is_int32(lse)) return PISA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return PISA_ERR_INVALID_ARG;
  const size_t need = packed_scratch(d, 256).total;
  const Area read[] = {area(q, Hq, T, d),
                       area(k_cache, num_pages, Hkv, page_size, d),
                       area(v_cache, num_pages, Hkv, page_size, d),
                       area(block_table, 4ll * B * width),
                       area(cu_seqlens, 4ll * (B + 1)),
                       area(kv_lens, 4ll * B)};
  const Area written[] = {area(out, Hq, T, d), area(lse, 4ll * Hq * T), area(workspace, need)};
  PISA_TRY(check_apart(written, 2, read, 6));
  if (ws_bytes < need) return PISA_ERR_WORKSPACE;
  PISA_TRY(check_apart(written, 3, read, 6, 2));
  const PackedProblem p = problem(cu_seqlens, kv_lens, B, T, Hq, Hkv, 1, (long long)width * page_size);
  const PagedKV cache{block_table, width, page_size, num_pages};
  const PackedOut o{out.data, out.head_stride, out.row_stride, lse, nullptr};
  const float s = scale == 0.f ? 1.f / std::sqrt((float)d) : scale;
  unsigned char *ws = (unsigned char *)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PISA_BF16)
    return d == 128 ? run_paged<__nv_bfloat16, 128>(p, cache, q, k_cache, v_cache, s, o, ws, st)
                    : run_paged<__nv_bfloat16, 64>(p, cache, q, k_cache, v_cache, s, o, ws, st);
  return d == 128 ? run_paged<__half, 128>(p, cache, q, k_cache, v_cache, s, o, ws, st)
                  : run_paged<__half, 64>(p, cache, q, k_cache, v_cache, s, o, ws, st);
}

pisa_status pisa_page_plan(const pisa_page_step *step, pisa_stream_t stream) {
  PISA_TRY(check_step(step));
  PagePlan p{};
  p.past = step->past_lens;
  p.fresh = step->new_lens;
  p.B = step->B;
  p.T = step->T;
  p.width = step->width;
  p.page_size = step->page_size;
  p.table = step->block_table;
  p.free_pages = step->free_pages;
  p.free_cap = step->free_cap;
  p.num_free = step->num_free;
  p.slots = step->slots;
  p.cu = step->cu_seqlens;
  p.kv_lens = step->kv_lens;
  p.num_free_out = step->num_free_out;
  const int smem = 2 * (p.B + 1) * (int)sizeof(int);
  PISA_CUDA(cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * (kPlanMaxB + 1) * (int)sizeof(int)));
  const int work = std::max(p.T, p.B + 1);
  const int grid = std::max(1, std::min(ceil_div(work, kPlanThreads), kPackedCtas));
  return launch_after(page_plan_kernel, dim3(grid), kPlanThreads, smem, (cudaStream_t)stream, p);
}

pisa_status pisa_page_write(pisa_rows k, pisa_rows v, pisa_dtype dtype, const int64_t *slots, int T, int Hkv,
                            int d, pisa_pages k_cache, pisa_pages v_cache, int num_pages, int page_size,
                            pisa_stream_t stream) {
  PISA_TRY(check_heads(1, T, Hkv, Hkv, d, dtype));
  if (num_pages < 1 || page_size < 1) return PISA_ERR_INVALID_ARG;
  if (!page_size_ok(page_size)) return PISA_ERR_UNSUPPORTED;
  if (T == 0) return PISA_OK;
  if (!slots || ((uintptr_t)slots & 7u)) return PISA_ERR_INVALID_ARG;
  PISA_TRY(check_rows(k, Hkv, T, d, false));
  PISA_TRY(check_rows(v, Hkv, T, d, false));
  PISA_TRY(check_pages(k_cache, Hkv, page_size, num_pages, d, true));
  PISA_TRY(check_pages(v_cache, Hkv, page_size, num_pages, d, true));
  const Area read[] = {area(k, Hkv, T, d), area(v, Hkv, T, d), area(slots, 8ll * T)};
  const Area written[] = {area(k_cache, num_pages, Hkv, page_size, d), area(v_cache, num_pages, Hkv, page_size, d)};
  PISA_TRY(check_apart(written, 2, read, 3));
  PageWrite w{};
  const pisa_rows r[2] = {k, v};
  const pisa_pages c[2] = {k_cache, v_cache};
  for (int i = 0; i < 2; ++i) {
    w.src[i] = (const unsigned char *)r[i].data;
    w.src_head[i] = r[i].head_stride * 2;
    w.src_row[i] = r[i].row_stride * 2;
    w.dst[i] = (unsigned char *)c[i].data;
    w.dst_page[i] = c[i].page_stride * 2;
    w.dst_head[i] = c[i].head_stride * 2;
    w.dst_row[i] = c[i].row_stride * 2;
  }
  w.slots = slots;
  w.T = T;
  w.H = Hkv;
  w.page_size = page_size;
  w.num_slots = (long long)num_pages * page_size;
  const int per = kWriteThreads / (d / 8) * kWriteRows;
  const dim3 grid(std::min(ceil_div(T, per), 65535), Hkv, 2);
  if (d == 128) return launch_after(page_write_kernel<16>, grid, kWriteThreads, 0, (cudaStream_t)stream, w);
  return launch_after(page_write_kernel<8>, grid, kWriteThreads, 0, (cudaStream_t)stream, w);
}

pisa_status pisa_paged_step(const pisa_page_step *step, pisa_rows q, pisa_rows k, pisa_rows v,
                            pisa_pages k_cache, pisa_pages v_cache, pisa_dtype dtype, int num_pages, int Hq,
                            int Hkv, int d, float scale, pisa_rows out, float *lse, void *workspace,
                            size_t ws_bytes, pisa_stream_t stream) {
  PISA_TRY(check_step(step));
  // everything is checked before the plan changes the table
  const int B = step->B, T = step->T, ps = step->page_size;
  PISA_TRY(check_heads(B, T, Hq, Hkv, d, dtype));
  if (num_pages < 1 || !(scale >= 0.f) || !std::isfinite(scale)) return PISA_ERR_INVALID_ARG;
  if (lse && !is_int32(lse)) return PISA_ERR_INVALID_ARG;
  if (T) {
    PISA_TRY(check_rows(q, Hq, T, d, false));
    PISA_TRY(check_rows(k, Hkv, T, d, false));
    PISA_TRY(check_rows(v, Hkv, T, d, false));
    PISA_TRY(check_rows(out, Hq, T, d, true));
    PISA_TRY(check_pages(k_cache, Hkv, ps, num_pages, d, true));
    PISA_TRY(check_pages(v_cache, Hkv, ps, num_pages, d, true));
    if (!aligned16(workspace)) return PISA_ERR_INVALID_ARG;
    const size_t need = packed_scratch(d, 256).total;
    const StepRead sr = step_read(*step);
    const StepWritten sw = step_written(*step);
    const Area read[] = {sr.a[0], sr.a[1], sr.a[2], sr.a[3], area(q, Hq, T, d), area(k, Hkv, T, d), area(v, Hkv, T, d)};
    const Area written[] = {sw.a[0], sw.a[1], sw.a[2], sw.a[3], sw.a[4],
                            area(k_cache, num_pages, Hkv, ps, d), area(v_cache, num_pages, Hkv, ps, d),
                            area(out, Hq, T, d), area(lse, 4ll * Hq * T), area(workspace, need)};
    PISA_TRY(check_apart(written, 9, read, 7));
    if (ws_bytes < need) return PISA_ERR_WORKSPACE;
    PISA_TRY(check_apart(written, 10, read, 7, 9));
  }
  PISA_TRY(pisa_page_plan(step, stream));
  PISA_TRY(pisa_page_write(k, v, dtype, step->slots, T, Hkv, d, k_cache, v_cache, num_pages, ps, stream));
  return pisa_paged_attention(q, k_cache, v_cache, dtype, num_pages, ps, step->block_table, step->width,
                              step->cu_seqlens, step->kv_lens, B, T, Hq, Hkv, d, scale, out, lse, workspace,
                              ws_bytes, stream);
}

}  // extern "C"
