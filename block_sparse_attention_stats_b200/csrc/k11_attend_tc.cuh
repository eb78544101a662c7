// Attention of many packed rows on the sm_100a tensor cores: whole prompts
// (causal or not, sequences of any lengths) and chunks of new tokens over a
// paged cache, with grouped query heads.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(s q_r . k_j),  j below row r's limit
// with the running maximum and sum of the softmax, one pass over the keys.
// Bound: the tensor cores (4 D flops a row and key) and, close behind, the
// special-function units: a 128 x 128 tile takes 1024 cycles of products at D =
// 128 and 1024 cycles of ex2 at 16 a cycle and SM.
//
// Work unit (packed_schedule.cuh): two subtiles of 128 rows, each 128 / G tokens
// with the G query heads of one key head (token-major), so K and V are read once
// for a group.  Keys come in tiles of 128 and are worked on in halves of 64.
// Roles (352 threads, one CTA per SM, persistent over its range of tiles):
//   warp 0      copies: Q of both subtiles, then K and V tiles into a ring;
//   warps 1, 10 (1: TMEM) issue S_ih = Q_i K_h^T and O_i += P_ih V_h (P read from TMEM)
//               for subtile 0 and 1 and half h of a tile;
//   warps 2-5   softmax of subtile 0, one thread a row (TMEM lane);
//   warps 6-9   softmax of subtile 1.
// TMEM columns: S_ih [128 i + 64 h, + 64), O_0 [256, 256 + D), O_1 after it; P
// (16-bit) overwrites the first 32 columns of its S.  While the softmax works on
// one half, the products of the other run: P V, then S of the next tile's same
// half.  With whole tiles a subtile's softmax waited 1200 of 3200 cycles for its
// own P V and S; with halves and one issuing warp, that warp waited for one
// subtile's weights while the other's were ready.  Measured, whole tiles / halves /
// halves and two issuing warps: 880 / 952 / 853 us on 12000 + 700 + 4608 tokens (24 /
// 8 heads, causal), 125 / 110 / 100 us on 16 x 1000 (16 / 16 heads).
// S_ih of the next tile is issued after P_ih V_h of this one by the same thread, and one
// thread's products run in order, so no barrier guards the overwrite.
// Pages of 16 (D = 128): a page comes in one copy of 4 KB, its two 64-column boxes one
// after the other, instead of two of 2 KB (32 copies a tile took as long as its products).
// Groups of 8 keys are then 4 KB apart only if a half takes the same 8 rows of every
// page: half h is the keys 16 g + 8 h + (0 .. 7), g = 0 .. 7, of the tile.  The order of
// keys is free, and S, P and V follow the same one.  185 against 220 us on 2048 tokens
// after 6952, 24 / 8 heads; pages of 64 take 180.
// The running maximum moves only when it grows by more than 2^8 (f16: 2^4); a softmax
// thread then waits for the product before, and rescales O_i itself.  f16 weights are
// formed 2^11 times as large (Half16, packed_schedule.cuh), so they stay below 2^15,
// keep their precision down to 2^-25 of the largest and vanish below 2^-36.  (A growth of
// 2^8 / 2^4 / 2^2 / 2 leaves a factor of 2^7 / 2^11 / 2^13 / 2^14 and takes 884 / 902 / 1006 / 1020
// us on 12000 + 700 + 4608 f16 tokens, 24 / 8 heads; with 2^7 a tail of weights 2^-24 is off by
// up to 2^-8.  Where queries are large and maxima move often it costs more: 315 / 349 us at 2^8 /
// 2^4 on 8000 + 3000 tokens, 16 / 4 heads, scores of deviation 4.)
// Every wait is bounded; on a timeout the CTA records the error, stops issuing,
// drains its copies and products, frees TMEM and exits.
#pragma once

#include "k10_attend_rows.cuh"
#include "packed_primitives.cuh"
#include "packed_schedule.cuh"

namespace pisa {

template <int D> struct AttendCfg {
  static constexpr int kThreads = 352;
  static constexpr int kRows = 256;                      // rows of a unit
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kTileBytes = kKeyTile * D * 2;    // K or V tile, or Q of a subtile
  static constexpr int kBoxBytes = kKeyTile * 128;       // one 64-column box of 128 rows
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffStage = kOffKV + kStages * kTileBytes;   // 4 KB a softmax warp
  static constexpr int kOffMisc = kOffStage + 8 * 4096;
  static constexpr int kSmem = kOffMisc + 1024 + 1024;   // + alignment slack
  static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarFull = 2, kBarEmpty = kBarFull + kStages;
  static constexpr int kBarS = kBarEmpty + kStages;      // + 2 half + subtile
  static constexpr int kBarP = kBarS + 4;                // + 2 half + subtile
  static constexpr int kBarPV = kBarP + 4;               // + subtile: a half's product is in O
  static constexpr int kBarO = kBarPV + 2;               // + subtile: O complete
  static constexpr int kBarOFree = kBarO + 2;            // + subtile: O read
  static constexpr int kBarTeardown = kBarOFree + 2;
  static_assert(kBarTeardown < 48 && kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
};

// Where the keys are: rows of a packed tensor, pages whose boxes are copied one by one, or
// pages of 16 copied whole, with the halves of a tile spread over them (D = 128)
enum KeySource { kPackedKeys, kPages, kSpreadPages };

// tq1 tokens of a subtile; rows of subtile i, and its halves of key tiles
struct SubTile {
  int rows, nh;
};
__device__ __forceinline__ SubTile subtile(const PackedProblem &p, const PackedSegment &s, int tq1, int i,
                                           bool spread) {
  SubTile x;
  const int tok = s.rt * p.tq + i * tq1;
  x.rows = max(min(s.r.n - tok, tq1), 0) * p.G;
  const int len = x.rows == 0 ? 0 : RowCost::length(p, s.r.n, s.r.kv, tq1, 2 * s.rt + i);
  // (spread: the second half of the last tile begins with its key 8)
  const int nt = packed_tiles(len);
  x.nh = spread ? 2 * nt - (nt > 0 && len - (nt - 1) * kKeyTile <= 8) : (len + 63) / 64;
  return x;
}

// One row's part of 64 keys: scores from TMEM, running maximum and sum, weights
// back as 16 bits over the scores' first 32 columns, O rescaled where the maximum
// has moved (once `pv_done` says that the product before is in it).  `seen` columns
// are visible; SPREAD: those whose key, 16 (c / 8) + c % 8, is below `seen`.
// All exponentials are on the special-function units.  (A quarter of them as a polynomial on
// the multiply-add units took 918 against 893 us on 12000 + 700 + 4608 causal tokens in an
// earlier form of this kernel, with whole tiles and one issuing warp; not measured in this one.)
// The sum is of the float32 weights.  ROUNDED (where the float32 output is wanted
// too): for the backward the output is divided by the sum of the rounded weights:
// dout_t . o_t is then the mean of dP under the weights themselves, and does not lose
// dP - Delta to their rounding where one key holds nearly all the weight; lse still
// comes from the float32 weights, summed beside.
template <typename T, int D, bool ROUNDED, bool SPREAD, typename Wait>
__device__ __forceinline__ bool softmax_half(uint32_t s_addr, uint32_t o_addr, float sl2, int seen, Wait pv_done,
                                             float &m_run, float &l_run, float &e_run) {
  using namespace sm100;
  uint32_t r[64];
  tmem_ld_x32(s_addr, reinterpret_cast<uint32_t(&)[32]>(r[0]));
  tmem_ld_x32(s_addr + 32, reinterpret_cast<uint32_t(&)[32]>(r[32]));
  tmem_wait_ld();
  auto sv = [&](int c) -> float { return __uint_as_float(r[c]); };
  if (__any_sync(0xffffffffu, seen < (SPREAD ? 120 : 64))) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // bit c: column 32 w + c is visible
      uint32_t m;
      if (SPREAD) {
        m = 0u;
#pragma unroll
        for (int g = 0; g < 4; ++g) m |= ((1u << min(max(seen - 64 * w - 16 * g, 0), 8)) - 1u) << (8 * g);
      } else {
        const int n = seen - 32 * w;
        m = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) r[32 * w + c] = (m >> c) & 1u ? r[32 * w + c] : 0xff800000u;
    }
  }
  float mx[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) mx[c] = max3f(sv(c), sv(c + 8), sv(c + 16));
#pragma unroll
  for (int k = 24; k < 56; k += 16)
#pragma unroll
    for (int c = 0; c < 8; ++c) mx[c] = max3f(mx[c], sv(c + k), sv(c + k + 8));
#pragma unroll
  for (int c = 0; c < 8; ++c) mx[c] = fmaxf(mx[c], sv(c + 56));
  const float tmax = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
  // m_run is what is subtracted: the maximum, less the factor of f16 weights.  Both roundings go
  // up, and the growth is a difference: however large scores are, where their float32 spacing is
  // whole powers of two, no weight leaves the type's range (to nearest, weights became infinite there)
  constexpr float kGrow = Half16<T>::kBf16 ? 8.f : 4.f;
  float m_t = __fmul_ru(tmax, sl2);
  if constexpr (!Half16<T>::kBf16) m_t = __fsub_ru(m_t, Half16<T>::kRoom - kGrow);
  const bool grow = m_t - m_run > kGrow;
  const bool need_o = grow && m_run != -INFINITY;
  if (__any_sync(0xffffffffu, need_o)) {
    if (!pv_done()) return false;
    tc_fence_after();
    const float f = need_o ? ex2_approx(m_run - m_t) : 1.0f;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      tmem_ld_x32(o_addr + 32 * c, ov);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
      tmem_st_x32(o_addr + 32 * c, ov);
    }
    l_run *= f;
    if (ROUNDED) e_run *= f;
  }
  if (grow) m_run = m_t;
  const float neg = m_run == -INFINITY ? 0.f : -m_run;   // no key seen yet: every weight is zero
  const float2 sl2x2 = make_float2(sl2, sl2), neg2 = make_float2(neg, neg);
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float2 exact[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t pk[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 z = fma2(make_float2(sv(2 * k), sv(2 * k + 1)), sl2x2, neg2);
    const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
    pk[k] = Half16<T>::pack(e.x, e.y);
    acc[k & 1] = add2(acc[k & 1], ROUNDED ? Half16<T>::unpack(pk[k]) : e);
    if (ROUNDED) exact[k & 1] = add2(exact[k & 1], e);
  }
  tmem_st_x32(s_addr, pk);
  const float2 a2 = add2(acc[0], acc[1]);
  l_run += a2.x + a2.y;
  if (ROUNDED) {
    const float2 e2 = add2(exact[0], exact[1]);
    e_run += e2.x + e2.y;
  }
  tmem_wait_st();
  return true;
}

template <typename T, int D, KeySource KEYS, bool ROUNDED>
__global__ void __launch_bounds__(352, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PackedProblem p,
                     const PagedKV cache, float scale, const PackedOut o,
                     PackedCut *__restrict__ cuts, float *__restrict__ part) {
  using C = AttendCfg<D>;
  using namespace sm100;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char *smem = smem_raw + (sbase - raw);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffMisc + 8 * i; };
  PackedStart *start = reinterpret_cast<PackedStart *>(smem + C::kOffMisc + 384);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 448);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc + 464);
  long long *wsum = reinterpret_cast<long long *>(smem + C::kOffMisc + 512);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int tq1 = p.tq / 2, sub_rows = tq1 * p.G;
  constexpr bool PAGED = KEYS != kPackedKeys, spread = KEYS == kSpreadPages;
  static_assert(!spread || D == 128, "one box a page otherwise");

  if (warp == 1) {
    tmem_alloc(sbase + C::kOffMisc + 464, C::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bar(C::kBarQFull), 1);
    mbar_init(bar(C::kBarQEmpty), 2);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(C::kBarS + i), 1);
      mbar_init(bar(C::kBarP + i), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarPV + i), 1);
      mbar_init(bar(C::kBarO + i), 1);
      mbar_init(bar(C::kBarOFree + i), 128);
    }
    mbar_init(bar(C::kBarTeardown), 1);
    mbar_init(bar(C::kBarTeardown + 1), 1);
    fence_mbar_init();
    *abort = 0;
  }
  if (tid == 32) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // rows of the Q tiles that no copy fills (128 is no multiple of G): zero
  for (int e = tid; e < 2 * (128 - sub_rows) * (D / 8); e += C::kThreads) {
    const int ch = e % (D / 8), row = sub_rows + (e / (D / 8)) % (128 - sub_rows), i = e / ((D / 8) * (128 - sub_rows));
    *reinterpret_cast<uint4 *>(smem + C::kOffQ + i * C::kTileBytes + (ch >> 3) * C::kBoxBytes + row * 128 +
                               ((ch & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  tc_fence_before();
  wait_for_launches_before();
  if (tid == 0) cuts[blockIdx.x].valid = 0;
  packed_locate<RowCost>(p, blockIdx.x, gridDim.x, tid, C::kThreads, wsum, start);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PackedWalk<RowCost> w;
  w.begin(p, *start);

  auto uwait = [&](uint32_t b_addr, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(b_addr, parity));
  };
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort != 0); };

  if (warp == 0) {
    // ======================= copies ============================================
    const int page_rows = PAGED ? min(cache.page_size, kKeyTile) : kKeyTile;
    int slot = 0;        // ring slots used: K and V of a tile take one each
    int seg = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      const PackedSegment &s = w.s;
      if (aborted() || (seg > 0 && !uwait(bar(C::kBarQEmpty), (seg - 1) & 1))) {
        ok = false;
        break;
      }
      if (elect_one()) {
        mbar_expect_tx(bar(C::kBarQFull), 2 * sub_rows * D * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
            tma_load_4d(sbase + C::kOffQ + i * C::kTileBytes + b * C::kBoxBytes, &tm_q,
                        bar(C::kBarQFull), 64 * b, 0, s.r.first + s.rt * p.tq + i * tq1, s.h);
      }
      __syncwarp();
      ++seg;
      int page = PAGED ? lane_page(cache, s.b, s.ta * kKeyTile, s.r.kv, page_rows, lane) : 0;
      for (int t = s.ta; ok && t < s.tb; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x, ++slot) {
          const int st = slot % C::kStages;
          if (aborted() || (slot >= C::kStages &&
                            !uwait(bar(C::kBarEmpty + st), ((slot / C::kStages) - 1) & 1))) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + C::kOffKV + st * C::kTileBytes;
          if constexpr (PAGED) {
            issue_pages<D>(x ? &tm_v : &tm_k, bar(C::kBarFull + st), dst, t * kKeyTile, s.r.kv, s.h, page, page_rows,
                           cache.page_size, spread, lane);
          } else {
            if (elect_one()) {
              mbar_expect_tx(bar(C::kBarFull + st), C::kTileBytes);
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
                tma_load_3d(dst + b * C::kBoxBytes, x ? &tm_v : &tm_k, bar(C::kBarFull + st), 64 * b,
                            s.r.first + t * kKeyTile, s.h);
            }
            __syncwarp();
          }
        }
        if (PAGED)
          page = t + 1 < s.tb
                     ? lane_page(cache, s.b, (t + 1) * kKeyTile, s.r.kv, page_rows, lane)
                     : -1;
      }
    }
    if (!ok) {
      *abort = 1;
      // copies in flight land before the CTA exits
      if (seg > 0) uwait(bar(C::kBarQFull), (seg - 1) & 1);
      for (int i = max(slot - C::kStages, 0); i < slot; ++i)
        uwait(bar(C::kBarFull + i % C::kStages), (i / C::kStages) & 1);
    }
  } else if (warp == 1 || warp == 10) {
    // ======================= products ==========================================
    constexpr bool kBf = Half16<T>::kBf16;
    constexpr uint32_t kIdS = idesc_16_f32<kBf>(128, 64, 0, 0);
    constexpr uint32_t kIdO = idesc_16_f32<kBf>(128, D, 0, 1);
    auto step = [](int k) -> uint64_t {   // K step of a K-major operand: 32 bytes of a box row
      return (uint64_t)(((k >> 2) * C::kBoxBytes + (k & 3) * 32) >> 4);
    };
    const int i = warp == 1 ? 0 : 1;   // subtile
    int slot = 0, seg = 0;
    int np[2] = {0, 0};                // P of each half waited for
    int no = 0;                        // segments that used O
    // S_ih of the tile whose K is in ring slot `ks`
    auto issue_s = [&](int h, int ks) {
      const uint64_t qd = smem_desc_sw128(sbase + C::kOffQ + i * C::kTileBytes, 16, 1024);
      const uint64_t kd = smem_desc_sw128(
          sbase + C::kOffKV + (ks % C::kStages) * C::kTileBytes + h * (spread ? 1024 : 64 * 128), 16,
          spread ? 4096 : 1024);
      const uint64_t kbox = (spread ? 2048 : C::kBoxBytes) >> 4;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + C::kColS + 128 * i + 64 * h, qd + step(k), kd + (k >> 2) * kbox + (k & 3) * 2, kIdS,
                 k > 0 ? 1u : 0u);
        tc_commit(bar(C::kBarS + 2 * h + i));
      }
      __syncwarp();
    };
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
      __syncwarp();
    };
    auto full = [&](int sl) { return uwait(bar(C::kBarFull + sl % C::kStages), (sl / C::kStages) & 1); };
    // a segment: first tile, end, key positions of the request, end of the subtile's halves
    struct Part {
      int ta, tb, kv, nh;
    };
    auto take = [&](Part &x) -> bool {
      if (!w.next(p)) return false;
      x.ta = w.s.ta;
      x.tb = w.s.tb;
      x.kv = w.s.r.kv;
      x.nh = min(subtile(p, w.s, tq1, i, spread).nh, 2 * x.tb);
      return true;
    };
    // S of a segment's first tile
    auto first_scores = [&](const Part &x, int ks) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * x.ta + h < x.nh) issue_s(h, ks);
    };
    Part cur, nxt;
    bool have = take(cur), ok = true;
    if (have) {
      ok = uwait(bar(C::kBarQFull), 0) && full(0);
      tc_fence_after();
      if (ok) {
        first_scores(cur, 0);
        commit(C::kBarEmpty + 0);
        if (cur.ta + 1 == cur.tb) commit(C::kBarQEmpty);
      }
    }
    while (ok && have) {
      if (aborted()) {
        ok = false;
        break;
      }
      bool have_n = false;
      for (int t = cur.ta; t < cur.tb; ++t, slot += 2) {
        const bool last = t + 1 == cur.tb;
        bool have_v = false, have_k = false;
#pragma unroll
        for (int h = 0; ok && h < 2; ++h) {
          if (2 * t + h >= cur.nh) continue;
          if (!uwait(bar(C::kBarP + 2 * h + i), np[h] & 1)) {
            ok = false;
            break;
          }
          ++np[h];
          if (!have_v) {
            have_v = true;
            if (!full(slot + 1)) {
              ok = false;
              break;
            }
            const int live = cur.kv - t * kKeyTile;
            if (live < kKeyTile) {
              // rows past the sequence's last key may hold anything: zero, so that 0 x Inf or
              // NaN never reaches a sum (both warps write the same zeros, each before its product)
              const int z0 = max(live, 0);
              unsigned char *v = smem + C::kOffKV + ((slot + 1) % C::kStages) * C::kTileBytes;
              for (int e = lane; e < (kKeyTile - z0) * (D / 8); e += 32) {
                const int row = z0 + e / (D / 8), ch = e % (D / 8);
                *reinterpret_cast<uint4 *>(v + (spread ? page_chunk<D>(row, ch, 4)
                                                       : (ch >> 3) * C::kBoxBytes + row * 128 +
                                                             (((ch & 7) ^ (row & 7)) << 4))) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async();
              __syncwarp();
            }
          }
          const bool first = t == cur.ta && h == 0;
          if (first) {
            // the first product of a unit overwrites O: its rows have been read
            if (no > 0 && !uwait(bar(C::kBarOFree + i), (no - 1) & 1)) {
              ok = false;
              break;
            }
            ++no;
          }
          tc_fence_after();
          const uint64_t vd = smem_desc_sw128(
              sbase + C::kOffKV + ((slot + 1) % C::kStages) * C::kTileBytes + h * (spread ? 1024 : 4 * 2048),
              spread ? 2048 : C::kBoxBytes, spread ? 4096 : 1024);
          const uint64_t vstep = (spread ? 8192 : 2048) >> 4;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + C::kColO + D * i, tmem + C::kColS + 128 * i + 64 * h + 8 * k,
                     vd + k * vstep, kIdO, (!first || k > 0) ? 1u : 0u);
            tc_commit(bar(C::kBarPV + i));
            if (2 * t + h + 1 == cur.nh) tc_commit(bar(C::kBarO + i));
          }
          __syncwarp();
          if (2 * (t + 1) + h < cur.nh) {
            if (!have_k) {
              have_k = true;
              if (!full(slot + 2)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
            issue_s(h, slot + 2);
          }
        }
        if (!ok) break;
        // (slots that this subtile had no use for are given back once they have come)
        if ((!have_v && !full(slot + 1)) || (!last && !have_k && !full(slot + 2))) {
          ok = false;
          break;
        }
        commit(C::kBarEmpty + (slot + 1) % C::kStages);
        // (after P V of both halves: the next unit's Q may still be on its way)
        if (last) have_n = take(nxt);
        const bool more = !last || have_n;
        if (last && have_n) {
          if (!uwait(bar(C::kBarQFull), (seg + 1) & 1) || !full(slot + 2)) {
            ok = false;
            break;
          }
          tc_fence_after();
          first_scores(nxt, slot + 2);
        }
        if (more) {
          commit(C::kBarEmpty + (slot + 2) % C::kStages);
          if (last ? nxt.ta + 1 == nxt.tb : t + 2 == cur.tb) commit(C::kBarQEmpty);
        }
      }
      if (!ok) break;
      ++seg;
      have = have_n;
      cur = nxt;
    }
    if (!ok) {
      *abort = 1;
      // every product issued so far must finish before TMEM is released
      commit(C::kBarTeardown + i);
      uwait(bar(C::kBarTeardown + i), 0);
    }
  } else {
    // ======================= softmax ===========================================
    const int i = (warp - 2) >> 2;             // subtile
    const int sp = warp & 3;                   // TMEM sub-partition of this warp
    const int row = sp * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(sp * 32) << 16);
    const uint32_t s_addr = lane_addr + C::kColS + 128 * i, o_addr = lane_addr + C::kColO + D * i;
    const float sl2 = scale * kLog2e;
    unsigned char *stage = smem + C::kOffStage + (warp - 2) * 4096;
    int ns[2] = {0, 0};      // S of each half waited for
    int nv = 0, no = 0;      // halves worked on, segments that used O
    bool ok = true;
    while (ok && w.next(p)) {
      const PackedSegment s = w.s;
      const SubTile x = subtile(p, s, tq1, i, spread);
      const int tok = s.rt * p.tq + i * tq1 + row / p.G;     // token of this row in its sequence
      // keys this row sees: positions below lim (rows past the tile's go along with the last one)
      const int ltok = min(tok, s.r.n - 1);
      const int lim = p.causal ? max(min(s.r.past + ltok + 1, s.r.kv), 0) : s.r.kv;
      const int nh = min(x.nh, 2 * s.tb);
      float m_run = -INFINITY, l_run = 0.f, e_run = 0.f;
      for (int u = 2 * s.ta; u < nh; ++u, ++nv) {
        const int h = u & 1;
        if (!uwait(bar(C::kBarS + 2 * h + i), (h ? ns[1] : ns[0]) & 1)) {
          ok = false;
          break;
        }
        ns[0] += h == 0;
        ns[1] += h;
        tc_fence_after();
        // the product of the half before: the one before that came before this S
        auto pv_done = [&]() { return uwait(bar(C::kBarPV + i), (nv - 1) & 1); };
        const int seen = lim - (spread ? (u >> 1) * kKeyTile + 8 * h : u * 64);
        if (!softmax_half<T, D, ROUNDED, spread>(s_addr + 64 * h, o_addr, sl2, seen, pv_done, m_run, l_run, e_run)) {
          ok = false;
          break;
        }
        tc_fence_before();
        mbar_arrive(bar(C::kBarP + 2 * h + i));
      }
      if (!ok) break;
      // ---- epilogue of the segment ----------------------------------------------
      const bool used = 2 * s.ta < nh;
      if (used) {
        if (aborted() || !uwait(bar(C::kBarO + i), no & 1)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after();
      }
      const bool store = row < x.rows, whole = s.whole();
      const int head = s.h * p.G + row % p.G, token = s.r.first + tok;
      const float inv = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;
      const size_t hr = (size_t)head * p.T + token;
      const int prow = i * sub_rows + row;
      float *slot = part + ((size_t)blockIdx.x * 2 + s.slot()) * packed_slot_floats<D>(C::kRows);
      if (store) {
        const float le = ROUNDED ? e_run : l_run;
        if (!whole) {
          slot[prow] = m_run;
          slot[C::kRows + prow] = l_run;
          slot[2 * C::kRows + prow] = le;
        } else if (o.lse) {
          o.lse[hr] = le == 0.f ? -INFINITY : (m_run + log2f(le)) * 0.6931471805599453f;
        }
      }
      if (used) {
        // rows of the warp that are stored, and where each goes
        const int nrow = min(max(x.rows - sp * 32, 0), 32);
        const long long at = (long long)head * o.head + (long long)token * o.row;
        // (a loop, not unrolled: units of a few tiles come back to this code often enough that its
        // length is paid for in instruction fetches)
        float4 *ps = reinterpret_cast<float4 *>(slot + 3 * C::kRows) + prow;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld_x32(o_addr + 32 * c, ov);
          tmem_wait_ld();
          if (c + 1 == D / 32) {
            tc_fence_before();
            mbar_arrive(bar(C::kBarOFree + i));    // the next unit's products may start
          }
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * inv);
            if (ROUNDED)
              store_rows<8>(stage, lane, nrow, (long long)hr * D + 32 * c, o.f32,
                            [&](int k) { return make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]); });
#pragma unroll
            for (int k = 0; k < 16; ++k)
              ov[k] = Half16<T>::pack(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1]));
            store_rows<4>(stage, lane, nrow, at + 32 * c, reinterpret_cast<T *>(o.out),
                          [&](int k) { return make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]); });
          } else if (store) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              ps[(size_t)(8 * c + k) * C::kRows] =
                  make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                              __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
          }
        }
      }
      if (!whole && s.ta == 0 && tid == 64) cuts[blockIdx.x] = packed_cut(p, *start, s, gridDim.x);
    }
    if (!ok) *abort = 1;
  }

  // ---- teardown -----------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace pisa
