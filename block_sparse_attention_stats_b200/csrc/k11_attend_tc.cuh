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
// for a group.  Keys come in tiles of 128.
// Roles (384 threads, one CTA per SM, persistent over its range of tiles):
//   warp 0      copies: Q of both subtiles, then K and V tiles into a ring;
//   warp 1      TMEM; issues S_i = Q_i K^T and O_i += P_i V (P read from TMEM);
//               subtile 0's products run while subtile 1's softmax does, and back;
//   warps 4-7   softmax of subtile 0, one thread a row (TMEM lane);
//   warps 8-11  softmax of subtile 1.
// A softmax thread holds 128 scores: its warpgroups take 200 registers a thread,
// the first (whose warps 2 and 3 have nothing to do) keeps 104: with the launch's
// 168 for all, the scores spilled.
// TMEM columns: S_0 [0, 128), S_1 [128, 256), O_0 [256, 256 + D), O_1 after it;
// P (16-bit) overwrites the first 64 columns of its S.  S_i of the next tile is
// issued after P_i V of this one by the same thread, and one thread's products
// run in issue order, so no barrier guards the overwrite; the commit that tells
// the softmax of S_i also says that O_i is complete up to the tile before, so a
// softmax thread may rescale O_i itself.  That is rare: the running maximum moves
// only when it grows by more than 2^8 (weights stay below 2^8, in range of both
// 16-bit types).
// Every wait is bounded; on a timeout the CTA records the error, stops issuing,
// drains its copies and products, frees TMEM and exits.
#pragma once

#include "k10_attend_rows.cuh"
#include "packed_primitives.cuh"
#include "packed_schedule.cuh"

namespace pisa {

template <int D> struct AttendCfg {
  static constexpr int kThreads = 384;
  static constexpr int kRegsSoftmax = 200, kRegsOther = 104;   // of 168 at launch
  static_assert(2 * kRegsSoftmax + kRegsOther == 3 * 168, "registers");
  static constexpr int kRows = 256;                      // rows of a unit
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kTileBytes = kKeyTile * D * 2;    // K or V tile, or Q of a subtile
  static constexpr int kBoxBytes = kKeyTile * 128;       // one 64-column box of 128 rows
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffMisc = kOffKV + kStages * kTileBytes;
  static constexpr int kSmem = kOffMisc + 1024 + 1024;   // + alignment slack
  static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarFull = 2, kBarEmpty = kBarFull + kStages;
  static constexpr int kBarS = kBarEmpty + kStages;      // + subtile
  static constexpr int kBarP = kBarS + 2;
  static constexpr int kBarO = kBarP + 2;                // O complete
  static constexpr int kBarOFree = kBarO + 2;            // O read
  static constexpr int kBarTeardown = kBarOFree + 2;
  static_assert(kBarTeardown < 32 && kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
};

// tq1 tokens of a subtile; rows of subtile i, and its key tiles
struct SubTile {
  int rows, nt;
};
__device__ __forceinline__ SubTile subtile(const PackedProblem &p, const PackedSegment &s, int tq1, int i) {
  SubTile x;
  const int tok = s.rt * p.tq + i * tq1;
  x.rows = max(min(s.r.n - tok, tq1), 0) * p.G;
  x.nt = x.rows == 0 ? 0 : RowCost<kKeyTile>::tiles(p, s.r.n, s.r.kv, tq1, 2 * s.rt + i);
  return x;
}

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(384, 1)
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
  PackedStart *start = reinterpret_cast<PackedStart *>(smem + C::kOffMisc + 256);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 320);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc + 336);
  long long *wsum = reinterpret_cast<long long *>(smem + C::kOffMisc + 384);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int tq1 = p.tq / 2, sub_rows = tq1 * p.G;

  if (warp == 1) {
    tmem_alloc(sbase + C::kOffMisc + 336, C::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bar(C::kBarQFull), 1);
    mbar_init(bar(C::kBarQEmpty), 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarS + i), 1);
      mbar_init(bar(C::kBarP + i), 128);
      mbar_init(bar(C::kBarO + i), 1);
      mbar_init(bar(C::kBarOFree + i), 128);
    }
    mbar_init(bar(C::kBarTeardown), 1);
    fence_mbar_init();
    *abort = 0;
    cuts[blockIdx.x].valid = 0;
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
  packed_locate<RowCost<kKeyTile>>(p, blockIdx.x, gridDim.x, tid, C::kThreads, wsum, start);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PackedWalk<RowCost<kKeyTile>> w;
  w.begin(p, *start);

  auto uwait = [&](uint32_t b_addr, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(b_addr, parity));
  };
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort != 0); };

  if (warp < 4) {
  regs_shrink<C::kRegsOther>();
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
            issue_pages<D>(x ? &tm_v : &tm_k, nullptr, bar(C::kBarFull + st), dst, 0, C::kBoxBytes,
                           t * kKeyTile, s.r.kv, s.h, page, page_rows, cache.page_size, lane);
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
  } else if (warp == 1) {
    // ======================= products ==========================================
    constexpr bool kBf = Half16<T>::kBf16;
    constexpr uint32_t kIdS = idesc_16_f32<kBf>(128, 128, 0, 0);
    constexpr uint32_t kIdO = idesc_16_f32<kBf>(128, D, 0, 1);
    auto step = [](int k) -> uint64_t {   // K step of a K-major operand: 32 bytes of a box row
      return (uint64_t)(((k >> 2) * C::kBoxBytes + (k & 3) * 32) >> 4);
    };
    int slot = 0, seg = 0;
    int np[2] = {0, 0};      // P tiles waited for
    int no[2] = {0, 0};      // segments that used O
    bool ok = true;
    // S_i of the tile whose K is in ring slot `ks`
    auto issue_s = [&](int i, int ks) {
      const uint64_t qd = smem_desc_sw128(sbase + C::kOffQ + i * C::kTileBytes, 16, 1024);
      const uint64_t kd = smem_desc_sw128(sbase + C::kOffKV + (ks % C::kStages) * C::kTileBytes, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + C::kColS + 128 * i, qd + step(k), kd + step(k), kIdS, k > 0 ? 1u : 0u);
        tc_commit(bar(C::kBarS + i));
      }
      __syncwarp();
    };
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
      __syncwarp();
    };
    auto full = [&](int sl) { return uwait(bar(C::kBarFull + sl % C::kStages), (sl / C::kStages) & 1); };
    while (ok && w.next(p)) {
      const PackedSegment &s = w.s;
      const int nt0 = min(subtile(p, s, tq1, 0).nt, s.tb), nt1 = min(subtile(p, s, tq1, 1).nt, s.tb);
      if (aborted() || !uwait(bar(C::kBarQFull), seg & 1) || !full(slot)) {
        ok = false;
        break;
      }
      ++seg;
      tc_fence_after();
      if (s.ta < nt0) issue_s(0, slot);
      if (s.ta < nt1) issue_s(1, slot);
      commit(C::kBarEmpty + slot % C::kStages);
      if (s.ta + 1 >= s.tb) commit(C::kBarQEmpty);
      for (int t = s.ta; ok && t < s.tb; ++t, slot += 2) {
        const bool more = t + 1 < s.tb;
        bool have_v = false, have_k = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int nt = i ? nt1 : nt0;
          if (t >= nt) continue;
          if (aborted() || !uwait(bar(C::kBarP + i), np[i] & 1)) {
            ok = false;
            break;
          }
          ++np[i];
          if (!have_v) {
            have_v = true;
            if (!full(slot + 1)) {
              ok = false;
              break;
            }
            const int live = s.r.kv - t * kKeyTile;
            if (live < kKeyTile) {
              // rows past the sequence's last key may hold anything: zero, so that 0 x Inf or
              // NaN never reaches a sum
              const int z0 = max(live, 0);
              unsigned char *v = smem + C::kOffKV + ((slot + 1) % C::kStages) * C::kTileBytes;
              for (int e = lane; e < (kKeyTile - z0) * (D / 8); e += 32) {
                const int row = z0 + e / (D / 8), ch = e % (D / 8);
                *reinterpret_cast<uint4 *>(v + (ch >> 3) * C::kBoxBytes + row * 128 +
                                           (((ch & 7) ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async();
              __syncwarp();
            }
          }
          if (t == s.ta) {
            // the first product of a unit overwrites O: its rows have been read
            if (no[i] > 0 && !uwait(bar(C::kBarOFree + i), (no[i] - 1) & 1)) {
              ok = false;
              break;
            }
            ++no[i];
          }
          tc_fence_after();
          const uint64_t vd = smem_desc_sw128(
              sbase + C::kOffKV + ((slot + 1) % C::kStages) * C::kTileBytes, C::kBoxBytes, 1024);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeyTile / 16; ++k)
              mma_ts(tmem + C::kColO + D * i, tmem + C::kColS + 128 * i + 8 * k,
                     vd + (uint64_t)((k * 2048) >> 4), kIdO, (t > s.ta || k > 0) ? 1u : 0u);
            if (t + 1 >= nt) tc_commit(bar(C::kBarO + i));
          }
          __syncwarp();
          if (t + 1 < nt) {
            if (!have_k) {
              have_k = true;
              if (!full(slot + 2)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
            issue_s(i, slot + 2);
          }
        }
        if (!ok) break;
        if (!have_v && !full(slot + 1)) {   // a tile of no subtile (cannot happen): keep the ring going
          ok = false;
          break;
        }
        commit(C::kBarEmpty + (slot + 1) % C::kStages);
        if (more) {
          if (!have_k && !full(slot + 2)) {
            ok = false;
            break;
          }
          commit(C::kBarEmpty + (slot + 2) % C::kStages);
          if (t + 2 >= s.tb) commit(C::kBarQEmpty);
        }
      }
    }
    if (!ok) {
      *abort = 1;
      // every product issued so far must finish before TMEM is released
      commit(C::kBarTeardown);
      uwait(bar(C::kBarTeardown), 0);
    }
  }
  } else {
    // ======================= softmax ===========================================
    regs_grow<C::kRegsSoftmax>();
    const int i = (warp - 4) >> 2;             // subtile
    const int sp = warp & 3;                   // TMEM sub-partition of this warp
    const int row = sp * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(sp * 32) << 16);
    const uint32_t s_addr = lane_addr + C::kColS + 128 * i, o_addr = lane_addr + C::kColO + D * i;
    const float sl2 = scale * kLog2e;
    int ns = 0, no = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      const PackedSegment s = w.s;
      const SubTile x = subtile(p, s, tq1, i);
      const int tok = s.rt * p.tq + i * tq1 + row / p.G;     // token of this row in its sequence
      // keys this row sees: positions below lim (rows past the tile's go along with the last one)
      const int ltok = min(tok, s.r.n - 1);
      const int lim = p.causal ? max(min(s.r.past + ltok + 1, s.r.kv), 0) : s.r.kv;
      const int t1 = min(x.nt, s.tb);
      float m_run = -INFINITY, l_run = 0.f;
      for (int t = s.ta; t < t1; ++t, ++ns) {
        if (aborted() || !uwait(bar(C::kBarS + i), ns & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[128];
        {
          uint32_t r[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_x32(s_addr + 32 * c, r[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = __uint_as_float(r[c >> 5][c & 31]);
        }
        const int seen = lim - t * kKeyTile;
        if (__any_sync(0xffffffffu, seen < kKeyTile)) {
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = c < seen ? sv[c] : -INFINITY;
        }
        float mx[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = max3f(sv[c], sv[c + 8], sv[c + 16]);
#pragma unroll
        for (int k = 24; k < 120; k += 16)
#pragma unroll
          for (int c = 0; c < 8; ++c) mx[c] = max3f(mx[c], sv[c + k], sv[c + k + 8]);
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = fmaxf(mx[c], sv[c + 120]);
        const float tmax = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
        const float m_t = tmax * sl2;
        const bool grow = m_t > m_run + 8.0f;
        const bool need_o = grow && m_run != -INFINITY;
        const float f = grow ? ex2_approx(m_run - m_t) : 1.0f;
        if (__any_sync(0xffffffffu, need_o)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(o_addr + 32 * c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
            tmem_st_x32(o_addr + 32 * c, ov);
          }
        }
        if (grow) {
          m_run = m_t;
          l_run *= f;
        }
        const float neg = m_run == -INFINITY ? 0.f : -m_run;   // no key seen yet: every weight is zero
        const float2 sl2x2 = make_float2(sl2, sl2), neg2 = make_float2(neg, neg);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // P is rounded to 16 bits for its product; the sum keeps the float32 weights
          uint32_t pk[32];
          if (PAGED || o.f32 == nullptr) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 z = fma2(make_float2(sv[64 * h + 2 * k], sv[64 * h + 2 * k + 1]), sl2x2, neg2);
              const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
              acc[k & 3] = add2(acc[k & 3], e);
              pk[k] = Half16<T>::pack(e.x, e.y);
            }
          } else {
            // for the backward the sum takes the rounded weights: dout_t . o_t is then the mean of
            // dP under the weights themselves, and does not lose dP - Delta to their rounding
            // where one key holds nearly all the weight
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 z = fma2(make_float2(sv[64 * h + 2 * k], sv[64 * h + 2 * k + 1]), sl2x2, neg2);
              pk[k] = Half16<T>::pack(ex2_approx(z.x), ex2_approx(z.y));
              acc[k & 3] = add2(acc[k & 3], Half16<T>::unpack(pk[k]));
            }
          }
          tmem_st_x32(s_addr + 32 * h, pk);
        }
        const float2 a2 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l_run += a2.x + a2.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::kBarP + i));
      }
      if (!ok) break;
      // ---- epilogue of the segment ----------------------------------------------
      const bool used = s.ta < t1;
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
        if (!whole) {
          slot[prow] = m_run;
          slot[C::kRows + prow] = l_run;
        } else if (o.lse) {
          o.lse[hr] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
        }
      }
      if (used) {
        T *dst = reinterpret_cast<T *>(o.out) + head * o.head + token * o.row;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld_x32(o_addr + 32 * c, ov);
          tmem_wait_ld();
          if (!store) continue;
          if (whole) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(ov[k]) * inv;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4 *>(dst + 32 * c)[k] = make_uint4(
                  Half16<T>::pack(v[8 * k], v[8 * k + 1]), Half16<T>::pack(v[8 * k + 2], v[8 * k + 3]),
                  Half16<T>::pack(v[8 * k + 4], v[8 * k + 5]), Half16<T>::pack(v[8 * k + 6], v[8 * k + 7]));
            if (o.f32) {
              float4 *d32 = reinterpret_cast<float4 *>(o.f32 + hr * D + 32 * c);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                d32[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          } else {
            float4 *ps = reinterpret_cast<float4 *>(slot + 2 * C::kRows);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              ps[(size_t)(8 * c + k) * C::kRows + prow] =
                  make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                              __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
          }
        }
        tc_fence_before();
        mbar_arrive(bar(C::kBarOFree + i));
      }
      if (!whole && s.ta == 0 && tid == 128) cuts[blockIdx.x] = packed_cut(*start, s);
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
