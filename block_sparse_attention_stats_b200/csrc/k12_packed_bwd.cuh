// Gradients of attention over packed sequences (causal or not, grouped heads),
// on the sm_100a tensor cores.  With P_tj = exp(s q_t . k_j - lse_t), dP_tj =
// dout_t . v_j and Delta_t = dout_t . o_t (= sum_j P_tj dP_tj):
//   dq_t = s sum_j P_tj (dP_tj - Delta_t) k_j
//   dk_j = s sum_t P_tj (dP_tj - Delta_t) q_t,   dv_j = sum_t P_tj dout_t
// where t runs over the rows of every query head of the key head's group.
// Bound: the tensor cores, seven products of 2 D flops a row and key (S and dP
// are formed in both kernels).  One kernel with five would have to add dq from
// every key tile: float32 atomics, whose order changes results, or a wait of
// CTAs on one another.  Two kernels keep every sum in one CTA in a fixed order.
//
// Both keep a pair of 128-row tiles (dq: Q and dout; dk, dv: K and V) and stream
// the other pair through a ring, 128 rows at a time; both are cut evenly over the
// SMs (packed_schedule.cuh), and packed_sum_kernel joins what a range's end cuts.
// dq keeps its pair in TMEM, as the A operands of S and dP: its products then read
// half as much shared memory, and the ring has six tiles instead of four (with
// four, K of the next tile arrived 600 cycles late).  dk, dv have two accumulators
// and no TMEM left: their pair stays in shared memory.
// Roles (352 threads): warp 0 copies; warps 1 and 10 issue the products; warps 2-5
// take columns 0 .. 63 of each 128 x 128 tile (half 0), warps 6-9 columns 64 .. 127
// (half 1), one thread a row (TMEM lane).
// The halves go their own ways, in this order each (h: half, u: tile):
//   dq      warp 1: S_uh as soon as S_u-1,h is in registers
//           warp 10: dQ += dS_uh K_uh, then dP_u+1,h
//   dk, dv  warp 1: dV += P_uh dout_uh, then S_u+1,h
//           warp 10: dK += dS_uh Q_uh, then dP_u+1,h
// so one half's products run while the other half's weights are formed, and one
// product's warp does not wait for the other product's operands.  Measured against
// whole tiles with one issuing warp: 214 against 236 us at d = 64 (4096 + 2048 tokens,
// 16 / 4 heads); at d = 128 level (1931 / 1938 us on 8192 + 4608 + 1500 tokens, 24 / 8
// heads, in a loop at the 1 kW cap, where the halves' narrower products read more
// shared memory).
// 16-bit dS is written over the dP columns it was formed from, 16-bit P over its S
// columns.  An overwrite is safe because the product that reads and the one that
// overwrites come from one thread, whose products run in order.
// Rounding: P and dS are rounded to bf16 for their products (the tensor cores
// take no more), everything else is float32.
#pragma once

#include "packed_primitives.cuh"
#include "packed_schedule.cuh"

namespace pisa {

// lse2 = lse log2 e and Delta, [Hq, T]: one warp a row
template <int D>
__global__ void __launch_bounds__(256)
    packed_delta_kernel(const __nv_bfloat16 *dout, long long head_stride, long long row_stride,
                        const float *out, const float *lse, int Hq, int T,
                        const int32_t *cu, int B, float *__restrict__ lse2,
                        float *__restrict__ delta) {
  sm100::allow_next_launch();
  sm100::wait_for_launches_before();
  const int lane = threadIdx.x & 31;
  const int end = min(max(sm100::ld_int(cu + B), 0), T);      // rows behind the last sequence are not read
  const long long rows = (long long)Hq * T;
  for (long long r = (blockIdx.x * 256ll + threadIdx.x) >> 5; r < rows; r += gridDim.x * 8ll) {
    const int h = (int)(r / T), t = (int)(r % T);
    if (t >= end) continue;
    float s = 0.f;
    if (lane < D / 4) {
      const float4 o = __ldcg(reinterpret_cast<const float4 *>(out + r * D) + lane);
      const uint2 g =
          __ldcg(reinterpret_cast<const uint2 *>(dout + h * head_stride + t * row_stride + 4 * lane));
      const float2 a = Half16<__nv_bfloat16>::unpack(g.x), b = Half16<__nv_bfloat16>::unpack(g.y);
      s = fmaf(o.x, a.x, fmaf(o.y, a.y, fmaf(o.z, b.x, o.w * b.y)));
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) {
      delta[r] = s;
      lse2[r] = __ldcg(lse + r) * kLog2e;
    }
  }
}

template <int D, bool KV> struct PackedBwdCfg {
  static constexpr int kThreads = 352;
  static constexpr int kStages = D == 128 ? (KV ? 4 : 6) : (KV ? 8 : 12);
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kOffA = 0;                          // the resident pair (KV)
  static constexpr int kOffRing = KV ? 2 * kTileBytes : 0;
  static constexpr int kOffStage = kOffRing + kStages * kTileBytes;   // 2 KB a warp that stores rows
  static constexpr int kVecs = KV ? (D == 128 ? 4 : 6) : 1;           // lse and Delta of streamed rows (KV)
  static constexpr int kOffVec = kOffStage + 8 * 2048;
  static constexpr int kOffMisc = kOffVec + kVecs * 1024;
  static constexpr int kSmem = kOffMisc + 1024 + 1024;     // + alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // kBarAFull: the resident pair is in shared memory (KV) or in TMEM; kBarAEmpty: KV only.  S, dP, P
  // (dq: S is in registers) and Z (dS): + half
  static constexpr int kBarAFull = 0, kBarAEmpty = 1, kBarS = 2, kBarDP = 4, kBarP = 6, kBarZ = 8, kBarAcc = 10,
                       kBarAccFree = 11, kBarTeardown = 12, kBarFull = 14, kBarEmpty = kBarFull + kStages;
  static_assert(kBarEmpty + kStages <= 48, "barrier slots");
  static constexpr uint32_t kTmemCols = 512, kColS = 0, kColDP = 128, kColAcc = 256, kColA = 384;
};

// KV = false: dq.  The unit's rows are 128 / G tokens with the G heads of a key
// head (token-major), streamed pairs are K and V of a key tile.
// KV = true: dk, dv.  The unit's rows are 128 keys, streamed pairs are Q and dout
// of 128 tokens of one query head; tiles run over the heads, then the tokens.
template <int D, bool KV>
__global__ void __launch_bounds__(352, 1)
    packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const PackedProblem p, float scale, const float *lse2, const float *delta,
                      __nv_bfloat16 *__restrict__ out0,
                      long long out0_head, long long out0_row, __nv_bfloat16 *__restrict__ out1,
                      long long out1_head, long long out1_row, PackedCut *__restrict__ cuts,
                      float *__restrict__ part) {
  using C = PackedBwdCfg<D, KV>;
  using Cost = typename std::conditional<KV, KeyCost, RowCost>::type;
  using namespace sm100;
  constexpr int kStages = C::kStages, kMisc = C::kOffMisc;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char *smem = smem_raw + (sbase - raw);
  auto bar = [&](int i) -> uint32_t { return sbase + kMisc + 8 * i; };
  PackedStart *start = reinterpret_cast<PackedStart *>(smem + kMisc + 384);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kMisc + 448);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + kMisc + 464);
  long long *wsum = reinterpret_cast<long long *>(smem + kMisc + 512);
  float *vec = reinterpret_cast<float *>(smem + C::kOffVec);      // [kVecs][lse 128, Delta 128] (KV)
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int sub_rows = KV ? 128 : p.tq * p.G;

  if (warp == 1) {
    tmem_alloc(sbase + kMisc + 464, C::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bar(C::kBarAFull), KV ? 1 : 256);
    mbar_init(bar(C::kBarAEmpty), 2);
    for (int h = 0; h < 2; ++h) {
      mbar_init(bar(C::kBarS + h), 1);
      mbar_init(bar(C::kBarDP + h), 1);
      mbar_init(bar(C::kBarP + h), 128);
      mbar_init(bar(C::kBarZ + h), 128);
      mbar_init(bar(C::kBarTeardown + h), 1);
    }
    mbar_init(bar(C::kBarAcc), KV ? 2 : 1);
    mbar_init(bar(C::kBarAccFree), 256);
    for (int s = 0; s < kStages; ++s) {
      // dq: K (even slots) is read for S and for dQ, V for dP; dk, dv: Q for S and for dK, dout for dP and dV
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), KV || s % 2 == 0 ? 2 : 1);
    }
    fence_mbar_init();
    *abort = 0;
  }
  if (tid == 32) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_do);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  wait_for_launches_before();
  if (tid == 0) cuts[blockIdx.x].valid = 0;
  packed_locate<Cost>(p, blockIdx.x, gridDim.x, tid, C::kThreads, wsum, start);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PackedWalk<Cost> w;
  w.begin(p, *start);

  auto uwait = [&](uint32_t b_addr, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(b_addr, parity));
  };
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort != 0); };
  // streamed tile t of a unit: the query head inside the group (KV), the first
  // token or key of its 128 rows
  auto tile_at = [&](const PackedSegment &s, int t, int &g) -> int {
    if (!KV) return t * 128;
    const int per = s.nt / p.G;
    g = t / per;
    return (t % per + (p.causal ? s.rt : 0)) * 128;
  };

  if (warp == 0) {
    // ======================= copies ============================================
    int slot = 0, seg = 0, tile = 0;
    bool ok = true;
    auto room = [&]() -> bool {
      return !aborted() && (slot < kStages || uwait(bar(C::kBarEmpty + slot % kStages), ((slot / kStages) - 1) & 1));
    };
    while (ok && w.next(p)) {
      const PackedSegment &s = w.s;
      if constexpr (KV) {
        if (aborted() || (seg > 0 && !uwait(bar(C::kBarAEmpty), (seg - 1) & 1))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t a = bar(C::kBarAFull);
          mbar_expect_tx(a, 2 * C::kTileBytes);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_3d(sbase + C::kOffA + x * C::kTileBytes + b * C::kBoxBytes, x ? &tm_v : &tm_k, a, 64 * b,
                          s.r.first + s.rt * 128, s.h);
        }
        __syncwarp();
        ++seg;
      } else {
        // Q and dout pass through two ring slots on their way to TMEM
#pragma unroll
        for (int x = 0; ok && x < 2; ++x) {
          if (!room()) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint32_t full = bar(C::kBarFull + slot % kStages);
            mbar_expect_tx(full, sub_rows * D * 2);
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_4d(sbase + C::kOffRing + (slot % kStages) * C::kTileBytes + b * C::kBoxBytes,
                          x ? &tm_do : &tm_q, full, 64 * b, 0, s.r.first + s.rt * p.tq, s.h);
          }
          __syncwarp();
          ++slot;
        }
      }
      for (int t = s.ta; ok && t < s.tb; ++t, ++tile) {
        int g = 0;
        const int row0 = tile_at(s, t, g);
        const int head = KV ? s.h * p.G + g : s.h;
        float lv[4], dv[4];
        if constexpr (KV) {
          // lse and Delta of the tile's rows: asked for before the wait for room
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = lane + 32 * k;
            const bool in = row0 + r < s.r.n;
            const size_t at = (size_t)head * p.T + s.r.first + row0 + r;
            lv[k] = in ? __ldcg(lse2 + at) : INFINITY;     // exp2(x - inf) = 0: a row that is not there
            dv[k] = in ? __ldcg(delta + at) : 0.f;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x, ++slot) {
          if (!room()) {
            ok = false;
            break;
          }
          const int st = slot % kStages;
          if (KV && x == 0) {
            // handed over with the slot's arrival.  Buffer tile % kVecs was last read for tile -
            // kVecs, whose dS came before the products that freed this slot
            float *v = vec + (tile % C::kVecs) * 256;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[lane + 32 * k] = lv[k];
              v[128 + lane + 32 * k] = dv[k];
            }
            __syncwarp();
          }
          if (elect_one()) {
            const uint32_t dst = sbase + C::kOffRing + st * C::kTileBytes;
            mbar_expect_tx(bar(C::kBarFull + st), C::kTileBytes);
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_3d(dst + b * C::kBoxBytes, KV ? (x ? &tm_do : &tm_q) : (x ? &tm_v : &tm_k),
                          bar(C::kBarFull + st), 64 * b, s.r.first + row0, head);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) {
      *abort = 1;
      // copies in flight land before the CTA exits
      if (KV && seg > 0) uwait(bar(C::kBarAFull), (seg - 1) & 1);
      for (int i = max(slot - kStages, 0); i < slot; ++i)
        uwait(bar(C::kBarFull + i % kStages), (i / kStages) & 1);
    }
  } else if (warp == 1 || warp == 10) {
    // ======================= products ==========================================
    constexpr uint32_t kIdS = idesc_bf16_f32(128, 64, 0, 0);
    constexpr uint32_t kIdAcc = idesc_bf16_f32(128, D, 0, 1);
    auto step = [](int k) -> uint64_t {
      return (uint64_t)(((k >> 2) * C::kBoxBytes + (k & 3) * 32) >> 4);
    };
    auto ring = [&](int sl) -> uint32_t { return sbase + C::kOffRing + (sl % kStages) * C::kTileBytes; };
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
      __syncwarp();
    };
    // waits for a ring slot; rows past the sequence's last may hold anything: zero, so that
    // 0 x Inf or NaN never reaches a sum
    auto take = [&](int sl, int live) -> bool {
      if (!uwait(bar(C::kBarFull + sl % kStages), (sl / kStages) & 1)) return false;
      if (live < 128) {
        unsigned char *v = smem + C::kOffRing + (sl % kStages) * C::kTileBytes;
        for (int e = lane; e < (128 - live) * (D / 8); e += 32) {
          const int row = live + e / (D / 8), ch = e % (D / 8);
          *reinterpret_cast<uint4 *>(v + (ch >> 3) * C::kBoxBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
      }
      tc_fence_after();
      return true;
    };
    // warp 1 (x = 0): S, and dV of what is laid over it; warp 10 (x = 1): dP, and dK or dQ
    const int x = warp == 1 ? 0 : 1;
    const bool reads = KV || x == 1;
    const uint32_t col = x ? C::kColDP : C::kColS;
    const uint32_t acc = tmem + C::kColAcc + (KV && x == 0 ? D : 0);   // dQ or dK, dV after it
    const int own = x, other = KV ? 1 - x : 0;   // slots of the pair: for S or dP, for the accumulator
    const uint64_t ad = smem_desc_sw128(sbase + C::kOffA + x * C::kTileBytes, 16, 1024);
    // half h of S or dP from ring slot sl
    auto issue_s = [&](int h, int sl) {
      const uint64_t bd = smem_desc_sw128(ring(sl) + h * 64 * 128, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (KV)
            mma_ss(tmem + col + 64 * h, ad + step(k), bd + step(k), kIdS, k > 0 ? 1u : 0u);
          else
            mma_ts(tmem + col + 64 * h, tmem + C::kColA + 64 * x + 8 * k, bd + step(k), kIdS, k > 0 ? 1u : 0u);
        }
        tc_commit(bar((x ? C::kBarDP : C::kBarS) + h));
      }
      __syncwarp();
    };
    // the accumulator += 16-bit half h times rows 64 h .. 64 h + 63 of ring slot sl
    auto issue_acc = [&](int h, int sl, bool first) {
      const uint64_t bd = smem_desc_sw128(ring(sl) + h * 64 * 128, C::kBoxBytes, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(acc, tmem + col + 64 * h + 8 * k, bd + (uint64_t)((k * 2048) >> 4), kIdAcc,
                 (!first || k > 0) ? 1u : 0u);
      }
      __syncwarp();
    };
    int slot = 0, seg = 0, u = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      const PackedSegment &s = w.s;
      int g = 0;
      auto live = [&](int t) { return max(min(s.r.n - tile_at(s, t, g), 128), 0); };
      if (aborted() || !uwait(bar(C::kBarAFull), seg & 1)) {
        ok = false;
        break;
      }
      if (!KV) {
        // Q and dout are in TMEM: their ring slots are free
        if (elect_one()) {
          mbar_arrive(bar(C::kBarEmpty + slot % kStages));
          if (x) mbar_arrive(bar(C::kBarEmpty + (slot + 1) % kStages));
        }
        __syncwarp();
        slot += 2;
      }
      int lv = live(s.ta);
      for (int h = 0; ok && h < 2; ++h) {
        // S of dq's first tile overwrites scores that the unit before has read
        if ((!KV && x == 0 && u > 0 && !uwait(bar(C::kBarP + h), (u - 1) & 1)) ||
            (h == 0 && !take(slot + own, lv))) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_s(h, slot + own);
      }
      if (!ok) break;
      commit(C::kBarEmpty + (slot + own) % kStages);
      if (KV && s.ta + 1 == s.tb) commit(C::kBarAEmpty);
      for (int t = s.ta; ok && t < s.tb; ++t, slot += 2, ++u) {
        const bool more = t + 1 < s.tb, first = t == s.ta;
        const int lnext = more ? live(t + 1) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (reads) {
            if ((h == 0 && !take(slot + other, lv)) ||
                !uwait(bar((x ? C::kBarZ : C::kBarP) + h), u & 1) ||
                // the accumulators of the unit before have been read
                (first && h == 0 && seg > 0 && !uwait(bar(C::kBarAccFree), (seg - 1) & 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_acc(h, slot + other, first && h == 0);
            if (h == 1) {
              commit(C::kBarEmpty + (slot + other) % kStages);
              if (!more) commit(C::kBarAcc);
            }
          }
          if (more) {
            if ((!reads && !uwait(bar(C::kBarP + h), u & 1)) ||    // S_uh is in registers
                (h == 0 && !take(slot + 2 + own, lnext))) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(h, slot + 2 + own);
            if (h == 1) {
              commit(C::kBarEmpty + (slot + 2 + own) % kStages);
              if (KV && t + 2 == s.tb) commit(C::kBarAEmpty);
            }
          }
        }
        lv = lnext;
      }
      ++seg;
    }
    if (!ok) {
      *abort = 1;
      commit(C::kBarTeardown + x);
      uwait(bar(C::kBarTeardown + x), 0);
    }
  } else {
    // ======================= weights ===========================================
    const int gw = (warp - 2) >> 2;              // columns 64 gw .. 64 gw + 63
    const int sp = warp & 3;
    const int row = sp * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(sp * 32) << 16);
    const uint32_t s_addr = lane_addr + C::kColS + 64 * gw, dp_addr = lane_addr + C::kColDP + 64 * gw;
    const float sl2 = scale * kLog2e;
    unsigned char *stage = smem + C::kOffStage + (warp - 2) * 2048;
    int u = 0, seg = 0, slot = 0;
    // this thread's row of Q (warpgroup 0) or dout (warpgroup 1) from the ring slots of segment
    // w.s into TMEM, as packed pairs, once no product reads the pair before
    auto load_pair = [&]() -> bool {
      const int sl = slot + gw;
      if (!uwait(bar(C::kBarFull + sl % kStages), (sl / kStages) & 1)) return false;
      const unsigned char *box = smem + C::kOffRing + (sl % kStages) * C::kTileBytes + row * 128;
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        uint32_t x[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row < sub_rows) v = *reinterpret_cast<const uint4 *>(box + b * C::kBoxBytes + ((c ^ (row & 7)) << 4));
          x[4 * c] = v.x;
          x[4 * c + 1] = v.y;
          x[4 * c + 2] = v.z;
          x[4 * c + 3] = v.w;
        }
        tmem_st_x32(lane_addr + C::kColA + 64 * gw + 32 * b, x);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(C::kBarAFull));
      slot += 2 + 2 * (w.s.tb - w.s.ta);
      return true;
    };
    bool have = w.next(p), ok = true;
    if (!KV && have) ok = load_pair();
    while (ok && have) {
      const PackedSegment s = w.s;
      int g = 0;
      // dq: this row's token, lse and Delta.  dk, dv: this row's key
      const int tok = KV ? s.rt * 128 + row : s.rt * p.tq + row / p.G;
      const bool valid = tok < s.r.n && row < sub_rows;
      const int qhead = s.h * p.G + row % p.G;
      const size_t hr = (size_t)qhead * p.T + s.r.first + tok;
      const float lrow = !KV && valid ? __ldcg(lse2 + hr) : 0.f, drow = !KV && valid ? __ldcg(delta + hr) : 0.f;
      for (int t = s.ta; t < s.tb; ++t, ++u) {
        const int row0 = tile_at(s, t, g);
        const float *ls = vec + (u % C::kVecs) * 256 + 64 * gw, *dl = ls + 128;
        // visible columns [c0, c1) of this thread's 64
        int c0 = 0, c1 = 64;
        if (KV) {
          if (p.causal) c0 = tok - row0 - 64 * gw;             // tokens at or behind the key
        } else {
          c1 = (p.causal ? min(tok, s.r.n - 1) + 1 : s.r.n) - row0 - 64 * gw;
        }
        if (!uwait(bar(C::kBarS + gw), u & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float pv[64];
        {
          uint32_t r[2][32];
          tmem_ld_x32(s_addr, r[0]);
          tmem_ld_x32(s_addr + 32, r[1]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; ++c) pv[c] = __uint_as_float(r[c >> 5][c & 31]);
        }
        if (!KV) {
          tc_fence_before();
          mbar_arrive(bar(C::kBarP + gw));          // S may be overwritten
        }
        if (KV) {
          // (the slot's arrival also hands over lse and Delta)
          if (!uwait(bar(C::kBarFull + (2 * u) % kStages), (2 * u / kStages) & 1)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4 *>(ls + c);
            pv[c] = ex2_approx(fmaf(pv[c], sl2, -l4.x));
            pv[c + 1] = ex2_approx(fmaf(pv[c + 1], sl2, -l4.y));
            pv[c + 2] = ex2_approx(fmaf(pv[c + 2], sl2, -l4.z));
            pv[c + 3] = ex2_approx(fmaf(pv[c + 3], sl2, -l4.w));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) pv[c] = ex2_approx(fmaf(pv[c], sl2, -lrow));
        }
        if (__any_sync(0xffffffffu, c0 > 0 || c1 < 64)) {
#pragma unroll
          for (int c = 0; c < 64; ++c) pv[c] = c >= c0 && c < c1 ? pv[c] : 0.f;
        }
        if (KV) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(pv[2 * c], pv[2 * c + 1]);
          tmem_st_x32(s_addr, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(C::kBarP + gw));
        }
        if (!uwait(bar(C::kBarDP + gw), u & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        {
          uint32_t r[2][32], pk[32];
          tmem_ld_x32(dp_addr, r[0]);
          tmem_ld_x32(dp_addr + 32, r[1]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            float4 d4 = make_float4(drow, drow, drow, drow);
            if (KV) d4 = *reinterpret_cast<const float4 *>(dl + c);
            pk[c / 2] = pack_bf16x2(pv[c] * (__uint_as_float(r[c >> 5][c & 31]) - d4.x),
                                    pv[c + 1] * (__uint_as_float(r[c >> 5][(c & 31) + 1]) - d4.y));
            pk[c / 2 + 1] = pack_bf16x2(pv[c + 2] * (__uint_as_float(r[c >> 5][(c & 31) + 2]) - d4.z),
                                        pv[c + 3] * (__uint_as_float(r[c >> 5][(c & 31) + 3]) - d4.w));
          }
          tmem_st_x32(dp_addr, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar(C::kBarZ + gw));
      }
      if (!ok) break;
      // ---- epilogue: dq = s dQ (half of the columns a warpgroup); dk = s dK, dv = dV (one each) ----
      if (aborted() || !uwait(bar(C::kBarAcc), seg & 1)) {
        ok = false;
        break;
      }
      ++seg;
      tc_fence_after();
      // every product of the unit is done: the next one's pair may take TMEM, and its S and dP run
      // while this unit's rows are stored
      have = w.next(p);
      if (!KV && have && !load_pair()) {
        ok = false;
        break;
      }
      const bool whole = s.whole();
      constexpr int kCols = KV ? D : D / 2;
      const int col0 = KV ? 0 : gw * (D / 2);
      const float f = KV && gw == 1 ? 1.f : scale;
      const uint32_t acc = lane_addr + C::kColAcc + (KV ? D * gw : col0);
      // KV: warpgroup 0 holds dK (accumulator 0), warpgroup 1 dV (accumulator 1)
      const bool second = KV && gw == 1;
      __nv_bfloat16 *dst = second ? out1 : out0;
      const long long to = (KV ? s.h : qhead) * (second ? out1_head : out0_head) +
                           (long long)(s.r.first + tok) * (second ? out1_row : out0_row) + col0;
      const int nrow = __popc(__ballot_sync(0xffffffffu, valid));   // the warp's first rows
      float4 *ps = reinterpret_cast<float4 *>(part) +
                   ((size_t)blockIdx.x * 2 + s.slot()) * ((KV ? 2 : 1) * 128 * (D / 4)) +
                   (KV ? gw * 128 * (D / 4) : 0);
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        uint32_t r[32];
        tmem_ld_x32(acc + 32 * c, r);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = f * __uint_as_float(r[k]);
        if (whole) {
          store_rows<4>(stage, lane, nrow, to + 32 * c, dst, [&](int k) {
            return make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                              pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
          });
        } else if (valid) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            ps[(size_t)(col0 / 4 + 8 * c + k) * 128 + row] =
                make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(C::kBarAccFree));
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

struct PackedSums {
  PackedProblem p;
  const PackedCut *cuts[2];      // of dq, and of dk and dv
  const float *part[2];
  __nv_bfloat16 *out[3];         // dq, dk, dv
  long long head[3], row[3];
  int clear;
};

// Joins the partial sums of the unit that CTA blockIdx.x's range cuts, in
// ascending CTA order.  blockIdx.z: dq, dk or dv.
template <int D> __global__ void __launch_bounds__(128) packed_sum_kernel(const PackedSums a) {
  sm100::allow_next_launch();
  sm100::wait_for_launches_before();
  const int z = blockIdx.z, kv = z > 0;
  const PackedProblem &p = a.p;
  __nv_bfloat16 *out = a.out[z];
  const long long hs = a.head[z], rs = a.row[z];
  if (a.clear)
    clear_unused<D>(p, kv ? p.Hkv : p.Hq, out, hs, rs,
                    ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                    (long long)gridDim.x * gridDim.y * blockDim.x);
  const PackedCut cut = packed_cut_at(a.cuts[kv], blockIdx.x);
  if (!cut.valid) return;
  int bad = 0;
  const PackedRequest r = packed_request(p, cut.b, bad);
  const int per = kv ? 128 : p.tq, g = kv ? 1 : p.G, tok0 = cut.rt * per;
  const int rows = min(r.n - tok0, per) * g;
  const int c0 = blockIdx.x, n = cut.last - c0 + 1;
  const size_t kSlot = (size_t)(kv ? 2 : 1) * 128 * (D / 4);
  const float4 *base = reinterpret_cast<const float4 *>(a.part[kv]) + (z == 2 ? 128 * (D / 4) : 0);
  for (int e = blockIdx.y * blockDim.x + threadIdx.x; e < rows * (D / 16); e += gridDim.y * blockDim.x) {
    const int row = e % rows, c16 = e / rows;
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 4) {
      float4 x[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = min(i0 + k, n - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[k][j] = __ldcg(base + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * kSlot + (size_t)(4 * c16 + j) * 128 + row);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + k >= n) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[4 * j] += x[k][j].x;
          acc[4 * j + 1] += x[k][j].y;
          acc[4 * j + 2] += x[k][j].z;
          acc[4 * j + 3] += x[k][j].w;
        }
      }
    }
    const long long at = (cut.h * g + row % g) * hs + (long long)(r.first + tok0 + row / g) * rs + 16 * c16;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      reinterpret_cast<uint4 *>(out + at)[j] =
          make_uint4(pack_bf16x2(acc[8 * j], acc[8 * j + 1]), pack_bf16x2(acc[8 * j + 2], acc[8 * j + 3]),
                     pack_bf16x2(acc[8 * j + 4], acc[8 * j + 5]), pack_bf16x2(acc[8 * j + 6], acc[8 * j + 7]));
  }
}

}  // namespace pisa
