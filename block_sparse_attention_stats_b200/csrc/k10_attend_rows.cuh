// Attention of a few packed rows (decoding: one or a few new tokens a request)
// over a paged key/value cache.
//
// For row r of a unit (token i of n new ones of a request with m positions):
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(s q_r . k_j),  j <= m - n + i
// in one pass over the keys with the running maximum and sum of the softmax.
// Bound: HBM.  Every live page is read once; at R = 16 rows a key costs 2 D
// bytes x 2 and 4 D R flops, 16 flops a byte, far under the tensor cores' 240.
// So the kernel is built around the loads: one warp brings pages by TMA into a
// ring that holds most of an SM's shared memory (three 64 KB tiles of 128 keys
// at D = 128), eight warps work on the tiles, and the key range of the whole
// batch is cut evenly over the SMs (packed_schedule.cuh), so one long request
// and a batch of short ones both fill the machine.
//
// Per tile, warp w forms S for keys 16 w .. 16 w + 15 (mma.sync m16n8k16; the
// rows are 16 at least, which a 128-row tcgen05 product would fill to an eighth,
// and its accumulator would cross TMEM for every key), the warps agree on the
// row maxima and lay down P (16-bit) through shared memory, and warp w adds
// P V for its own D / 8 output columns, so the output needs no merge of warps.
// A tile takes the warps 1600 cycles, less than its 64 KB take to arrive when all
// SMs load (2900); Q comes with a unit's first tile and stays in registers.
// Measured (graph replays): 48 requests of 1 to 8000 keys, 40 / 8 heads, d = 128,
// pages of 64 (957 MB) 151 us, 6.35 TB/s or 0.97 of a plain copy's rate; two requests of
// 131072 and 90001 keys, 32 / 4 heads (453 MB) 78 us, of which the join of the parts and
// the start are 7; one request of 777 keys, 8 heads, d = 64: 9.0 us, two launches; 300
// requests of 1 to 300 keys (185 MB) 61 us, where a unit's start and end (a tile's time)
// count as much as its tiles.
#pragma once

#include "packed_schedule.cuh"
#include "packed_primitives.cuh"

namespace pisa {

template <int D, int R> struct RowsCfg {
  static constexpr int kConsumers = 256, kThreads = 288;
  static constexpr int kTileBytes = kKeyTile * D * 2;       // K or V of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kQBytes = R * D * 2, kPBytes = R * kKeyTile * 2;
  static constexpr int kFixed = kPBytes + 8 * R * 4 + 1024;
  static constexpr int kMaxStages = (227 * 1024 - 1024 - kFixed) / (kStageBytes + kQBytes);
  static constexpr int kStages = kMaxStages < 6 ? kMaxStages : 6;
  static constexpr int kOffQ = kStages * kStageBytes;       // Q of a unit, with its first tile's stage
  static constexpr int kOffP = kOffQ + kStages * kQBytes;
  static constexpr int kOffRed = kOffP + kPBytes;           // [8][R] f32
  static constexpr int kOffMisc = kOffRed + 8 * R * 4;      // barriers, schedule
  static constexpr int kSmem = kOffMisc + 1024 + 1024;      // + alignment slack
  static_assert(kStages >= 2 && kSmem <= 227 * 1024, "shared memory");
};

// Pages of a key/value cache as the loads see them.
struct PagedKV {
  const int32_t *table;      // [B, width]
  int width, page_size, num_pages;
};

// Issues the copies of one tile's pages: the keys key0 .. key0 + 127 of request b
// that lie below kv.  All 32 lanes; lane i brings the i-th page, whose number
// `page` it already holds.  A copy brings `rows` = min(page_size, 128) keys; a page
// number outside the cache reads as zeros (the copy's own bounds check).
// expect_pages: announces them, and `more` bytes on the same barrier; returns their number
template <int D>
__device__ __forceinline__ int expect_pages(uint32_t bar, int key0, int kv, int rows, int tensors, int more,
                                            int lane) {
  const int live = kv - key0 <= 0 ? 0 : min((kv - key0 + rows - 1) / rows, kKeyTile / rows);
  if (lane == 0) sm100::mbar_expect_tx(bar, (uint32_t)(live * rows * D * 2 * tensors + more));
  __syncwarp();
  return live;
}
// K or V: 64-column boxes of all 128 keys one after the other, as tcgen05 reads them,
// or (`whole`) page by page
template <int D>
__device__ __forceinline__ void issue_pages(const CUtensorMap *m, uint32_t bar, uint32_t dst, int key0, int kv,
                                            int head, int page, int rows, int page_size, bool whole, int lane) {
  if (lane < expect_pages<D>(bar, key0, kv, rows, 1, 0, lane)) {
    const int row = (key0 + lane * rows) % page_size;
    if (whole)
      sm100::tma_load_5d(dst + lane * rows * D * 2, m, bar, 0, row, 0, head, page);
    else
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        sm100::tma_load_5d(dst + b * kKeyTile * 128 + lane * rows * 128, m, bar, 0, row, b, head, page);
  }
  __syncwarp();
}
// K and V page by page, the 64-column boxes of a page together: one copy each.
// Small copies are what small pages wait for: 48 requests of 4000 keys in pages
// of 16 took 163 us with a copy a box, 138 with these.
template <int D>
__device__ __forceinline__ void issue_pages_whole(const CUtensorMap *mk, const CUtensorMap *mv, uint32_t bar,
                                                  uint32_t dst, uint32_t v_off, int key0, int kv, int head,
                                                  int page, int rows, int page_size, int more, int lane) {
  if (lane < expect_pages<D>(bar, key0, kv, rows, 2, more, lane)) {
    const int row = (key0 + lane * rows) % page_size;
    const uint32_t d = dst + lane * rows * D * 2;
    sm100::tma_load_5d(d, mk, bar, 0, row, 0, head, page);
    sm100::tma_load_5d(d + v_off, mv, bar, 0, row, 0, head, page);
  }
  __syncwarp();
}
// Byte offset of 16-byte chunk c of key `row` in a tile brought page by page
// (1 << lg keys a page)
template <int D> __device__ __forceinline__ uint32_t page_chunk(int row, int c, int lg) {
  const int in = row & ((1 << lg) - 1);
  return (uint32_t)(((row >> lg) << lg) * D * 2 + ((((c >> 3) << lg) + in) << 7) + (((c & 7) ^ (row & 7)) << 4));
}

// Page number of lane's page of the tile at key0, or -1 where there is none.
__device__ __forceinline__ int lane_page(const PagedKV &c, int b, int key0, int kv, int rows, int lane) {
  const int key = key0 + lane * rows;
  if (lane >= kKeyTile / rows || key >= kv) return -1;
  const int page = sm100::ld_int(c.table + (size_t)b * c.width + key / c.page_size);
  if (page < 0 || page >= c.num_pages) {
    report_device_error(kDevErrRange);
    return -1;
  }
  return page;
}

template <typename T> __device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4],
                                                                uint32_t b0, uint32_t b1) {
  if constexpr (Half16<T>::kBf16)
    mma_bf16_16816(c, a, b0, b1);
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <typename T, int D, int R>
__global__ void __launch_bounds__(RowsCfg<D, R>::kThreads, 1)
    attend_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PackedProblem p,
                       const PagedKV cache, float scale, const PackedOut o, PackedCut *__restrict__ cuts,
                       float *__restrict__ part) {
  using C = RowsCfg<D, R>;
  using namespace sm100;
  constexpr int RT = R / 16;            // m16 tiles
  constexpr int NT = D / 64;            // n8 tiles of a warp's output columns
  constexpr int kStep = NT == 2 ? 1 : 2;   // 16 keys a step of P V
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char *smem = smem_raw + (sbase - raw);
  const uint32_t bars = sbase + C::kOffMisc;                       // full[s], empty[s]
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (C::kStages + s); };
  PackedStart *start = reinterpret_cast<PackedStart *>(smem + C::kOffMisc + 128);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 256);
  long long *wsum = reinterpret_cast<long long *>(smem + C::kOffMisc + 384);   // 9 warps
  float *red = reinterpret_cast<float *>(smem + C::kOffRed);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 8);
    }
    fence_mbar_init();
    *abort = 0;
  }
  if (tid == 32) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  wait_for_launches_before();
  if (tid == 0) cuts[blockIdx.x].valid = 0;
  packed_locate<RowCost>(p, blockIdx.x, gridDim.x, tid, C::kThreads, wsum, start);
  PackedWalk<RowCost> w;
  w.begin(p, *start);
  const int page_rows = min(cache.page_size, kKeyTile), lg = 31 - __clz(page_rows);

  if (warp == 8) {
    // ======================= page loads =======================================
    int it = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      const PackedSegment &s = w.s;
      int page = lane_page(cache, s.b, s.ta * kKeyTile, s.r.kv, page_rows, lane);
      for (int t = s.ta; t < s.tb; ++t, ++it) {
        const int st = it % C::kStages;
        if (it >= C::kStages &&
            !__all_sync(0xffffffffu, mbar_wait(empty(st), ((it / C::kStages) - 1) & 1))) {
          ok = false;
          break;
        }
        if (__any_sync(0xffffffffu, *abort != 0)) {
          ok = false;
          break;
        }
        const bool first = t == s.ta;   // Q comes with it
        issue_pages_whole<D>(&tm_k, &tm_v, full(st), sbase + st * C::kStageBytes, C::kTileBytes,
                             t * kKeyTile, s.r.kv, s.h, page, page_rows, cache.page_size,
                             first ? p.tq * p.G * D * 2 : 0, lane);
        if (first && elect_one()) {
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
            tma_load_4d(sbase + C::kOffQ + st * C::kQBytes + b * R * 128, &tm_q, full(st), 64 * b, 0,
                        s.r.first + s.rt * p.tq, s.h);
        }
        __syncwarp();
        page = t + 1 < s.tb
                   ? lane_page(cache, s.b, (t + 1) * kKeyTile, s.r.kv, page_rows, lane)
                   : -1;
      }
    }
    if (!ok) *abort = 1;
    // copies in flight land before the CTA exits, whatever the consumers do
    for (int i = max(it - C::kStages, 0); i < it; ++i) mbar_wait(full(i % C::kStages), (i / C::kStages) & 1);
    return;
  }

  // ======================= the eight working warps ============================
  const float sl2 = scale * kLog2e;
  // weights are at most 1 here (the maximum is of all keys so far), so all of the type's room is theirs:
  // f16 weights keep their precision down to 2^-29 of the largest, and vanish below 2^-40
  constexpr float kLift = (float)Half16<T>::kRoom, kLower = 1.f / (float)(1 << Half16<T>::kRoom);
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  int it = 0;
  while (w.next(p)) {
    const PackedSegment s = w.s;
    const int tok0 = s.rt * p.tq, rows = min(s.r.n - tok0, p.tq) * p.G;
    // Q of the unit as product operands, read once (rows past the tile's hold anything: their
    // scores are masked, and a product's rows do not mix)
    uint32_t qa[RT][D / 16][4];
    // keys each of this thread's rows sees: positions below lim
    int lim[RT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = 16 * i + g + 8 * x;
        lim[i][x] = row >= rows ? 0 : max(min(s.r.past + tok0 + row / p.G + 1, s.r.kv), 0);
      }
    float m[RT][2], l[RT][2], acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][n][x] = 0.f;
    }
    consumers_sync();   // every warp has read the last unit's sums from `red`
    for (int t = s.ta; t < s.tb; ++t, ++it) {
      const int st = it % C::kStages;
      // a warp that gives up goes on through the same barriers, so that no other waits for it;
      // its results are not used: the error word says so
      if (!__any_sync(0xffffffffu, *abort != 0) &&
          !__all_sync(0xffffffffu, mbar_wait(full(st), (it / C::kStages) & 1)))
        *abort = 1;
      const uint32_t ks = sbase + st * C::kStageBytes, vs = ks + C::kTileBytes;
      if (t == s.ta) {
        const uint32_t qs = sbase + C::kOffQ + st * C::kQBytes;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int row = 16 * i + (lane & 15), c = 2 * k + (lane >> 4);
            ldmatrix_x4(qs + (c >> 3) * R * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4), qa[i][k][0], qa[i][k][1],
                        qa[i][k][2], qa[i][k][3]);
          }
      }
      const int key0 = t * kKeyTile;
      const int live = s.r.kv - key0;    // keys of the tile that exist
      if (live < kKeyTile) {
        // the rest of V may hold anything: zero, so that 0 x Inf or NaN never reaches a sum (up to
        // the end of a step of the product: those behind are not read)
        const int z0 = max(live, 0), z1 = (z0 + 16 * kStep - 1) & ~(16 * kStep - 1);
        for (int e = tid; e < (z1 - z0) * (D / 8); e += C::kConsumers) {
          const int row = z0 + e / (D / 8), ch = e % (D / 8);
          *reinterpret_cast<uint4 *>(smem + st * C::kStageBytes + C::kTileBytes + page_chunk<D>(row, ch, lg)) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
      }
      // S = Q K^T for this warp's 16 keys
      float sc[RT][2][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[i][n][x] = 0.f;
      if (16 * warp < live)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        const int krow = 16 * warp + ((lane >> 4) << 3) + (lane & 7), kc = 2 * k + ((lane >> 3) & 1);
        ldmatrix_x4(ks + page_chunk<D>(krow, kc, lg), b[0], b[1], b[2], b[3]);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          mma_16816<T>(sc[i][0], qa[i][k], b[0], b[1]);
          mma_16816<T>(sc[i][1], qa[i][k], b[2], b[3]);
        }
      }
      // scores in units of log2; the row maximum of these 16 keys
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = key0 + 16 * warp + 8 * n + c2 + y;
              float &v = sc[i][n][2 * x + y];
              v = key < lim[i][x] ? v * sl2 : -INFINITY;
              mx = fmaxf(mx, v);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          if ((lane & 3) == 0) red[warp * R + 16 * i + g + 8 * x] = mx;
        }
      consumers_sync();
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 16 * i + g + 8 * x;
          float mt = red[row];
#pragma unroll
          for (int j = 1; j < 8; ++j) mt = fmaxf(mt, red[j * R + row]);
          const float mn = fmaxf(m[i][x], mt);
          const float base = mn == -INFINITY ? 0.f : mn;   // no key seen yet: every weight is zero
          const float f = ex2_approx(m[i][x] - base);
          m[i][x] = mn;
          l[i][x] *= f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[i][n][2 * x] *= f;
            acc[i][n][2 * x + 1] *= f;
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            // P is rounded to 16 bits for the product (the tensor cores take no more); the sum
            // keeps the float32 weights, so only the weights' own rounding enters the output
            float z0 = sc[i][n][2 * x] - base, z1 = sc[i][n][2 * x + 1] - base;
            if constexpr (Half16<T>::kRoom != 0) {
              z0 += kLift;
              z1 += kLift;
            }
            const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
            l[i][x] += p0 + p1;
            *reinterpret_cast<uint32_t *>(smem + C::kOffP +
                                          SwizzledTile<kKeyTile>::offset(row, 16 * warp + 8 * n + c2)) =
                Half16<T>::pack(p0, p1);
          }
        }
      consumers_sync();
      // O += P V for this warp's D / 8 columns, 16 kStep keys at a time
      auto add = [&](int k) {
        uint32_t b[4];
        if (NT == 2) {
          const int vrow = 16 * k + (lane & 15), vc = 2 * warp + (lane >> 4);
          ldmatrix_x4_trans(vs + page_chunk<D>(vrow, vc, lg), b[0], b[1], b[2], b[3]);
        } else {
          const int vrow = 16 * k + lane;
          ldmatrix_x4_trans(vs + page_chunk<D>(vrow, warp, lg), b[0], b[1], b[2], b[3]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          uint32_t a[4];
          const uint32_t prow = 16 * i + (lane & 15);
          ldmatrix_x4(sbase + C::kOffP + SwizzledTile<kKeyTile>::offset(prow, 16 * k + (lane >> 4) * 8),
                      a[0], a[1], a[2], a[3]);
          mma_16816<T>(acc[i][0], a, b[0], b[1]);
          if constexpr (NT == 2) {
            mma_16816<T>(acc[i][1], a, b[2], b[3]);
          } else {
            ldmatrix_x4(sbase + C::kOffP +
                            SwizzledTile<kKeyTile>::offset(prow, 16 * (k + 1) + (lane >> 4) * 8),
                        a[0], a[1], a[2], a[3]);
            mma_16816<T>(acc[i][0], a, b[2], b[3]);
          }
        }
      };
      if (live >= kKeyTile) {
#pragma unroll
        for (int k = 0; k < kKeyTile / 16; k += kStep) add(k);
      } else {
#pragma unroll 1
        for (int k = 0; 16 * k < live; k += kStep) add(k);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }
    // l over the 4 lanes of a row and the 8 warps
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[i][x] += __shfl_xor_sync(0xffffffffu, l[i][x], 1);
        l[i][x] += __shfl_xor_sync(0xffffffffu, l[i][x], 2);
        if ((lane & 3) == 0) red[warp * R + 16 * i + g + 8 * x] = l[i][x];
      }
    consumers_sync();
    float *slot = part + ((size_t)blockIdx.x * 2 + s.slot()) * packed_slot_floats<D>(R);
    const bool whole = s.whole();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = 16 * i + g + 8 * x;
        float ls = red[row];
#pragma unroll
        for (int j = 1; j < 8; ++j) ls += red[j * R + row];
        if (row >= rows) continue;
        const bool head_lane = warp == 0 && (lane & 3) == 0;
        if (whole) {
          const float inv = ls > 0.f ? 1.f / ls : ls == 0.f ? 0.f : ls;
          const int token = s.r.first + tok0 + row / p.G, head = s.h * p.G + row % p.G;
          T *dst = reinterpret_cast<T *>(o.out) + head * o.head + token * o.row;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<uint32_t *>(dst + warp * (D / 8) + 8 * n + c2) =
                Half16<T>::pack(acc[i][n][2 * x] * inv, acc[i][n][2 * x + 1] * inv);
          if (head_lane && o.lse)
            o.lse[(size_t)head * p.T + token] =
                ls == 0.f ? -INFINITY : (m[i][x] + log2f(ls * kLower)) * 0.6931471805599453f;
        } else {
          // (a power of two: exact)
          if (head_lane) {
            slot[row] = m[i][x];
            slot[R + row] = ls * kLower;
            slot[2 * R + row] = ls * kLower;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int col = warp * (D / 8) + 8 * n + c2;
            *reinterpret_cast<float2 *>(slot + 3 * R + ((size_t)(col >> 2) * R + row) * 4 + (col & 3)) =
                make_float2(acc[i][n][2 * x] * kLower, acc[i][n][2 * x + 1] * kLower);
          }
        }
      }
    if (!whole && s.ta == 0 && tid == 0) cuts[blockIdx.x] = packed_cut(p, *start, s, gridDim.x);
  }
}

}  // namespace pisa
