// How the kernels of packed rows and paged caches share out their work.
//
// A batch is B sequences of new tokens, packed: sequence b holds rows cu[b] ..
// cu[b+1] - 1 of q, and its tokens are the last n of its kv positions (for
// packed prompts kv = n).  A unit is (sequence, row tile, key head): tq tokens
// times the G query heads of the key head, G rows a token, against the key
// tiles of 128 positions that the tile's last token sees.  All units' key
// tiles, laid end to end, are cut into as many equal ranges as there are CTAs,
// so every CTA gets the same number of tiles whatever the lengths are.  Nothing
// is read on the host: the cut depends on lengths in device memory alone, and
// the grid on the device alone, so a captured launch serves any lengths.
// A unit counts unit_cost tiles more than it has, for what its start and its end
// take: without, a CTA that got many short units ran twice as long as the others.
// A cut that would fall into these is moved to the unit's start.
// A unit inside one range is written by its CTA.  A unit cut by a range's end
// leaves float32 partial sums, and combine_kernel joins them in ascending CTA
// order (no atomics: the same inputs give the same bits).
#pragma once

#include <math.h>

#include "packed_primitives.cuh"

namespace pisa {

constexpr int kKeyTile = 128;   // key positions of a tile

struct PackedProblem {
  const int32_t *cu;        // [B + 1] first row of each sequence
  const int32_t *kv_lens;   // [B] key positions, or nullptr: the sequences' own lengths
  int B, T;                 // sequences, rows of q
  int Hq, Hkv, G;           // query heads, key heads, Hq / Hkv
  int causal;
  int tq;                   // tokens of a row tile
  int max_kv;               // most key positions a sequence can have (table width x page size)
  int min_tiles;            // no range is cut shorter than this
  int unit_cost;            // what a unit takes beside its tiles, in tiles
};

struct PackedRequest {
  int first, n, kv, past;   // first row, tokens, key positions, positions before the first token
};

// Offsets and lengths are device data: whatever they hold, rows stay inside
// [0, T) and positions inside [0, max_kv].
__device__ __forceinline__ PackedRequest packed_request(const PackedProblem &p, int b) {
  PackedRequest r;
  const int lo = sm100::ld_int(p.cu + b), hi = sm100::ld_int(p.cu + b + 1);
  r.first = min(max(lo, 0), p.T);
  r.n = max(min(hi, p.T) - r.first, 0);
  r.kv = r.n;
  if (p.kv_lens) r.kv = min(max(sm100::ld_int(p.kv_lens + b), 0), p.max_kv);
  r.past = r.kv - r.n;
  return r;
}

__device__ __forceinline__ bool packed_request_malformed(const PackedProblem &p, int b) {
  const int lo = sm100::ld_int(p.cu + b), hi = sm100::ld_int(p.cu + b + 1);
  bool bad = lo < 0 || hi < lo || hi > p.T;
  if (p.kv_lens) {
    const int kv = sm100::ld_int(p.kv_lens + b);
    bad = bad || kv < 0 || kv > p.max_kv;
  }
  return bad;
}

// sum of floor((a i + b) / m) for i = 0 .. n - 1 (the Euclidean recursion on
// the lattice points under a line); a, m <= 2^8, b < 2^31, a n < 2^31
__host__ __device__ inline long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long s = 0;
  while (n) {
    s += (long long)(a / m) * ((long long)n * (n - 1) / 2) + (long long)(b / m) * n;
    a %= m;
    b %= m;
    const unsigned y = a * n + b;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
    if (m == 0) break;
  }
  return s;
}

// What a unit costs, in tiles.  RowCost<KT>: a unit is a row tile of tq tokens,
// its tiles are the KT-key tiles that the last token sees (at least one: a row
// without keys is still written).  KeyCost: a unit is a tile of 128 keys of a
// sequence over itself, its tiles are the 128-token tiles of every query head
// that see it.  before(..., rt): the tiles of units 0 .. rt - 1 of a key head.
template <int KT> struct RowCost {
  static __host__ __device__ int units(const PackedProblem &p, int n) { return n > 0 ? (n - 1) / p.tq + 1 : 0; }
  static __host__ __device__ int tiles(const PackedProblem &p, int n, int kv, int tq, int rt) {
    const long long past = kv > n ? kv - n : 0;
    const long long upto = (long long)(rt + 1) * tq;
    const long long end = p.causal ? past + (n < upto ? n : upto) : (kv > 1 ? kv : 1);
    return (int)((end + KT - 1) / KT);
  }
  static __host__ __device__ int tiles(const PackedProblem &p, int n, int kv, int rt) {
    return tiles(p, n, kv, p.tq, rt);
  }
  static __host__ __device__ long long before(const PackedProblem &p, int n, int kv, int rt) {
    const int R = units(p, n);
    if (rt <= 0 || R == 0) return 0;
    if (!p.causal) return (long long)rt * tiles(p, n, kv, 0);
    const int past = kv > n ? kv - n : 0;
    const int whole = rt < R ? rt : R - 1;   // units of tq tokens
    long long s = floor_sum((unsigned)whole, KT, (unsigned)p.tq, (unsigned)past + (unsigned)p.tq + KT - 1);
    if (rt >= R) s += tiles(p, n, kv, R - 1);
    return s;
  }
};
struct KeyCost {
  static __host__ __device__ int units(const PackedProblem &, int n) { return (n + kKeyTile - 1) / kKeyTile; }
  static __host__ __device__ int tiles(const PackedProblem &p, int n, int, int rt) {
    return p.G * (units(p, n) - (p.causal ? rt : 0));
  }
  static __host__ __device__ long long before(const PackedProblem &p, int n, int, int rt) {
    const long long N = units(p, n);
    return p.G * (rt * N - (p.causal ? (long long)rt * (rt - 1) / 2 : 0));
  }
};

// what all key heads' units before row tile rt count
template <class Cost>
__host__ __device__ __forceinline__ long long packed_before(const PackedProblem &p, const PackedRequest &r, int rt) {
  return p.Hkv * (Cost::before(p, r.n, r.kv, rt) + (long long)rt * p.unit_cost);
}

template <class Cost>
__device__ __forceinline__ long long packed_cost(const PackedProblem &p, const PackedRequest &r) {
  return packed_before<Cost>(p, r, Cost::units(p, r.n));
}

struct PackedStart {
  long long total;    // key tiles of the whole problem
  long long w0, w1;   // this CTA's range
  long long rem;      // w0's distance from the first tile of sequence b
  int b, ctas;        // sequence of w0; CTAs that have a range
};

__host__ __device__ __forceinline__ long long packed_range_start(long long total, int ctas, int c) {
  return total * c / ctas;
}

// One call by all `threads` threads of a CTA (a multiple of 32, at most 512):
// fills *out (shared memory).  Contains two CTA barriers.
template <class Cost>
__device__ __forceinline__ void packed_locate(const PackedProblem &p, int cta, int grid, int tid,
                                              int threads, long long *warp_sum, PackedStart *out) {
  const int per = (p.B + threads - 1) / threads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long own = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    own += packed_cost<Cost>(p, packed_request(p, b));
    bad = bad || packed_request_malformed(p, b);
  }
  if (bad && cta == 0) report_device_error(kDevErrRange);
  const int lane = tid & 31, warp = tid >> 5;
  long long incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - own, total = 0;
  for (int w = 0; w < threads / 32; ++w) {
    const long long s = warp_sum[w];
    if (w < warp) before += s;
    total += s;
  }
  const long long want = total / p.min_tiles;
  const int ctas = want < 1 ? 1 : want < grid ? (int)want : grid;
  const long long w0 = cta < ctas ? packed_range_start(total, ctas, cta) : total;
  const long long w1 = cta < ctas ? packed_range_start(total, ctas, cta + 1) : total;
  if (tid == 0 && w0 >= total) {
    out->total = total;
    out->w0 = out->w1 = total;
    out->rem = 0;
    out->b = p.B;
    out->ctas = ctas;
  }
  if (own > 0 && w0 >= before && w0 < before + own) {
    long long rem = w0 - before;
    int b = b0;
    for (;; ++b) {
      const long long c = packed_cost<Cost>(p, packed_request(p, b));
      if (rem < c) break;
      rem -= c;
    }
    out->total = total;
    out->w0 = w0;
    out->w1 = w1;
    out->rem = rem;
    out->b = b;
    out->ctas = ctas;
  }
  __syncthreads();
}

// The part [ta, tb) of one unit's key tiles [0, nt)
struct PackedSegment {
  PackedRequest r;
  int b, rt, h, nt, ta, tb;
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == nt; }
  // partial slot of the CTA: 0 holds a unit begun by an earlier CTA, 1 one that goes on in the next
  __device__ __forceinline__ int slot() const { return ta != 0 ? 0 : 1; }
};

// Walks a CTA's range segment by segment.  Every warp keeps its own (all lanes
// hold the same values), so no role waits for another to learn what comes next.
template <class Cost> struct PackedWalk {
  PackedSegment s;
  long long left;   // of the range, counted like the units
  int at;           // where the next segment starts in its unit, counted like the unit
  static constexpr int kDone = -1;
  // all 32 lanes of a converged warp
  __device__ __forceinline__ void begin(const PackedProblem &p, const PackedStart &st) {
    left = st.w1 - st.w0;
    at = 0;
    s.b = st.b;
    s.rt = 0;
    s.h = 0;
    if (left <= 0) return;
    s.r = packed_request(p, s.b);
    // last row tile that starts at or before rem: 32-way search
    int lo = 0, hi = Cost::units(p, s.r.n);   // answer in [lo, hi)
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, x = lo + lane * step;
      const bool ok = x < hi && packed_before<Cost>(p, s.r, x) <= st.rem;
      const unsigned m = __ballot_sync(0xffffffffu, ok);   // lane 0 always holds
      const int last = 31 - __clz(m);
      lo += last * step;
      hi = min(hi, lo + step);
    }
    s.rt = lo;
    s.nt = Cost::tiles(p, s.r.n, s.r.kv, lo);
    const long long in = st.rem - packed_before<Cost>(p, s.r, lo);
    s.h = (int)(in / (s.nt + p.unit_cost));
    at = (int)(in % (s.nt + p.unit_cost));
  }
  __device__ __forceinline__ bool next(const PackedProblem &p) {
    if (left <= 0) return false;
    if (at == kDone) {
      at = 0;
      if (++s.h == p.Hkv) {
        s.h = 0;
        if (++s.rt >= Cost::units(p, s.r.n)) {
          s.rt = 0;
          do {
            if (++s.b >= p.B) return false;   // cannot happen while tiles are left
            s.r = packed_request(p, s.b);
          } while (s.r.n == 0);
        }
        s.nt = Cost::tiles(p, s.r.n, s.r.kv, s.rt);
      }
    }
    const int all = s.nt + p.unit_cost;
    const int end = (int)(left < all - at ? at + left : all);
    left -= end - at;
    s.ta = max(at - p.unit_cost, 0);
    s.tb = max(end - p.unit_cost, 0);
    at = end == all ? kDone : end;
    return s.tb > s.ta;   // else the range ends before the unit's first tile: the next CTA has it all
  }
};

// What a CTA says about the unit that its range's end cuts (slot 1)
struct PackedCut {
  int valid, b, rt, h, last;   // last: the CTA that holds the unit's last tile
};

__device__ __forceinline__ PackedCut packed_cut_at(const PackedCut *cuts, int c) {
  const int *x = reinterpret_cast<const int *>(cuts + c);
  return PackedCut{__ldcg(x), __ldcg(x + 1), __ldcg(x + 2), __ldcg(x + 3), __ldcg(x + 4)};
}

__device__ __forceinline__ PackedCut packed_cut(const PackedStart &st, const PackedSegment &s) {
  PackedCut c;
  c.valid = 1;
  c.b = s.b;
  c.rt = s.rt;
  c.h = s.h;
  const long long end = st.w1 + (s.nt - s.tb) - 1;   // the unit's last tile
  c.last = (int)(((end + 1) * st.ctas - 1) / st.total);
  return c;
}

// partial slot: R rows of m and l, then the unnormalised output as [D / 4][R] float4
template <int D> __host__ __device__ constexpr size_t packed_slot_floats(int R) {
  return (size_t)R * (D + 2);
}

template <typename T> struct Half16;
template <> struct Half16<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
};
template <> struct Half16<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<__half2 *>(&x));
  }
};

// A warp's 32 rows of CH 16-byte chunks (lane r holds row r: chunk(k)) to global
// memory, whole rows side by side, by way of 512 CH bytes of shared memory: a
// store of 16 bytes a row would touch 32 lines an instruction.  `at`: this lane's
// row as an offset into dst; the first `rows` rows are written.
template <int CH, typename E, typename F>
__device__ __forceinline__ void store_rows(unsigned char *stage, int lane, int rows, long long at, E *dst,
                                           F chunk) {
  static_assert(CH == 4 || CH == 8, "chunks of a row");
  // 16-byte slot of chunk k of row r: eight rows of one chunk fall into eight different bank groups
  auto slot = [&](int r, int k) { return CH == 8 ? r * 8 + (k ^ (r & 7)) : r * 4 + (k ^ ((r >> 1) & 3)); };
  __syncwarp();
#pragma unroll
  for (int k = 0; k < CH; ++k) *reinterpret_cast<uint4 *>(stage + 16 * slot(lane, k)) = chunk(k);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int r = k * (32 / CH) + lane / CH, c = lane % CH;
    const long long a = __shfl_sync(0xffffffffu, at, r);
    const uint4 v = *reinterpret_cast<const uint4 *>(stage + 16 * slot(r, c));
    if (r < rows) *reinterpret_cast<uint4 *>(dst + a + c * (16 / (int)sizeof(E))) = v;
  }
}

struct PackedOut {
  void *out;                // 16-bit rows
  long long head, row;      // strides in elements
  float *lse;               // [Hq, T] or nullptr
  float *f32;               // [Hq, T, D] or nullptr
};

// Zeros rows [cu[B], T) of a 16-bit tensor of H heads: rows that belong to no
// sequence.  All threads of a grid of `threads` threads, this one the `me`-th.
template <int D>
__device__ __forceinline__ void clear_tail(const PackedProblem &p, int H, void *out, long long head_stride,
                                           long long row_stride, long long me, long long threads) {
  const int end = min(max(sm100::ld_int(p.cu + p.B), 0), p.T);
  const long long n = (long long)H * (p.T - end) * (D / 8);
  for (long long e = me; e < n; e += threads) {
    const long long r = e / (D / 8);
    const int h = (int)(r / (p.T - end)), t = end + (int)(r % (p.T - end));
    reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + h * head_stride + t * row_stride)[e % (D / 8)] =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// Joins the partials of the unit that CTA blockIdx.x's range cuts:
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  o = sum_i O_i 2^(m_i - m) / l
// (m in units of log2).  One thread per (row, 16 columns): neighbouring threads
// read neighbouring rows.
template <typename T, int D>
__global__ void __launch_bounds__(128)
    packed_combine_kernel(const PackedProblem p, const PackedCut *cuts,
                          const float *part, int R, const PackedOut o, int clear) {
  sm100::wait_for_launches_before();
  if (clear)
    clear_tail<D>(p, p.Hq, o.out, o.head, o.row,
                  ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                  (long long)gridDim.x * gridDim.y * blockDim.x);
  const PackedCut cut = packed_cut_at(cuts, blockIdx.x);
  if (!cut.valid) return;
  const PackedRequest r = packed_request(p, cut.b);
  const int tok0 = cut.rt * p.tq, rows = min(r.n - tok0, p.tq) * p.G;
  const size_t slot = packed_slot_floats<D>(R);
  const int c0 = blockIdx.x, n = cut.last - c0 + 1;
  for (int e = blockIdx.y * blockDim.x + threadIdx.x; e < rows * (D / 16); e += gridDim.y * blockDim.x) {
    const int row = e % rows, c16 = e / rows;
    float base = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    // four partials at a time: their loads are in flight together
    for (int i0 = 0; i0 < n; i0 += 4) {
      float m[4], ls[4];
      float4 x[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = min(i0 + k, n - 1);
        // partial i: slot 1 of the first CTA, slot 0 of the later ones
        const float *s = part + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * slot;
        m[k] = __ldcg(s + row);
        ls[k] = __ldcg(s + R + row);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[k][j] = __ldcg(reinterpret_cast<const float4 *>(s + 2 * R) + (size_t)(4 * c16 + j) * R + row);
        if (i0 + k >= n) m[k] = -INFINITY;
      }
      const float top = fmaxf(fmaxf(base, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
      const float from = top == -INFINITY ? 0.f : top;
      const float f0 = exp2f(base - from);
      l *= f0;
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[j] *= f0;
      base = top;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = exp2f(m[k] - from);
        if (f == 0.f) continue;   // no weight (and, of a tile without keys, no output either)
        l = fmaf(f, ls[k], l);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[4 * j] = fmaf(f, x[k][j].x, acc[4 * j]);
          acc[4 * j + 1] = fmaf(f, x[k][j].y, acc[4 * j + 1]);
          acc[4 * j + 2] = fmaf(f, x[k][j].z, acc[4 * j + 2]);
          acc[4 * j + 3] = fmaf(f, x[k][j].w, acc[4 * j + 3]);
        }
      }
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a row without keys is zero; NaN stays
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] *= inv;
    const int token = r.first + tok0 + row / p.G, head = cut.h * p.G + row % p.G;
    uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<T *>(o.out) + head * o.head + token * o.row + 16 * c16);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      dst[j] = make_uint4(Half16<T>::pack(acc[8 * j], acc[8 * j + 1]), Half16<T>::pack(acc[8 * j + 2], acc[8 * j + 3]),
                          Half16<T>::pack(acc[8 * j + 4], acc[8 * j + 5]),
                          Half16<T>::pack(acc[8 * j + 6], acc[8 * j + 7]));
    const size_t hr = (size_t)head * p.T + token;
    if (o.f32)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4 *>(o.f32 + hr * D + 16 * c16)[j] =
            make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
    if (o.lse && c16 == 0) o.lse[hr] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
  }
}

}  // namespace pisa
