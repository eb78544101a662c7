// How the kernels of packed rows and paged caches share out their work.
//
// A batch is B sequences of new tokens, packed: sequence b holds rows cu[b] ..
// cu[b+1] - 1 of q, and its tokens are the last n of its kv positions (for
// packed prompts kv = n).  A unit is (sequence, row tile, key head): tq tokens
// times the G query heads of the key head, G rows a token, against the key
// positions that the tile's last token sees, in tiles of 128.  All units, each as
// long as its positions and a constant (unit_cost), are laid end to end, and the
// line is cut into ranges of equal length, one a CTA; a cut counts for the tile that
// it falls into, in a short unit for the unit's nearer end.  So CTAs get equal
// lengths to within a tile or a short unit, not equal numbers of tiles: many short units
// have fewer than one long one, and where there is little work (min_range) some CTAs
// have none.  Nothing is read on the host: the cut depends on lengths in device
// memory alone, and the grid on the device alone, so a captured launch serves any
// lengths.
// Lengths in positions, not in tiles, make what lies before a unit a polynomial of
// its number, so a CTA finds its place with a few multiplications.  (Exact sums of
// rounded tiles, with 64-bit divisions, took 4 us at the start of every kernel.)
// A unit counts unit_cost positions more than it has, for what its start and its
// end take: without, a CTA that got many short units ran twice as long as the
// others.  A cut that falls into these is one at the unit's start.
// A unit inside one range is written by its CTA.  A unit cut by a range's end
// leaves float32 partial sums, and packed_combine_kernel joins them in ascending
// CTA order (no atomics: the same inputs give the same bits).
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
  int unit_cost;            // what a unit takes beside its positions, in positions
  int min_range;            // no range is shorter than this, at least a tile
  int whole;                // units of this many positions or fewer are not cut
};

struct PackedRequest {
  int first, n, kv, past;   // first row, tokens, key positions, positions before the first token
};

// Offsets and lengths are device data: whatever they hold, rows stay inside
// [0, T) and positions inside [0, max_kv]; `bad` says where they did not.
enum : int { kBadOffsets = 1, kBadLengths = 2 };
__device__ __forceinline__ PackedRequest packed_request(const PackedProblem &p, int b, int &bad) {
  PackedRequest r;
  const int lo = sm100::ld_int(p.cu + b), hi = sm100::ld_int(p.cu + b + 1);
  const int kv = p.kv_lens ? sm100::ld_int(p.kv_lens + b) : 0;
  r.first = min(max(lo, 0), p.T);
  r.n = max(min(hi, p.T) - r.first, 0);
  r.kv = p.kv_lens ? min(max(kv, 0), p.max_kv) : r.n;
  r.past = r.kv - r.n;
  bad |= (lo < 0 || hi < lo || hi > p.T ? kBadOffsets : 0) | (kv < 0 || kv > p.max_kv ? kBadLengths : 0);
  return r;
}

// Units of a sequence, the length of one (without unit_cost), the lengths of those
// before it, and about which one starts y positions on.  RowCost: a unit is a row
// tile of tq tokens.  KeyCost: a unit is a tile of 128 keys of a sequence over
// itself, its length the 128-token tiles of every query head that see it.
struct RowCost {
  static __host__ __device__ int units(const PackedProblem &p, int n) { return n > 0 ? (n - 1) / p.tq + 1 : 0; }
  // positions that row tile rt of tq tokens sees (at least one: a row without keys is still written)
  static __host__ __device__ int length(const PackedProblem &p, int n, int kv, int tq, int rt) {
    const int past = kv > n ? kv - n : 0;
    return p.causal ? past + (n - rt * tq < tq ? n : (rt + 1) * tq) : (kv > 1 ? kv : 1);
  }
  static __host__ __device__ int length(const PackedProblem &p, int n, int kv, int rt) {
    return length(p, n, kv, p.tq, rt);
  }
  static __host__ __device__ long long before(const PackedProblem &p, int n, int kv, int rt) {
    const int past = kv > n ? kv - n : 0;
    if (!p.causal) return (long long)rt * (kv > 1 ? kv : 1);
    return (long long)rt * past + (long long)p.tq * ((long long)rt * (rt + 1) / 2);
  }
  static __device__ int guess(const PackedProblem &p, int n, int kv, float y) {
    if (!p.causal) return (int)(y / (float)((kv > 1 ? kv : 1) + p.unit_cost));
    const float b = (float)(kv > n ? kv - n : 0) + p.unit_cost + 0.5f * p.tq;
    return (int)(2.f * y / (b + sqrtf(fmaf(b, b, 2.f * p.tq * y))));
  }
};
struct KeyCost {
  static __host__ __device__ int units(const PackedProblem &, int n) { return (n + kKeyTile - 1) / kKeyTile; }
  static __host__ __device__ int length(const PackedProblem &p, int n, int, int rt) {
    return kKeyTile * p.G * (units(p, n) - (p.causal ? rt : 0));
  }
  static __host__ __device__ long long before(const PackedProblem &p, int n, int, int rt) {
    const long long N = units(p, n);
    return kKeyTile * p.G * (rt * N - (p.causal ? (long long)rt * (rt - 1) / 2 : 0));
  }
  static __device__ int guess(const PackedProblem &p, int n, int, float y) {
    const float g = (float)kKeyTile * p.G, N = (float)units(p, n);
    if (!p.causal) return (int)(y / (g * N + p.unit_cost));
    const float b = g * (N + 0.5f) + p.unit_cost;
    return (int)(2.f * y / (b + sqrtf(fmaxf(fmaf(b, b, -2.f * g * y), 0.f))));
  }
};
__host__ __device__ inline int packed_tiles(int length) { return (length + kKeyTile - 1) / kKeyTile; }

// what units 0 .. rt - 1 of a sequence count, over all key heads
template <class Cost>
__host__ __device__ __forceinline__ long long packed_before(const PackedProblem &p, const PackedRequest &r, int rt) {
  return p.Hkv * (Cost::before(p, r.n, r.kv, rt) + (long long)rt * p.unit_cost);
}
template <class Cost>
__host__ __device__ __forceinline__ long long packed_cost(const PackedProblem &p, const PackedRequest &r) {
  const int R = Cost::units(p, r.n);
  if (R == 0) return 0;
  return packed_before<Cost>(p, r, R - 1) + p.Hkv * (long long)(Cost::length(p, r.n, r.kv, R - 1) + p.unit_cost);
}

// Where a CTA's range starts: `at` positions into unit (b, rt, h), `left` positions long
struct PackedStart {
  long long left, end, chunk;   // end: the range's end on the line; chunk: the length of a range
  int b, rt, h, at;
  PackedRequest r;
};

// Row tile, key head and offset of the point `rem` positions into sequence r.
template <class Cost>
__device__ __forceinline__ void packed_point(const PackedProblem &p, const PackedRequest &r, long long rem,
                                             int &rt, int &h, int &at) {
  const int R = Cost::units(p, r.n);
  int x = min(max(Cost::guess(p, r.n, r.kv, (float)rem / (float)p.Hkv), 0), R - 1);
  while (x > 0 && packed_before<Cost>(p, r, x) > rem) --x;
  while (x + 1 < R && packed_before<Cost>(p, r, x + 1) <= rem) ++x;
  const long long in = rem - packed_before<Cost>(p, r, x);
  const int all = Cost::length(p, r.n, r.kv, x) + p.unit_cost;
  int y = min(max((int)((float)in / (float)all), 0), p.Hkv - 1);
  while (y > 0 && (long long)y * all > in) --y;
  while (y + 1 < p.Hkv && (long long)(y + 1) * all <= in) ++y;
  rt = x;
  h = y;
  at = (int)(in - (long long)y * all);
}

// One call by all `threads` threads of a CTA (a multiple of 32, at most 512):
// fills *out (shared memory).  Contains two CTA barriers.  Where offsets are out of order or
// range nothing is worked on: clamped one by one, B of them could each name all T rows, and a
// launch take B times as long as a batch of that size (minutes, of a buffer that was never filled).
template <class Cost>
__device__ __forceinline__ void packed_locate(const PackedProblem &p, int cta, int grid, int tid, int threads,
                                              long long *warp_sum, PackedStart *out) {
  const int per = (p.B + threads - 1) / threads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long own = 0;
  int bad = 0;
  PackedRequest r{};
  for (int b = b0; b < b1; ++b) {
    r = packed_request(p, b, bad);
    own += packed_cost<Cost>(p, r);
  }
  if (bad && cta == 0) report_device_error(kDevErrRange);
  const int lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  long long incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  const bool skip = __syncthreads_or(bad & kBadOffsets);
  // sums of the warps before this one, and of all
  long long sum = lane < warps ? warp_sum[lane] : 0;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  const long long all = __shfl_sync(0xffffffffu, sum, warps - 1), total = skip ? 0 : all;
  const long long up_to = __shfl_sync(0xffffffffu, sum, max(warp - 1, 0));
  const long long before = (warp ? up_to : 0) + incl - own;
  long long chunk = (long long)((double)total * (1.0 / grid)) + 1;
  if (chunk < p.min_range) chunk = p.min_range;
  const long long w0 = chunk * cta < total ? chunk * cta : total;
  const long long w1 = cta + 1 < grid && chunk * (cta + 1) < total ? chunk * (cta + 1) : total;
  if (w0 >= total) {
    if (tid == 0) out->left = 0;
  } else if (own > 0 && w0 >= before && w0 < before + own) {
    long long rem = w0 - before;
    int b = b0;
    if (per > 1)
      for (;; ++b) {
        r = packed_request(p, b, bad);
        const long long c = packed_cost<Cost>(p, r);
        if (rem < c) break;
        rem -= c;
      }
    packed_point<Cost>(p, r, rem, out->rt, out->h, out->at);
    out->left = w1 - w0;
    out->end = w1;
    out->chunk = chunk;
    out->b = b;
    out->r = r;
  }
  __syncthreads();
}

// The part [ta, tb) of one unit's tiles [0, nt)
struct PackedSegment {
  PackedRequest r;
  int b, rt, h, nt, ta, tb;
  int end;   // where the segment ends in its unit, in positions
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == nt; }
  // partial slot of the CTA: 0 holds a unit begun by an earlier CTA, 1 one that goes on in the next
  __device__ __forceinline__ int slot() const { return ta != 0 ? 0 : 1; }
};

// Walks a CTA's range segment by segment.  Every warp keeps its own (all lanes
// hold the same values), so no role waits for another to learn what comes next.
template <class Cost> struct PackedWalk {
  PackedSegment s;
  long long left;   // positions of the range
  int at, len;      // where the next segment starts in its unit, and the unit's length
  __device__ __forceinline__ void begin(const PackedProblem &p, const PackedStart &st) {
    left = st.left;
    if (left <= 0) return;
    s.b = st.b;
    s.rt = st.rt;
    s.h = st.h;
    s.r = st.r;
    at = st.at;
    len = Cost::length(p, s.r.n, s.r.kv, s.rt);
    s.nt = packed_tiles(len);
  }
  // tiles of the unit that lie before its position x
  __device__ __forceinline__ int tiles_before(const PackedProblem &p, int x) const {
    if (len <= p.whole) return 2 * x < len + p.unit_cost ? 0 : s.nt;
    return x <= p.unit_cost ? 0 : packed_tiles(x - p.unit_cost);
  }
  __device__ __forceinline__ bool next(const PackedProblem &p) {
    while (left > 0) {
      const int all = len + p.unit_cost;
      if (at == all) {   // the next unit
        at = 0;
        if (++s.h == p.Hkv) {
          s.h = 0;
          if (++s.rt >= Cost::units(p, s.r.n)) {
            s.rt = 0;
            int bad = 0;   // (packed_locate has recorded it)
            do {
              if (++s.b >= p.B) return false;   // cannot happen while positions are left
              s.r = packed_request(p, s.b, bad);
            } while (s.r.n == 0);
          }
          len = Cost::length(p, s.r.n, s.r.kv, s.rt);
          s.nt = packed_tiles(len);
        }
        continue;
      }
      s.end = (int)(left < all - at ? at + left : all);
      s.ta = tiles_before(p, at);
      s.tb = tiles_before(p, s.end);
      left -= s.end - at;
      at = s.end;
      if (s.tb > s.ta) return true;   // else both ends fall into one tile, or before the first
    }
    return false;
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

// (a range is at least a tile long, so every CTA between the first and the last has a part)
__device__ __forceinline__ PackedCut packed_cut(const PackedProblem &p, const PackedStart &st,
                                                const PackedSegment &s, int grid) {
  PackedCut c;
  c.valid = 1;
  c.b = s.b;
  c.rt = s.rt;
  c.h = s.h;
  const long long start = st.end - s.end;   // the unit's, on the line
  const long long tile = (start + p.unit_cost + (long long)(s.nt - 1) * kKeyTile) / st.chunk;
  c.last = tile < grid ? (int)tile : grid - 1;
  return c;
}

// partial slot: R rows of m, l and the sum for lse, then the unnormalised output as [D / 4][R] float4
template <int D> __host__ __device__ constexpr size_t packed_slot_floats(int R) {
  return (size_t)R * (D + 3);
}

// A softmax weight is rounded to T for its product with the values.  bf16 has float32's range; f16's
// spacing stops shrinking at 2^-14 and ends at 2^-24, so of a weight far below the largest little or
// nothing would be left there, while the sum has all of it: of one key 2^17.4 above 131071 others,
// whose values are 1, came 0.9964.  So f16 weights are formed larger by a power of two, where the
// type still has room above (kRoom), and the factor, common to the weights and their sum, cancels.
template <typename T> struct Half16;
template <> struct Half16<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static constexpr int kRoom = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
};
template <> struct Half16<__half> {
  static constexpr bool kBf16 = false;
  static constexpr int kRoom = 15;   // the largest weight is 2^15 at most
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
  uint4 v[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k)
    v[k] = *reinterpret_cast<const uint4 *>(stage + 16 * slot(k * (32 / CH) + lane / CH, lane % CH));
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int r = k * (32 / CH) + lane / CH;
    const long long a = __shfl_sync(0xffffffffu, at, r);
    if (r < rows) *reinterpret_cast<uint4 *>(dst + a + (lane % CH) * (16 / (int)sizeof(E))) = v[k];
  }
}

struct PackedOut {
  void *out;                // 16-bit rows
  long long head, row;      // strides in elements
  float *lse;               // [Hq, T] or nullptr
  float *f32;               // [Hq, T, D] or nullptr
};

// Zeros rows [0, cu[0]) and [cu[B], T) of a 16-bit tensor of H heads: rows that belong to no
// sequence.  All threads of a grid of `threads` threads, this one the `me`-th.
template <int D>
__device__ __forceinline__ void clear_unused(const PackedProblem &p, int H, void *out, long long head_stride,
                                             long long row_stride, long long me, long long threads) {
  const int first = min(max(sm100::ld_int(p.cu), 0), p.T);
  const int end = max(min(sm100::ld_int(p.cu + p.B), p.T), first);
  const int rows = first + p.T - end;
  const long long n = (long long)H * rows * (D / 8);
  for (long long e = me; e < n; e += threads) {
    const long long r = e / (D / 8);
    const int h = (int)(r / rows), i = (int)(r % rows), t = i < first ? i : end + i - first;
    reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + h * head_stride + t * row_stride)[e % (D / 8)] =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// Joins the partials of the unit that CTA blockIdx.x's range cuts:
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  o = sum_i O_i 2^(m_i - m) / l
// (m in units of log2).  One thread per (row, 4 V columns): neighbouring threads
// read neighbouring rows, and a thread's loads of 16 / V partials are in flight
// together.  V = 4 where units have many rows; V = 2 where they have few, and a long
// request tens of parts (V = 4 / 2 / 1: 80.0 / 78.0 / 78.4 us on 131072 and 90001 keys, 9.5 /
// 9.0 / 9.3 us on one request of 777, 150 / 150 / 151 us on 48 of 1 to 8000).
template <typename T, int D, int V>
__global__ void __launch_bounds__(128)
    packed_combine_kernel(const PackedProblem p, const PackedCut *cuts,
                          const float *part, int R, const PackedOut o, int clear) {
  constexpr int kBatch = 16 / V;
  sm100::wait_for_launches_before();
  if (clear)
    clear_unused<D>(p, p.Hq, o.out, o.head, o.row,
                    ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                    (long long)gridDim.x * gridDim.y * blockDim.x);
  const PackedCut cut = packed_cut_at(cuts, blockIdx.x);
  if (!cut.valid) return;
  int bad = 0;
  const PackedRequest r = packed_request(p, cut.b, bad);
  const int tok0 = cut.rt * p.tq, rows = min(r.n - tok0, p.tq) * p.G;
  const size_t slot = packed_slot_floats<D>(R);
  const int c0 = blockIdx.x, n = cut.last - c0 + 1;
  for (int e = blockIdx.y * blockDim.x + threadIdx.x; e < rows * (D / (4 * V)); e += gridDim.y * blockDim.x) {
    const int row = e % rows, c = e / rows;
    float base = -INFINITY, l = 0.f, le = 0.f;
    float4 acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float m[kBatch], ls[kBatch], es[kBatch];
      float4 x[kBatch][V];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = min(i0 + k, n - 1);
        // partial i: slot 1 of the first CTA, slot 0 of the later ones
        const float *s = part + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * slot;
        m[k] = __ldcg(s + row);
        ls[k] = __ldcg(s + R + row);
        es[k] = __ldcg(s + 2 * R + row);
#pragma unroll
        for (int j = 0; j < V; ++j)
          x[k][j] = __ldcg(reinterpret_cast<const float4 *>(s + 3 * R) + (size_t)(V * c + j) * R + row);
        if (i0 + k >= n) {
          m[k] = -INFINITY;
          ls[k] = 0.f;
        }
      }
      float top = base;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, m[k]);
      const float from = top == -INFINITY ? 0.f : top;
      const float f0 = exp2f(base - from);
      l *= f0;
      le *= f0;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = make_float4(acc[j].x * f0, acc[j].y * f0, acc[j].z * f0, acc[j].w * f0);
      base = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        // no key seen (of a tile without keys the slot holds no output either).  A sum of NaN comes
        // with no maximum too, where every score is NaN, and is not passed over
        if (m[k] == -INFINITY && ls[k] == 0.f) continue;
        const float f = exp2f(m[k] - from);
        l = fmaf(f, ls[k], l);
        le = fmaf(f, es[k], le);
#pragma unroll
        for (int j = 0; j < V; ++j)
          acc[j] = make_float4(fmaf(f, x[k][j].x, acc[j].x), fmaf(f, x[k][j].y, acc[j].y),
                               fmaf(f, x[k][j].z, acc[j].z), fmaf(f, x[k][j].w, acc[j].w));
      }
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a row without keys is zero; NaN stays
    const int token = r.first + tok0 + row / p.G, head = cut.h * p.G + row % p.G;
    const size_t hr = (size_t)head * p.T + token;
    T *dst = reinterpret_cast<T *>(o.out) + head * o.head + token * o.row + 4 * V * c;
    uint2 w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      acc[j] = make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
      w[j] = make_uint2(Half16<T>::pack(acc[j].x, acc[j].y), Half16<T>::pack(acc[j].z, acc[j].w));
      if (o.f32) reinterpret_cast<float4 *>(o.f32 + hr * D + 4 * V * c)[j] = acc[j];
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      reinterpret_cast<uint4 *>(dst)[j] = make_uint4(w[2 * j].x, w[2 * j].y, w[2 * j + 1].x, w[2 * j + 1].y);
    if (o.lse && c == 0) o.lse[hr] = le == 0.f ? -INFINITY : (base + log2f(le)) * 0.6931471805599453f;
  }
}

}  // namespace pisa
