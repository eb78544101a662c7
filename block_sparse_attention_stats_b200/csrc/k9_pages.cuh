// Bookkeeping of a paged key/value cache: one step's block tables, slots and
// offsets from the requests' lengths, and the write of new keys and values.
//
// Plan.  Request b holds past_b positions and gets new_b.  With have_b =
// ceil(past_b / ps), want_b = ceil((past_b + new_b) / ps) and need_b = want_b -
// have_b, the n-th fresh page of the batch (requests in order) is
// free[num_free - 1 - n]; row r of request b sits at position pos = past_b + r -
// cu_b, in slot page(pos / ps) * ps + pos % ps.
// Bound: a launch (a few thousand integers are read, 8 bytes a row written).
// Every CTA sums the whole batch by itself, into prefix sums in shared memory,
// instead of a second launch or a wait between CTAs: at 1500 requests that is
// 6 KB of lengths from L2 and one CTA-wide scan.  A row finds its request by
// binary search; a slot on a fresh page comes from the free list, not from the
// table, so no CTA waits for another's table entries.  Replayed from a graph it
// takes 3.8 us for 7 requests of up to 40 new tokens and 7.7 us for 1500 of up to 90.
#pragma once

#include "packed_primitives.cuh"

namespace pisa {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 16384;   // two prefix sums of B + 1 in shared memory: 128 KB

struct PagePlan {
  const int32_t *past, *fresh;   // [B] lengths before the step, new tokens
  int B, T, width, page_size;    // T: rows that `slots` holds
  int32_t *table;                // [B, width]
  const int32_t *free_pages;     // [free_cap]
  int free_cap;
  const int32_t *num_free;       // [1]
  int64_t *slots;                // [T]
  int32_t *cu, *kv_lens, *num_free_out;
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlan p) {
  extern __shared__ int plan_sm[];
  int *cu = plan_sm, *need = plan_sm + p.B + 1;   // exclusive prefix sums
  __shared__ long long wsum[2][kPlanThreads / 32];
  __shared__ int wbad[kPlanThreads / 32];
  sm100::allow_next_launch();
  sm100::wait_for_launches_before();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long sn = 0, sp = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const long long past = sm100::ld_int(p.past + b), fresh = sm100::ld_int(p.fresh + b);
    bad = bad || past < 0 || fresh < 0 || past + fresh > 0x7fffffffll;
    const long long want = (past + fresh + p.page_size - 1) / p.page_size;
    bad = bad || want > p.width;
    sn += fresh;
    sp += want - (past + p.page_size - 1) / p.page_size;
  }
  long long in = sn, ip = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, in, o), y = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      in += x;
      ip += y;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 31) {
    wsum[0][warp] = in;
    wsum[1][warp] = ip;
    wbad[warp] = bad;
  }
  __syncthreads();
  long long an = in - sn, ap = ip - sp, tn = 0, tp = 0;
  int anybad = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      an += wsum[0][w];
      ap += wsum[1][w];
    }
    tn += wsum[0][w];
    tp += wsum[1][w];
    anybad |= wbad[w];
  }
  const int nf = sm100::ld_int(p.num_free);
  // all or nothing: a step that does not fit changes no table and gives no slot
  const bool ok = !anybad && tn <= p.T && nf >= 0 && nf <= p.free_cap && tp <= nf;
  const int gid = blockIdx.x * kPlanThreads + tid, gsz = gridDim.x * kPlanThreads;
  if (!ok) {
    if (gid == 0) {
      report_device_error(kDevErrRange);
      *p.num_free_out = nf;
      p.cu[p.B] = 0;
    }
    for (int b = gid; b < p.B; b += gsz) {
      p.cu[b] = 0;
      p.kv_lens[b] = sm100::ld_int(p.past + b);
    }
    for (int r = gid; r < p.T; r += gsz) p.slots[r] = -1;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    cu[b] = (int)an;
    need[b] = (int)ap;
    const int past = sm100::ld_int(p.past + b), fresh = sm100::ld_int(p.fresh + b);
    an += fresh;
    ap += (past + (long long)fresh + p.page_size - 1) / p.page_size -
          (past + (long long)p.page_size - 1) / p.page_size;
  }
  if (tid == 0) {
    cu[p.B] = (int)tn;
    need[p.B] = (int)tp;
  }
  __syncthreads();
  // last b with prefix[b] <= x: requests that hold nothing are passed over
  auto find = [&](const int *prefix, int x) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  for (int r = gid; r < p.T; r += gsz) {
    long long slot = -1;
    if (r < (int)tn) {
      const int b = find(cu, r);
      const long long past = sm100::ld_int(p.past + b), pos = past + r - cu[b];
      const int have = (int)((past + p.page_size - 1) / p.page_size);
      const int at = (int)(pos / p.page_size);
      const int page = at < have ? sm100::ld_int(p.table + (size_t)b * p.width + at)
                                 : sm100::ld_int(p.free_pages + (nf - 1 - (need[b] + at - have)));
      if (page >= 0) slot = (long long)page * p.page_size + pos % p.page_size;
      else report_device_error(kDevErrRange);
    }
    p.slots[r] = slot;
  }
  for (int n = gid; n < (int)tp; n += gsz) {
    const int b = find(need, n);
    const int have = (int)(((long long)sm100::ld_int(p.past + b) + p.page_size - 1) / p.page_size);
    p.table[(size_t)b * p.width + have + n - need[b]] = sm100::ld_int(p.free_pages + (nf - 1 - n));
  }
  for (int b = gid; b <= p.B; b += gsz) {
    p.cu[b] = cu[b];
    if (b < p.B) p.kv_lens[b] = sm100::ld_int(p.past + b) + sm100::ld_int(p.fresh + b);
  }
  if (gid == 0) *p.num_free_out = nf - (int)tp;
}

// Write.  Row t of k and v goes to row slots[t] % ps of page slots[t] / ps, head
// by head; rows whose slot is negative are left out.
// Bound: HBM (each byte read once and written once).  One thread moves 16 bytes
// of kWriteRows rows, so that that many loads are in flight before the first store.
// 65000 rows of 8 heads, d = 128 (532 MB): 84 us, 6.3 TB/s, 0.97 of a plain copy's
// rate.  33 rows: 1.8 us, the launch.
struct PageWrite {
  const unsigned char *src[2];          // k, v
  long long src_head[2], src_row[2];    // strides in bytes
  unsigned char *dst[2];                // the caches
  long long dst_page[2], dst_head[2], dst_row[2];
  const int64_t *slots;
  int T, H, page_size;
  long long num_slots;
};

constexpr int kWriteThreads = 256, kWriteRows = 4;

// CH: 16-byte chunks of a row (d / 8).  blockIdx.y: head, blockIdx.z: k or v.
template <int CH> __global__ void __launch_bounds__(kWriteThreads) page_write_kernel(const PageWrite p) {
  sm100::allow_next_launch();
  sm100::wait_for_launches_before();
  constexpr int kPer = kWriteThreads / CH;   // rows that the CTA's threads cover at once
  const int x = blockIdx.z, h = blockIdx.y;
  const int c = threadIdx.x % CH, r0 = threadIdx.x / CH;
  const unsigned char *src = p.src[x] + h * p.src_head[x] + 16 * c;
  unsigned char *dst = p.dst[x] + h * p.dst_head[x] + 16 * c;
  for (long long t0 = (long long)blockIdx.x * kPer * kWriteRows; t0 < p.T;
       t0 += (long long)gridDim.x * kPer * kWriteRows) {
    uint4 v[kWriteRows];
    long long slot[kWriteRows];
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const long long t = t0 + i * kPer + r0;
      slot[i] = t < p.T ? __ldcg(reinterpret_cast<const long long *>(p.slots) + t) : -1;
      if (t < p.T) v[i] = __ldcg(reinterpret_cast<const uint4 *>(src + t * p.src_row[x]));
    }
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      if (slot[i] < 0) continue;
      if (slot[i] >= p.num_slots) {
        report_device_error(kDevErrRange);
        continue;
      }
      const long long page = slot[i] / p.page_size;
      const int row = (int)(slot[i] - page * p.page_size);
      *reinterpret_cast<uint4 *>(dst + page * p.dst_page[x] + row * p.dst_row[x]) = v[i];
    }
  }
}

}  // namespace pisa
