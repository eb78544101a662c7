// Host-side helpers of the packed and paged entry points: argument checks and
// tensor maps of strided 16-bit tensors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "pisa_common.cuh"

namespace pisa {

// CTAs of the persistent kernels: one per SM of a B200.  No CTA waits for
// another, so any other number of SMs runs them too.
constexpr int kPackedCtas = 148;

#define PISA_TRY(expr)                         \
  do {                                         \
    pisa_status _s = (expr);                   \
    if (_s != PISA_OK) return _s;              \
  } while (0)

#define PISA_CUDA(expr)                        \
  do {                                         \
    cudaError_t _e = (expr);                   \
    if (_e != cudaSuccess) {                   \
      set_last_error(_e);                      \
      return PISA_ERR_CUDA;                    \
    }                                          \
  } while (0)

// Launches a kernel that may be set up while the kernel before it on the stream still runs (it
// waits for that one by itself, see wait_for_launches_before): between the short kernels of a
// decode step the gap is most of the time.
template <typename... P, typename... A>
inline pisa_status launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st,
                                const A &...args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  PISA_CUDA(cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...));
  return PISA_OK;
}

inline bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// [H][T] rows of d elements at the given strides: 16-byte aligned, rows of one
// tensor that is written must not share memory.  The stride of an extent of one
// is never used.
inline pisa_status check_rows(const pisa_rows &r, int H, int T, int d, bool written) {
  if (!aligned16(r.data)) return PISA_ERR_INVALID_ARG;
  if (H > 1 && (r.head_stride < d || r.head_stride % 8 || r.head_stride >= (1ll << 38)))
    return PISA_ERR_INVALID_ARG;
  if (T > 1 && (r.row_stride < d || r.row_stride % 8 || r.row_stride >= (1ll << 38)))
    return PISA_ERR_INVALID_ARG;
  if (written && H > 1 && T > 1 && r.head_stride < (int64_t)(T - 1) * r.row_stride + d &&
      r.row_stride < (int64_t)(H - 1) * r.head_stride + d)
    return PISA_ERR_INVALID_ARG;
  return PISA_OK;
}

// ---- operands that share memory ---------------------------------------------------------
// The memory of one operand: rows of `size` bytes, n[i] of them stride[i] bytes apart, outermost
// (widest stride) first, neighbouring dimensions merged where one fills the other's stride, so a
// dense tensor is one row.  `nested`: no block reaches into the next, so no two rows share memory.
struct Area {
  const char *data, *end;   // from the first row to behind the last
  __int128 size, stride[3], n[3];
  int dims;
  bool nested;
  __int128 span(int from = 0) const {
    __int128 s = size;
    for (int i = from; i < dims; ++i) s += (n[i] - 1) * stride[i];
    return s;
  }
};
inline Area area(const void *data, int64_t bytes) {
  Area a{};
  a.data = (const char *)data;
  a.size = data ? bytes : 0;
  a.end = a.data + (int64_t)a.size;
  a.nested = true;
  return a;
}
// counts and strides (elements of two bytes) of `dims` dimensions in any order, over rows of d elements
inline Area area(const void *data, int d, int dims, const int64_t *n, const int64_t *stride) {
  Area a = area(data, 2ll * d);
  for (int i = 0; i < dims; ++i) {
    if (n[i] <= 0) a.size = 0;
    if (n[i] <= 1) continue;
    int at = a.dims++;
    for (; at > 0 && a.stride[at - 1] < 2 * (__int128)stride[i]; --at) {
      a.stride[at] = a.stride[at - 1];
      a.n[at] = a.n[at - 1];
    }
    a.stride[at] = 2 * (__int128)stride[i];
    a.n[at] = n[i];
  }
  while (a.dims && a.stride[a.dims - 1] == a.size) a.size *= a.n[--a.dims];
  __int128 span = a.size;
  for (int i = a.dims - 1; i >= 0; --i) {
    a.nested = a.nested && a.stride[i] >= span;
    span += (a.n[i] - 1) * a.stride[i];
  }
  // (past the address space, strides that no memory has: as far as it goes)
  const __int128 end = (__int128)(uintptr_t)data + span;
  a.end = (const char *)(end > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end);
  return a;
}
inline Area area(const pisa_rows &r, int H, int T, int d) {
  const int64_t n[] = {H, T}, s[] = {r.head_stride, r.row_stride};
  return area(r.data, d, 2, n, s);
}
inline Area area(const pisa_pages &c, int pages, int H, int ps, int d) {
  const int64_t n[] = {pages, H, ps}, s[] = {c.page_stride, c.head_stride, c.row_stride};
  return area(c.data, d, 3, n, s);
}

// Whether dimensions i on of a and j on of b, at[b] - at[a] = off, share a byte.  Exact where the outer
// strides are equal (slices of one tensor) or one of the two is dense; other layouts, whose rows may
// lie between one another's, count as apart.
inline bool areas_meet(const Area &a, int i, const Area &b, int j, __int128 off) {
  if (off >= a.span(i) || -off >= b.span(j)) return false;
  if (i == a.dims && j == b.dims) return true;
  auto down = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };
  if (i < a.dims && j < b.dims) {
    const __int128 s = a.stride[i];
    if (s != b.stride[j]) return false;
    // block x of a and y of b lie off + (y - x) s apart: the few differences k at which they can meet
    __int128 k0 = down(-off - b.span(j + 1), s) + 1, k1 = down(a.span(i + 1) - 1 - off, s);
    if (k0 < 1 - a.n[i]) k0 = 1 - a.n[i];
    if (k1 > b.n[j] - 1) k1 = b.n[j] - 1;
    for (__int128 k = k0; k <= k1; ++k)
      if (areas_meet(a, i + 1, b, j + 1, off + k * s)) return true;
    return false;
  }
  if (i < a.dims) return areas_meet(b, j, a, i, -off);
  // a dense: the blocks of b that reach into it; of three, the middle one lies inside
  const __int128 s = b.stride[j];
  __int128 k0 = down(-off - b.span(j + 1), s) + 1, k1 = down(a.span(i) - 1 - off, s);
  if (k0 < 0) k0 = 0;
  if (k1 > b.n[j] - 1) k1 = b.n[j] - 1;
  if (k1 - k0 >= 2) return true;
  for (__int128 k = k0; k <= k1; ++k)
    if (areas_meet(a, i, b, j + 1, off + k * s)) return true;
  return false;
}
inline bool share_memory(const Area &a, const Area &b) {
  if (a.end <= b.data || b.end <= a.data || a.size == 0 || b.size == 0) return false;
  if (a.data == b.data) return true;
  if (!a.nested || !b.nested) return false;
  return areas_meet(a, 0, b, 0, (__int128)(intptr_t)b.data - (__int128)(intptr_t)a.data);
}
// What a call writes may share memory neither with what it reads nor with anything else it writes
// (`from`: those before have been looked at).
inline pisa_status check_apart(const Area *written, int nw, const Area *read, int nr, int from = 0) {
  for (int i = from; i < nw; ++i) {
    for (int j = 0; j < nr; ++j)
      if (share_memory(written[i], read[j])) return PISA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (share_memory(written[i], written[j])) return PISA_ERR_INVALID_ARG;
  }
  return PISA_OK;
}

// 16-bit tensor of `rank` dimensions, innermost contiguous, read in boxes of 64
// columns with the 128-byte swizzle; what lies outside reads as zero.
inline pisa_status map16(CUtensorMap *m, const void *base, bool bf16, int rank, const uint64_t *dims,
                         const uint64_t *stride_elems, const uint32_t *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_tiled();
  if (!enc) {
    set_last_error_text("cuTensorMapEncodeTiled is not available from the driver");
    return PISA_ERR_CUDA;
  }
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], e[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    e[i] = 1;
    if (i) s[i - 1] = (dims[i] > 1 ? stride_elems[i] : dims[0]) * 2;   // an extent of one: any legal stride
  }
  const CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                         const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_last_error_text("cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r));
    return PISA_ERR_CUDA;
  }
  return PISA_OK;
}

// rows of one head: (column, row, head)
inline pisa_status map_rows(CUtensorMap *m, const pisa_rows &r, bool bf16, int d, int T, int H, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)T, (uint64_t)H};
  const uint64_t st[3] = {1, (uint64_t)r.row_stride, (uint64_t)r.head_stride};
  const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
  return map16(m, r.data, bf16, 3, dims, st, box);
}

// rows of a group of heads, token by token: (column, head of the group, row, key head)
inline pisa_status map_query(CUtensorMap *m, const pisa_rows &r, bool bf16, int d, int G, int T, int Hkv,
                             int tokens) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)G, (uint64_t)T, (uint64_t)Hkv};
  const uint64_t st[4] = {1, (uint64_t)r.head_stride, (uint64_t)r.row_stride, (uint64_t)r.head_stride * G};
  const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)tokens, 1};
  return map16(m, r.data, bf16, 4, dims, st, box);
}

// rows of a page: (column of 64, row, 64 columns, head, page), boxes of one page's rows (128 at
// most) and `halves` times 64 columns
inline pisa_status map_pages(CUtensorMap *m, const pisa_pages &c, bool bf16, int d, int page_size, int H,
                             int pages, int halves) {
  const uint64_t dims[5] = {64, (uint64_t)page_size, (uint64_t)d / 64, (uint64_t)H, (uint64_t)pages};
  const uint64_t st[5] = {1, (uint64_t)c.row_stride, 64, (uint64_t)c.head_stride, (uint64_t)c.page_stride};
  const uint32_t box[5] = {64, (uint32_t)(page_size < 128 ? page_size : 128), (uint32_t)halves, 1, 1};
  return map16(m, c.data, bf16, 5, dims, st, box);
}

}  // namespace pisa
