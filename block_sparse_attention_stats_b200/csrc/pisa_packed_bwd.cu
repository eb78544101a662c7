// libpisa C ABI, third translation unit: gradients of attention over packed
// sequences.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "packed_host.cuh"
#include "packed_schedule.cuh"
#include "k12_packed_bwd.cuh"

namespace pisa {

pisa_status take_packed_bwd_status(unsigned *bits) { return take_status_word(&g_device_status, bits); }

struct PackedBwdLayout {
  size_t lse2, delta, cuts[2], part[2], total;   // cuts and partial sums of dq, and of dk and dv
};
static PackedBwdLayout packed_bwd_layout(int T, int Hq, int d) {
  PackedBwdLayout l;
  const size_t rows = align_up((size_t)Hq * T * sizeof(float), 256);
  l.lse2 = 0;
  l.delta = rows;
  size_t at = 2 * rows;
  for (int i = 0; i < 2; ++i) {
    l.cuts[i] = at;
    at += align_up(kPackedCtas * sizeof(PackedCut), 256);
    l.part[i] = at;
    at += (size_t)kPackedCtas * 2 * (i + 1) * 128 * d * sizeof(float);
  }
  l.total = at;
  return l;
}

template <int D>
static pisa_status launch_packed_bwd(PackedProblem p, const pisa_rows &q, const pisa_rows &k, const pisa_rows &v,
                                     const pisa_rows &dout, const float *lse, const float *out_f32, float scale,
                                     const pisa_rows &dq, const pisa_rows &dk, const pisa_rows &dv,
                                     int clear, unsigned char *ws, cudaStream_t st) {
  using Cq = PackedBwdCfg<D, false>;
  using Ck = PackedBwdCfg<D, true>;
  const PackedBwdLayout l = packed_bwd_layout(p.T, p.Hq, D);
  float *lse2 = (float *)(ws + l.lse2), *delta = (float *)(ws + l.delta);
  PackedSums s{};
  const pisa_rows *out[3] = {&dq, &dk, &dv};
  for (int i = 0; i < 3; ++i) {
    s.out[i] = (__nv_bfloat16 *)out[i]->data;
    s.head[i] = out[i]->head_stride;
    s.row[i] = out[i]->row_stride;
  }
  PackedCut *cuts[2];
  float *part[2];
  for (int i = 0; i < 2; ++i) {
    s.cuts[i] = cuts[i] = (PackedCut *)(ws + l.cuts[i]);
    s.part[i] = part[i] = (float *)(ws + l.part[i]);
  }
  s.clear = clear;
  const long long rows = (long long)p.Hq * p.T;
  PISA_TRY(launch_after(packed_delta_kernel<D>, dim3((unsigned)std::min<long long>((rows + 7) / 8, 148 * 8)), 256, 0, st,
      (const __nv_bfloat16 *)dout.data, dout.head_stride, dout.row_stride, out_f32, lse, p.Hq, p.T, p.cu, p.B,
      lse2, delta));
  p.tq = 128 / p.G;
  // a unit's start and end in tiles, measured at 1.5 / 2.5 / 4: 2383 / 2228 / 2230 us a training step on 8192 +
  // 4608 + 1500 tokens, 322 / 301 / 306 us on 4096 + 2048 at d = 64.  The shortest range at 1 / 3 / 6 tiles: 60 /
  // 56 / 62 us on 512 + 100 tokens, where most units are cut
  p.unit_cost = 5 * kKeyTile / 2;
  p.min_range = 3 * kKeyTile;
  p.whole = 4 * kKeyTile;
  s.p = p;
  CUtensorMap mq, mdo, mk, mv;
  PISA_TRY(map_query(&mq, q, true, D, p.G, p.T, p.Hkv, p.tq));
  PISA_TRY(map_query(&mdo, dout, true, D, p.G, p.T, p.Hkv, p.tq));
  PISA_TRY(map_rows(&mk, k, true, D, p.T, p.Hkv, 128));
  PISA_TRY(map_rows(&mv, v, true, D, p.T, p.Hkv, 128));
  PISA_CUDA(cudaFuncSetAttribute(packed_bwd_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cq::kSmem));
  PISA_TRY(launch_after(packed_bwd_kernel<D, false>, dim3(kPackedCtas), Cq::kThreads, Cq::kSmem, st,
      mq, mdo, mk, mv, p, scale, lse2, delta, s.out[0], s.head[0], s.row[0], nullptr, 0, 0, cuts[0], part[0]));
  // dk, dv: Q and dout one head at a time
  PISA_TRY(map_rows(&mq, q, true, D, p.T, p.Hq, 128));
  PISA_TRY(map_rows(&mdo, dout, true, D, p.T, p.Hq, 128));
  PISA_CUDA(cudaFuncSetAttribute(packed_bwd_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Ck::kSmem));
  PISA_TRY(launch_after(packed_bwd_kernel<D, true>, dim3(kPackedCtas), Ck::kThreads, Ck::kSmem, st,
      mq, mdo, mk, mv, p, scale, lse2, delta, s.out[1], s.head[1], s.row[1], s.out[2], s.head[2], s.row[2],
      cuts[1], part[1]));
  return launch_after(packed_sum_kernel<D>, dim3(kPackedCtas, D / 16, 3), 128, 0, st, s);
}

}  // namespace pisa

using namespace pisa;

extern "C" {

size_t pisa_varlen_attention_bwd_workspace_bytes(int T, int Hq, int Hkv, int d) {
  if (T < 1 || T > (1 << 24) || pisa_varlen_attention_workspace_bytes(Hq, Hkv, d) == 0) return 0;
  return packed_bwd_layout(T, Hq, d).total;
}

pisa_status pisa_varlen_attention_bwd(pisa_rows q, pisa_rows k, pisa_rows v, pisa_rows dout, pisa_dtype dtype,
                                      const float *lse, const float *out_f32, const int32_t *cu_seqlens, int B,
                                      int T, int Hq, int Hkv, int d, float scale, int flags, pisa_rows dq,
                                      pisa_rows dk, pisa_rows dv, void *workspace, size_t ws_bytes,
                                      pisa_stream_t stream) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv) return PISA_ERR_INVALID_ARG;
  if (dtype != PISA_BF16 && dtype != PISA_F16 && dtype != PISA_F32) return PISA_ERR_INVALID_ARG;
  if (dtype != PISA_BF16 || (d != 64 && d != 128)) return PISA_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hq / Hkv > 128 || T > (1 << 24) || B > (1 << 16)) return PISA_ERR_UNSUPPORTED;
  // a key tile's length, the 128-row tiles of its whole group, is counted in 32 bits
  if ((long long)ceil_div(T, 128) * 128 * (Hq / Hkv) > (1 << 30)) return PISA_ERR_UNSUPPORTED;
  if (!(scale >= 0.f) || !std::isfinite(scale) || (flags & ~(PISA_CAUSAL | PISA_ZERO_TAIL))) return PISA_ERR_INVALID_ARG;
  if (!cu_seqlens || ((uintptr_t)cu_seqlens & 3u)) return PISA_ERR_INVALID_ARG;
  if (T == 0) return PISA_OK;
  PISA_TRY(check_rows(q, Hq, T, d, false));
  PISA_TRY(check_rows(k, Hkv, T, d, false));
  PISA_TRY(check_rows(v, Hkv, T, d, false));
  PISA_TRY(check_rows(dout, Hq, T, d, false));
  PISA_TRY(check_rows(dq, Hq, T, d, true));
  PISA_TRY(check_rows(dk, Hkv, T, d, true));
  PISA_TRY(check_rows(dv, Hkv, T, d, true));
  if (!lse || ((uintptr_t)lse & 3u) || !aligned16(out_f32) || !aligned16(workspace)) return PISA_ERR_INVALID_ARG;
  const size_t need = packed_bwd_layout(T, Hq, d).total;
  const Area read[] = {area(q, Hq, T, d),           area(k, Hkv, T, d),  area(v, Hkv, T, d),
                       area(dout, Hq, T, d),        area(lse, 4ll * Hq * T), area(out_f32, 4ll * Hq * T * d),
                       area(cu_seqlens, 4ll * (B + 1))};
  const Area written[] = {area(dq, Hq, T, d), area(dk, Hkv, T, d), area(dv, Hkv, T, d), area(workspace, need)};
  PISA_TRY(check_apart(written, 3, read, 7));
  if (ws_bytes < need) return PISA_ERR_WORKSPACE;
  PISA_TRY(check_apart(written, 4, read, 7, 3));
  PackedProblem p{};
  p.cu = cu_seqlens;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.causal = flags & PISA_CAUSAL;
  p.max_kv = T;
  const float s = scale == 0.f ? 1.f / std::sqrt((float)d) : scale;
  unsigned char *ws = (unsigned char *)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  const int clear = flags & PISA_ZERO_TAIL;
  if (d == 128) return launch_packed_bwd<128>(p, q, k, v, dout, lse, out_f32, s, dq, dk, dv, clear, ws, st);
  return launch_packed_bwd<64>(p, q, k, v, dout, lse, out_f32, s, dq, dk, dv, clear, ws, st);
}

}  // extern "C"
