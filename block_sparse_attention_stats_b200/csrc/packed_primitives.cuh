// sm_100a primitives of the packed and paged kernels beyond sm100_primitives.cuh.
#pragma once

#include "sm100_primitives.cuh"

namespace pisa {
namespace sm100 {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
      : "memory");
}
// Programmatic dependent launch: the next kernel of the stream may be set up from here on; and
// wait until the kernels before this one are complete and their writes are seen.  Every kernel
// that launch_after starts waits before it touches global memory, and reads what kernels before
// it may have written with ld_int (an ordinary load: the wait makes their writes visible to it) or
// __ldcg, never through the read-only path: it has been running while they wrote.
__device__ __forceinline__ void allow_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launches_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ int ld_int(const int32_t *p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// generic-proxy writes to shared memory, made visible to the tensor cores and TMA
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// kind::f16 instruction descriptor with f16 or bf16 A and B, f32 accumulator
template <bool kBf16> __host__ __device__ constexpr uint32_t idesc_16_f32(int M, int N, int a_mn, int b_mn) {
  return kBf16 ? idesc_bf16_f32(M, N, a_mn, b_mn)
               : idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

}  // namespace sm100
}  // namespace pisa
