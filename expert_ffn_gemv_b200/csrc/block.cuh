// block.cuh -- what the block operators (norms.cu, adapters.cu, ffn.cu) share.
#pragma once

#include <atomic>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {

// Whether the handle adapts d -> d on this device and takes n tokens a call (adapters.cu).
bool adapters_match(const moe_adapters *h, int d, int device, int n);

// Reads and clears the norms' error word on the current device (norms.cu).
cudaError_t take_norm_error(uint32_t *err);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SMs of the current device (asked once per device).
inline cudaError_t current_sm_count(int *nsm) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int v = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (!v) {
    e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) known[dev].store(v, std::memory_order_relaxed);
  }
  *nsm = v;
  return cudaSuccess;
}

// D += A B, mma.sync m16n8k16, bf16 operands, fp32 accumulators
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Two floats as N bf16 pairs (the first float in the low half) that add up to them: to 2^-16 of a
// value for N = 2, exactly (but for subnormal parts) for N = 3.  All parts but the last are cut, not
// rounded, so that a large finite value never becomes an infinity.  An infinity has one part.
template <int N>
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t (&out)[N]) {
  const bool xi = (__float_as_uint(x) & 0x7FFFFFFFu) == 0x7F800000u, yi = (__float_as_uint(y) & 0x7FFFFFFFu) == 0x7F800000u;
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) {
    const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
    out[i] = __byte_perm(xb, yb, 0x7632);
    x = xi ? 0.f : x - __uint_as_float(xb & 0xFFFF0000u);
    y = yi ? 0.f : y - __uint_as_float(yb & 0xFFFF0000u);
  }
  const __nv_bfloat162 l = __floats2bfloat162_rn(x, y);
  out[N - 1] = *reinterpret_cast<const uint32_t *>(&l);
}

}  // namespace moe
