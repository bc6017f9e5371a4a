// block.cuh -- what the block operators (norms.cu, adapters.cu, ffn.cu) share.
#pragma once

#include <atomic>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {

// Whether the handle adapts d -> d on this device and takes n tokens a call (adapters.cu).
bool adapters_match(const moe_adapters *h, int d, int device, int n);
// What kernels of earlier calls on the handle reported, once; and moe_adapters_apply without asking for it
// (adapters.cu): a run of layers asks before its first launch, since what a layer of the run itself
// reports may or may not be there when the next one is enqueued.
moe_status adapters_pending(moe_adapters *h);
moe_status adapters_run(moe_adapters *h, const void *x, int32_t x_dtype, int64_t x_stride, const void *base, int64_t base_stride,
                        void *out, int64_t out_stride, int32_t out_dtype, const int32_t *ids, int32_t n_tokens, void *stream,
                        bool pending);

// The current device's error word of the norms and the dense block: host memory that kernels write, so
// that the host can read and clear it in one step (norms.cu).  A first use allocates the words of all
// devices, also while a stream is captured.
struct BlockWord {
  uint32_t *host = nullptr, *dev = nullptr;
};
cudaError_t block_word(BlockWord *w);
// MOE_ERR_TIMEOUT, once, where a kernel of an earlier call on this device set its word.
moe_status block_pending();

// The operators' entries with an error word of the caller's (norms.cu, ffn.cu): a bounded wait that runs out
// sets it in place of the device's, and the device's is not asked for what earlier calls left there.
moe_status norm_in_run(const void *x, int32_t x_dtype, int64_t x_stride, const void *weight, int32_t w_dtype, float eps,
                       int32_t unit_offset, void *h, int32_t h_dtype, int64_t h_stride, int32_t n_tokens, int32_t d_model,
                       void *stream, uint32_t *err);
moe_status norm_out_run(const moe_norm_out_args *args, void *stream, uint32_t *err);
moe_status ffn_forward_run(const moe_ffn_args *args, void *stream, uint32_t *err);

// Limits that they check.
constexpr int kNormMaxD = 8192;
constexpr int kFfnMaxDim = 65536;
inline bool bad_ffn_dim(int v) { return v < 8 || v % 8 || v > kFfnMaxDim; }

// Clock cycles that a wait of a bulk-copy ring (norms.cu, adapters.cu) may take, and for which a ring's
// first copies are held back (norms.cu): none, but where a test has the waits run out.
struct RingSpin {
  uint64_t limit, hold;
};
RingSpin ring_spin();

__device__ __forceinline__ void hold_back(uint64_t clocks) {
  const long long t0 = clock64();
  while (static_cast<uint64_t>(clock64() - t0) < clocks) {
  }
}

// The status of a call whose own CUDA call returned e; an error is not left for whoever asks next.
inline moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : MOE_ERR_CUDA;
}

// An output in the place of an input, whose rows or values lie elsewhere: rows would be written before they
// are read.
inline bool misplaced(const void *out, int64_t out_ld, int out_dt, const void *in, int64_t in_ld, int in_dt, int n) {
  return out && out == in && (out_dt != in_dt || (n > 1 && out_ld != in_ld));
}

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

// 1 / (1 + exp(-z)) by the approximate power and reciprocal.  Relative error: the power's argument is the
// rounded z log2 e, so that exp(-z) is off by up to 1.25 |z| 2^-24 and the instruction's 2^-22; the reciprocal's
// 2^-23 and the sum's 2^-24 come on top: (1.25 |z| + 7) 2^-24 for negative z, less for
// positive z, where exp(-z) counts little.  Below z = -87 it falls to 0 (1 / inf = 0).  Four instructions: an
// IEEE division takes ten, an exponential that keeps subnormals three more.
__device__ __forceinline__ float fast_sigmoid(float z, float &e) {  // e: exp(-z)
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
__device__ __forceinline__ float fast_sigmoid(float z) {
  float e;
  return fast_sigmoid(z, e);
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

// A float as the sum of bf16 parts, two floats at a time (a pair, the first in the low half): cut_bf16x2
// takes the upper halves of the floats and leaves the rest in f, round_bf16x2 rounds what is left.  One
// cut and one rounding keep a value to 2^-16 of its magnitude, two cuts and one rounding exactly (but
// for subnormal parts).  A part that is cut, not rounded, never becomes an infinity; an infinity (inf:
// one may be among the values) has no rest.
__device__ __forceinline__ uint32_t cut_bf16x2(float2 &f, bool inf) {
  const uint32_t x = __float_as_uint(f.x), y = __float_as_uint(f.y), r = __byte_perm(x, y, 0x7632);
  const float hx = __uint_as_float(x & 0xFFFF0000u), hy = __uint_as_float(y & 0xFFFF0000u);
  f.x = inf && (x & 0x7FFFFFFFu) == 0x7F800000u ? 0.f : f.x - hx;
  f.y = inf && (y & 0x7FFFFFFFu) == 0x7F800000u ? 0.f : f.y - hy;
  return r;
}
__device__ __forceinline__ uint32_t round_bf16x2(const float2 &f) {
  const __nv_bfloat162 l = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&l);
}

}  // namespace moe
