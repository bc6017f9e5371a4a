// ffn.cu -- dense gated feed-forward block from bf16 weights and its gradients:
//   g = x Wg^T   u = x Wu^T   h = silu(g) * u   y = h Wd^T (+ add)
//   dh = dy Wd   dg = dh u silu'(g)   du = dh silu(g)
//   dx = dg Wg + du Wu   dWg = dg^T x   dWu = du^T x   dWd = dy^T h
// x, dy n x d; Wg, Wu f x d; Wd d x f; all products of bf16 values with fp32 accumulators, each
// result rounded once.  h, dg and du are operands of the next products and so in bf16: their rounding
// (2^-9 of a value) is no more than that of the bf16 results.  g and u, from which the backward
// computes h, dg and du again, are saved in fp32: in bf16 their rounding would come on top of it
// (gradients 3.5e-3 off, relative 2-norm, against 2.4e-3).
//
// Few tokens: the weights stream once through mma.sync operands (k_ffn_up, k_ffn_down), bound by
// their bytes.  More tokens: one warp-specialised tcgen05 kernel (k_ffn_gemm) for every product,
// D[M][N] = sum_k A[m][k] B[n][k]; an operand is read as it lies in memory, along k (K-major) or
// along its rows (MN-major), so no transpose is ever written.
#include <mutex>

#include "block.cuh"
#include "tc05.cuh"

using namespace moe;

namespace {

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kStages = 4;
constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2, kStageBytes = kABytes + kBBytes;
constexpr int kGemmSmem = 1024 + 1024 + kStages * kStageBytes;
constexpr int kGemmThreads = 192;  // warps 0..3 epilogue, 4 TMA producer, 5 MMA
constexpr uint64_t kSpin = 2000000000ull;  // about a second
constexpr int kMaxProb = 4, kMaxMaps = 5;

// Set by a kernel whose bounded wait ran out; moe_ffn_check reads and clears it.
__device__ uint32_t g_ffn_err;

enum { kEpiPlain = 0, kEpiSwiglu = 1, kEpiDswiglu = 2 };

struct GemmProb {
  int m, n, k, segs;       // segs products over k added up (operands a[i], b[i])
  int tiles_n, tile0;      // tiles along n, first tile of this product in the launch
  int a[2], b[2];          // tensor map numbers
  int a_mn, b_mn;          // 1: the operand lies along its rows
  void *out;               // plain: [m][ld]
  const void *add;         // plain: added to the result, or NULL
  int64_t ld, add_ld;
  int out_bf16, add_bf16;
};

struct GemmArgs {
  CUtensorMap map[kMaxMaps];
  GemmProb p[kMaxProb];
  int n_prob, tiles;
  // gated epilogues: n columns of f values
  float *g, *u;                // swiglu: saved unless NULL; dswiglu: read
  __nv_bfloat16 *h, *dg, *du;  // swiglu: h; dswiglu: all three
  int64_t f_ld;
};

struct GemmTile {
  int p, m0, n0, steps;
};
__device__ __forceinline__ GemmTile gemm_tile(const GemmArgs &a, int t) {
  GemmTile r;
  r.p = 0;
  while (r.p + 1 < a.n_prob && t >= a.p[r.p + 1].tile0) ++r.p;
  const GemmProb &p = a.p[r.p];
  const int i = t - p.tile0;
  r.m0 = i / p.tiles_n * kBM;
  r.n0 = i % p.tiles_n;  // in tiles
  r.steps = p.segs * ((p.k + kBK - 1) / kBK);
  return r;
}

// MN-major operand, 128-byte swizzle: blocks of 64 rows x 64 k, each k one 128-byte line of 64
// rows; 8 k make 1024 bytes (stride offset), the next 64 rows lie 8192 bytes on (leading offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight values to or from a row; whole vectors only (f and the strides are multiples of 8).
__device__ __forceinline__ void put8(__nv_bfloat16 *p, const float *v) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void get8(const __nv_bfloat16 *p, float *v) {
  const uint4 q = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void put8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void get8(const float *p, float *v) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <int EPI>
__global__ void __launch_bounds__(kGemmThreads, 1) k_ffn_gemm(const __grid_constant__ GemmArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + kStages, *acc_full = empty + kStages,
           *acc_empty = acc_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + 512);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 516);
  unsigned char *stages = smem + 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t *err = &g_ffn_err;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 128);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
        const GemmTile tl = gemm_tile(a, t);
        const GemmProb &p = a.p[tl.p];
        const int per = tl.steps / p.segs;
        for (int s = 0; s < tl.steps; ++s, ++it) {
          const int st = it % kStages;
          if (it >= kStages && !(ok = pf_wait(&empty[st], ((it / kStages) - 1) & 1u, kSpin, abort_flag, err))) break;
          const int seg = s >= per, k0 = (s - seg * per) * kBK;
          unsigned char *sa = stages + st * kStageBytes, *sb = sa + kABytes;
          mbar_arrive_expect_tx(&full[st], kStageBytes);
          const CUtensorMap *ma = &a.map[p.a[seg]];
          if (p.a_mn)
            for (int i = 0; i < kBM / 64; ++i) tma_load_2d(sa + i * 8192, ma, tl.m0 + 64 * i, k0, &full[st]);
          else
            tma_load_2d(sa, ma, k0, tl.m0, &full[st]);
          if (EPI == kEpiSwiglu) {  // 128 rows of Wg, then the same rows of Wu
            tma_load_2d(sb, &a.map[p.b[0]], k0, tl.n0 * 128, &full[st]);
            tma_load_2d(sb + kBBytes / 2, &a.map[p.b[1]], k0, tl.n0 * 128, &full[st]);
          } else {
            const CUtensorMap *mb = &a.map[p.b[seg]];
            if (p.b_mn) {
              for (int i = 0; i < kBN / 64; ++i) tma_load_2d(sb + i * 8192, mb, tl.n0 * kBN + 64 * i, k0, &full[st]);
            } else {
              tma_load_2d(sb, mb, k0, tl.n0 * kBN, &full[st]);
              tma_load_2d(sb + kBBytes / 2, mb, k0, tl.n0 * kBN + 128, &full[st]);
            }
          }
        }
      }
      // leave only once every copy has landed
      for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
        mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1u, kDrainLimit);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x, ++n) {
        const GemmTile tl = gemm_tile(a, t);
        const GemmProb &p = a.p[tl.p];
        const int b = n & 1;
        if (n >= 2 && !(ok = pf_wait(&acc_empty[b], ((n >> 1) - 1) & 1u, kSpin, abort_flag, err))) break;
        tc_fence_after();
        const uint32_t idesc = idesc_bf16(kBN) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u);
        const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
        for (int s = 0; s < tl.steps; ++s, ++it) {
          const int st = it % kStages;
          if (!(ok = pf_wait(&full[st], (it / kStages) & 1u, kSpin, abort_flag, err))) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(stages + st * kStageBytes), sb = sa + kABytes;
          const uint64_t ad = p.a_mn ? mn_desc(sa) : sw128_desc(sa), bd = p.b_mn ? mn_desc(sb) : sw128_desc(sb);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tmem + b * kBN, ad + kk * a_step, bd + kk * b_step, idesc, s > 0 || kk > 0);
          tc_commit(&empty[st]);
        }
        if (ok) tc_commit(&acc_full[b]);
      }
      if (it > 0) mbar_wait_bounded(&empty[(it - 1) % kStages], ((it - 1) / kStages) & 1u, kDrainLimit);
    }
  } else {
    uint32_t n = 0;
    for (int t = blockIdx.x; t < a.tiles; t += gridDim.x, ++n) {
      const GemmTile tl = gemm_tile(a, t);
      const GemmProb &p = a.p[tl.p];
      const int b = n & 1;
      if (!pf_wait(&acc_full[b], (n >> 1) & 1u, kSpin, abort_flag, err)) break;
      tc_fence_after();
      const int row = tl.m0 + 32 * warp + lane;
      const uint32_t acc = tmem + b * kBN + (static_cast<uint32_t>(32 * warp) << 16);
      if (EPI == kEpiSwiglu) {
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t g[32], u[32];
          tmem_ld32_nowait(acc + c0, g);
          tmem_ld32_nowait(acc + 128 + c0, u);
          tmem_wait_ld();
          const int col = tl.n0 * 128 + c0;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (row >= p.m || col + i >= p.n) continue;
            const int64_t at = static_cast<int64_t>(row) * a.f_ld + col + i;
            float gv[8], uv[8], hv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              gv[k] = __uint_as_float(g[i + k]);
              uv[k] = __uint_as_float(u[i + k]);
              hv[k] = gv[k] * sigmoid_f(gv[k]) * uv[k];
            }
            put8(a.h + at, hv);
            if (a.g) {
              put8(a.g + at, gv);
              put8(a.u + at, uv);
            }
          }
        }
      } else {
        for (int c0 = 0; c0 < kBN; c0 += 32) {
          uint32_t v[32];
          tmem_ld32_nowait(acc + c0, v);
          tmem_wait_ld();
          const int col = tl.n0 * kBN + c0;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (row >= p.m || col + i >= p.n) continue;
            float d[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = __uint_as_float(v[i + k]);
            if (EPI == kEpiDswiglu) {
              const int64_t at = static_cast<int64_t>(row) * a.f_ld + col + i;
              float gv[8], uv[8], hv[8], dg[8], du[8];
              get8(a.g + at, gv);
              get8(a.u + at, uv);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float sg = sigmoid_f(gv[k]), sl = gv[k] * sg;
                hv[k] = sl * uv[k];
                du[k] = d[k] * sl;
                dg[k] = d[k] * uv[k] * (sg * (1.f + gv[k] * (1.f - sg)));
              }
              put8(a.h + at, hv);
              put8(a.dg + at, dg);
              put8(a.du + at, du);
            } else {
              if (p.add) {
                const int64_t at = static_cast<int64_t>(row) * p.add_ld + col + i;
                float e[8];
                if (p.add_bf16)
                  get8(static_cast<const __nv_bfloat16 *>(p.add) + at, e);
                else
                  get8(static_cast<const float *>(p.add) + at, e);
#pragma unroll
                for (int k = 0; k < 8; ++k) d[k] += e[k];
              }
              const int64_t at = static_cast<int64_t>(row) * p.ld + col + i;
              if (p.out_bf16)
                put8(static_cast<__nv_bfloat16 *>(p.out) + at, d);
              else
                put8(static_cast<float *>(p.out) + at, d);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[b]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------------------
// few tokens: mma.sync m16n8k16 with the weights as the 16-row operand, straight from global
// memory (a lane's 16-byte load is its operand of two MMAs: the order of k inside 32 is the same
// on both sides, so it does not matter), the tokens as the 8-column operand.  The block's warps
// take interleaved pieces of 32 k; their sums meet in shared memory and are added in warp order.
// ------------------------------------------------------------------------------------------
constexpr int kSmThreads = 256, kSmWarps = 8;
constexpr int kSmallMax = 32;  // tokens

struct SmallArgs {
  const __nv_bfloat16 *x, *wg, *wu, *wd;
  const void *add;
  void *y;
  __nv_bfloat16 *h;
  float *g, *u;
  int64_t x_ld, add_ld, y_ld;
  int n, d, f, add_bf16, y_bf16;
};

// acc[t] += rows r0 (lanes' g) and r1 (g + 8) of 16 weight rows times the tokens' rows x
template <int NT>
__device__ __forceinline__ void small_mma(const __nv_bfloat16 *r0, const __nv_bfloat16 *r1, bool ok0, bool ok1,
                                          const __nv_bfloat16 *x, int64_t x_ld, int n, int k_all, float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int kb = warp; kb < (k_all + 31) / 32; kb += kSmWarps) {
    const int k = 32 * kb + 8 * q;
    const bool in = k < k_all;
    const uint4 w0 = ok0 && in ? __ldg(reinterpret_cast<const uint4 *>(r0 + k)) : zero;
    const uint4 w1 = ok1 && in ? __ldg(reinterpret_cast<const uint4 *>(r1 + k)) : zero;
    const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = 8 * t + g;
      const uint4 b = row < n && in ? __ldg(reinterpret_cast<const uint4 *>(x + row * x_ld + k)) : zero;
      mma_bf16(acc[t], a0, b.x, b.y);
      mma_bf16(acc[t], a1, b.z, b.w);
    }
  }
}

// Sum over the block's warps, in warp order, of warp 0's view: red [warps - 1][NT * 4][32].
template <int NT>
__device__ __forceinline__ bool small_reduce(float (&acc)[NT][4], float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp)
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) red[((warp - 1) * NT * 4 + i) * 32 + lane] = acc[i >> 2][i & 3];
  __syncthreads();
  if (warp) return false;
  for (int w = 0; w < kSmWarps - 1; ++w)
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) acc[i >> 2][i & 3] += red[(w * NT * 4 + i) * 32 + lane];
  return true;
}

// Block: 8 rows of Wg (operand rows 0..7) and the same 8 of Wu (8..15): a lane gets g and u of the
// same row and tokens.
template <int NT>
__global__ void __launch_bounds__(kSmThreads) k_ffn_up(SmallArgs a) {
  __shared__ float red[(kSmWarps - 1) * NT * 4 * 32];
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, row = blockIdx.x * 8 + g;
  float acc[NT][4] = {};
  const bool ok = row < a.f;
  small_mma<NT>(a.wg + static_cast<int64_t>(row) * a.d, a.wu + static_cast<int64_t>(row) * a.d, ok, ok, a.x, a.x_ld, a.n,
                a.d, acc);
  if (!small_reduce<NT>(acc, red) || !ok) return;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tok = 8 * t + 2 * q + e;
      if (tok >= a.n) continue;
      const float gv = acc[t][e], uv = acc[t][2 + e];
      const int64_t at = static_cast<int64_t>(tok) * a.f + row;
      a.h[at] = __float2bfloat16_rn(gv * sigmoid_f(gv) * uv);
      if (a.g) {
        a.g[at] = gv;
        a.u[at] = uv;
      }
    }
}

// Block: 16 rows of Wd.
template <int NT>
__global__ void __launch_bounds__(kSmThreads) k_ffn_down(SmallArgs a) {
  __shared__ float red[(kSmWarps - 1) * NT * 4 * 32];
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, r0 = blockIdx.x * 16 + g, r1 = r0 + 8;
  float acc[NT][4] = {};
  small_mma<NT>(a.wd + static_cast<int64_t>(r0) * a.f, a.wd + static_cast<int64_t>(r1) * a.f, r0 < a.d, r1 < a.d, a.h,
                a.f, a.n, a.f, acc);
  if (!small_reduce<NT>(acc, red)) return;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = 8 * t + 2 * q + (e & 1), row = e < 2 ? r0 : r1;
      if (tok >= a.n || row >= a.d) continue;
      float v = acc[t][e];
      if (a.add) {
        const int64_t at = tok * a.add_ld + row;
        v += a.add_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.add)[at]) : static_cast<const float *>(a.add)[at];
      }
      const int64_t at = tok * a.y_ld + row;
      if (a.y_bf16)
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
      else
        static_cast<float *>(a.y)[at] = v;
    }
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Once per device, with it current: the encoder's address and the kernels' shared-memory limit.
cudaError_t ffn_setup(EncodeFn *out) {
  constexpr int kMaxDevices = 64;
  static std::mutex mutex;
  static EncodeFn encode = nullptr;
  static bool ready[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorNotSupported;
  std::lock_guard<std::mutex> lock(mutex);
  if (!encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    encode = reinterpret_cast<EncodeFn>(fn);
  }
  if (!ready[dev]) {
    const void *ks[] = {(const void *)k_ffn_gemm<kEpiPlain>, (const void *)k_ffn_gemm<kEpiSwiglu>,
                        (const void *)k_ffn_gemm<kEpiDswiglu>};
    for (const void *k : ks)
      if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem)) != cudaSuccess) return e;
    ready[dev] = true;
  }
  *out = encode;
  return cudaSuccess;
}

// bf16 [rows][cols] with a row stride of ld values, boxes of 64 columns x box_rows rows, 128-byte
// swizzle; what lies outside reads as zeros.
struct Maps {
  EncodeFn encode;
  GemmArgs &a;
  int n = 0;
  bool ok = true;
  int add(const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    ok = ok && n < kMaxMaps &&
         encode(&a.map[n], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    return n++;
  }
};

GemmProb &add_prob(GemmArgs &a, int m, int n, int k, int tile_n) {
  GemmProb &p = a.p[a.n_prob++];
  p.m = m, p.n = n, p.k = k, p.segs = 1;
  p.tiles_n = (n + tile_n - 1) / tile_n;
  p.tile0 = a.tiles;
  a.tiles += (m + kBM - 1) / kBM * p.tiles_n;
  return p;
}

template <int EPI>
cudaError_t launch_gemm(const GemmArgs &a, int nsm, cudaStream_t st) {
  k_ffn_gemm<EPI><<<a.tiles < nsm ? a.tiles : nsm, kGemmThreads, kGemmSmem, st>>>(a);
  return cudaGetLastError();
}

constexpr int kMaxDim = 65536;
bool bad_mat(const void *p) { return !p || !aligned16(p); }
bool bad_act(const void *p, int64_t ld, int d, int n, int bytes) {
  return !p || !aligned16(p) || ld * bytes % 16 || (n > 1 && ld < d);
}
bool bad_shape(int n, int d, int f) {
  return n < 1 || d < 8 || d % 8 || d > kMaxDim || f < 8 || f % 8 || f > kMaxDim;
}
uint64_t align_ws(uint64_t v) { return (v + 255) & ~uint64_t(255); }

}  // namespace

extern "C" uint64_t moe_ffn_workspace(int32_t n_tokens, int32_t d_model, int32_t d_ff, int32_t backward) {
  if (bad_shape(n_tokens, d_model, d_ff)) return 0;
  const uint64_t nf = align_ws(static_cast<uint64_t>(n_tokens) * d_ff * 2);
  return backward ? 3 * nf : nf;
}

extern "C" moe_status moe_ffn_forward(const moe_ffn_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_ffn_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model, f = p->d_ff;
  if (bad_shape(n, d, f) || bad_act(p->x, p->x_stride, d, n, 2) || bad_mat(p->w_gate) || bad_mat(p->w_up) ||
      bad_mat(p->w_down) || (p->y_dtype != MOE_F32 && p->y_dtype != MOE_BF16) ||
      bad_act(p->y, p->y_stride, d, n, p->y_dtype == MOE_BF16 ? 2 : 4) ||
      (p->add && ((p->add_dtype != MOE_F32 && p->add_dtype != MOE_BF16) ||
                  bad_act(p->add, p->add_stride, d, n, p->add_dtype == MOE_BF16 ? 2 : 4))) ||
      (p->save_gate != nullptr) != (p->save_up != nullptr) || (p->save_gate && (bad_mat(p->save_gate) || bad_mat(p->save_up))) ||
      bad_mat(p->workspace) || p->workspace_bytes < moe_ffn_workspace(n, d, f, 0))
    return MOE_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(p->workspace);
  cudaError_t e;
  if (n <= kSmallMax) {
    SmallArgs s{};
    s.x = static_cast<const __nv_bfloat16 *>(p->x), s.x_ld = p->x_stride;
    s.wg = static_cast<const __nv_bfloat16 *>(p->w_gate), s.wu = static_cast<const __nv_bfloat16 *>(p->w_up);
    s.wd = static_cast<const __nv_bfloat16 *>(p->w_down);
    s.add = p->add, s.add_ld = p->add_stride, s.add_bf16 = p->add_dtype == MOE_BF16;
    s.y = p->y, s.y_ld = p->y_stride, s.y_bf16 = p->y_dtype == MOE_BF16;
    s.h = h, s.g = static_cast<float *>(p->save_gate), s.u = static_cast<float *>(p->save_up);
    s.n = n, s.d = d, s.f = f;
    const int gu = (f + 7) / 8, gd = (d + 15) / 16;
    if (n <= 8)
      k_ffn_up<1><<<gu, kSmThreads, 0, st>>>(s), k_ffn_down<1><<<gd, kSmThreads, 0, st>>>(s);
    else if (n <= 16)
      k_ffn_up<2><<<gu, kSmThreads, 0, st>>>(s), k_ffn_down<2><<<gd, kSmThreads, 0, st>>>(s);
    else
      k_ffn_up<4><<<gu, kSmThreads, 0, st>>>(s), k_ffn_down<4><<<gd, kSmThreads, 0, st>>>(s);
    e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  EncodeFn encode = nullptr;
  int nsm = 0;
  if ((e = ffn_setup(&encode)) != cudaSuccess || (e = current_sm_count(&nsm)) != cudaSuccess) {
    cudaGetLastError();
    return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : MOE_ERR_CUDA;
  }
  GemmArgs a{};
  {
    Maps m{encode, a};
    GemmProb &q = add_prob(a, n, f, d, 128);
    q.a[0] = m.add(p->x, n, d, p->x_stride, kBM);
    q.b[0] = m.add(p->w_gate, f, d, d, 128);
    q.b[1] = m.add(p->w_up, f, d, d, 128);
    a.h = h, a.g = static_cast<float *>(p->save_gate), a.u = static_cast<float *>(p->save_up);
    a.f_ld = f;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
  }
  if ((e = launch_gemm<kEpiSwiglu>(a, nsm, st)) != cudaSuccess) return MOE_ERR_CUDA;
  GemmArgs b{};
  {
    Maps m{encode, b};
    GemmProb &q = add_prob(b, n, d, f, kBN);
    q.a[0] = m.add(h, n, f, f, kBM);
    q.b[0] = m.add(p->w_down, d, f, f, 128);
    q.out = p->y, q.ld = p->y_stride, q.out_bf16 = p->y_dtype == MOE_BF16;
    q.add = p->add, q.add_ld = p->add_stride, q.add_bf16 = p->add_dtype == MOE_BF16;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
  }
  e = launch_gemm<kEpiPlain>(b, nsm, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_ffn_backward(const moe_ffn_bwd_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_ffn_bwd_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model, f = p->d_ff;
  if (bad_shape(n, d, f) || bad_act(p->dy, p->dy_stride, d, n, 2) || bad_act(p->x, p->x_stride, d, n, 2) ||
      bad_mat(p->w_gate) || bad_mat(p->w_up) || bad_mat(p->w_down) || bad_mat(p->save_gate) || bad_mat(p->save_up) ||
      (p->dx && bad_act(p->dx, p->dx_stride, d, n, 2)) || (p->dw_gate != nullptr) != (p->dw_up != nullptr) ||
      (p->dw_gate && (bad_mat(p->dw_gate) || bad_mat(p->dw_up))) || (p->dw_down && bad_mat(p->dw_down)) ||
      (!p->dx && !p->dw_gate && !p->dw_down) || bad_mat(p->workspace) ||
      p->workspace_bytes < moe_ffn_workspace(n, d, f, 1))
    return MOE_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  EncodeFn encode = nullptr;
  int nsm = 0;
  cudaError_t e;
  if ((e = ffn_setup(&encode)) != cudaSuccess || (e = current_sm_count(&nsm)) != cudaSuccess) {
    cudaGetLastError();
    return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : MOE_ERR_CUDA;
  }
  const uint64_t nf = align_ws(static_cast<uint64_t>(n) * f * 2) / 2;
  __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(p->workspace), *dg = h + nf, *du = dg + nf;
  {
    GemmArgs a{};
    Maps m{encode, a};
    GemmProb &q = add_prob(a, n, f, d, kBN);
    q.a[0] = m.add(p->dy, n, d, p->dy_stride, kBM);
    q.b[0] = m.add(p->w_down, d, f, f, kBK), q.b_mn = 1;
    a.g = static_cast<float *>(const_cast<void *>(p->save_gate)), a.u = static_cast<float *>(const_cast<void *>(p->save_up));
    a.h = h, a.dg = dg, a.du = du, a.f_ld = f;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
    if ((e = launch_gemm<kEpiDswiglu>(a, nsm, st)) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (p->dx) {
    GemmArgs a{};
    Maps m{encode, a};
    GemmProb &q = add_prob(a, n, d, f, kBN);
    q.segs = 2;
    q.a[0] = m.add(dg, n, f, f, kBM), q.a[1] = m.add(du, n, f, f, kBM);
    q.b[0] = m.add(p->w_gate, f, d, d, kBK), q.b[1] = m.add(p->w_up, f, d, d, kBK), q.b_mn = 1;
    q.out = p->dx, q.ld = p->dx_stride, q.out_bf16 = 1;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
    if ((e = launch_gemm<kEpiPlain>(a, nsm, st)) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (p->dw_gate || p->dw_down) {
    GemmArgs a{};
    Maps m{encode, a};
    const int mh = p->dw_down ? m.add(h, n, f, f, kBK) : 0, mdy = p->dw_down ? m.add(p->dy, n, d, p->dy_stride, kBK) : 0;
    if (p->dw_gate) {
      const int mx = m.add(p->x, n, d, p->x_stride, kBK);
      for (int i = 0; i < 2; ++i) {
        GemmProb &q = add_prob(a, f, d, n, kBN);
        q.a[0] = m.add(i ? du : dg, n, f, f, kBK), q.b[0] = mx, q.a_mn = q.b_mn = 1;
        q.out = i ? p->dw_up : p->dw_gate, q.ld = d, q.out_bf16 = 1;
      }
    }
    if (p->dw_down) {
      GemmProb &q = add_prob(a, d, f, n, kBN);
      q.a[0] = mdy, q.b[0] = mh, q.a_mn = q.b_mn = 1;
      q.out = p->dw_down, q.ld = f, q.out_bf16 = 1;
    }
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
    if ((e = launch_gemm<kEpiPlain>(a, nsm, st)) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

extern "C" moe_status moe_ffn_check(void) {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_ffn_err, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (!v) return MOE_OK;
  v = 0;
  if (cudaMemcpyToSymbol(g_ffn_err, &v, sizeof v) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_ERR_TIMEOUT;
}
