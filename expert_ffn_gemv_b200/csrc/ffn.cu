// ffn.cu -- dense gated feed-forward block from bf16 weights and its gradients:
//   g = x Wg^T   u = x Wu^T   h = silu(g) * u   y = h Wd^T (+ add)
//   dh = dy Wd   dg = dh u silu'(g)   du = dh silu(g)
//   dx = dg Wg + du Wu   dWg = dg^T x   dWu = du^T x   dWd = dy^T h
// x, dy n x d; Wg, Wu f x d; Wd d x f; all products of bf16 values with fp32 accumulators, each
// result rounded once.  h, dg and du are operands of the next products and so in bf16: their rounding (half
// a step, up to 2^-8 of a value) is of the size of the bf16 results' own and adds to it (forward 2.4e-3 off
// 64 bits in relative 2-norm, 1.7e-3 with all of them in fp32); a second bf16 part of each would double the
// products that take them.  g and u, from which the backward computes h, dg and du again, are saved in
// fp32: in bf16 their rounding would come on top of it (gradients 3.5e-3 off, relative 2-norm, against
// 2.4e-3).
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

constexpr int kBK = 64;
constexpr int kMaxBN = 256;
constexpr uint64_t kSpin = 2000000000ull;  // about a second
constexpr int kMaxProb = 4, kMaxMaps = 9;

enum { kEpiPlain = 0, kEpiSwiglu = 1, kEpiDswiglu = 2 };

struct GemmProb {
  int m, n, k, segs;       // segs products over k added up (operands a[i], b[i])
  int tiles_m, tiles_n;
  int a[2], b[2];          // tensor map numbers
  int a_mn, b_mn;          // 1: the operand lies along its rows
  int a_rows;              // K-major A: rows of a box, all that the one tile of up to 128 rows has, or 128
  void *out;               // plain: [m][ld]
  const void *add;         // plain: added to the result, or NULL
  int64_t ld, add_ld;
  int out_bf16, add_bf16;
};

struct GemmArgs {
  CUtensorMap map[kMaxMaps];
  GemmProb p[kMaxProb];    // p[0] is dealt out first, then the others as one list
  int n_prob, bn;          // bn: columns of a tile (swiglu: bn / 2 of g and of u)
  uint32_t *err;           // set where a bounded wait ran out (NULL at the launch: the device's word)
  // gated epilogues: n columns of f values
  float *g, *u;                // swiglu: saved unless NULL; dswiglu: read
  __nv_bfloat16 *h, *dg, *du;  // swiglu: h; dswiglu: all three
  int64_t f_ld;
};

// Threads: sixteen epilogue warps (TMEM lanes 32 (w % 4) .., 32-column chunks w / 4, w / 4 + 4), a TMA
// producer warp, an MMA warp.  A CTA holds 128 rows of A and up to 128 rows of B per stage: tiles of
// 128 x 64 or 128 x 128 for one CTA, of 256 x 128 or 256 x 256 for a pair (cta_group::2), whose CTAs share
// their halves of B (choose_form).
// With eight epilogue warps the arithmetic of the gated ones (some 30 instructions a value) took 25 us
// a tile of 256 x 256, its 2048-deep product 12 us, and the last tile's plain one 4.3 us.
// Bound by the tensor cores under the power cap: 8,192 x 2,048 x 8,192 forward 596 us, 1,384 TFLOP/s; small
// products by latency (1,180 x 2,048 x 1,000 forward 29 us, its flops 9).
constexpr int kEpiWarps = 16, kGemmThreads = 32 * (kEpiWarps + 2);
constexpr int kABytes = 128 * kBK * 2, kBBytes = 128 * kBK * 2, kStageBytes = kABytes + kBBytes, kStages = 5;
constexpr int kGemmSmem = 1024 + 1024 + kStages * kStageBytes + kEpiWarps * 4096;

struct GemmTile {
  int p, m0, n0, s0, steps;  // k steps s0 .. s0 + steps - 1
};

// The tiles of unit c of g (a unit: the CTAs of one tile): p[0]'s tiles c, c + g, ..; then the other
// products' tiles as one list.  Where p[0] leaves some units a tile short, these take as many of the
// list's tiles as that tile was worth first, then the list goes round.  Inside a product, bands of
// eight tile rows, so that the tiles in flight share operands in L2.
struct GemmWalk {
  int c, g, n0, rest, r, k0, i, phase;
  int cur;  // product whose numbers are held here: a tile is placed without loads or integer divisions
  int tiles_m, tiles_n, steps;
  float inv_band;
  __device__ GemmWalk(const GemmArgs &a, int c_, int g_) : c(c_), g(g_), i(0), phase(0), cur(-1) {
    n0 = a.p[0].tiles_m * a.p[0].tiles_n;
    rest = 0;
    for (int p = 1; p < a.n_prob; ++p) rest += a.p[p].tiles_m * a.p[p].tiles_n;
    r = n0 % g;
    k0 = 0;
    if (rest) {
      const int s0 = a.p[0].segs * a.p[0].k, s1 = a.p[1].k;
      k0 = r ? (s0 + s1 / 2) / s1 : 0;
      if (static_cast<int64_t>(k0) * (g - r) > rest) k0 = rest / (g - r);
    }
  }
  __device__ bool next(const GemmArgs &a, GemmTile &t) {
    if (phase == 0) {
      const int j = c + i * g;
      if (j < n0) {
        ++i;
        place(a, 0, j, t);
        return true;
      }
      phase = 1, i = 0;
    }
    if (phase == 1) {
      if (c >= r && i < k0) {
        const int j = (c - r) + i * (g - r);
        ++i;
        pick(a, j, t);
        return true;
      }
      phase = 2, i = 0;
    }
    const int j = k0 * (g - r) + c + i * g;
    ++i;
    if (j >= rest) return false;
    pick(a, j, t);
    return true;
  }
  __device__ void pick(const GemmArgs &a, int j, GemmTile &t) {
    int p = 1;
    while (p + 1 < a.n_prob && j >= a.p[p].tiles_m * a.p[p].tiles_n) j -= a.p[p].tiles_m * a.p[p].tiles_n, ++p;
    place(a, p, j, t);
  }
  // j / d for j < 2^24: the float quotient is off by less than one
  static __device__ int div(int j, int d, float inv) {
    int q = static_cast<int>(static_cast<float>(j) * inv);
    q += (q + 1) * d <= j;
    q -= q * d > j;
    return q;
  }
  __device__ void place(const GemmArgs &a, int pi, int j, GemmTile &t) {
    constexpr int kBand = 8;
    if (pi != cur) {
      const GemmProb &p = a.p[pi];
      cur = pi, tiles_m = p.tiles_m, tiles_n = p.tiles_n;
      steps = p.segs * ((p.k + kBK - 1) / kBK);
      inv_band = 1.f / (kBand * tiles_n);
    }
    t.p = pi;
    t.s0 = 0, t.steps = steps;
    const int band = div(j, kBand * tiles_n, inv_band), in = j - band * kBand * tiles_n;
    const int rows = min(kBand, tiles_m - band * kBand);
    t.n0 = rows == kBand ? in / kBand : in / rows;
    t.m0 = band * kBand + in - t.n0 * rows;
  }
};

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

// ---- the cta_group::2 forms of tc05.cuh's helpers
template <int CG>
__device__ __forceinline__ void g_tmem_alloc(uint32_t *dst) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, 512);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void g_tmem_dealloc(uint32_t t) {
  if constexpr (CG == 1)
    tmem_dealloc(t, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
}
template <int CG>
__device__ __forceinline__ void g_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1) {
    tc_mma(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
}
// arrives on `bar` of every CTA of the tile
template <int CG>
__device__ __forceinline__ void g_commit(uint64_t *bar) {
  if constexpr (CG == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ uint32_t leader_addr(const void *p) {  // the same place in CTA 0 of the cluster
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// a tile of this CTA's operands, counted on the leader's barrier
template <int CG>
__device__ __forceinline__ void g_load(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar, uint32_t leader) {
  if constexpr (CG == 1)
    tma_load_2d(dst, map, x, y, bar);
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float (&v)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ float4 get4(const void *p, int64_t i, int bf16) {
  if (!bf16) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i);
  return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u), __uint_as_float(q.y << 16),
                     __uint_as_float(q.y & 0xFFFF0000u));
}

// The epilogue turns chunks of 32 rows x 32 accumulator columns round in shared memory: a lane of the
// TMEM load holds a row, a lane of the global accesses four columns of a row, so that these are whole
// sectors of consecutive columns.  16-byte pieces are exchanged (piece ^ row % 8): no bank conflicts.
__device__ __forceinline__ void turn_in(float *s, const uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    reinterpret_cast<uint4 *>(s)[lane * 8 + (c ^ (lane & 7))] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ float4 turn_out(const float *s, int row, int c) {
  return reinterpret_cast<const float4 *>(s)[row * 8 + (c ^ (row & 7))];
}

// 32 rows x 32 columns of bf16 results, a row a lane, to global memory: turned in 2 KB, then a lane
// stores eight columns (16 bytes), four lanes a row.
__device__ __forceinline__ void store_bf16(float *scratch, const uint32_t (&v)[16], int lane, __nv_bfloat16 *out, int64_t ld,
                                           int row0, int rows, int col0, int cols) {
  uint4 *s = reinterpret_cast<uint4 *>(scratch);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    s[lane * 4 + (c ^ ((lane >> 1) & 3))] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  const int r0 = lane >> 2, c = lane & 3, col = col0 + 8 * c;
  uint4 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = s[(r0 + 8 * i) * 4 + (c ^ (((r0 + 8 * i) >> 1) & 3))];
  __nv_bfloat16 *p = out + (row0 + r0) * ld + col;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col < cols && row0 + r0 + 8 * i < rows) *reinterpret_cast<uint4 *>(p + 8 * i * ld) = q[i];
}
// The same for fp32: 4 KB, four columns a lane, eight lanes a row.
__device__ __forceinline__ void store_f32(float *scratch, const uint32_t (&v)[32], int lane, float *out, int64_t ld, int row0,
                                          int rows, int col0, int cols) {
  __syncwarp();
  turn_in(scratch, v, lane);
  __syncwarp();
  const int r0 = lane >> 3, c = lane & 7, col = col0 + 4 * c;
  float *p = out + (row0 + r0) * ld + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 q = turn_out(scratch, r0 + 4 * i, c);
    if (col < cols && row0 + r0 + 4 * i < rows) *reinterpret_cast<float4 *>(p + 4 * i * ld) = q;
  }
}

// h and the gradients of g and u, where the gradient of h is dh
__device__ __forceinline__ void dswiglu(float g, float u, float dh, float &h, float &dg, float &du) {
  const float sg = fast_sigmoid(g), sl = g * sg;
  h = sl * u;
  dg = dh * u * fmaf(sl, 1.f - sg, sg);
  du = dh * sl;
}

// SPLIT: the k range of a tile is dealt to the CTAs of a cluster, which then lay their sums in shared
// memory (the stages, no longer used), each as chunks of 32 x 32 values; every CTA adds up a share of the
// values over the cluster, in the order of its CTAs, and finishes them.  For products with fewer tiles than
// SMs: 64 tokens, d 4,096, f 768, forward 17 us, with the pieces of the down product alone split and added
// up through global memory 33; 64 x 2,208 x 752, all gradients, 25 us (39).  Of such a kernel's 5 us the
// first copies take 1.6, the cluster's meeting and parting 1.5, the sums 1.
__device__ __forceinline__ int chunk_at(int row, int c4, int bn) {  // float4 c4 of a row, in 16-byte pieces
  return ((row >> 5) * (bn >> 5) + (c4 >> 3)) * 256 + (row & 31) * 8 + ((c4 & 7) ^ (row & 7));
}
__device__ __forceinline__ float4 cluster_total(uint32_t base, int at, uint32_t ctas) {
  float4 q[8];
#pragma unroll
  for (uint32_t r = 0; r < 8; ++r) {
    if (r >= ctas) break;
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(base + 16 * at), "r"(r));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(q[r].x), "=f"(q[r].y), "=f"(q[r].z), "=f"(q[r].w)
                 : "r"(p)
                 : "memory");
  }
  float4 d = q[0];
#pragma unroll
  for (uint32_t r = 1; r < 8; ++r)
    if (r < ctas) d.x += q[r].x, d.y += q[r].y, d.z += q[r].z, d.w += q[r].w;
  return d;
}
template <int EPI>
__device__ __forceinline__ void split_epilogue(const GemmArgs &a, const GemmTile &tl, uint32_t base, uint32_t rank, uint32_t ctas,
                                               int tid) {
  const GemmProb &p = a.p[0];
  const int wide = EPI == kEpiSwiglu ? a.bn / 2 : a.bn, log4 = 29 - __clz(wide);  // values of a row, log2 of its float4s
  const int row0 = tl.m0 * 128, rows = min(128, p.m - row0), step = 32 * kEpiWarps;
  for (int e = rank * step + tid; e < rows << log4; e += ctas * step) {
    const int r = e >> log4, c4 = e & ((1 << log4) - 1), col = tl.n0 * wide + 4 * c4;
    if (col >= p.n) continue;
    const int64_t row = row0 + r;
    const float4 q = cluster_total(base, chunk_at(r, c4, a.bn), ctas);
    float d[4] = {q.x, q.y, q.z, q.w};
    if (EPI == kEpiSwiglu) {
      const float4 u = cluster_total(base, chunk_at(r, wide / 4 + c4, a.bn), ctas);
      const int64_t at = row * a.f_ld + col;
      if (a.g) {
        *reinterpret_cast<float4 *>(a.g + at) = q;
        *reinterpret_cast<float4 *>(a.u + at) = u;
      }
      const float w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = d[k] * fast_sigmoid(d[k]) * w[k];
      put4(a.h + at, d);
    } else if (EPI == kEpiPlain) {
      if (p.add) {
        const float4 x = get4(p.add, row * p.add_ld + col, p.add_bf16);
        d[0] += x.x, d[1] += x.y, d[2] += x.z, d[3] += x.w;
      }
      if (p.out_bf16)
        put4(static_cast<__nv_bfloat16 *>(p.out) + row * p.ld + col, d);
      else
        put4(static_cast<float *>(p.out) + row * p.ld + col, d);
    } else {
      const int64_t at = row * a.f_ld + col;
      const float4 g = *reinterpret_cast<const float4 *>(a.g + at), u = *reinterpret_cast<const float4 *>(a.u + at);
      const float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
      float h[4], dg[4], du[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) dswiglu(gv[k], uv[k], d[k], h[k], dg[k], du[k]);
      put4(a.h + at, h);
      put4(a.dg + at, dg);
      put4(a.du + at, du);
    }
  }
}

template <int EPI, int CG, bool SPLIT>
__global__ void __launch_bounds__(kGemmThreads, 1) k_ffn_gemm(const __grid_constant__ GemmArgs a) {
  constexpr int NS = kStages, EW = kEpiWarps;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + NS, *acc_full = empty + NS, *acc_empty = acc_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + 512);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 516);
  unsigned char *stages = smem + 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t part = 0, parts = 1;  // this CTA's piece of the k range
  if (SPLIT) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(part));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
  }
  const int size = SPLIT ? parts : CG, rank = CG == 2 ? blockIdx.x & 1 : 0, unit = blockIdx.x / size, units = gridDim.x / size;
  const int bn = a.bn, bl = bn / CG;  // columns of a tile, B rows of a CTA
  uint32_t *err = a.err;

  if (warp == EW && lane < kMaxMaps)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.map[lane])) : "memory");
  GemmWalk walk(a, unit, units);
  GemmTile tl;
  auto next = [&]() {
    if (!walk.next(a, tl)) return false;
    if (SPLIT) {
      tl.s0 = static_cast<int>(tl.steps * part / parts);
      tl.steps = static_cast<int>(tl.steps * (part + 1) / parts) - tl.s0;
    }
    return true;
  };
  bool have = next();  // the first tile is placed while the barriers and TMEM are set up

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], EW * CG);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) g_tmem_alloc<CG>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == EW) {
    // ---------------- producer: this CTA's rows of both operands.  Lane l issues the step's copy l (the
    // one or two boxes of A, then those of B), with its map and coordinates worked out once a tile: one
    // lane that issued them all and looked them up spent 880 clocks a step on it, the MMAs take 512.
    uint32_t it = 0;
    bool ok = true;
    bool waited = false;
    for (; ok && have; have = next()) {
      const GemmProb &p = a.p[tl.p];
      const uint32_t tx = CG * ((p.a_mn ? kABytes : p.a_rows * kBK * 2) + bl * kBK * 2);
      const int per = (p.k + kBK - 1) / kBK, m0 = (tl.m0 * CG + rank) * 128, na = p.a_mn ? 2 : 1;
      const bool is_a = lane < na, mine = lane < na + bl / 64, mn = is_a ? p.a_mn : p.b_mn;
      const int box = is_a ? lane : lane - na;
      const uint32_t off = is_a ? box * 8192 : kABytes + box * 8192;
      int row = is_a ? m0 + 64 * box : rank * bl + 64 * box, m_first = is_a ? p.a[0] : p.b[0], m_then = is_a ? p.a[1] : p.b[1];
      if (!is_a && EPI == kEpiSwiglu) {
        // the first half of the tile's B rows are Wg's, the second half the same rows of Wu
        const int half = bn / 2, up = row >= half;
        m_first = up ? m_then : m_first;
        row = tl.n0 * half + row - up * half;
      } else if (!is_a) {
        row += tl.n0 * bn;
      }
      const CUtensorMap *map = &a.map[m_first];
      const CUtensorMap *then = &a.map[m_then];
      if (tl.s0 > per) map = then;
      int k = (tl.s0 > per ? tl.s0 - per : tl.s0) * kBK;
      if (!waited) {
        griddep_wait();
        griddep_launch();
        waited = true;
      }
      for (int s = tl.s0; s < tl.s0 + tl.steps; ++s, ++it) {
        const int st = it % NS;
        const bool got = it < NS || pf_wait(&empty[st], ((it / NS) - 1) & 1u, kSpin, abort_flag, err);
        if (!(ok = __all_sync(0xffffffffu, got))) break;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&full[st], tx);
        __syncwarp();
        if (s == per) map = then, k = 0;
        if (mine)
          g_load<CG>(stages + st * kStageBytes + off, map, mn ? row : k, mn ? k : row, &full[st],
                     CG == 2 ? leader_addr(&full[st]) : 0);
        k += kBK;
      }
    }
    __syncwarp();
    // leave only once every copy has landed (the leader's barriers count both CTAs' copies) and every
    // stage's commit has arrived
    if (lane == 0)
      for (uint32_t k = it > NS ? it - NS : 0; k < it; ++k) {
        if (rank == 0) mbar_wait_bounded(&full[k % NS], (k / NS) & 1u, kDrainLimit);
        if (ok) mbar_wait_bounded(&empty[k % NS], (k / NS) & 1u, kDrainLimit);
      }
  } else if (warp == EW + 1) {
    // ---------------- MMA issue (one thread of the leader)
    if (lane == 0 && rank == 0) {
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (; ok && have; have = next(), ++n) {
        const GemmProb &p = a.p[tl.p];
        const int b = n & 1;
        if (n >= 2 && !(ok = pf_wait(&acc_empty[b], ((n >> 1) - 1) & 1u, kSpin, abort_flag, err))) break;
        tc_fence_after();
        const uint32_t idesc = (idesc_bf16(bn) & 0x00FFFFFFu) | (static_cast<uint32_t>(128 * CG >> 4) << 24) |
                               (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u);
        const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
        const uint32_t sa = smem_u32(stages), sb = sa + kABytes;
        const uint64_t ad0 = p.a_mn ? mn_desc(sa) : sw128_desc(sa), bd0 = p.b_mn ? mn_desc(sb) : sw128_desc(sb);
        const uint32_t acc = tmem + b * kMaxBN;
        for (int s = 0; s < tl.steps; ++s, ++it) {
          const int st = it % NS;
          if (!(ok = pf_wait(&full[st], (it / NS) & 1u, kSpin, abort_flag, err))) break;
          tc_fence_after();
          const uint64_t ad = ad0 + (st * kStageBytes >> 4), bd = bd0 + (st * kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            g_mma<CG>(acc, ad + kk * a_step, bd + kk * b_step, idesc, s > 0 || kk > 0);
          g_commit<CG>(&empty[st]);
        }
        if (ok) g_commit<CG>(&acc_full[b]);
      }
      if (it > 0) mbar_wait_bounded(&empty[(it - 1) % NS], ((it - 1) / NS) & 1u, kDrainLimit);
    }
  } else if (SPLIT) {
    // ---------------- epilogue, one tile: the sums to shared memory
    const int c0 = 32 * (warp >> 2);
    griddep_wait();
    griddep_launch();
    if (have && __all_sync(0xffffffffu, pf_wait(&acc_full[0], 0u, kSpin, abort_flag, err)) && c0 < bn) {
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32_nowait(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c0, v);
      tmem_wait_ld();
      turn_in(reinterpret_cast<float *>(stages) + ((warp & 3) * (bn / 32) + c0 / 32) * 1024, v, lane);
    }
  } else {
    // ---------------- epilogue
    float *scratch = reinterpret_cast<float *>(stages + NS * kStageBytes + warp * 4096);
    const uint32_t quad = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    uint32_t n = 0;
    griddep_wait();  // nothing before this touched global memory (nor do the MMA warp's lanes)
    griddep_launch();
    for (; have; have = next()) {
      const int b = n & 1, rows = a.p[tl.p].m, cols = a.p[tl.p].n;
      const int row0 = (tl.m0 * CG + rank) * 128 + 32 * (warp & 3), first = 32 * (warp >> 2);
      const uint32_t acc = tmem + b * kMaxBN + quad;
      // dswiglu: a lane takes eight columns of a row of g, u and the results; the first g and u are on
      // their way while the accumulators are waited for
      float4 gq[2][2], uq[2][2];
      const int c = lane & 3, r0 = lane >> 2;
      auto fetch = [&](int c0, int h) {  // rows 16 h + 8 i + lane / 4 of the chunk at column c0
        const int col = tl.n0 * bn + c0 + 8 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = row0 + 16 * h + 8 * i + r0;
          if (row < rows && col < cols) {
            const float4 *gp = reinterpret_cast<const float4 *>(a.g + row * a.f_ld + col);
            const float4 *up = reinterpret_cast<const float4 *>(a.u + row * a.f_ld + col);
            gq[i][0] = gp[0], gq[i][1] = gp[1], uq[i][0] = up[0], uq[i][1] = up[1];
          }
        }
      };
      if (EPI == kEpiDswiglu && first < bn) fetch(first, 0);
      if (!__all_sync(0xffffffffu, pf_wait(&acc_full[b], (n >> 1) & 1u, kSpin, abort_flag, err))) break;
      ++n;
      tc_fence_after();
      // the accumulators are handed back as soon as this warp's last chunk is in registers, before its
      // stores: a release at cluster scope after them would wait for all of them (2,000 clocks)
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(&acc_empty[b])) : "memory");
          else
            mbar_arrive(&acc_empty[b]);
        }
      };
      if (EPI == kEpiSwiglu) {
        const int half = bn / 2, col = tl.n0 * half + first;  // at most one chunk of g and u a warp
        if (first < half) {
          uint32_t v[32], w[32];
          tmem_ld32_nowait(acc + first, v);
          tmem_ld32_nowait(acc + half + first, w);
          tmem_wait_ld();
          release();
          if (a.g) {
            store_f32(scratch, v, lane, a.g, a.f_ld, row0, rows, col, cols);
            store_f32(scratch, w, lane, a.u, a.f_ld, row0, rows, col, cols);
          }
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float g0 = __uint_as_float(v[2 * i]), g1 = __uint_as_float(v[2 * i + 1]);
            h[i] = pack2(g0 * fast_sigmoid(g0) * __uint_as_float(w[2 * i]), g1 * fast_sigmoid(g1) * __uint_as_float(w[2 * i + 1]));
          }
          store_bf16(scratch, h, lane, a.h, a.f_ld, row0, rows, col, cols);
        } else {
          release();
        }
      } else if (EPI == kEpiPlain) {
        const void *add = a.p[tl.p].add;
        void *out = a.p[tl.p].out;
        const int64_t ld = a.p[tl.p].ld, add_ld = a.p[tl.p].add_ld;
        const int out_bf16 = a.p[tl.p].out_bf16, add_bf16 = a.p[tl.p].add_bf16;
        if (first >= bn) release();
        for (int c0 = first; c0 < bn; c0 += 8 * EW) {
          uint32_t v[32];
          tmem_ld32_nowait(acc + c0, v);
          tmem_wait_ld();
          if (c0 + 8 * EW >= bn) release();
          const int col = tl.n0 * bn + c0;
          if (add) {
            // added a row a lane: whole sectors of that row
            const int row = row0 + lane;
            if (row < rows) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (col + i < cols) {
                  const float4 e = get4(add, row * add_ld + col + i, add_bf16);
                  const float f[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) v[i + k] = __float_as_uint(__uint_as_float(v[i + k]) + f[k]);
                }
            }
            __syncwarp();
          }
          if (out_bf16) {
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            store_bf16(scratch, h, lane, static_cast<__nv_bfloat16 *>(out), ld, row0, rows, col, cols);
          } else {
            store_f32(scratch, v, lane, static_cast<float *>(out), ld, row0, rows, col, cols);
          }
        }
      } else {
        if (first >= bn) release();
        for (int c0 = first; c0 < bn; c0 += 8 * EW) {
          if (c0 != first) fetch(c0, 0);
          uint32_t v[32];
          tmem_ld32_nowait(acc + c0, v);
          tmem_wait_ld();
          if (c0 + 8 * EW >= bn) release();
          __syncwarp();
          turn_in(scratch, v, lane);
          __syncwarp();
          const int col = tl.n0 * bn + c0 + 8 * c;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h) fetch(c0, 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 16 * h + 8 * i + r0, row = row0 + r;
              const float4 d0 = turn_out(scratch, r, 2 * c), d1 = turn_out(scratch, r, 2 * c + 1);
              if (row >= rows || col >= cols) continue;
              const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
              const float gv[8] = {gq[i][0].x, gq[i][0].y, gq[i][0].z, gq[i][0].w, gq[i][1].x, gq[i][1].y, gq[i][1].z, gq[i][1].w};
              const float uv[8] = {uq[i][0].x, uq[i][0].y, uq[i][0].z, uq[i][0].w, uq[i][1].x, uq[i][1].y, uq[i][1].z, uq[i][1].w};
              uint32_t hv[4], dg[4], du[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float x[2][3];
#pragma unroll
                for (int e = 0; e < 2; ++e) dswiglu(gv[2 * k + e], uv[2 * k + e], d[2 * k + e], x[e][0], x[e][1], x[e][2]);
                hv[k] = pack2(x[0][0], x[1][0]), dg[k] = pack2(x[0][1], x[1][1]), du[k] = pack2(x[0][2], x[1][2]);
              }
              const int64_t at = row * a.f_ld + col;
              *reinterpret_cast<uint4 *>(a.h + at) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
              *reinterpret_cast<uint4 *>(a.dg + at) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
              *reinterpret_cast<uint4 *>(a.du + at) = make_uint4(du[0], du[1], du[2], du[3]);
            }
          }
        }
      }
    }
  }
  __syncwarp();
  if (SPLIT) {
    cluster_sync();  // the sums of all CTAs are there
    if (warp < EW) split_epilogue<EPI>(a, tl, smem_u32(stages), part, parts, tid);
    __syncwarp();
    cluster_sync();  // and have been read
  }
  tc_fence_before();
  __syncthreads();
  // a CTA's shared memory is read by the pair's MMAs and its barriers are arrived on by the other CTA
  if (CG == 2) cluster_sync();
  if (warp == 0) g_tmem_dealloc<CG>(tmem);
}

// ------------------------------------------------------------------------------------------
// few tokens: mma.sync m16n8k16 with the weights as the 16-row operand, straight from global
// memory (a lane's 16-byte load is its operand of two MMAs: the order of k inside 32 is the same
// on both sides, so it does not matter), the tokens as the 8-column operand.  A cluster of CL blocks
// has 16 rows; its blocks take runs of k, their warps interleaved pieces of 64 k (128 bytes of a row);
// the sums meet in shared memory, then over the cluster, and are added in warp and block order.
// Bound by the weights' bytes: what counts is loads on their way, so there are up to eight small blocks
// an SM and eight weight loads a lane.  8 tokens, d 2,048, f 8,192 (100 MB of weights): 29 us, 3.4 TB/s;
// with one block an SM in the down product 41, with four blocks of eight warps 31, with twelve of four
// warps and half the loads 30, with two persistent blocks fed by cp.async 38.
// ------------------------------------------------------------------------------------------
constexpr int kSmThreads = 128, kSmWarps = 4;
constexpr int kSmallMax = 8;  // tokens: the MMA's columns (16 in two column groups took 38 us; k_ffn_gemm takes 28.5 for 12)

struct SmallArgs {
  const __nv_bfloat16 *x, *wg, *wu, *wd;
  const void *add;
  void *y;
  __nv_bfloat16 *h;
  float *g, *u;
  int64_t x_ld, add_ld, y_ld;
  int n, d, f, add_bf16, y_bf16;
};

// acc = rows r0 (lanes' g) and r1 (g + 8) of 16 weight rows times the tokens' rows x, summed over
// the cluster; true in the lanes that hold the result (warp 0 of block 0).  `ready` is called before x
// is read.
template <typename F>
__device__ __forceinline__ bool small_product(const __nv_bfloat16 *r0, const __nv_bfloat16 *r1, bool ok0, bool ok1,
                                              const __nv_bfloat16 *x, int64_t x_ld, int n, int k_all, float (&acc)[4], F ready) {
  __shared__ float red[kSmWarps - 1][4][32];
  __shared__ float part[4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  uint32_t cl, cr;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(cr));
  const int pieces = (k_all + 63) / 64, p0 = static_cast<int>(pieces * cr / cl) + warp, p1 = static_cast<int>(pieces * (cr + 1) / cl);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int AHEAD = 2;  // pieces of weights on their way
  uint4 w[AHEAD][2][2];
  auto fetch = [&](int p, uint4 (&to)[2][2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = 64 * p + 32 * s + 8 * q;
      const bool in = p < p1 && k < k_all;
      to[0][s] = ok0 && in ? __ldg(reinterpret_cast<const uint4 *>(r0 + k)) : zero;
      to[1][s] = ok1 && in ? __ldg(reinterpret_cast<const uint4 *>(r1 + k)) : zero;
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(p0 + i * kSmWarps, w[i]);
  ready();
  for (int p = p0; p < p1; p += AHEAD * kSmWarps) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int at = p + i * kSmWarps;
      uint4 b[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = 64 * at + 32 * s + 8 * q;
        b[s] = g < n && at < p1 && k < k_all ? *reinterpret_cast<const uint4 *>(x + g * x_ld + k) : zero;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t a0[4] = {w[i][0][s].x, w[i][1][s].x, w[i][0][s].y, w[i][1][s].y};
        const uint32_t a1[4] = {w[i][0][s].z, w[i][1][s].z, w[i][0][s].w, w[i][1][s].w};
        mma_bf16(acc, a0, b[s].x, b[s].y);
        mma_bf16(acc, a1, b[s].z, b[s].w);
      }
      fetch(at + AHEAD * kSmWarps, w[i]);
    }
  }
  if (warp)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp - 1][i][lane] = acc[i];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int v = 0; v < kSmWarps - 1; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += red[v][i][lane];
  }
  if (cl == 1) return warp == 0;
  if (warp == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i][lane] = acc[i];
  cluster_sync();
  const bool mine = warp == 0 && cr == 0;
  if (mine)
    for (uint32_t c = 1; c < cl; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t at;
        float v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&part[i][lane])), "r"(c));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
        acc[i] += v;
      }
  cluster_sync();  // a block's sums are read before it leaves
  return mine;
}

// Cluster: 8 rows of Wg (operand rows 0..7) and the same 8 of Wu (8..15): a lane gets g and u of the
// same row and tokens.
__global__ void __launch_bounds__(kSmThreads, 8) k_ffn_up(SmallArgs a, int cl) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, row = blockIdx.x / cl * 8 + g;
  float acc[4] = {};
  const bool ok = row < a.f;
  griddep_wait();
  griddep_launch();
  const bool mine = small_product(a.wg + static_cast<int64_t>(row) * a.d, a.wu + static_cast<int64_t>(row) * a.d, ok, ok, a.x,
                                      a.x_ld, a.n, a.d, acc, [] {});
  if (!mine || !ok) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int tok = 2 * q + e;
    if (tok >= a.n) continue;
    const float gv = acc[e], uv = acc[2 + e];
    const int64_t at = static_cast<int64_t>(tok) * a.f + row;
    a.h[at] = __float2bfloat16_rn(gv * fast_sigmoid(gv) * uv);
    if (a.g) {
      a.g[at] = gv;
      a.u[at] = uv;
    }
  }
}

// Cluster: 16 rows of Wd.  Launched while k_ffn_up ends (which began when everything before it had
// completed), it has weights on their way before it waits for h.
__global__ void __launch_bounds__(kSmThreads, 8) k_ffn_down(SmallArgs a, int cl) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, r0 = blockIdx.x / cl * 16 + g, r1 = r0 + 8;
  float acc[4] = {};
  const bool mine = small_product(a.wd + static_cast<int64_t>(r0) * a.f, a.wd + static_cast<int64_t>(r1) * a.f, r0 < a.d, r1 < a.d,
                                      a.h, a.f, a.n, a.f, acc, [] {
                                        griddep_wait();
                                        griddep_launch();
                                      });
  if (!mine) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int tok = 2 * q + (e & 1), row = e < 2 ? r0 : r1;
    if (tok >= a.n || row >= a.d) continue;
    float v = acc[e];
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

template <int EPI>
cudaError_t configure_gemm() {
  for (const void *k : {reinterpret_cast<const void *>(k_ffn_gemm<EPI, 1, false>), reinterpret_cast<const void *>(k_ffn_gemm<EPI, 2, false>),
                        reinterpret_cast<const void *>(k_ffn_gemm<EPI, 1, true>)}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Launch configuration: clusters of cg CTAs, programmatic stream serialization (the kernel may begin
// while the one before it ends; it waits for that one's results itself).
struct Config {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  Config(int grid, int threads, int smem, int cg, cudaStream_t st) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cg;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cg > 1 ? 2 : 1;
  }
};

constexpr int kMaxParts = 8;
struct FfnDevice {
  EncodeFn encode;
  int nsm, pairs;              // CTA pairs the device holds at once
  int clusters[kMaxParts + 1];  // and clusters of so many CTAs of a split product
};

// Once per device, with it current: the encoder's address, the kernels' shared-memory limit, sizes.
cudaError_t ffn_setup(FfnDevice *out) {
  constexpr int kMaxDevices = 64;
  static std::mutex mutex;
  static FfnDevice known[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorNotSupported;
  std::lock_guard<std::mutex> lock(mutex);
  FfnDevice &k = known[dev];
  if (!k.encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    e = current_sm_count(&k.nsm);
    if (e == cudaSuccess) e = configure_gemm<kEpiPlain>();
    if (e == cudaSuccess) e = configure_gemm<kEpiSwiglu>();
    if (e == cudaSuccess) e = configure_gemm<kEpiDswiglu>();
    if (e != cudaSuccess) return e;
    const Config two(2, kGemmThreads, kGemmSmem, 2, nullptr);
    e = cudaOccupancyMaxActiveClusters(&k.pairs, k_ffn_gemm<kEpiPlain, 2, false>, &two.cfg);
    for (int c = 2; e == cudaSuccess && c <= kMaxParts; ++c) {
      const Config of(c, kGemmThreads, kGemmSmem, c, nullptr);
      e = cudaOccupancyMaxActiveClusters(&k.clusters[c], k_ffn_gemm<kEpiPlain, 1, true>, &of.cfg);
    }
    if (e != cudaSuccess) return e;
    if (k.pairs > k.nsm / 2) k.pairs = k.nsm / 2;
    k.encode = reinterpret_cast<EncodeFn>(fn);
  }
  *out = k;
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

int box_rows(int m) { return m < 128 ? (m + 7) & ~7 : 128; }
GemmProb &add_prob(GemmArgs &a, int m, int n, int k) {
  GemmProb &p = a.p[a.n_prob++];
  p.m = m, p.n = n, p.k = k, p.segs = 1, p.a_rows = box_rows(m);
  return p;
}

// How a launch is tiled: a unit is one CTA on tiles of 128 x bn, a pair of CTAs on tiles of 256 x bn, which
// read half as many operand bytes for their products, or (one product alone) a cluster of `parts` CTAs that
// share the k range of a tile.  The rule takes what fills the device in the least time, by the clocks of a
// 64-deep step of each tile (all gradients, mean of 56 shapes: kJoin 1 40.2 us, 4 39.2, 8 39.9).
struct Form {
  int cg, bn, parts;
  double clocks;
};
template <int EPI>
Form choose_form(const GemmProb *prob, int n_prob, const FfnDevice &dev, bool split = true) {
  constexpr struct { int cg, bn, step; } forms[] = {{2, 256, 800}, {2, 128, 560}, {1, 128, 560}, {1, 64, 420}};
  constexpr int kFill = 4, kJoin = 4;  // steps' worth of filling and draining, of adding up over a cluster
  Form best{};
  for (const auto &c : forms) {
    if (EPI == kEpiSwiglu && c.bn == 64) continue;  // 64 rows each of two matrices at least
    const int cols = EPI == kEpiSwiglu ? c.bn / 2 : c.bn;
    for (int parts = 1; parts <= (split && c.cg == 1 && n_prob == 1 ? kMaxParts : 1); ++parts) {
      const int units = parts > 1 ? dev.clusters[parts] : c.cg == 2 ? dev.pairs : dev.nsm;
      if (units < 1) continue;
      double steps = 0, longest = 0;  // of all tiles and of the longest
      bool fits = true;
      for (int i = 0; i < n_prob; ++i) {
        const GemmProb &p = prob[i];
        const int deep = p.segs * ((p.k + kBK - 1) / kBK);
        const double len = parts > 1 ? (deep + parts - 1) / parts + kFill + kJoin : deep + kFill;
        const double tiles = static_cast<double>((p.m + 128 * c.cg - 1) / (128 * c.cg)) * ((p.n + cols - 1) / cols);
        fits = fits && (parts == 1 || (deep >= parts && tiles * parts <= dev.nsm));
        // alone, whole rounds of tiles; among others, what is left over is filled up
        steps += n_prob == 1 ? len * units * static_cast<int>((tiles + units - 1) / units) : len * tiles;
        longest = longest > len ? longest : len;
      }
      const double t = (steps / units > longest ? steps / units : longest) * c.step;
      if (fits && (!best.cg || t < best.clocks)) best = Form{c.cg, c.bn, parts, t};
    }
  }
  return best;
}

// Whether dx is split over its k range in a launch of its own: where that takes less than its tiles beside
// those of the weights' gradients.  By the sizes alone: dx has the same bits whatever else is asked for.
bool dx_apart(int n, int d, int f, const FfnDevice &dev) {
  constexpr double kLaunch = 4000;  // clocks
  GemmProb p[4] = {};
  p[0].m = n, p[0].n = d, p[0].k = f, p[0].segs = 2;
  for (int i = 1; i < 4; ++i) p[i].m = i < 3 ? f : d, p[i].n = i < 3 ? d : f, p[i].k = n, p[i].segs = 1;
  const Form alone = choose_form<kEpiPlain>(p, 1, dev), rest = choose_form<kEpiPlain>(p + 1, 3, dev);
  // (a list of unlike tiles takes some 15 % longer than its sums say)
  return alone.parts > 1 && alone.clocks + rest.clocks + kLaunch < 1.15 * choose_form<kEpiPlain>(p, 4, dev).clocks;
}

template <int EPI>
cudaError_t launch_gemm(GemmArgs &a, const FfnDevice &dev, cudaStream_t st, bool split = true) {
  const Form f = choose_form<EPI>(a.p, a.n_prob, dev, split);
  a.bn = f.bn;
  if (!a.err) {
    BlockWord word;
    const cudaError_t e = block_word(&word);
    if (e != cudaSuccess) return e;
    a.err = word.dev;
  }
  const int cols = EPI == kEpiSwiglu ? f.bn / 2 : f.bn;
  int tiles = 0;
  for (int i = 0; i < a.n_prob; ++i) {
    GemmProb &p = a.p[i];
    p.tiles_m = (p.m + 128 * f.cg - 1) / (128 * f.cg);
    p.tiles_n = (p.n + cols - 1) / cols;
    tiles += p.tiles_m * p.tiles_n;
  }
  const int units = f.parts > 1 ? tiles : f.cg == 2 ? dev.pairs : dev.nsm, size = f.cg * f.parts;
  const Config c((tiles < units ? tiles : units) * size, kGemmThreads, kGemmSmem, size, st);
  if (f.parts > 1) return cudaLaunchKernelEx(&c.cfg, k_ffn_gemm<EPI, 1, true>, a);
  return f.cg == 1 ? cudaLaunchKernelEx(&c.cfg, k_ffn_gemm<EPI, 1, false>, a) : cudaLaunchKernelEx(&c.cfg, k_ffn_gemm<EPI, 2, false>, a);
}

// Blocks of a cluster over k: enough clusters x blocks for four an SM, each of eight pieces of 64 at
// least (two for every warp; with one, 2,048 x 768 takes 9.6 us in place of 8.3).
int small_cluster(int tiles, int k) {
  int cl = 1;
  while (cl < 8 && tiles * cl < 4 * 148 && (k + 63) / 64 >= 16 * cl) cl *= 2;
  return cl;
}

cudaError_t launch_small(const SmallArgs &s, cudaStream_t st) {
  const int up = (s.f + 7) / 8, down = (s.d + 15) / 16, cu = small_cluster(up, s.d), cd = small_cluster(down, s.f);
  const Config u(up * cu, kSmThreads, 0, cu, st), d(down * cd, kSmThreads, 0, cd, st);
  const cudaError_t e = cudaLaunchKernelEx(&u.cfg, k_ffn_up, s, cu);
  return e == cudaSuccess ? cudaLaunchKernelEx(&d.cfg, k_ffn_down, s, cd) : e;
}

constexpr int kMaxRows = 1 << 20;  // at most 2^23 tiles
bool bad_mat(const void *p) { return !p || !aligned16(p); }
bool bad_act(const void *p, int64_t ld, int d, int n, int bytes) {
  return !p || !aligned16(p) || ld * bytes % 16 || (n > 1 && ld < d);
}
bool bad_shape(int n, int d, int f) {
  return n < 1 || n > kMaxRows || bad_ffn_dim(d) || bad_ffn_dim(f);
}
uint64_t align_ws(uint64_t v) { return (v + 255) & ~uint64_t(255); }

}  // namespace

extern "C" uint64_t moe_ffn_workspace(int32_t n_tokens, int32_t d_model, int32_t d_ff, int32_t backward) {
  if (bad_shape(n_tokens, d_model, d_ff)) return 0;
  const uint64_t nf = align_ws(static_cast<uint64_t>(n_tokens) * d_ff * 2);
  return backward ? 3 * nf : nf;
}

namespace moe {
moe_status ffn_forward_run(const moe_ffn_args *p, void *stream, uint32_t *err) {
  if (!p || p->struct_size != sizeof(moe_ffn_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model, f = p->d_ff;
  if (bad_shape(n, d, f) || bad_act(p->x, p->x_stride, d, n, 2) || bad_mat(p->w_gate) || bad_mat(p->w_up) ||
      bad_mat(p->w_down) || (p->y_dtype != MOE_F32 && p->y_dtype != MOE_BF16) ||
      bad_act(p->y, p->y_stride, d, n, p->y_dtype == MOE_BF16 ? 2 : 4) ||
      (p->add && ((p->add_dtype != MOE_F32 && p->add_dtype != MOE_BF16) ||
                  bad_act(p->add, p->add_stride, d, n, p->add_dtype == MOE_BF16 ? 2 : 4))) ||
      misplaced(p->y, p->y_stride, p->y_dtype, p->add, p->add_stride, p->add_dtype, n) ||
      (p->save_gate != nullptr) != (p->save_up != nullptr) || (p->save_gate && (bad_mat(p->save_gate) || bad_mat(p->save_up))) ||
      bad_mat(p->workspace) || p->workspace_bytes < moe_ffn_workspace(n, d, f, 0))
    return MOE_ERR_INVALID_ARGUMENT;
  if (const moe_status s = err ? MOE_OK : block_pending()) return s;
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
    return cuda_status(launch_small(s, st));
  }
  FfnDevice dev{};
  if ((e = ffn_setup(&dev)) != cudaSuccess) return cuda_status(e);
  GemmArgs a{};
  {
    Maps m{dev.encode, a};
    GemmProb &q = add_prob(a, n, f, d);
    q.a[0] = m.add(p->x, n, d, p->x_stride, box_rows(n));
    q.b[0] = m.add(p->w_gate, f, d, d, 64);
    q.b[1] = m.add(p->w_up, f, d, d, 64);
    a.h = h, a.g = static_cast<float *>(p->save_gate), a.u = static_cast<float *>(p->save_up);
    a.f_ld = f, a.err = err;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
  }
  if ((e = launch_gemm<kEpiSwiglu>(a, dev, st)) != cudaSuccess) return cuda_status(e);
  GemmArgs b{};
  {
    Maps m{dev.encode, b};
    GemmProb &q = add_prob(b, n, d, f);
    q.a[0] = m.add(h, n, f, f, box_rows(n));
    q.b[0] = m.add(p->w_down, d, f, f, 64);
    q.out = p->y, q.ld = p->y_stride, q.out_bf16 = p->y_dtype == MOE_BF16;
    q.add = p->add, q.add_ld = p->add_stride, q.add_bf16 = p->add_dtype == MOE_BF16;
    b.err = err;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
  }
  return cuda_status(launch_gemm<kEpiPlain>(b, dev, st));
}
}  // namespace moe

extern "C" moe_status moe_ffn_forward(const moe_ffn_args *p, void *stream) { return ffn_forward_run(p, stream, nullptr); }

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
  if (const moe_status s = block_pending()) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  FfnDevice dev{};
  cudaError_t e;
  if ((e = ffn_setup(&dev)) != cudaSuccess) return cuda_status(e);
  const uint64_t nf = align_ws(static_cast<uint64_t>(n) * f * 2) / 2;
  __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(p->workspace), *dg = h + nf, *du = dg + nf;
  {
    GemmArgs a{};
    Maps m{dev.encode, a};
    GemmProb &q = add_prob(a, n, f, d);
    q.a[0] = m.add(p->dy, n, d, p->dy_stride, box_rows(n));
    q.b[0] = m.add(p->w_down, d, f, f, kBK), q.b_mn = 1;
    a.g = static_cast<float *>(const_cast<void *>(p->save_gate)), a.u = static_cast<float *>(const_cast<void *>(p->save_up));
    a.h = h, a.dg = dg, a.du = du, a.f_ld = f;
    if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
    if ((e = launch_gemm<kEpiDswiglu>(a, dev, st)) != cudaSuccess) return cuda_status(e);
  }
  // everything else in one launch: dx (its tiles run over both matrices), then the weights' gradients; few
  // tokens: dx before them
  GemmArgs a{};
  Maps m{dev.encode, a};
  if (p->dx) {
    GemmProb &q = add_prob(a, n, d, f);
    q.segs = 2;
    q.a[0] = m.add(dg, n, f, f, box_rows(n)), q.a[1] = m.add(du, n, f, f, box_rows(n));
    q.b[0] = m.add(p->w_gate, f, d, d, kBK), q.b[1] = m.add(p->w_up, f, d, d, kBK), q.b_mn = 1;
    q.out = p->dx, q.ld = p->dx_stride, q.out_bf16 = 1;
    const bool apart = dx_apart(n, d, f, dev);
    if (apart || (!p->dw_gate && !p->dw_down)) {
      if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
      if ((e = launch_gemm<kEpiPlain>(a, dev, st, apart)) != cudaSuccess) return cuda_status(e);
      a.n_prob = m.n = 0;
    }
  }
  if (p->dw_gate) {
    const int mx = m.add(p->x, n, d, p->x_stride, kBK);
    const int rows[2] = {m.add(dg, n, f, f, kBK), m.add(du, n, f, f, kBK)};
    for (int i = 0; i < 2; ++i) {
      GemmProb &q = add_prob(a, f, d, n);
      q.a[0] = rows[i], q.b[0] = mx, q.a_mn = q.b_mn = 1;
      q.out = i ? p->dw_up : p->dw_gate, q.ld = d, q.out_bf16 = 1;
    }
  }
  if (p->dw_down) {
    GemmProb &q = add_prob(a, d, f, n);
    q.a[0] = m.add(p->dy, n, d, p->dy_stride, kBK), q.b[0] = m.add(h, n, f, f, kBK), q.a_mn = q.b_mn = 1;
    q.out = p->dw_down, q.ld = f, q.out_bf16 = 1;
  }
  if (!m.ok) return MOE_ERR_INVALID_ARGUMENT;
  return cuda_status(a.n_prob ? launch_gemm<kEpiPlain>(a, dev, st, false) : cudaSuccess);
}

extern "C" moe_status moe_block_check(void) {
  BlockWord w;
  cudaError_t e = cudaDeviceSynchronize();  // every stream of the device, also those that no other waits for
  if (e == cudaSuccess) e = block_word(&w);
  if (e != cudaSuccess) return cuda_status(e);
  return __atomic_exchange_n(w.host, 0u, __ATOMIC_ACQ_REL) ? MOE_ERR_TIMEOUT : MOE_OK;
}
