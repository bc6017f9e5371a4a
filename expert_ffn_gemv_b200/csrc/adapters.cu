// adapters.cu -- low-rank adapters of many requests beside a shared projection or block:
//   out_t = base_t + s_i B_i (A_i x_t),  i = ids[t];  no adapter (-1): out_t = base_t
// A_i rank x d_in, B_i d_out x rank in bf16; x, base and out in bf16 or fp32.
//
// The tokens are grouped by adapter into tiles of at most TM tokens of one adapter; a cluster of CL
// blocks runs both products of a tile in one kernel: block c takes a slice of d_in for
// v = A_i x (mma.sync, warps on interleaved 32-column pieces, the x rows read from global memory
// straight into the operand registers), the blocks' partial v meet over distributed shared memory
// and are added in block order, then block c multiplies its slice of d_out by v and adds the base.
// So x, base and out cross HBM once and v never leaves the SMs.
//
// Precision: products of bf16 values with fp32 accumulators.  What is not bf16 by itself (fp32 x, and
// v between the two products) enters as bf16 parts that add up to it: two where out is bf16 (2^-16 of
// a value, far below the rounding of out), three where out is fp32 (exact).
#include <new>
#include <string>

#include "block.cuh"

using namespace moe;

namespace {

constexpr int kAdThreads = 256, kAdWarps = kAdThreads / 32;
constexpr int kAdMaxRank = 128;
constexpr int kAdMaxTokens = 8192;
constexpr int kAdMaxSlots = 4096;
constexpr int kAdMaxD = 65536;
constexpr int kAdInKernel = 256;    // up to this many tokens every block groups the ids itself
constexpr int kAdGroups = 8;        // n8 rank groups of one pass over x: 64 ranks
constexpr int kRedLd = 8 * kAdGroups + 8;

struct AdMeta {
  int rank;     // 0: slot not loaded
  float scale;
};

struct AdArgs {
  const void *x, *base;
  void *out;
  const int *ids;
  const __nv_bfloat16 *a, *b;  // packed, slot strides a_slot / b_slot (elements)
  const AdMeta *meta;
  const int4 *tiles;           // more than kAdInKernel tokens: first place in order, tokens, adapter
  const int *order;            // tokens grouped by adapter
  const int *n_tiles;
  uint32_t *err;
  int64_t x_ld, base_ld, out_ld, a_slot, b_slot;
  int n, d_in, d_out, slots, max_rank16;
  int x_bf16, io_bf16, in_place;
};

__host__ __device__ constexpr int round16(int r) { return (r + 15) & ~15; }

struct AdSmem {
  int red, part, v, v_part, total, v_ld;  // v: VP parts of v_part bytes
};
template <int TM, int VP>
__host__ __device__ AdSmem ad_smem(int r16) {
  AdSmem s;
  s.v_ld = r16 + 8;
  s.red = 0;
  s.part = s.red + kAdWarps * TM * kRedLd * 4;
  s.v = s.part + TM * r16 * 4;
  s.v_part = TM * s.v_ld * 2;
  s.total = s.v + VP * s.v_part;
  return s;
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float ld_cluster_f32(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// The adapter a token asks for: slots stands for "none" (id -1), and for ids out of range or of a
// slot that is not loaded, which raise the error word.
__device__ __forceinline__ int ad_id(const AdArgs &a, int t, bool report) {
  const int id = a.ids[t];
  if (id == -1) return a.slots;
  if (id < 0 || id >= a.slots || a.meta[id].rank == 0) {
    if (report) flag_error(a.err, kErrBadIndex);
    return a.slots;
  }
  return id;
}

// Few tokens: finds tile `want` of the grouped order and writes its tokens to rows[]; every block
// of a cluster comes to the same answer.  Tiles are numbered by their group's first token.
// Returns the tile's token count (0: no such tile) and its adapter.
template <int TM>
__device__ int ad_find_tile(const AdArgs &a, int want, bool report, int *rows, int &adapter) {
  __shared__ int s_id[kAdInKernel], s_warp[kAdWarps], s_got[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int id = -1;
  if (tid < a.n) id = ad_id(a, tid, report);
  s_id[tid] = id;
  if (tid < 2) s_got[tid] = 0;
  __syncthreads();
  int before = 0, size = 0;
  if (tid < a.n)
    for (int t = 0; t < a.n; ++t) {
      const int same = s_id[t] == id;
      size += same;
      before += same & (t < tid);
    }
  const bool live = tid < a.n && !(id == a.slots && a.in_place);
  const int mine = live && before == 0 ? (size + TM - 1) / TM : 0;  // tiles of the group I lead
  int scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  int first = scan - mine;
  for (int w = 0; w < warp; ++w) first += s_warp[w];
  __shared__ int s_sel[2];  // adapter, tile inside the group
  if (tid == 0) s_sel[0] = -1;
  __syncthreads();
  if (mine && want >= first && want < first + mine) {
    s_sel[0] = id;
    s_sel[1] = want - first;
  }
  __syncthreads();
  adapter = s_sel[0];
  if (adapter < 0) return 0;
  const int lo = s_sel[1] * TM;
  if (tid < a.n && id == adapter && before >= lo && before < lo + TM) {
    rows[before - lo] = tid;
    if (before == lo) s_got[0] = min(TM, size - lo);
  }
  __syncthreads();
  return s_got[0];
}

// Eight consecutive values of a row as XP parts of four operand words (bf16 pairs); XP = 1: bf16 x.
template <int XP>
__device__ __forceinline__ void load_x8(const void *x, int64_t i, bool ok, uint32_t (&w)[XP][4]) {
  if constexpr (XP == 1) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(x) + i));
    w[0][0] = v.x; w[0][1] = v.y; w[0][2] = v.z; w[0][3] = v.w;
  } else {
    float4 u = make_float4(0, 0, 0, 0), v = u;
    if (ok) {
      const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
      u = __ldg(p);
      v = __ldg(p + 1);
    }
    const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t parts[XP];
      split_bf16x2<XP>(f[2 * k], f[2 * k + 1], parts);
#pragma unroll
      for (int i2 = 0; i2 < XP; ++i2) w[i2][k] = parts[i2];
    }
  }
}

template <int TM, int XP, int VP>
__global__ void __launch_bounds__(kAdThreads) k_adapter(const __grid_constant__ AdArgs a) {
  constexpr int MT = TM / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int rows[TM];
  const AdSmem S = ad_smem<TM, VP>(a.max_rank16);
  float *red = reinterpret_cast<float *>(smem + S.red), *part = reinterpret_cast<float *>(smem + S.part);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int cl = cluster_nctarank(), cr = cluster_ctarank(), tile = blockIdx.x / cl;

  int adapter, cnt;
  if (a.n <= kAdInKernel) {
    cnt = ad_find_tile<TM>(a, tile, blockIdx.x == 0, rows, adapter);
  } else {
    cnt = 0, adapter = -1;
    if (tile < *a.n_tiles) {
      const int4 ti = a.tiles[tile];
      cnt = ti.y, adapter = ti.z;
      if (tid < cnt) rows[tid] = a.order[ti.x + tid];
    }
    __syncthreads();
  }
  if (cnt == 0) return;  // the same for every block of the cluster
  AdMeta meta{0, 0.f};
  if (adapter < a.slots) meta = a.meta[adapter];
  const int r16 = round16(meta.rank), ng = r16 / 8;

  // row numbers of this lane's operand rows (16m + g and 16m + g + 8)
  int row[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * m + 8 * h + g;
      row[m][h] = i < cnt ? rows[i] : -1;
    }

  // ---- v = A_i x over this block's slice of d_in, 64 ranks a pass
  const int kb_all = (a.d_in + 31) / 32, kb0 = kb_all * cr / cl, kb1 = kb_all * (cr + 1) / cl;
  const __nv_bfloat16 *ap = a.a + a.a_slot * adapter;
  for (int g0 = 0; g0 < ng; g0 += kAdGroups) {
    const int nj = min(kAdGroups, ng - g0);
    float acc[MT][kAdGroups][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < kAdGroups; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][j][k] = 0.f;
#pragma unroll 2
    for (int kb = kb0 + warp; kb < kb1; kb += kAdWarps) {
      const int k = 32 * kb + 8 * q;
      uint32_t xw[MT][2][XP][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          load_x8<XP>(a.x, row[m][h] * a.x_ld + k, row[m][h] >= 0 && k < a.d_in, xw[m][h]);
      const uint4 *w = reinterpret_cast<const uint4 *>(ap) + (static_cast<int64_t>(kb) * ng + g0) * 32 + lane;
      uint4 bw[kAdGroups];
#pragma unroll
      for (int j = 0; j < kAdGroups; ++j)
        if (j < nj) bw[j] = __ldg(w + 32 * j);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < XP; ++i) {
          const uint32_t a0[4] = {xw[m][0][i][0], xw[m][1][i][0], xw[m][0][i][1], xw[m][1][i][1]};
          const uint32_t a1[4] = {xw[m][0][i][2], xw[m][1][i][2], xw[m][0][i][3], xw[m][1][i][3]};
#pragma unroll
          for (int j = 0; j < kAdGroups; ++j)
            if (j < nj) {
              mma_bf16(acc[m][j], a0, bw[j].x, bw[j].y);
              mma_bf16(acc[m][j], a1, bw[j].z, bw[j].w);
            }
        }
    }
    // the warps' sums meet in shared memory, added in warp order
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < kAdGroups; ++j)
        if (j < nj) {
          float *p = red + (warp * TM + 16 * m + g) * kRedLd + 8 * j + 2 * q;
          *reinterpret_cast<float2 *>(p) = make_float2(acc[m][j][0], acc[m][j][1]);
          *reinterpret_cast<float2 *>(p + 8 * kRedLd) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
    __syncthreads();
    for (int i = tid; i < TM * 8 * nj; i += kAdThreads) {
      const int t = i / (8 * nj), r = i - t * (8 * nj);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kAdWarps; ++w) s += red[(w * TM + t) * kRedLd + r];
      part[t * r16 + 8 * g0 + r] = s;
    }
    __syncthreads();
  }
  // ---- the blocks' partial v, added in block order; s v in bf16 parts
  if (cl > 1) {
    cluster_arrive();
    cluster_wait();
  }
  for (int i = tid; i < TM * r16; i += kAdThreads) {
    const int t = i / r16, r = i - t * r16;
    float s = 0.f;
    if (cl > 1)
      for (int c = 0; c < cl; ++c) s += ld_cluster_f32(smem_u32(part + i), c);
    else
      s = part[i];
    if (r >= meta.rank) s = 0.f;  // padded ranks: 0 even where x holds infinities
    uint32_t w[VP];
    split_bf16x2<VP>(s * meta.scale, 0.f, w);
#pragma unroll
    for (int k = 0; k < VP; ++k)
      reinterpret_cast<uint16_t *>(smem + S.v + k * S.v_part)[t * S.v_ld + r] = static_cast<uint16_t>(w[k]);
  }
  __syncthreads();
  if (cl > 1) cluster_arrive();  // done with the other blocks' shared memory; waited for at the end

  // ---- out = base + B_i v over this block's slice of d_out, 32 columns a warp and step; a lane
  // holds eight consecutive columns of its rows (the packed B orders the MMA columns so)
  const int nb_all = (a.d_out + 31) / 32, nb0 = nb_all * cr / cl, nb1 = nb_all * (cr + 1) / cl;
  const uint4 *bp = reinterpret_cast<const uint4 *>(a.b + a.b_slot * adapter);
  const int nk = r16 / 16;
  const uint32_t vaddr = smem_u32(smem + S.v) + ((lane & 15) * S.v_ld + (lane >> 4) * 8) * 2;
  for (int nb = nb0 + warp; nb < nb1; nb += kAdWarps) {
    const int col = 32 * nb + 8 * q;
    float acc[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][j][k] = 0.f;
    for (int k = 0; k < nk; ++k) {
      const uint4 *w = bp + ((static_cast<int64_t>(nb) * nk + k) * 32 + lane) * 2;
      const uint4 w0 = __ldg(w), w1 = __ldg(w + 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          uint32_t v[4];
          ldmatrix_x4(v, vaddr + i * S.v_part + (16 * m * S.v_ld + 16 * k) * 2);
          mma_bf16(acc[m][0], v, w0.x, w0.y);
          mma_bf16(acc[m][1], v, w0.z, w0.w);
          mma_bf16(acc[m][2], v, w1.x, w1.y);
          mma_bf16(acc[m][3], v, w1.z, w1.w);
        }
      }
    }
    if (col >= a.d_out) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = row[m][h];
        if (t < 0) continue;
        const int64_t ib = t * a.base_ld + col, io = t * a.out_ld + col;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = acc[m][j][2 * h];
          v[2 * j + 1] = acc[m][j][2 * h + 1];
        }
        if (a.io_bf16) {
          const uint4 b = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.base) + ib);
          const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(bw[j] << 16) + v[2 * j],
                                                           __uint_as_float(bw[j] & 0xFFFF0000u) + v[2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t *>(&p);
          }
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + io) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          const float4 *b = reinterpret_cast<const float4 *>(static_cast<const float *>(a.base) + ib);
          const float4 b0 = b[0], b1 = b[1];
          float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + io);
          o[0] = make_float4(b0.x + v[0], b0.y + v[1], b0.z + v[2], b0.w + v[3]);
          o[1] = make_float4(b1.x + v[4], b1.y + v[5], b1.z + v[6], b1.w + v[7]);
        }
      }
  }
  if (cl > 1) cluster_wait();
}

// Counting sort of the tokens by adapter and the list of tiles (more than kAdInKernel tokens); one
// block.  The order inside a group is the order of arrival, which no result depends on: every row
// is computed by itself.
__global__ void __launch_bounds__(1024) k_adapter_group(AdArgs a, int4 *tiles, int *order, int *n_tiles, int tm) {
  extern __shared__ int s_cnt[];  // [slots + 1] counts, then cursors
  __shared__ int s_rows[32], s_tiles[32], s_base[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = a.slots + 1;
  for (int i = tid; i < groups; i += 1024) s_cnt[i] = 0;
  if (tid < 2) s_base[tid] = 0;
  __syncthreads();
  for (int t = tid; t < a.n; t += 1024) atomicAdd(&s_cnt[ad_id(a, t, true)], 1);
  __syncthreads();
  for (int i0 = 0; i0 < groups; i0 += 1024) {
    const int i = i0 + tid, c = i < groups ? s_cnt[i] : 0;
    const int nt = i == a.slots && a.in_place ? 0 : (c + tm - 1) / tm;
    int sr = c, st = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sr, o), v = __shfl_up_sync(0xffffffffu, st, o);
      if (lane >= o) sr += u, st += v;
    }
    if (lane == 31) s_rows[warp] = sr, s_tiles[warp] = st;
    __syncthreads();
    int r0 = s_base[0] + sr - c, t0 = s_base[1] + st - nt;
    for (int w = 0; w < warp; ++w) r0 += s_rows[w], t0 += s_tiles[w];
    for (int k = 0; k < nt; ++k) tiles[t0 + k] = make_int4(r0 + k * tm, min(tm, c - k * tm), i, 0);
    if (i < groups) s_cnt[i] = r0;
    __syncthreads();
    if (tid == 1023) s_base[0] = r0 + c, s_base[1] = t0 + nt;
    __syncthreads();
  }
  if (tid == 0) *n_tiles = s_base[1];
  for (int t = tid; t < a.n; t += 1024) order[atomicAdd(&s_cnt[ad_id(a, t, false)], 1)] = t;
}

// A (rank x d_in) and B (d_out x rank) into the kernels' operand order, padded with zeros to 16
// ranks and 32 columns.
//   A: [k / 32][rank / 8][lane][8]: lane 4g + q holds A[8j + g][32 kb + 8q + e]
//   B: [col / 32][rank / 16][lane][j][2][2]: MMA j, lane 4g + q, register h, element e holds column
//      32 nb + 8 (g / 2) + 2j + g % 2 of rank 16 k + 8h + 2q + e
__global__ void __launch_bounds__(256) k_adapter_pack(const __nv_bfloat16 *src, __nv_bfloat16 *dst, int is_b, int rank, int d) {
  const int r16 = round16(rank), d32 = (d + 31) / 32 * 32;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(r16) * d32) return;
  int r, c;
  if (is_b) {
    const int e = i & 1, h = (i >> 1) & 1, j = (i >> 2) & 3, lane = (i >> 4) & 31;
    const int64_t blk = i >> 9;
    const int nk = r16 / 16, k = blk % nk, nb = blk / nk, g = lane >> 2, q = lane & 3;
    r = 16 * k + 8 * h + 2 * q + e;
    c = 32 * nb + 8 * (g >> 1) + 2 * j + (g & 1);
  } else {
    const int e = i & 7, lane = (i >> 3) & 31;
    const int64_t blk = i >> 8;
    const int ng = r16 / 8, j = blk % ng, kb = blk / ng;
    r = 8 * j + (lane >> 2);
    c = 32 * kb + 8 * (lane & 3) + e;
  }
  const bool in = r < rank && c < d;
  dst[i] = in ? (is_b ? src[static_cast<int64_t>(c) * rank + r] : src[static_cast<int64_t>(r) * d + c]) : __float2bfloat16_rn(0.f);
}

__global__ void k_adapter_meta(AdMeta *m, AdMeta v) { *m = v; }

struct Device {
  int prev = -1;
  bool ok = false;
  explicit Device(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) return;
    ok = prev == dev || cudaSetDevice(dev) == cudaSuccess;
    if (prev == dev) prev = -1;
  }
  ~Device() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

}  // namespace

struct moe_adapters {
  moe_adapters_config cfg;
  int r16 = 0, nsm = 0;
  int64_t a_slot = 0, b_slot = 0;  // elements
  uint64_t bytes = 0;
  void *mem = nullptr;
  __nv_bfloat16 *a = nullptr, *b = nullptr, *stage = nullptr;
  AdMeta *meta = nullptr;
  int4 *tiles = nullptr;
  int *order = nullptr, *n_tiles = nullptr;
  uint32_t *err_host = nullptr, *err_dev = nullptr;
  std::string last_error;
};

namespace moe {
bool adapters_match(const moe_adapters *h, int d, int device, int n) {
  return h->cfg.d_in == d && h->cfg.d_out == d && h->cfg.device == device && n <= h->cfg.max_tokens;
}
}  // namespace moe

namespace {

moe_status ad_fail(moe_adapters *h, moe_status s, const char *msg) {
  h->last_error = msg;
  return s;
}
moe_status ad_cuda(moe_adapters *h, cudaError_t e, const char *what) {
  cudaGetLastError();
  h->last_error = std::string(what) + ": " + cudaGetErrorString(e);
  return e == cudaErrorMemoryAllocation ? MOE_ERR_OUT_OF_MEMORY : MOE_ERR_CUDA;
}

moe_status ad_pending(moe_adapters *h) {
  const uint32_t e = __atomic_exchange_n(h->err_host, 0u, __ATOMIC_ACQ_REL);
  return e ? ad_fail(h, MOE_ERR_DEVICE_FAULT, "an adapter id of an earlier call was out of range or not loaded") : MOE_OK;
}

int tile_rows(int n) { return n > 1024 ? 32 : 16; }
int64_t most_tiles(int n, int tm, int slots) { return n / tm + (n < slots + 1 ? n : slots + 1); }

template <int TM, int XP, int VP>
cudaError_t launch_adapter(const AdArgs &a, int clusters, int cl, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clusters * cl);
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = ad_smem<TM, VP>(a.max_rank16).total;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_adapter<TM, XP, VP>, a);
}

template <int TM>
cudaError_t launch_adapter_types(const AdArgs &a, int clusters, int cl, cudaStream_t st) {
  if (a.io_bf16) return a.x_bf16 ? launch_adapter<TM, 1, 2>(a, clusters, cl, st) : launch_adapter<TM, 2, 2>(a, clusters, cl, st);
  return a.x_bf16 ? launch_adapter<TM, 1, 3>(a, clusters, cl, st) : launch_adapter<TM, 3, 3>(a, clusters, cl, st);
}

template <int TM, int XP, int VP>
cudaError_t configure_adapter() {
  return cudaFuncSetAttribute(k_adapter<TM, XP, VP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              ad_smem<TM, VP>(kAdMaxRank).total);
}
template <int TM>
cudaError_t configure_adapters() {
  cudaError_t e = configure_adapter<TM, 1, 2>();
  if (e == cudaSuccess) e = configure_adapter<TM, 2, 2>();
  if (e == cudaSuccess) e = configure_adapter<TM, 1, 3>();
  return e == cudaSuccess ? configure_adapter<TM, 3, 3>() : e;
}

bool host_ptr(const void *p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return true;
  }
  return at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged;
}

}  // namespace

extern "C" {

moe_status moe_adapters_create(const moe_adapters_config *cfg, moe_adapters **out) {
  if (!out) return MOE_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (!cfg || cfg->struct_size != sizeof(moe_adapters_config)) return MOE_ERR_INVALID_ARGUMENT;
  const moe_adapters_config &g = *cfg;
  if (g.d_in < 8 || g.d_in % 8 || g.d_in > kAdMaxD || g.d_out < 8 || g.d_out % 8 || g.d_out > kAdMaxD ||
      g.max_adapters < 1 || g.max_adapters > kAdMaxSlots || g.max_rank < 1 || g.max_rank > kAdMaxRank ||
      g.max_tokens < 1 || g.max_tokens > kAdMaxTokens || g.device < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || g.device >= ndev) {
    cudaGetLastError();
    return MOE_ERR_INVALID_ARGUMENT;
  }
  Device dev(g.device);
  if (!dev.ok) return MOE_ERR_CUDA;
  moe_adapters *h = new (std::nothrow) moe_adapters();
  if (!h) return MOE_ERR_OUT_OF_MEMORY;
  h->cfg = g;
  h->r16 = round16(g.max_rank);
  h->a_slot = static_cast<int64_t>(h->r16) * ((g.d_in + 31) / 32 * 32);
  h->b_slot = static_cast<int64_t>(h->r16) * ((g.d_out + 31) / 32 * 32);
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = (off + bytes + 255) & ~uint64_t(255);
    return at;
  };
  const uint64_t d_max = g.d_in > g.d_out ? g.d_in : g.d_out;
  const uint64_t oa = take(h->a_slot * 2 * g.max_adapters), ob = take(h->b_slot * 2 * g.max_adapters);
  const uint64_t os = take(d_max * g.max_rank * 2), om = take(sizeof(AdMeta) * g.max_adapters);
  const uint64_t ot = take(16 * (g.max_tokens / 16 + g.max_adapters + 2)), oo = take(4ull * g.max_tokens), on = take(4);
  cudaError_t e = cudaMalloc(&h->mem, off);
  moe_status s = MOE_OK;
  if (e != cudaSuccess) {
    h->mem = nullptr;
    s = ad_cuda(h, e, "adapters");
  } else {
    h->bytes = off;
    char *p = static_cast<char *>(h->mem);
    h->a = reinterpret_cast<__nv_bfloat16 *>(p + oa);
    h->b = reinterpret_cast<__nv_bfloat16 *>(p + ob);
    h->stage = reinterpret_cast<__nv_bfloat16 *>(p + os);
    h->meta = reinterpret_cast<AdMeta *>(p + om);
    h->tiles = reinterpret_cast<int4 *>(p + ot);
    h->order = reinterpret_cast<int *>(p + oo);
    h->n_tiles = reinterpret_cast<int *>(p + on);
    e = cudaMemset(h->meta, 0, sizeof(AdMeta) * g.max_adapters);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess)
      e = cudaHostAlloc(reinterpret_cast<void **>(&h->err_host), sizeof(uint32_t), cudaHostAllocMapped);
    if (e == cudaSuccess) {
      *h->err_host = 0;
      e = cudaHostGetDevicePointer(reinterpret_cast<void **>(&h->err_dev), h->err_host, 0);
    }
    if (e == cudaSuccess) e = current_sm_count(&h->nsm);
    if (e == cudaSuccess) e = configure_adapters<16>();
    if (e == cudaSuccess) e = configure_adapters<32>();
    if (e != cudaSuccess) s = ad_cuda(h, e, "adapters");
  }
  if (s != MOE_OK) {
    moe_adapters_destroy(h);
    return s;
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_adapters_destroy(moe_adapters *h) {
  if (!h) return MOE_OK;
  Device dev(h->cfg.device);
  cudaDeviceSynchronize();
  if (h->mem) cudaFree(h->mem);
  if (h->err_host) cudaFreeHost(h->err_host);
  cudaGetLastError();
  delete h;
  return MOE_OK;
}

const char *moe_adapters_last_error(const moe_adapters *h) { return h ? h->last_error.c_str() : "no handle"; }

uint64_t moe_adapters_device_bytes(const moe_adapters *h) { return h ? h->bytes : 0; }

moe_status moe_adapters_check(moe_adapters *h) { return h ? ad_pending(h) : MOE_ERR_INVALID_ARGUMENT; }

moe_status moe_adapters_load(moe_adapters *h, int32_t slot, const void *a, const void *b, int32_t rank, float scale,
                             void *stream) {
  if (!h) return MOE_ERR_INVALID_ARGUMENT;
  const moe_adapters_config &g = h->cfg;
  if (slot < 0 || slot >= g.max_adapters) return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "slot out of range");
  if (rank < 0 || rank > g.max_rank) return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "rank out of range");
  if (rank && (!a || !b)) return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "missing adapter matrix");
  Device dev(g.device);
  if (!dev.ok) return ad_fail(h, MOE_ERR_CUDA, "set device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  bool host = false;
  for (int m = 0; m < 2 && rank && e == cudaSuccess; ++m) {
    const int d = m ? g.d_out : g.d_in;
    const void *src = m ? b : a;
    if (host_ptr(src)) {  // both matrices pass through one buffer in stream order
      host = true;
      e = cudaMemcpyAsync(h->stage, src, static_cast<size_t>(rank) * d * 2, cudaMemcpyHostToDevice, st);
      src = h->stage;
      if (e != cudaSuccess) break;
    }
    const int64_t count = static_cast<int64_t>(round16(rank)) * ((d + 31) / 32 * 32);
    k_adapter_pack<<<static_cast<unsigned>((count + 255) / 256), 256, 0, st>>>(
        static_cast<const __nv_bfloat16 *>(src), m ? h->b + h->b_slot * slot : h->a + h->a_slot * slot, m, rank, d);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    k_adapter_meta<<<1, 1, 0, st>>>(h->meta + slot, AdMeta{rank, scale});
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && host) e = cudaStreamSynchronize(st);
  return e == cudaSuccess ? MOE_OK : ad_cuda(h, e, "adapter load");
}

moe_status moe_adapters_apply(moe_adapters *h, const void *x, int32_t x_dtype, int64_t x_stride, const void *base,
                              int64_t base_stride, void *out, int64_t out_stride, int32_t out_dtype, const int32_t *ids,
                              int32_t n_tokens, void *stream) {
  if (!h) return MOE_ERR_INVALID_ARGUMENT;
  const moe_adapters_config &g = h->cfg;
  if (!x || !base || !out || !ids || n_tokens < 1 || n_tokens > g.max_tokens || (x_dtype != MOE_F32 && x_dtype != MOE_BF16) ||
      (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
    return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "bad apply arguments");
  // rows are read and written 16 bytes at a time
  const int xs = x_dtype == MOE_BF16 ? 2 : 4, os = out_dtype == MOE_BF16 ? 2 : 4;
  if (!aligned16(x) || !aligned16(base) || !aligned16(out) || x_stride * xs % 16 || base_stride * os % 16 ||
      out_stride * os % 16 || reinterpret_cast<uintptr_t>(ids) % 4)
    return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "a pointer or row stride is not a multiple of 16 bytes");
  if (n_tokens > 1 && (x_stride < g.d_in || base_stride < g.d_out || out_stride < g.d_out))
    return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "a row stride is smaller than a row");
  moe_status s = ad_pending(h);
  if (s != MOE_OK) return s;
  Device dev(g.device);
  if (!dev.ok) return ad_fail(h, MOE_ERR_CUDA, "set device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AdArgs a{};
  a.x = x, a.base = base, a.out = out, a.ids = ids;
  a.a = h->a, a.b = h->b, a.meta = h->meta, a.a_slot = h->a_slot, a.b_slot = h->b_slot;
  a.tiles = h->tiles, a.order = h->order, a.n_tiles = h->n_tiles, a.err = h->err_dev;
  a.x_ld = x_stride, a.base_ld = base_stride, a.out_ld = out_stride;
  a.n = n_tokens, a.d_in = g.d_in, a.d_out = g.d_out, a.slots = g.max_adapters, a.max_rank16 = h->r16;
  a.x_bf16 = x_dtype == MOE_BF16, a.io_bf16 = out_dtype == MOE_BF16;
  a.in_place = base == out && base_stride == out_stride;
  const int tm = tile_rows(n_tokens);
  const int64_t tiles = most_tiles(n_tokens, tm, g.max_adapters);
  cudaError_t e = cudaSuccess;
  if (n_tokens > kAdInKernel) {
    k_adapter_group<<<1, 1024, (g.max_adapters + 1) * 4, st>>>(a, h->tiles, h->order, h->n_tiles, tm);
    e = cudaGetLastError();
  }
  int cl = 8;
  while (cl > 1 && tiles * cl > 2 * h->nsm) cl >>= 1;
  if (e == cudaSuccess)
    e = tm == 16 ? launch_adapter_types<16>(a, tiles, cl, st) : launch_adapter_types<32>(a, tiles, cl, st);
  return e == cudaSuccess ? MOE_OK : ad_cuda(h, e, "adapter launch");
}

}  // extern "C"
