// adapters.cu -- low-rank adapters of many requests beside a shared projection or block:
//   out_t = base_t + s_i B_i (A_i x_t),  i = ids[t];  no adapter (-1): out_t = base_t
// A_i rank x d_in, B_i d_out x rank in bf16; x, base and out in bf16 or fp32.
//
// The tokens are grouped by adapter into tiles of at most TM tokens of one adapter; a cluster of CL
// blocks runs both products of a tile in one kernel: block c takes a slice of d_in for
// v = A_i x (mma.sync), the blocks' partial v meet over distributed shared memory and are added in
// block order, then block c multiplies its slice of d_out by v and adds the base.  So x, base and out
// cross HBM once and v never leaves the SMs.  A warp has 16 of the tile's tokens (TM / 16 groups of
// warps, whose equal weight loads meet in L1) and every KG-th 32-deep piece.
//
// What bounds it is latency: a piece is a few MMAs behind its loads.  So everything comes through
// rings in shared memory, several pieces ahead: x and base by cp.async, in which every lane copies just
// the 16-byte words that it takes out itself (no barrier: a thread waits for its own groups), and the
// weights, packed in operand order, by bulk copies of the block's ninth warp, one ring for the warps
// that share them.  8,192 tokens, 2,048 -> 4,096, rank 64, bf16: 64 us, 2.6 TB/s (with weights loaded one
// piece ahead into registers a piece took 1.6 us, by bulk copies 0.9).
//
// Precision: products of bf16 values with fp32 accumulators.  What is not bf16 by itself (fp32 x, and
// v between the two products) enters as bf16 parts that add up to it: two where out is bf16 (2^-16 of
// a value, far below the rounding of out), three where out is fp32 (exact).
#include <cstdio>
#include <mutex>
#include <new>

#include "block.cuh"

using namespace moe;

namespace {

constexpr int kAdThreads = 256, kAdWarps = kAdThreads / 32;  // that compute; one more warp feeds them
constexpr int kAdBlock = kAdThreads + 32;
constexpr int kAdMaxRank = 128;
constexpr int kSmSmem = 228 * 1024;  // of an SM, 1 KB of it taken by each block
constexpr int kAdMaxTokens = 8192;
constexpr int kAdMaxSlots = 4096;
constexpr int kAdMaxD = 65536;
// Up to this many tokens ids are compared with one another, beyond counted (mean over shapes, us, compared and
// counted: 64 tokens 9.0, 9.9; 128 9.75, 10.1; 160 10.8, 10.2; 256 15.4, 11.9).
constexpr int kAdInKernel = 128;
constexpr int kAdGroups = 8;        // n8 rank groups of one pass over x: 64 ranks
constexpr int kRedLd = 8 * kAdGroups + 8;
// Pieces of x and base, and of weights, on their way: what fits two blocks on an SM at 32 ranks (RC = 0)
// and at 64 (RC = 1).  In bytes they are what bounds long prompts: 64 KB an SM gave 3 TB/s.
template <int XP, int VP, int RC>
__host__ __device__ constexpr int ad_depth() { return XP == 1 && VP == 2 ? 4 : RC == 0 ? 4 : 3; }
constexpr int kWDepth = 2;

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
  uint32_t *err;
  int64_t x_ld, base_ld, out_ld, a_slot, b_slot;
  int n, d_in, d_out, slots, max_rank16;
  int x_bf16, io_bf16, in_place;
  RingSpin spin;
};

__host__ __device__ constexpr int round16(int r) { return (r + 15) & ~15; }

// Shared memory: barriers; the rings of x, then base, and the warps' sums [KG][TM][kRedLd] between them
// in one place; the block's partial v; s v as VP bf16 parts; the weights' rings, a stage r16 x 64 bytes.
struct AdSmem {
  int ring, part, v, v_part, w, total, v_ld;
};
template <int TM, int XP, int VP, int RC>
__host__ __device__ AdSmem ad_smem(int r16) {
  constexpr int ring = ad_depth<XP, VP, RC>() * kAdThreads * 16 * (XP == 1 && VP == 2 ? 2 : 4), red = kAdWarps * 16 * kRedLd * 4;
  AdSmem s;
  s.v_ld = r16 + 8;
  s.ring = 512;
  s.part = s.ring + (ring > red ? ring : red);
  s.v = s.part + TM * r16 * 4;
  s.v_part = TM * s.v_ld * 2;
  s.w = (s.v + VP * s.v_part + 127) / 128 * 128;
  s.total = s.w + kAdWarps / (TM / 16) * kWDepth * r16 * 64;
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

// The adapter a token asks for: slots stands for "none" (id -1), and for ids out of range, which raise
// the error word.  (Whether the slot is loaded is seen once a tile.)
__device__ __forceinline__ int ad_id(const AdArgs &a, int id, bool report) {
  const bool in = id >= 0 && id < a.slots;
  if (!in && id != -1 && report) flag_error(a.err, kErrBadIndex);
  return in ? id : a.slots;
}

// Few tokens: finds tile `want` of the grouped order and writes its tokens to rows[]; every block
// of a cluster comes to the same answer.  Tiles are numbered by their group's first token.
// Returns the tile's token count (0: no such tile) and its adapter.
template <int TM>
__device__ int ad_find_tile(const AdArgs &a, int want, bool report, int *rows, int &adapter) {
  __shared__ int s_id[kAdInKernel], s_warp[kAdWarps + 1], s_got[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int id = -1;
  if (tid < a.n) id = ad_id(a, a.ids[tid], report);
  if (tid < kAdInKernel) s_id[tid] = id;
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

// Many tokens: the same, with the tiles numbered by slot (the tokens without an adapter last).  Every
// block counts the ids of all tokens for itself (counters and the ids it read in `scratch`): reading
// them takes less time than a launch that would sort them for all, and a call needs no workspace.
template <int TM>
__device__ int ad_find_tile_many(const AdArgs &a, int want, bool report, unsigned char *scratch, int *rows, int &adapter) {
  __shared__ int s_warp[kAdWarps], s_sel[3], s_base;
  int *count = reinterpret_cast<int *>(scratch);                                 // [slots + 1]
  uint16_t *ids = reinterpret_cast<uint16_t *>(scratch + (kAdMaxSlots + 64) * 4);  // [n]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = a.slots + 1;
  for (int i = tid; i < groups; i += kAdBlock) count[i] = 0;
  if (tid == 0) s_base = 0, s_sel[0] = -1;
  __syncthreads();
  // warp w has tokens w * each .. of a run; a warp's lanes with the same id make one atomic (a few long
  // prompts put every token on one counter)
  const int each = (a.n + 32 * kAdWarps - 1) / (32 * kAdWarps) * 32, t0 = warp * each;
  if (warp < kAdWarps)
    for (int b = t0 + lane; b < t0 + each; b += 8 * 32) {  // eight loads on their way
      int id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) id[k] = __ldg(a.ids + min(b + 32 * k, a.n - 1));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = b + 32 * k;
        id[k] = t < t0 + each && t < a.n ? ad_id(a, id[k], report) : -1;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (id[k] >= 0) ids[b + 32 * k] = static_cast<uint16_t>(id[k]);
        const uint32_t same = __match_any_sync(0xffffffffu, id[k]);
        if (id[k] >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[id[k]], __popc(same));
      }
    }
  __syncthreads();
  for (int i0 = 0; i0 < groups; i0 += kAdThreads) {
    const int i = i0 + tid, c = tid < kAdThreads && i < groups ? count[i] : 0;
    const int nt = i == a.slots && a.in_place ? 0 : (c + TM - 1) / TM;
    int scan = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31 && warp < kAdWarps) s_warp[warp] = scan;
    __syncthreads();
    int first = s_base + scan - nt;
    for (int w = 0; w < warp && w < kAdWarps; ++w) first += s_warp[w];
    if (nt && want >= first && want < first + nt) s_sel[0] = i, s_sel[1] = (want - first) * TM, s_sel[2] = c;
    __syncthreads();
    if (tid == kAdThreads - 1) s_base = first + nt;
    __syncthreads();
    if (s_sel[0] >= 0) break;
  }
  adapter = s_sel[0];
  if (adapter < 0) return 0;
  // the tile's tokens: places lo .. of the adapter's tokens in their order
  int mine = 0;
  if (warp < kAdWarps)
#pragma unroll 8
    for (int t = t0 + lane; t < t0 + each; t += 32) mine += __popc(__ballot_sync(0xffffffffu, t < a.n && ids[t] == adapter));
  if (lane == 0 && warp < kAdWarps) s_warp[warp] = mine;
  __syncthreads();
  const int lo = s_sel[1];
  if (warp < kAdWarps) {
    int at = -lo;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    for (int t = t0 + lane; t < t0 + each && at < TM; t += 32) {
      const bool is = t < a.n && ids[t] == adapter;
      const uint32_t all = __ballot_sync(0xffffffffu, is);
      const int place = at + __popc(all & ((1u << lane) - 1u));
      if (is && place >= 0 && place < TM) rows[place] = t;
      at += __popc(all);
    }
  }
  __syncthreads();
  return min(TM, s_sel[2] - lo);
}

// 16 bytes to this thread's slot; zeros where there is no source
__device__ __forceinline__ void ad_copy(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ad_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int DEPTH>
__device__ __forceinline__ void ad_wait() {  // all but the last DEPTH - 1 groups
  asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
}
__device__ __forceinline__ void ad_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kAdThreads) : "memory"); }
__device__ __forceinline__ void ad_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// What both products of a tile share: a thread's place, its rows, its slots of the rings.
struct AdLane {
  int q, lane, row[2];  // row numbers of this lane's operand rows (16 mg + g and 16 mg + g + 8), or -1
  uint32_t slot;        // this thread's first slot; the others lie kAdThreads * 16 bytes apart
};
constexpr uint32_t kSlots = kAdThreads * 16;

// cp.async of a piece's 2 rows x 32 values of B bytes a quad of lanes into `stage`; one group.  A lane
// takes 16 bytes at a time, so that a quad's requests are whole sectors (its values of fp32 are two runs
// of four, 4q and 16 + 4q, of bf16 one of eight, 8q: half sectors were fetched twice).
template <int B>
__device__ __forceinline__ void ad_piece(const AdLane &l, const char *const (&row)[2], int piece, int limit, int width, int stage) {
  if (piece < limit) {
#pragma unroll
    for (int c = 0; c < B / 2; ++c) {
      const int k = 32 * piece + (B == 2 ? 8 * l.q : 16 * c + 4 * l.q);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = l.row[h] >= 0 && k < width;
        ad_copy(l.slot + (stage * B + h * (B / 2) + c) * kSlots, ok ? row[h] + k * B : row[h], ok);
      }
    }
  }
  ad_commit();
}

// The operand words of a piece of x: XP parts of rows g (0) and g + 8 (1), four words of two values.
template <int XP>
__device__ __forceinline__ void ad_operands(uint32_t src, uint32_t (&p)[XP][2][4]) {
  if constexpr (XP == 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = lds_u128(src + h * kSlots);
      p[0][h][0] = u.x, p[0][h][1] = u.y, p[0][h][2] = u.z, p[0][h][3] = u.w;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 f[4];
      float most = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 u = lds_u128(src + (2 * h + c) * kSlots);
        f[2 * c] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        f[2 * c + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        most = fmaxf(most, fmaxf(fmaxf(fabsf(f[2 * c].x), fabsf(f[2 * c].y)), fmaxf(fabsf(f[2 * c + 1].x), fabsf(f[2 * c + 1].y))));
      }
      const bool inf = most == __int_as_float(0x7F800000);
#pragma unroll
      for (int i = 0; i < XP; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) p[i][h][k] = i + 1 < XP ? cut_bf16x2(f[k], inf) : round_bf16x2(f[k]);
    }
  }
}

// A ring of weights: stages of `bytes`, filled in order; one for the warps of a kg.
template <int DEPTH>
struct AdRing {
  uint64_t *full, *empty;
  unsigned char *base;
  int bytes, stage = 0, phase = 0;
  __device__ AdRing(unsigned char *smem, const AdSmem &S, int r16, int kg, int kgs)
      : full(reinterpret_cast<uint64_t *>(smem) + kg * DEPTH), empty(full + kgs * DEPTH), base(smem + S.w + kg * DEPTH * r16 * 64),
        bytes(r16 * 64) {}
  __device__ __forceinline__ void next() {
    if (++stage == DEPTH) stage = 0, phase ^= 1;
  }
  // feeding lane: a piece of n bytes, when the stage is free and the copy of its last fill has landed (the
  // second follows from the first but where a wait of the warps ran out)
  __device__ __forceinline__ bool put(const void *src, int n, uint64_t limit) {
    if (!mbar_wait_bounded(&empty[stage], phase ^ 1, limit) || !mbar_wait_bounded(&full[stage], phase ^ 1, kDrainLimit))
      return false;
    mbar_arrive_expect_tx(&full[stage], n);
    bulk_g2s(base + stage * bytes, src, n, &full[stage]);
    next();
    return true;
  }
  // feeding lane, at its end: nothing may be on its way to the block's shared memory when it leaves
  __device__ __forceinline__ void drain() const {
    for (int s = 0; s < DEPTH; ++s) mbar_wait_bounded(&full[s], s < stage ? phase : phase ^ 1, kDrainLimit);
  }
  // A thread whose wait ran out sets the error word and does not wait again: what it then multiplies is
  // in bounds, and every barrier is still reached.
  __device__ __forceinline__ uint32_t take(uint64_t &limit, uint32_t *err) const {
    if (!mbar_wait_bounded(&full[stage], phase, limit)) {
      limit = 0;
      flag_error(err, kErrTimeout);
    }
    return smem_u32(base + stage * bytes);
  }
  __device__ __forceinline__ void give() {  // this warp is done with the stage
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[stage]);
    next();
  }
};

// acc += A_i x over pieces kb, kb + KG, .. of x, for nj (2, 4, 6 or 8) groups of 8 ranks
template <int KG, int XP, int VP, int RC, typename R>
__device__ __forceinline__ void ad_shrink(const AdLane &l, const char *const (&row)[2], int kb, int kb1, int d_in, R &ring, int nj,
                                          float (&acc)[kAdGroups][4], uint64_t &limit, uint32_t *err) {
  constexpr int B = XP == 1 ? 2 : 4, D = ad_depth<XP, VP, RC>();
#pragma unroll
  for (int i = 0; i < D - 1; ++i) ad_piece<B>(l, row, kb + i * KG, kb1, d_in, i);
  int stage = 0;
  for (; kb < kb1; kb += KG) {
    ad_piece<B>(l, row, kb + (D - 1) * KG, kb1, d_in, stage == 0 ? D - 1 : stage - 1);
    ad_wait<D>();
    uint32_t p[XP][2][4];
    ad_operands<XP>(l.slot + stage * B * kSlots, p);
    const uint32_t w = ring.take(limit, err) + (XP == 1 ? l.lane * 16 : (l.lane & ~3) * 16 + l.q * 8);
#pragma unroll
    for (int j = 0; j < kAdGroups; j += 2)
      if (j < nj) {
        uint4 u, v;
        if (XP == 1) {
          u = lds_u128(w + 512 * j), v = lds_u128(w + 512 * j + 512);
        } else {  // the weights of fp32's order of k: half of two other lanes' words each
          const uint2 a = lds_u64(w + 512 * j), b = lds_u64(w + 512 * j + 32);
          const uint2 c = lds_u64(w + 512 * j + 512), d = lds_u64(w + 512 * j + 544);
          u = make_uint4(a.x, a.y, b.x, b.y), v = make_uint4(c.x, c.y, d.x, d.y);
        }
#pragma unroll
        for (int i = 0; i < XP; ++i) {
          const uint32_t a0[4] = {p[i][0][0], p[i][1][0], p[i][0][1], p[i][1][1]};
          const uint32_t a1[4] = {p[i][0][2], p[i][1][2], p[i][0][3], p[i][1][3]};
          mma_bf16(acc[j], a0, u.x, u.y), mma_bf16(acc[j], a1, u.z, u.w);
          mma_bf16(acc[j + 1], a0, v.x, v.y), mma_bf16(acc[j + 1], a1, v.z, v.w);
        }
      }
    ring.give();
    stage = stage == D - 1 ? 0 : stage + 1;
  }
  ad_wait_all();
}

// out = base + B_i v over columns 32 nb .., nb + KG, ..: a lane holds eight columns of its rows, 8q ..
// for bf16 as the packed B orders the MMA columns, 4q .. and 16 + 4q .. for fp32 by taking other lanes'
// words; nk 16-rank steps; the first pieces of base are on their way already.
template <int KG, int XP, int VP, int RC, typename R>
__device__ __forceinline__ void ad_expand(const AdLane &l, const char *const (&base)[2], char *const (&out)[2], int nb, int nb1,
                                          int d_out, R &ring, int nk, uint32_t vaddr, int v_part, uint64_t &limit, uint32_t *err) {
  constexpr int B = VP == 2 ? 2 : 4, D = ad_depth<XP, VP, RC>();
  int stage = 0;
  const int g = l.lane >> 2;
  const uint32_t mine = B == 2 ? l.lane * 16 : ((g >> 1) & 1) * 512 + (4 * (2 * (g >> 2) + (g & 1)) + l.q) * 16;
  for (; nb < nb1; nb += KG) {
    ad_piece<B>(l, base, nb + (D - 1) * KG, nb1, d_out, stage == 0 ? D - 1 : stage - 1);
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    const uint32_t w = ring.take(limit, err) + mine;
#pragma unroll 4
    for (int k = 0; k < nk; ++k) {
      const uint4 wa = lds_u128(w + 1024 * k), wb = lds_u128(w + 1024 * k + (B == 2 ? 512 : 256));
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        uint32_t v[4];
        ldmatrix_x4(v, vaddr + i * v_part + 32 * k);
        mma_bf16(acc[0], v, wa.x, wa.y);
        mma_bf16(acc[1], v, wa.z, wa.w);
        mma_bf16(acc[2], v, wb.x, wb.y);
        mma_bf16(acc[3], v, wb.z, wb.w);
      }
    }
    ring.give();
    ad_wait<D>();
#pragma unroll
    for (int c = 0; c < B / 2; ++c) {
      const int col = 32 * nb + (B == 2 ? 8 * l.q : 16 * c + 4 * l.q);
      if (col >= d_out) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (l.row[h] < 0) continue;
        const uint4 b = lds_u128(l.slot + (stage * B + h * (B / 2) + c) * kSlots);
        const uint32_t b4[4] = {b.x, b.y, b.z, b.w};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (B == 2) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(__uint_as_float(b4[j] << 16) + acc[j][2 * h],
                                                           __uint_as_float(b4[j] & 0xFFFF0000u) + acc[j][2 * h + 1]);
            r[j] = *reinterpret_cast<const uint32_t *>(&q);
          } else {
            r[j] = __float_as_uint(__uint_as_float(b4[j]) + acc[2 * c + (j >> 1)][2 * h + (j & 1)]);
          }
        }
        *reinterpret_cast<uint4 *>(out[h] + col * B) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
    stage = stage == D - 1 ? 0 : stage + 1;
  }
  ad_wait_all();
}

// out = base: tokens without an adapter
template <int KG, int B>
__device__ __forceinline__ void ad_plain_rows(const AdLane &l, char *const (&out)[2], int nb, int nb1, int d_out,
                                              const char *const (&base)[2]) {
  ad_wait_all();
  for (; nb < nb1; nb += KG) {
    const int col = 32 * nb + 8 * l.q;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (l.row[h] >= 0 && col < d_out)
#pragma unroll
        for (int c = 0; c < B / 2; ++c)
          reinterpret_cast<uint4 *>(out[h] + col * B)[c] = reinterpret_cast<const uint4 *>(base[h] + col * B)[c];
  }
}

template <int TM, int XP, int VP, int RC>
__global__ void __launch_bounds__(kAdBlock, 2) k_adapter(const __grid_constant__ AdArgs a) {
  constexpr int MG = TM / 16, KG = kAdWarps / MG;
  constexpr int XB = XP == 1 ? 2 : 4, IO = VP == 2 ? 2 : 4;  // bytes of a value of x; of base and out
  constexpr int DW = kWDepth;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int rows[TM];
  const AdSmem S = ad_smem<TM, XP, VP, RC>(a.max_rank16);
  float *red = reinterpret_cast<float *>(smem + S.ring), *part = reinterpret_cast<float *>(smem + S.part);
  const int tid = threadIdx.x, warp = tid >> 5, mg = warp % MG, kg = warp / MG;
  const int cl = cluster_nctarank(), cr = cluster_ctarank(), tile = blockIdx.x / cl;
  if (tid == 0) {
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);
    for (int i = 0; i < KG * DW; ++i) {
      mbar_init(&bars[i], 1);
      mbar_init(&bars[KG * DW + i], MG);
    }
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch();

  int adapter, cnt;
  if (a.n <= kAdInKernel)
    cnt = ad_find_tile<TM>(a, tile, blockIdx.x == 0, rows, adapter);
  else
    cnt = ad_find_tile_many<TM>(a, tile, blockIdx.x == 0, smem + S.ring, rows, adapter);
  if (cnt == 0) return;  // the same for every block of the cluster
  AdMeta meta{0, 0.f};
  if (adapter < a.slots) {
    meta = a.meta[adapter];
    if (meta.rank == 0 && cr == 0 && tid == 0) flag_error(a.err, kErrBadIndex);  // the slot is empty: as none
  }
  const int r16 = round16(meta.rank), ng = r16 / 8, nk = r16 / 16;
  const int kb_all = (a.d_in + 31) / 32, kb0 = kb_all * cr / cl, kb1 = kb_all * (cr + 1) / cl;
  const int nb_all = (a.d_out + 31) / 32, nb0 = nb_all * cr / cl, nb1 = nb_all * (cr + 1) / cl;

  if (warp == kAdWarps) {
    // ---- the feeding warp: lane kg fills the ring of the warps kg
    const int lane = tid & 31;
    const bool mine = lane < KG;
    AdRing<DW> ring(smem, S, a.max_rank16, mine ? lane : 0, KG);
    bool ok = mine;
    if (a.spin.hold) hold_back(a.spin.hold);
    const __nv_bfloat16 *ap = a.a + a.a_slot * adapter, *bp = a.b + a.b_slot * adapter;
    for (int g0 = 0; g0 < ng; g0 += kAdGroups) {
      const int nj = min(kAdGroups, ng - g0);
      for (int kb = kb0 + lane; kb < kb1 && ok; kb += KG) ok = ring.put(ap + (static_cast<int64_t>(kb) * ng + g0) * 256, nj * 512, a.spin.limit);
    }
    // the first pieces of the second product, then the block's part in the cluster's barriers
    int nb = nb0 + lane, first = 0;
    for (; nk && nb < nb1 && first < DW && ok; nb += KG, ++first) ok = ring.put(bp + static_cast<int64_t>(nb) * nk * 512, nk * 1024, a.spin.limit);
    __syncwarp();
    if (cl > 1) {
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
    }
    for (; nk && nb < nb1 && ok; nb += KG) ok = ring.put(bp + static_cast<int64_t>(nb) * nk * 512, nk * 1024, a.spin.limit);
    if (mine && !ok) flag_error(a.err, kErrTimeout);
    if (mine) ring.drain();
    __syncwarp();
    if (cl > 1) cluster_wait();
    return;
  }

  uint64_t limit = a.spin.limit;
  AdRing<DW> ring(smem, S, a.max_rank16, kg, KG);
  AdLane l;
  l.lane = tid & 31, l.q = tid & 3, l.slot = smem_u32(smem + S.ring) + tid * 16;
  const int g = l.lane >> 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) l.row[h] = 16 * mg + g + 8 * h < cnt ? rows[16 * mg + g + 8 * h] : -1;
  const int64_t at[2] = {l.row[0] < 0 ? 0 : l.row[0], l.row[1] < 0 ? 0 : l.row[1]};

  // ---- v = A_i x over this block's slice of d_in, 64 ranks a pass
  {
    const char *const xr[2] = {static_cast<const char *>(a.x) + at[0] * a.x_ld * XB, static_cast<const char *>(a.x) + at[1] * a.x_ld * XB};
    for (int g0 = 0; g0 < ng; g0 += kAdGroups) {
      const int nj = min(kAdGroups, ng - g0);
      float acc[kAdGroups][4];
#pragma unroll
      for (int j = 0; j < kAdGroups; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;
      ad_shrink<KG, XP, VP, RC>(l, xr, kb0 + kg, kb1, a.d_in, ring, nj, acc, limit, a.err);
      ad_sync();  // the rings are read: the warps' sums take their place
      // added in the order of kg
#pragma unroll
      for (int j = 0; j < kAdGroups; ++j)
        if (j < nj) {
          float *p = red + (kg * TM + 16 * mg + g) * kRedLd + 8 * j + 2 * l.q;
          *reinterpret_cast<float2 *>(p) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2 *>(p + 8 * kRedLd) = make_float2(acc[j][2], acc[j][3]);
        }
      ad_sync();
      for (int i = tid; i < TM * 2 * nj; i += kAdThreads) {
        const int t = i / (2 * nj), r = 4 * (i - t * (2 * nj));
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KG; ++w) {
          const float4 v = *reinterpret_cast<const float4 *>(red + (w * TM + t) * kRedLd + r);
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        *reinterpret_cast<float4 *>(part + t * r16 + 8 * g0 + r) = s;
      }
      ad_sync();
    }
  }

  // ---- the first pieces of base do not wait for v
  const char *const br[2] = {static_cast<const char *>(a.base) + at[0] * a.base_ld * IO,
                             static_cast<const char *>(a.base) + at[1] * a.base_ld * IO};
  char *const orow[2] = {static_cast<char *>(a.out) + at[0] * a.out_ld * IO, static_cast<char *>(a.out) + at[1] * a.out_ld * IO};
#pragma unroll
  for (int i = 0; i < ad_depth<XP, VP, RC>() - 1; ++i) ad_piece<IO>(l, br, nb0 + kg + i * KG, nb1, a.d_out, i);

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
    float2 f = make_float2(s * meta.scale, 0.f);
    const bool inf = fabsf(f.x) == __int_as_float(0x7F800000);
#pragma unroll
    for (int k = 0; k < VP; ++k)
      reinterpret_cast<uint16_t *>(smem + S.v + k * S.v_part)[t * S.v_ld + r] =
          static_cast<uint16_t>(k + 1 < VP ? cut_bf16x2(f, inf) : round_bf16x2(f));
  }
  ad_sync();
  if (cl > 1) cluster_arrive();  // done with the other blocks' shared memory; waited for at the end

  const uint32_t vaddr = smem_u32(smem + S.v) + ((16 * mg + (l.lane & 15)) * S.v_ld + (l.lane >> 4) * 8) * 2;
  if (nk)
    ad_expand<KG, XP, VP, RC>(l, br, orow, nb0 + kg, nb1, a.d_out, ring, nk, vaddr, S.v_part, limit, a.err);
  else if (a.in_place)
    ad_wait_all();
  else
    ad_plain_rows<KG, IO>(l, orow, nb0 + kg, nb1, a.d_out, br);
  __syncwarp();
  if (cl > 1) cluster_wait();
}

// A (rank x d_in) and B (d_out x rank) into the kernels' operand order, padded with zeros to 16
// ranks and 32 columns.
//   A: [k / 32][rank / 8][lane][8]: lane 4g + q holds A[8j + g][32 kb + 8q + e]
//   B: [col / 32][rank / 16][j / 2][lane][j % 2][2][2]: MMA j, lane 4g + q, register h, element e holds
//      column 32 nb + 8 (g / 2) + 2j + g % 2 of rank 16 k + 8h + 2q + e
// One launch packs both matrices (blocks from `blocks_a` on: B) and sets the slot's rank and scale.
__global__ void __launch_bounds__(256) k_adapter_pack(const __nv_bfloat16 *a, const __nv_bfloat16 *b, __nv_bfloat16 *pa, __nv_bfloat16 *pb,
                                                      AdMeta *meta, AdMeta m, int d_in, int d_out, int blocks_a) {
  const int rank = m.rank, r16 = round16(rank), block = blockIdx.x;
  if (block == 0 && threadIdx.x == 0) *meta = m;
  const bool is_b = block >= blocks_a;
  const int d = is_b ? d_out : d_in, d32 = (d + 31) / 32 * 32;
  const int64_t i = static_cast<int64_t>(is_b ? block - blocks_a : block) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(r16) * d32) return;
  int r, c;
  if (is_b) {
    const int e = i & 1, h = (i >> 1) & 1, lane = (i >> 3) & 31, j = ((i >> 2) & 1) + 2 * ((i >> 8) & 1);
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
  (is_b ? pb : pa)[i] = in ? (is_b ? b[static_cast<int64_t>(c) * rank + r] : a[static_cast<int64_t>(r) * d + c]) : __float2bfloat16_rn(0.f);
}

// Error words in host memory that every device can write: handed out from pages that stay with the
// process, since pinning one for each handle takes longer than everything else in its creation.
class ErrorWords {
 public:
  uint32_t *take() {
    std::lock_guard<std::mutex> lock(mutex_);
    if (!free_) {
      Word *page = nullptr;
      if (cudaHostAlloc(reinterpret_cast<void **>(&page), 4096, cudaHostAllocMapped | cudaHostAllocPortable) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
      }
      for (size_t i = 0; i < 4096 / sizeof(Word); ++i) page[i].next = free_, free_ = page + i;
    }
    Word *w = free_;
    free_ = w->next;
    w->err = 0;
    return &w->err;
  }
  void give(uint32_t *err) {
    std::lock_guard<std::mutex> lock(mutex_);
    Word *w = reinterpret_cast<Word *>(err);
    w->next = free_, free_ = w;
  }

 private:
  struct alignas(64) Word {
    uint32_t err;
    Word *next;  // of the words that no handle has
  };
  std::mutex mutex_;
  Word *free_ = nullptr;
};
ErrorWords g_error_words;

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
  uint32_t *err_host = nullptr, *err_dev = nullptr;
  char last_error[160] = "";
};

namespace moe {
bool adapters_match(const moe_adapters *h, int d, int device, int n) {
  return h->cfg.d_in == d && h->cfg.d_out == d && h->cfg.device == device && n <= h->cfg.max_tokens;
}
}  // namespace moe

namespace {

moe_status ad_fail(moe_adapters *h, moe_status s, const char *msg) {
  snprintf(h->last_error, sizeof h->last_error, "%s", msg);
  return s;
}
moe_status ad_cuda(moe_adapters *h, cudaError_t e, const char *what) {
  cudaGetLastError();
  snprintf(h->last_error, sizeof h->last_error, "%s: %s", what, cudaGetErrorString(e));
  return e == cudaErrorMemoryAllocation ? MOE_ERR_OUT_OF_MEMORY : MOE_ERR_CUDA;
}

moe_status ad_pending(moe_adapters *h) {
  const uint32_t e = __atomic_exchange_n(h->err_host, 0u, __ATOMIC_ACQ_REL);
  if (e & kErrTimeout) return ad_fail(h, MOE_ERR_TIMEOUT, "a device-side bounded wait ran out");
  return e ? ad_fail(h, MOE_ERR_DEVICE_FAULT, "an adapter id of an earlier call was out of range or not loaded") : MOE_OK;
}

// Clusters of a size that 148 SMs hold, at one block an SM.
struct Cluster {
  int size, held;
};
constexpr Cluster kClusters[] = {{8, 15}, {4, 33}, {3, 45}, {2, 74}};

int64_t most_tiles(int n, int tm, int slots) { return n / tm + (n < slots + 1 ? n : slots + 1); }

// Launch in clusters of cl blocks, with programmatic stream serialization (the kernels wait for the one
// before them themselves).
struct AdConfig {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  AdConfig(int grid, int threads, int smem, int cl, cudaStream_t st) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cl;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cl > 1 ? 2 : 1;
  }
};

// f(TM, XP, VP, RC) as constants, for every kernel
template <int TM, int RC, typename F>
cudaError_t each_type(F f) {
  constexpr std::integral_constant<int, TM> tm{};
  constexpr std::integral_constant<int, RC> rc{};
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 3> three{};
  cudaError_t e = f(tm, one, two, rc);
  if (e == cudaSuccess) e = f(tm, two, two, rc);
  if (e == cudaSuccess) e = f(tm, one, three, rc);
  return e == cudaSuccess ? f(tm, three, three, rc) : e;
}
template <typename F>
cudaError_t each_kernel(F f) {
  cudaError_t e = each_type<16, 0>(f);
  if (e == cudaSuccess) e = each_type<32, 0>(f);
  if (e == cudaSuccess) e = each_type<16, 1>(f);
  return e == cudaSuccess ? each_type<32, 1>(f) : e;
}

// The kernels' shared-memory limit, once per device, with it current.
cudaError_t configure_kernels(int dev) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[kMaxDevices];
  if (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = each_kernel([](auto tm, auto xp, auto vp, auto rc) {
    constexpr int TM = decltype(tm)::value, XP = decltype(xp)::value, VP = decltype(vp)::value, RC = decltype(rc)::value;
    return cudaFuncSetAttribute(k_adapter<TM, XP, VP, RC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ad_smem<TM, XP, VP, RC>(RC ? kAdMaxRank : 32).total);
  });
  if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
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

namespace moe {
moe_status adapters_pending(moe_adapters *h) { return ad_pending(h); }
}  // namespace moe

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
  const uint64_t oa = take(h->a_slot * 2 * g.max_adapters), ob = take(h->b_slot * 2 * g.max_adapters);
  const uint64_t os = take((static_cast<uint64_t>(g.d_in) + g.d_out) * g.max_rank * 2), om = take(sizeof(AdMeta) * g.max_adapters);
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
    e = cudaMemset(h->meta, 0, sizeof(AdMeta) * g.max_adapters);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) {
      h->err_host = g_error_words.take();
      e = h->err_host ? cudaHostGetDevicePointer(reinterpret_cast<void **>(&h->err_dev), h->err_host, 0) : cudaErrorMemoryAllocation;
    }
    if (e == cudaSuccess) e = current_sm_count(&h->nsm);
    if (e == cudaSuccess) e = configure_kernels(g.device);
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
  if (h->err_host) g_error_words.give(h->err_host);
  cudaGetLastError();
  delete h;
  return MOE_OK;
}

const char *moe_adapters_last_error(const moe_adapters *h) { return h ? h->last_error : "no handle"; }

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
  // host sources pass through the staging buffer, in stream order
  const void *src[2] = {a, b};
  bool host = false;
  for (int m = 0; m < 2 && rank && e == cudaSuccess; ++m) {
    if (!host_ptr(src[m])) continue;
    host = true;
    __nv_bfloat16 *to = h->stage + (m ? static_cast<size_t>(g.d_in) * g.max_rank : 0);
    e = cudaMemcpyAsync(to, src[m], static_cast<size_t>(rank) * (m ? g.d_out : g.d_in) * 2, cudaMemcpyHostToDevice, st);
    src[m] = to;
  }
  if (e == cudaSuccess) {
    const int64_t r16 = round16(rank);
    const int blocks_a = static_cast<int>((r16 * ((g.d_in + 31) / 32 * 32) + 255) / 256);
    const int blocks_b = static_cast<int>((r16 * ((g.d_out + 31) / 32 * 32) + 255) / 256);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rank ? blocks_a + blocks_b : 1);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    e = cudaLaunchKernelEx(&cfg, k_adapter_pack, static_cast<const __nv_bfloat16 *>(src[0]),
                           static_cast<const __nv_bfloat16 *>(src[1]), h->a + h->a_slot * slot, h->b + h->b_slot * slot,
                           h->meta + slot, AdMeta{rank, scale}, g.d_in, g.d_out, blocks_a);
  }
  if (e == cudaSuccess && host) e = cudaStreamSynchronize(st);
  return e == cudaSuccess ? MOE_OK : ad_cuda(h, e, "adapter load");
}

moe_status moe_adapters_apply(moe_adapters *h, const void *x, int32_t x_dtype, int64_t x_stride, const void *base,
                              int64_t base_stride, void *out, int64_t out_stride, int32_t out_dtype, const int32_t *ids,
                              int32_t n_tokens, void *stream) {
  return adapters_run(h, x, x_dtype, x_stride, base, base_stride, out, out_stride, out_dtype, ids, n_tokens, stream, true);
}

}  // extern "C"

moe_status moe::adapters_run(moe_adapters *h, const void *x, int32_t x_dtype, int64_t x_stride, const void *base,
                             int64_t base_stride, void *out, int64_t out_stride, int32_t out_dtype, const int32_t *ids,
                             int32_t n_tokens, void *stream, bool pending) {
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
  if (base == out && n_tokens > 1 && base_stride != out_stride)
    return ad_fail(h, MOE_ERR_INVALID_ARGUMENT, "out is base with another row stride");
  if (const moe_status s = pending ? ad_pending(h) : MOE_OK) return s;
  Device dev(g.device);
  if (!dev.ok) return ad_fail(h, MOE_ERR_CUDA, "set device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AdArgs a{};
  a.x = x, a.base = base, a.out = out, a.ids = ids;
  a.a = h->a, a.b = h->b, a.meta = h->meta, a.a_slot = h->a_slot, a.b_slot = h->b_slot;
  a.err = h->err_dev;
  a.x_ld = x_stride, a.base_ld = base_stride, a.out_ld = out_stride;
  a.n = n_tokens, a.d_in = g.d_in, a.d_out = g.d_out, a.slots = g.max_adapters, a.max_rank16 = h->r16;
  a.x_bf16 = x_dtype == MOE_BF16, a.io_bf16 = out_dtype == MOE_BF16;
  a.in_place = base == out;
  a.spin = ring_spin();
  const cudaError_t e = each_kernel([&](auto tmc, auto xp, auto vp, auto rc) {
    constexpr int TM = decltype(tmc)::value, XP = decltype(xp)::value, VP = decltype(vp)::value, RC = decltype(rc)::value;
    if ((RC == 0) != (h->r16 <= 32) || (VP == 2) != (a.io_bf16 != 0) || (XP == 1) != (a.x_bf16 != 0)) return cudaSuccess;
    // Tiles of 16 tokens, whose warps share k eight ways, where all of them fit on the device at once, else of
    // 32, which read a group's weights half as often (2,048 -> 2,048, us, 16 and 32: 1,180 tokens of rank 16
    // 13.0, 13.7; 4,096 of rank 64 25.6, 28.5; 8,192 58.9, 43.7; with tiles of 64: 48.9).
    const auto room = [&](int smem) { return static_cast<int64_t>(h->nsm) * (2 * (smem + 1024) <= kSmSmem ? 2 : 1); };
    const int small = ad_smem<16, XP, VP, RC>(a.max_rank16).total, smem = ad_smem<TM, XP, VP, RC>(a.max_rank16).total;
    if (TM != (most_tiles(n_tokens, 16, g.max_adapters) <= room(small) ? 16 : 32)) return cudaSuccess;
    // Blocks of a tile: as many as fit at once (clusters of two in two rounds took 28 us, single blocks in one
    // 19: 1,180 tokens, 20 adapters of rank 64, fp32 x; of three, 5 of rank 33, 19 us, of two 22).
    const int64_t tiles = most_tiles(n_tokens, TM, g.max_adapters), most = room(smem);
    int cl = 1;
    for (const Cluster &c : kClusters)
      if (cl == 1 && tiles * 148 <= most * c.held) cl = c.size;
    const AdConfig c(static_cast<int>(tiles) * cl, kAdBlock, smem, cl, st);
    return cudaLaunchKernelEx(&c.cfg, k_adapter<TM, XP, VP, RC>, a);
  });
  return e == cudaSuccess ? MOE_OK : ad_cuda(h, e, "adapter launch");
}
