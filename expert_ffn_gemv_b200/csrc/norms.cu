// norms.cu -- RMS norms before and after a block, fused with the block's gate, the residual scale
// and the residual add, and their gradients.
//
// Forward, per token (one thread block per row, the row held in registers between the passes):
//   q  = rsqrt(mean(o^2) + eps)             u = o q w   (no post norm: u = o)
//   r' = r + s a(g) u                       a = identity or sigmoid, g broadcast or full
//   p  = rsqrt(mean(r'^2) + eps')           h = r' p w'  (r' as it is stored)
// Backward of the post norm, per token, with dz = s dr':
//   t = dz a w       do = q (t - o q^2 mean(t o))       dw += dz a o q      dg = dz u a'(g)
// Backward of the input norm:
//   t = dh w'        dr = dr' + p (t - x p^2 mean(t x))  dw' += dh x p
// The products and sums that decide a stored value's last bits are rounded in the order written above,
// without fused multiply-adds: where a residual or gradient is then rounded to bf16 it falls on the side
// that the formula's fp32 evaluation gives, so that what is computed from it in fp32 (dw, do, dw') agrees
// to 2e-5.  With them contracted, one gradient in sixteen over random shapes was further off.
// Sums over columns are taken over the row's threads (shuffles, then the warps in order), sums over
// tokens (dw, the gradient of a channel gate) in two steps: every block of a grid that depends on the
// sizes and the device alone adds its rows in order, k_colsum adds the blocks' partial rows in order.  No
// atomics: the same call gives the same bits.
#include <math.h>
#include <string.h>

#include <initializer_list>
#include <mutex>

#include "block.cuh"

namespace moe {
namespace {

// V consecutive values (V = 1, 2, 4 or 8: the widest that width, pointers and strides allow)
template <int V>
__device__ __forceinline__ void load_v(const void *p, int64_t i, int bf16, float (&v)[V]) {
  if (bf16) {
    const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p) + i;
    if constexpr (V == 1) {
      v[0] = __bfloat162float(*b);
    } else {
      uint32_t w[V / 2];
      if constexpr (V == 8) {
        const uint4 q = *reinterpret_cast<const uint4 *>(b);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      } else if constexpr (V == 4) {
        const uint2 q = *reinterpret_cast<const uint2 *>(b);
        w[0] = q.x, w[1] = q.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t *>(b);
      }
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  } else {
    const float *f = static_cast<const float *>(p) + i;
    if constexpr (V == 1) {
      v[0] = *f;
    } else if constexpr (V == 2) {
      const float2 a = *reinterpret_cast<const float2 *>(f);
      v[0] = a.x, v[1] = a.y;
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(f + k);
        v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
      }
    }
  }
}

// Stores v rounded to the destination's type and leaves in v the values as they are stored.
template <int V>
__device__ __forceinline__ void store_v(void *p, int64_t i, int bf16, float (&v)[V]) {
  if (bf16) {
    __nv_bfloat16 *b = static_cast<__nv_bfloat16 *>(p) + i;
    if constexpr (V == 1) {
      const __nv_bfloat16 h = __float2bfloat16_rn(v[0]);
      *b = h;
      v[0] = __bfloat162float(h);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t *>(&h);
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
      if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(b) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(b) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t *>(b) = w[0];
    }
  } else {
    float *f = static_cast<float *>(p) + i;
    if constexpr (V == 1) {
      *f = v[0];
    } else if constexpr (V == 2) {
      *reinterpret_cast<float2 *>(f) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) *reinterpret_cast<float4 *>(f + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    }
  }
}

// A thread's values of a row: columns (256 c + thread) V .. + V - 1, c < NCH, below d <= kNormMaxD.  (A
// block of fewer threads holds its row in c = 0.)  One branch on the type for all of a row's loads.
constexpr int kNormMaxThreads = 256;
template <int V, int NCH>
__device__ __forceinline__ void load_row(const void *p, int64_t first, int bf16, int d, float (&v)[NCH][V]) {
  const int i0 = threadIdx.x * V;
  if (bf16) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p) + first + i0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (i0 + c * kNormMaxThreads * V < d) load_v<V>(q, c * kNormMaxThreads * V, 1, v[c]);
  } else {
    const float *q = static_cast<const float *>(p) + first + i0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (i0 + c * kNormMaxThreads * V < d) load_v<V>(q, c * kNormMaxThreads * V, 0, v[c]);
  }
}
template <int V, int NCH>
__device__ __forceinline__ void store_row(void *p, int64_t first, int bf16, int d, float (&v)[NCH][V]) {
  const int i0 = threadIdx.x * V;
  if (bf16) {
    __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(p) + first + i0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (i0 + c * kNormMaxThreads * V < d) store_v<V>(q, c * kNormMaxThreads * V, 1, v[c]);
  } else {
    float *q = static_cast<float *>(p) + first + i0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (i0 + c * kNormMaxThreads * V < d) store_v<V>(q, c * kNormMaxThreads * V, 0, v[c]);
  }
}
// f(value index in the thread) for all of them
#define MOE_EACH(c, k)             \
  _Pragma("unroll") for (int c = 0; c < NCH; ++c) _Pragma("unroll") for (int k = 0; k < V; ++k)

template <int V, int NCH>
__device__ __forceinline__ void fill(float (&v)[NCH][V], float x) {
  MOE_EACH(c, k) v[c][k] = x;
}

// Sums of NV values over `threads` threads of the block, in every one of them: shuffles, then the warps'
// sums in order.  red: [NV][8], zeros where there is no warp (clear_sums); calls take turns with two of
// them, so one barrier a call is enough.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float *red, int threads) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (threads == 32) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < NV; ++k) red[8 * k + (threadIdx.x >> 5)] = v[k];
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const float4 p = *reinterpret_cast<const float4 *>(red + 8 * k), q = *reinterpret_cast<const float4 *>(red + 8 * k + 4);
    v[k] = ((((((p.x + p.y) + p.z) + p.w) + q.x) + q.y) + q.z) + q.w;
  }
}
// Before the first sum; the caller's next barrier over the block comes after it.
template <int N>
__device__ __forceinline__ void clear_sums(float (&red)[N]) {
  for (int i = threadIdx.x; i < N; i += 32)
    if (threadIdx.x < 32) red[i] = 0.f;
  __syncthreads();
}

// a(g).  A gate of a row scales all its values, so that its last bit decides many roundings: it is taken
// with expf and a division.  Gates by the value take the fast form (8,192 x 4,096, a gate for every value:
// 56 us, 69 with the other).
__device__ __forceinline__ float gate_value(float g, int act) {
  return act == MOE_GATE_SIGMOID ? 1.0f / (1.0f + expf(-g)) : g;
}
// The slope of the sigmoid is sigmoid(g) sigmoid(-g).  With the second factor as 1 - a nothing would be left
// where a rounds to 1 (off by 1e-3 at g = 10, 0 from g = 17 on, where the slope is 4e-8), so it comes from
// the exponential.  Of a token's gate, a = gate_value(g):
__device__ __forceinline__ float gate_slope(float g, float a, int act) {
  return act == MOE_GATE_SIGMOID ? a * fminf(expf(-g) * a, 1.0f) : 1.f;  // (infinity times 0 gives 1)
}
// Both factors of a value's gate.
__device__ __forceinline__ void fast_sigmoids(float g, float &a, float &c) {
  float e;
  a = fast_sigmoid(g, e);
  c = fminf(e * a, 1.0f);  // infinity times 0: 1
}
// The same of a column's gate, kept in one register for all rows: the smaller factor, with the sign bit set
// where g is positive.
__device__ __forceinline__ float fold_sigmoid(float g) {
  float a, c;
  fast_sigmoids(g, a, c);
  return g > 0.f ? -c : a;
}
__device__ __forceinline__ float folded_value(float v) { return __float_as_int(v) < 0 ? 1.0f + v : v; }
__device__ __forceinline__ float folded_slope(float v) { return fmaf(-fabsf(v), fabsf(v), fabsf(v)); }

// 1 / sqrt(sum / d + eps)
__device__ __forceinline__ float root(float sum, float inv_d, float eps) { return rsqrtf(__fadd_rn(__fmul_rn(sum, inv_d), eps)); }

template <int V, int NCH>
__device__ __forceinline__ void gate_values(float (&g)[NCH][V], int act) {
  if (act == MOE_GATE_SIGMOID) MOE_EACH(c, k) g[c][k] = fast_sigmoid(g[c][k]);
}

struct NormFwd {
  const void *o, *res, *w, *gate, *next_w;
  void *res_out, *h;
  int64_t o_ld, res_ld, gate_ld, out_ld, h_ld;
  int o_bf16, res_bf16, out_bf16, w_bf16, gate_bf16, h_bf16;
  int gate_kind, gate_act, d;
  float eps, next_eps, scale, w_off, inv_d;
};

// A row's gate is per value (of its own, or one per column).
__device__ __forceinline__ bool gate_by_value(int kind) { return kind == MOE_GATE_CHANNEL || kind == MOE_GATE_FULL; }

// weight + unit offset; zeros past d
template <int V, int NCH>
__device__ __forceinline__ void load_weight(const void *p, int bf16, int d, float off, float (&w)[NCH][V]) {
  load_row<V, NCH>(p, 0, bf16, d, w);
  if (off != 0.f) {
    const int i0 = threadIdx.x * V;
    MOE_EACH(c, k) if (i0 + c * kNormMaxThreads * V < d) w[c][k] += off;
  }
}

// What follows a row's loads.  Values past d are zeros everywhere.  The weights come in registers (KEEP,
// with the offset added) or are loaded where they are used; `active`: g holds a(g) already.
template <int V, int NCH, bool KEEP>
__device__ __forceinline__ void fwd_row(const NormFwd &a, int64_t t, float (&r)[NCH][V], float (&o)[NCH][V], float (&g)[NCH][V],
                                        float (&w)[NCH][V], float (&wn)[NCH][V], float gt, float *red, int threads,
                                        bool active) {
  const int d = a.d;
  if (a.o) {
    const bool by_value = gate_by_value(a.gate_kind);
    if (a.w) {
      float ss[1] = {0.f};
      MOE_EACH(c, k) ss[0] = fmaf(o[c][k], o[c][k], ss[0]);
      if (!KEEP) load_weight<V, NCH>(a.w, a.w_bf16, d, a.w_off, w);
      block_sum<1>(ss, red, threads);
      const float q = root(ss[0], a.inv_d, a.eps);
      MOE_EACH(c, k) o[c][k] = __fmul_rn(__fmul_rn(o[c][k], q), w[c][k]);
    }
    if (by_value) {
      if (!active) gate_values<V, NCH>(g, a.gate_act);
      MOE_EACH(c, k) r[c][k] = __fadd_rn(r[c][k], __fmul_rn(a.scale, __fmul_rn(g[c][k], o[c][k])));
    } else {
      MOE_EACH(c, k) r[c][k] = __fadd_rn(r[c][k], __fmul_rn(a.scale, __fmul_rn(gt, o[c][k])));
    }
    store_row<V, NCH>(a.res_out, t * a.out_ld, a.out_bf16, d, r);
  }
  if (!a.h) return;
  float ss[1] = {0.f};
  MOE_EACH(c, k) ss[0] = fmaf(r[c][k], r[c][k], ss[0]);
  if (!KEEP) load_weight<V, NCH>(a.next_w, a.w_bf16, d, a.w_off, wn);
  block_sum<1>(ss, red + 8, threads);
  const float p = root(ss[0], a.inv_d, a.next_eps);
  MOE_EACH(c, k) r[c][k] = __fmul_rn(__fmul_rn(r[c][k], p), wn[c][k]);
  store_row<V, NCH>(a.h, t * a.h_ld, a.h_bf16, d, r);
}

// A token gate g and a(g), else 1
__device__ __forceinline__ float2 token_gates(const void *gate, int kind, int act, int64_t i, int bf16) {
  if (kind != MOE_GATE_TOKEN) return make_float2(1.f, 1.f);
  float g[1];
  load_v<1>(gate, i, bf16, g);
  return make_float2(g[0], gate_value(g[0], act));
}
__device__ __forceinline__ float token_gate(const void *gate, int kind, int act, int64_t i, int bf16) {
  return token_gates(gate, kind, act, i, bf16).y;
}

// One block per token, every load of the row on its way before the first sum.
template <int V, int NCH>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_fwd(const __grid_constant__ NormFwd a) {
  __shared__ __align__(16) float red[16];
  const int64_t t = blockIdx.x;
  const int d = a.d;
  griddep_wait();
  griddep_launch();
  float r[NCH][V], o[NCH][V], g[NCH][V], w[NCH][V], wn[NCH][V];
  fill<V, NCH>(r, 0.f), fill<V, NCH>(o, 0.f), fill<V, NCH>(g, 0.f), fill<V, NCH>(w, 0.f), fill<V, NCH>(wn, 0.f);
  load_row<V, NCH>(a.res, t * a.res_ld, a.res_bf16, d, r);
  if (a.o) load_row<V, NCH>(a.o, t * a.o_ld, a.o_bf16, d, o);
  if (gate_by_value(a.gate_kind))
    load_row<V, NCH>(a.gate, a.gate_kind == MOE_GATE_FULL ? t * a.gate_ld : 0, a.gate_bf16, d, g);
  const float gt = token_gate(a.gate, a.gate_kind, a.gate_act, t * a.gate_ld, a.gate_bf16);
  constexpr bool KEEP = V * NCH <= 8;
  if (KEEP && a.w) load_weight<V, NCH>(a.w, a.w_bf16, d, a.w_off, w);
  if (KEEP && a.h) load_weight<V, NCH>(a.next_w, a.w_bf16, d, a.w_off, wn);
  clear_sums(red);
  fwd_row<V, NCH, KEEP>(a, t, r, o, g, w, wn, gt, red, blockDim.x, false);
}

struct NormBwd {
  const void *x, *dy, *w, *gate, *dres;  // post norm: x = o, dy = dr'; input norm: x, dy = dh, dres
  void *dx, *dgate;
  float *dw_part, *dg_part;              // [blocks][d] sums over the block's rows, or NULL
  int64_t x_ld, dy_ld, gate_ld, dres_ld, dx_ld, dgate_ld;
  int x_bf16, dy_bf16, w_bf16, gate_bf16, dres_bf16, dx_bf16;
  int gate_kind, gate_act, d, n;
  float eps, scale, w_off, inv_d;
};

// What a block keeps from row to row: the sums over its rows (a channel gate's without its slope, which
// comes in at the end), and (KEEP) the weight and a gate by column.  For the slope a sigmoid's two factors are
// kept folded, or the gate is loaded again at the end.  The second costs up to 1 us (1,177 x 1,001: 12.9 us
// against 12.2), the first arithmetic in every row, which many rows feel (8,192 x 2,048: 43.5 us against 41),
// and registers, which cost eight values a thread half their blocks (1,177 x 2,001: 21.9 us against 18.0).
template <int V, int NCH, bool KEEP, bool RING>
struct BwdState {
  static constexpr bool FOLD = KEEP && !RING && V * NCH != 8;
  float dw[NCH][V], dg[NCH][V], w[NCH][V], gc[NCH][V];
  __device__ __forceinline__ explicit BwdState(const NormBwd &a) {
    fill<V, NCH>(dw, 0.f), fill<V, NCH>(dg, 0.f), fill<V, NCH>(w, a.w ? 0.f : 1.f), fill<V, NCH>(gc, 0.f);
    if (KEEP) columns(a);
  }
  __device__ __forceinline__ void columns(const NormBwd &a) {
    if (a.w) load_weight<V, NCH>(a.w, a.w_bf16, a.d, a.w_off, w);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      load_row<V, NCH>(a.gate, 0, a.gate_bf16, a.d, gc);
      if (FOLD && a.gate_act == MOE_GATE_SIGMOID) {
        MOE_EACH(c, k) gc[c][k] = fold_sigmoid(gc[c][k]);
      } else {
        gate_values<V, NCH>(gc, a.gate_act);
      }
    }
  }
  __device__ __forceinline__ void finish(const NormBwd &a) {
    if (a.dg_part && a.gate_act == MOE_GATE_SIGMOID) {
      if (!FOLD) {
        load_row<V, NCH>(a.gate, 0, a.gate_bf16, a.d, gc);
        MOE_EACH(c, k) gc[c][k] = fold_sigmoid(gc[c][k]);
      }
      MOE_EACH(c, k) dg[c][k] *= folded_slope(gc[c][k]);
    }
    if (a.dw_part) store_row<V, NCH>(a.dw_part, static_cast<int64_t>(blockIdx.x) * a.d, 0, a.d, dw);
    if (a.dg_part) store_row<V, NCH>(a.dg_part, static_cast<int64_t>(blockIdx.x) * a.d, 0, a.d, dg);
  }
};
template <int V, int NCH>
struct BwdRow {
  float x[NCH][V], dy[NCH][V], dres[NCH][V], g[NCH][V];
};

template <int V, int NCH, bool KEEP, bool RING>
__device__ __forceinline__ void bwd_row(const NormBwd &a, int64_t t, BwdRow<V, NCH> &q, BwdState<V, NCH, KEEP, RING> &st,
                                        float2 token, float *red, int threads) {
  const int d = a.d;
  const float gt = token.y;
  if (!KEEP) st.columns(a);
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL, full = a.gate_kind == MOE_GATE_FULL;
  const bool sigmoid = a.gate_act == MOE_GATE_SIGMOID, full_sigmoid = full && sigmoid;
  if (st.FOLD && channel && sigmoid) {
    MOE_EACH(c, k) q.g[c][k] = folded_value(st.gc[c][k]);
  } else if (channel) {
    MOE_EACH(c, k) q.g[c][k] = st.gc[c][k];
  }
  // sums of x^2 and of s dy a w x, the second without the gate where a row has only one
  const bool by_value = full || channel;
  float s[2] = {0.f, 0.f};
  MOE_EACH(c, k) {
    q.dy[c][k] = __fmul_rn(a.scale, q.dy[c][k]);
    s[0] = fmaf(q.x[c][k], q.x[c][k], s[0]);
  }
  if (full_sigmoid) {  // leaves s dy a in dy, the slope's other factor in g
    MOE_EACH(c, k) {
      float av, other;
      fast_sigmoids(q.g[c][k], av, other);
      q.dy[c][k] = __fmul_rn(q.dy[c][k], av);
      q.g[c][k] = other;
      s[1] = fmaf(__fmul_rn(q.dy[c][k], st.w[c][k]), q.x[c][k], s[1]);
    }
  } else if (by_value) {
    MOE_EACH(c, k) s[1] = fmaf(__fmul_rn(__fmul_rn(q.dy[c][k], q.g[c][k]), st.w[c][k]), q.x[c][k], s[1]);
  } else {
    MOE_EACH(c, k) s[1] = fmaf(__fmul_rn(q.dy[c][k], st.w[c][k]), q.x[c][k], s[1]);
  }
  block_sum<2>(s, red, threads);
  const float rt = a.w ? root(s[0], a.inv_d, a.eps) : 1.f;
  const float m = a.w ? (by_value ? s[1] : gt * s[1]) * a.inv_d * (rt * rt) : 0.f;
  if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && threadIdx.x == 0) {
    float v1[1] = {gate_slope(token.x, gt, a.gate_act) * rt * s[1]};
    store_v<1>(a.dgate, t * a.dgate_ld, a.gate_bf16, v1);
  }
  // dx in dres, the gradient of a value's own gate in g
  if (full_sigmoid) {
    MOE_EACH(c, k) {
      const float x = q.x[c][k], da = q.dy[c][k];
      q.dres[c][k] = __fadd_rn(q.dres[c][k], __fmul_rn(rt, fmaf(-x, m, __fmul_rn(da, st.w[c][k]))));
      st.dw[c][k] = fmaf(da * rt, x, st.dw[c][k]);
      q.g[c][k] = da * (x * rt * st.w[c][k]) * q.g[c][k];
    }
  } else if (by_value) {
    MOE_EACH(c, k) {
      const float x = q.x[c][k], da = __fmul_rn(q.dy[c][k], q.g[c][k]);
      q.dres[c][k] = __fadd_rn(q.dres[c][k], __fmul_rn(rt, fmaf(-x, m, __fmul_rn(da, st.w[c][k]))));
      st.dw[c][k] = fmaf(da * rt, x, st.dw[c][k]);
      const float gg = q.dy[c][k] * (x * rt * st.w[c][k]);
      st.dg[c][k] += gg;
      q.g[c][k] = gg;
    }
  } else {
    MOE_EACH(c, k) {
      const float x = q.x[c][k], da = __fmul_rn(q.dy[c][k], gt);
      q.dres[c][k] = __fadd_rn(q.dres[c][k], __fmul_rn(rt, fmaf(-x, m, __fmul_rn(da, st.w[c][k]))));
      st.dw[c][k] = fmaf(da * rt, x, st.dw[c][k]);
    }
  }
  store_row<V, NCH>(a.dx, t * a.dx_ld, a.dx_bf16, d, q.dres);
  if (full && a.dgate) store_row<V, NCH>(a.dgate, t * a.dgate_ld, a.gate_bf16, d, q.g);
}

// Persistent: block b takes rows b, b + grid, ...; where a thread holds few values of a row (NEXT) the
// next row is loaded while this one is summed (without it, a row took 6 us of latency after latency:
// 28 us for 4 rows a block).
template <int V, int NCH>
__global__ void __launch_bounds__(kNormMaxThreads, V * NCH <= 2 ? 3 : 0) k_norm_bwd(const __grid_constant__ NormBwd a) {
  constexpr bool NEXT = V * NCH <= 8;
  __shared__ __align__(16) float red[48];
  const int d = a.d, threads = blockDim.x;
  clear_sums(red);
  griddep_wait();
  griddep_launch();
  constexpr bool KEEP = V * NCH <= 16;
  BwdState<V, NCH, KEEP, false> st(a);
  auto load = [&](int64_t t, BwdRow<V, NCH> &q, float2 &gt) {
    fill<V, NCH>(q.x, 0.f), fill<V, NCH>(q.dy, 0.f), fill<V, NCH>(q.dres, 0.f), fill<V, NCH>(q.g, 0.f);
    if (t >= a.n) return;
    load_row<V, NCH>(a.x, t * a.x_ld, a.x_bf16, d, q.x);
    load_row<V, NCH>(a.dy, t * a.dy_ld, a.dy_bf16, d, q.dy);
    if (a.dres) load_row<V, NCH>(a.dres, t * a.dres_ld, a.dres_bf16, d, q.dres);
    if (a.gate_kind == MOE_GATE_FULL) load_row<V, NCH>(a.gate, t * a.gate_ld, a.gate_bf16, d, q.g);
    gt = token_gates(a.gate, a.gate_kind, a.gate_act, t * a.gate_ld, a.gate_bf16);
  };
  if (NEXT) {
    BwdRow<V, NCH> q0, q1;
    float2 g0{}, g1{};
    load(blockIdx.x, q0, g0);
    for (int64_t t = blockIdx.x; t < a.n; t += 2 * gridDim.x) {
      load(t + gridDim.x, q1, g1);
      bwd_row(a, t, q0, st, g0, red, threads);
      if (t + gridDim.x >= a.n) break;
      load(t + 2 * gridDim.x, q0, g0);
      bwd_row(a, t + gridDim.x, q1, st, g1, red + 24, threads);
    }
  } else {
    int k = 0;
    for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x, k ^= 1) {
      BwdRow<V, NCH> q;
      float2 gt{};
      load(t, q, gt);
      bwd_row(a, t, q, st, gt, red + 24 * k, threads);
    }
  }
  st.finish(a);
}

// ------------------------------------------------------------------------------------------
// Many rows of whole vectors: persistent blocks fed by a ring of bulk copies.  A stage holds the rows
// of one token that the kernel reads (contiguous runs of d values, 16-byte aligned); the block's last
// warp refills a stage when the others have its values in registers, so the copies of the next rows
// never wait for a row's sums, and a row costs its arithmetic, not its latencies.
// ------------------------------------------------------------------------------------------
constexpr uint64_t kRingSpin = 2000000000ull;  // about a second
std::atomic<uint64_t> g_ring_limit{0};         // of a test, 0: the default
constexpr int kRingMaxStages = 6, kRingMaxRows = 4;

struct RowSource {
  const void *p;
  int64_t ld;
  int bf16;
};
struct Ring {
  RowSource src[kRingMaxRows];
  int n_src, stages, stage_bytes;
  RingSpin spin;
  uint32_t *err;  // set where a bounded wait ran out
};

struct RingState {
  unsigned char *base;
  uint64_t *full, *empty;
  uint64_t limit;
  int threads;  // that compute: all warps but the last
  __device__ RingState(unsigned char *smem, const Ring &r) : base(smem + 128), limit(r.spin.limit), threads(blockDim.x - 32) {
    full = reinterpret_cast<uint64_t *>(smem);
    empty = full + kRingMaxStages;
    if (threadIdx.x == 0) {
      for (int s = 0; s < r.stages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], threads / 32);
      }
      fence_barrier_init();
    }
  }
  __device__ bool producer() const { return static_cast<int>(threadIdx.x) >= threads; }
  // The last warp: lane i copies row i of a token, k-th token of this block after the other.  A stage is
  // filled again when the others have given it back and the copies of its last fill have landed: the
  // second follows from the first but where a wait of the others ran out.
  __device__ void produce(const Ring &r, int d, int n) const {
    const int lane = threadIdx.x & 31;
    const bool mine = lane < r.n_src;
    const RowSource src = r.src[mine ? lane : 0];
    const int size = src.bf16 ? 2 : 4;
    int off = 0;
    for (int i = 0; i < lane && i < r.n_src; ++i) off += d * (r.src[i].bf16 ? 2 : 4);
    const char *p = static_cast<const char *>(src.p) + blockIdx.x * src.ld * size;
    const int64_t step = static_cast<int64_t>(gridDim.x) * src.ld * size;
    int s = 0, phase = 1;
    uint32_t armed = 0;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x, ++armed) {
      const bool free = mbar_wait_bounded(&empty[s], phase, r.spin.limit);
      const bool landed = armed < static_cast<uint32_t>(r.stages) || mbar_wait_bounded(&full[s], phase, kDrainLimit);
      if (!__all_sync(0xffffffffu, free && landed)) {
        if (lane == 0) flag_error(r.err, kErrTimeout);
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[s], r.stage_bytes);
      if (armed == 0 && r.spin.hold) hold_back(r.spin.hold);
      __syncwarp();
      if (mine) bulk_g2s(base + s * r.stage_bytes + off, p, d * size, &full[s]);
      p += step;
      if (++s == r.stages) s = 0, phase ^= 1;
    }
    // nothing may be on its way to the block's shared memory when it leaves: the last fill of every stage
    // is waited for here, whatever the other warps did
    __syncwarp();
    if (lane == 0)
      for (uint32_t k = armed > static_cast<uint32_t>(r.stages) ? armed - r.stages : 0; k < armed; ++k)
        mbar_wait_bounded(&full[k % r.stages], (k / r.stages) & 1u, kDrainLimit);
    __syncwarp();
  }
  // A thread whose wait ran out does not wait again: what it then reads and writes is in bounds, and every
  // barrier is still reached.  It sets the error word after its last row (in the loop over the rows that cost
  // 8,192 x 4,096 with a gate per value 3 us of 57).
  __device__ __forceinline__ const unsigned char *wait(const Ring &r, int s, int phase) {
    if (!mbar_wait_bounded(&full[s], phase, limit)) limit = 0;
    return base + s * r.stage_bytes;
  }
  __device__ __forceinline__ void report(const Ring &r) const {  // after the last row
    if (!limit) flag_error(r.err, kErrTimeout);
  }
  __device__ __forceinline__ void release(int s) const {  // this warp has the stage in registers
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
  }
};

constexpr int kRingThreads = kNormMaxThreads + 32;

template <int NCH>
__global__ void __launch_bounds__(kRingThreads, NCH == 1 ? 3 : NCH == 2 ? 2 : 1) k_norm_fwd_ring(const __grid_constant__ NormFwd a,
                                                                                 const __grid_constant__ Ring r, int n) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) float red[32];
  constexpr int V = 8;
  const int d = a.d;
  RingState ring(smem, r);
  clear_sums(red);
  griddep_wait();
  griddep_launch();
  if (ring.producer()) {
    ring.produce(r, d, n);
    return;
  }
  // in registers for a block's rows while they are few; from L1 where that would cost a block of the SM
  constexpr bool KEEP = NCH == 1;
  float w[NCH][V], wn[NCH][V], gc[NCH][V];
  fill<V, NCH>(w, 0.f), fill<V, NCH>(wn, 0.f), fill<V, NCH>(gc, 0.f);
  const bool full = a.gate_kind == MOE_GATE_FULL, channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (KEEP) {
    if (a.w) load_weight<V, NCH>(a.w, a.w_bf16, d, a.w_off, w);
    if (a.h) load_weight<V, NCH>(a.next_w, a.w_bf16, d, a.w_off, wn);
    if (channel) {
      load_row<V, NCH>(a.gate, 0, a.gate_bf16, d, gc);
      gate_values<V, NCH>(gc, a.gate_act);
    }
  }
  int s = 0, phase = 0, turn = 0;
  for (int64_t t = blockIdx.x; t < n; t += gridDim.x, turn ^= 16) {
    float x[NCH][V], o[NCH][V], g[NCH][V];
    fill<V, NCH>(x, 0.f), fill<V, NCH>(o, 0.f), fill<V, NCH>(g, 0.f);
    const float gt = token_gate(a.gate, a.gate_kind, a.gate_act, t * a.gate_ld, a.gate_bf16);
    const unsigned char *p = ring.wait(r, s, phase);
    load_row<V, NCH>(p, 0, a.res_bf16, d, x);
    p += d * (a.res_bf16 ? 2 : 4);
    if (a.o) {
      load_row<V, NCH>(p, 0, a.o_bf16, d, o);
      p += d * (a.o_bf16 ? 2 : 4);
      if (full)
        load_row<V, NCH>(p, 0, a.gate_bf16, d, g);
      else if (!KEEP && channel)
        load_row<V, NCH>(a.gate, 0, a.gate_bf16, d, g);
      else
        MOE_EACH(c, i) g[c][i] = gc[c][i];
    }
    ring.release(s);
    if (++s == r.stages) s = 0, phase ^= 1;
    fwd_row<V, NCH, KEEP>(a, t, x, o, g, w, wn, gt, red + turn, ring.threads, KEEP && channel);
  }
  ring.report(r);
}

template <int NCH>
__global__ void __launch_bounds__(kRingThreads, NCH == 1 ? 2 : 1) k_norm_bwd_ring(const __grid_constant__ NormBwd a,
                                                                                 const __grid_constant__ Ring r) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) float red[48];
  constexpr int V = 8;
  const int d = a.d;
  RingState ring(smem, r);
  clear_sums(red);
  griddep_wait();
  griddep_launch();
  if (ring.producer()) {
    ring.produce(r, d, a.n);
    return;
  }
  constexpr bool KEEP = NCH == 1;
  BwdState<V, NCH, KEEP, true> st(a);
  int s = 0, phase = 0, turn = 0;
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x, turn ^= 1) {
    BwdRow<V, NCH> q;
    fill<V, NCH>(q.x, 0.f), fill<V, NCH>(q.dy, 0.f), fill<V, NCH>(q.dres, 0.f), fill<V, NCH>(q.g, 0.f);
    const float2 gt = token_gates(a.gate, a.gate_kind, a.gate_act, t * a.gate_ld, a.gate_bf16);
    const unsigned char *p = ring.wait(r, s, phase);
    load_row<V, NCH>(p, 0, a.x_bf16, d, q.x);
    p += d * (a.x_bf16 ? 2 : 4);
    load_row<V, NCH>(p, 0, a.dy_bf16, d, q.dy);
    p += d * (a.dy_bf16 ? 2 : 4);
    if (a.dres) {
      load_row<V, NCH>(p, 0, a.dres_bf16, d, q.dres);
      p += d * (a.dres_bf16 ? 2 : 4);
    }
    if (a.gate_kind == MOE_GATE_FULL) load_row<V, NCH>(p, 0, a.gate_bf16, d, q.g);
    ring.release(s);
    if (++s == r.stages) s = 0, phase ^= 1;
    bwd_row(a, t, q, st, gt, red + 24 * turn, ring.threads);
  }
  ring.report(r);
  st.finish(a);
}

// out[i] = sum over rows of part[row][i]: warp y of a block adds every 32nd row of 32 columns in order,
// then one warp a column adds the 32 sums in a fixed tree; blockIdx.y picks one of two sums.
struct ColSum {
  const float *part[2];
  void *out[2];
  int bf16[2];
  int rows, d;
};
__global__ void __launch_bounds__(1024) k_colsum(ColSum a) {
  __shared__ float s[32][33];
  const int which = blockIdx.y, x = threadIdx.x, y = threadIdx.y, i = blockIdx.x * 32 + x;
  griddep_wait();
  griddep_launch();
  const float *part = a.part[which] + static_cast<int64_t>(y) * a.d + i;
  float v = 0.f;
  if (i < a.d) {
#pragma unroll 16
    for (int r = y; r < a.rows; r += 32, part += 32 * static_cast<int64_t>(a.d)) v += *part;
  }
  s[y][x] = v;
  __syncthreads();
  v = s[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + y;
  if (x == 0 && col < a.d) {
    float o[1] = {v};
    store_v<1>(a.out[which], col, a.bf16[which], o);
  }
}

// Values that can be read and written at once: the width, and every pointer and row stride, a
// multiple of v values.
struct VecRule {
  int v;
  explicit VecRule(int d) : v(d % 8 == 0 ? 8 : d % 4 == 0 ? 4 : d % 2 == 0 ? 2 : 1) {}
  void row(const void *p, int64_t ld, int bf16) {
    const int size = bf16 ? 2 : 4;
    if (p)
      while (v > 1 && (reinterpret_cast<uintptr_t>(p) % (v * size > 16 ? 16 : v * size) || ld % v)) v /= 2;
  }
};

int norm_threads(int d, int v) {
  const int need = (d + v - 1) / v, t = (need + 31) / 32 * 32;
  return t < kNormMaxThreads ? t : kNormMaxThreads;
}

// Launch with programmatic stream serialization: a kernel may begin while the one before it ends, and
// waits for its results itself.
template <typename... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t st, const P &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Calls f with the instantiation that holds a row of d <= kNormMaxD values, v at a time.
template <typename F>
cudaError_t pick_norm(int d, int v, F f) {
  const int threads = norm_threads(d, v), nch = (d + v * threads - 1) / (v * threads);
#define MOE_NORM_CASE(V, N) f(std::integral_constant<int, V>{}, std::integral_constant<int, N>{}, threads)
  if (v == 8) return nch <= 1 ? MOE_NORM_CASE(8, 1) : nch <= 2 ? MOE_NORM_CASE(8, 2) : MOE_NORM_CASE(8, 4);
  if (v == 4)
    return nch <= 1 ? MOE_NORM_CASE(4, 1) : nch <= 2 ? MOE_NORM_CASE(4, 2) : nch <= 4 ? MOE_NORM_CASE(4, 4) : MOE_NORM_CASE(4, 8);
  if (v == 2)
    return nch <= 2 ? MOE_NORM_CASE(2, 2) : nch <= 4 ? MOE_NORM_CASE(2, 4) : nch <= 8 ? MOE_NORM_CASE(2, 8) : MOE_NORM_CASE(2, 16);
  return nch <= 2 ? MOE_NORM_CASE(1, 2) : nch <= 4 ? MOE_NORM_CASE(1, 4) : nch <= 8 ? MOE_NORM_CASE(1, 8)
                                        : nch <= 16 ? MOE_NORM_CASE(1, 16) : MOE_NORM_CASE(1, 32);
#undef MOE_NORM_CASE
}

bool bad_dtype(int dt) { return dt != MOE_F32 && dt != MOE_BF16; }
bool bad_rows(const void *p, int64_t ld, int d, int n, int dt) {
  // a stride of fewer values than a row would make rows overlap; pointers keep their type's alignment
  return !p || bad_dtype(dt) || (n > 1 && ld < d) || reinterpret_cast<uintptr_t>(p) % (dt == MOE_BF16 ? 2 : 4);
}
bool bad_vec(const void *p, int dt) {
  return bad_dtype(dt) || reinterpret_cast<uintptr_t>(p) % (dt == MOE_BF16 ? 2 : 4);
}

moe_status check_gate(const void *gate, int kind, int act, int dt, int64_t ld, int d, int n) {
  if (kind < MOE_GATE_NONE || kind > MOE_GATE_FULL || (kind == MOE_GATE_NONE) != (gate == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (kind == MOE_GATE_NONE) return MOE_OK;
  if ((act != MOE_GATE_LINEAR && act != MOE_GATE_SIGMOID) || bad_vec(gate, dt)) return MOE_ERR_INVALID_ARGUMENT;
  if (n > 1 && ((kind == MOE_GATE_FULL && ld < d) || (kind == MOE_GATE_TOKEN && ld < 1))) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// The ring of a kernel over n rows (word: where its errors go, the device's if NULL), or stages = 0 where
// it does not pay: rows that are not whole 16-byte vectors, too long for two stages, or (backward) for the
// registers, or fewer than kRingRows for each of the blocks that fill the device (1,180 x 2,048, fp32:
// 12.5 us against 10.5; 8,192 x 4,096, bf16 with a gate of its own: 57 against 97).
constexpr int kRingBytes = 208 * 1024, kRingRows = 4, kMostBlocksPerSm = 16;
struct RingPlan {
  Ring r{};
  int blocks = 0, threads = 0, smem = 0;
  cudaError_t err = cudaSuccess;
  RingPlan(std::initializer_list<RowSource> src, int n, int d, int v, bool backward, uint32_t *word) {
    if (v != 8) return;
    for (const RowSource &s : src)
      if (s.p) r.src[r.n_src++] = s, r.stage_bytes += d * (s.bf16 ? 2 : 4);
    int nsm = 0;
    if ((err = current_sm_count(&nsm)) != cudaSuccess) return;
    threads = norm_threads(d, v);
    // as many blocks as the registers hold (72 a thread forward, 96 backward, all of them beyond), of at
    // least three stages each
    int per_sm = kRingBytes / (3 * r.stage_bytes);
    const int wide = d > 8 * kNormMaxThreads;
    const int most = wide ? (backward || d > 16 * kNormMaxThreads ? 1 : 2) : 65536 / ((backward ? 96 : 72) * (threads + 32));
    per_sm = per_sm > most ? most : per_sm;
    per_sm = per_sm > kMostBlocksPerSm ? kMostBlocksPerSm : per_sm < 1 ? 1 : per_sm;
    if (n < kRingRows * nsm * (per_sm < 3 ? per_sm : 3) || (backward && d > 16 * kNormMaxThreads)) return;
    if (per_sm > n / (kRingRows * nsm)) per_sm = n / (kRingRows * nsm);
    int stages = (kRingBytes / per_sm - 1024) / r.stage_bytes;
    if (stages > kRingMaxStages) stages = kRingMaxStages;
    r.spin = ring_spin();
    r.err = word;
    if (!word) {
      BlockWord own;
      if ((err = block_word(&own)) != cudaSuccess) return;
      r.err = own.dev;
    }
    blocks = per_sm * nsm;
    smem = 128 + stages * r.stage_bytes;
    if (stages >= 2) r.stages = stages;
  }
};

template <int MOST, typename F>
cudaError_t pick_ring(int d, F f) {
  const int nch = (d + 8 * kNormMaxThreads - 1) / (8 * kNormMaxThreads);
  if (nch <= 1) return f(std::integral_constant<int, 1>{});
  if constexpr (MOST == 4)
    if (nch > 2) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 2>{});
}

// Once per device, with it current.
cudaError_t configure_rings() {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kMaxDevices && done[dev].load(std::memory_order_acquire))) return e;
  const void *ks[] = {(const void *)k_norm_fwd_ring<1>, (const void *)k_norm_fwd_ring<2>, (const void *)k_norm_fwd_ring<4>,
                      (const void *)k_norm_bwd_ring<1>, (const void *)k_norm_bwd_ring<2>};
  for (const void *k : ks)
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes)) != cudaSuccess) return e;
  if (dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

moe_status launch_fwd(const NormFwd &a, int n, int v, cudaStream_t st, uint32_t *err) {
  const bool full = a.gate_kind == MOE_GATE_FULL;
  const RingPlan p({{a.res, a.res_ld, a.res_bf16}, {a.o, a.o_ld, a.o_bf16}, {full ? a.gate : nullptr, a.gate_ld, a.gate_bf16}}, n,
                   a.d, v, false, err);
  cudaError_t e = p.err;
  if (e == cudaSuccess && p.r.stages) {
    e = configure_rings();
    if (e == cudaSuccess)
      e = pick_ring<4>(a.d, [&](auto nch) { return launch(k_norm_fwd_ring<decltype(nch)::value>, p.blocks, p.threads + 32, p.smem, st, a, p.r, n); });
  } else if (e == cudaSuccess) {
    e = pick_norm(a.d, v, [&](auto vv, auto nch, int threads) {
      return launch(k_norm_fwd<decltype(vv)::value, decltype(nch)::value>, n, threads, 0, st, a);
    });
  }
  return cuda_status(e);
}

// Blocks of the backward grid: enough to fill the device, no more than rows; the partial sums need
// one row of d values for each.
constexpr int kBwdBlocksPerSm = 3;
cudaError_t bwd_blocks(int n, int *blocks) {
  int nsm = 0;
  const cudaError_t e = current_sm_count(&nsm);
  *blocks = n < nsm * kBwdBlocksPerSm ? n : nsm * kBwdBlocksPerSm;
  return e;
}

moe_status run_bwd(NormBwd &a, int v, void *dw, int dw_bf16, void *dg, int dg_bf16, void *ws, uint64_t ws_bytes,
                   cudaStream_t st) {
  const bool full = a.gate_kind == MOE_GATE_FULL;
  const RingPlan p({{a.x, a.x_ld, a.x_bf16}, {a.dy, a.dy_ld, a.dy_bf16}, {a.dres, a.dres_ld, a.dres_bf16},
                    {full ? a.gate : nullptr, a.gate_ld, a.gate_bf16}}, a.n, a.d, v, true, nullptr);
  int blocks = p.blocks;
  cudaError_t e = p.err;
  if (e == cudaSuccess && !p.r.stages) e = bwd_blocks(a.n, &blocks);
  if (e != cudaSuccess) return cuda_status(e);
  const int sums = (dw ? 1 : 0) + (dg ? 1 : 0);
  if (sums && (!ws || ws_bytes < moe_norm_workspace(a.n, a.d) || !aligned16(ws))) return MOE_ERR_INVALID_ARGUMENT;
  float *part = static_cast<float *>(ws);
  ColSum c{};
  c.rows = blocks;
  c.d = a.d;
  int k = 0;
  if (dw) {
    a.dw_part = part;
    c.part[k] = part, c.out[k] = dw, c.bf16[k] = dw_bf16, ++k;
    part += static_cast<int64_t>(blocks) * a.d;
  }
  if (dg) {
    a.dg_part = part;
    c.part[k] = part, c.out[k] = dg, c.bf16[k] = dg_bf16, ++k;
  }
  if (p.r.stages) {
    e = configure_rings();
    if (e == cudaSuccess)
      e = pick_ring<2>(a.d, [&](auto nch) { return launch(k_norm_bwd_ring<decltype(nch)::value>, p.blocks, p.threads + 32, p.smem, st, static_cast<const NormBwd &>(a), p.r); });
  } else {
    e = pick_norm(a.d, v, [&](auto vv, auto nch, int threads) {
      return launch(k_norm_bwd<decltype(vv)::value, decltype(nch)::value>, blocks, threads, 0, st, static_cast<const NormBwd &>(a));
    });
  }
  if (e == cudaSuccess && sums) e = launch(k_colsum, dim3((a.d + 31) / 32, sums), dim3(32, 32), 0, st, c);
  return cuda_status(e);
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace moe {
RingSpin ring_spin() {
  const uint64_t v = g_ring_limit.load(std::memory_order_relaxed);
  return v ? RingSpin{v, 4 * v} : RingSpin{kRingSpin, 0};
}

namespace {
constexpr int kMaxDevices = 64, kWordBytes = 64;
std::atomic<char *> g_words{nullptr};            // the words of all devices
std::atomic<char *> g_words_seen[kMaxDevices];   // the same as each device sees them
}  // namespace

moe_status block_pending() {
  char *page = g_words.load(std::memory_order_acquire);
  int dev = 0;
  if (!page || cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return MOE_OK;
  uint32_t *w = reinterpret_cast<uint32_t *>(page + dev * kWordBytes);
  if (!__atomic_load_n(w, __ATOMIC_RELAXED)) return MOE_OK;
  return __atomic_exchange_n(w, 0u, __ATOMIC_ACQ_REL) ? MOE_ERR_TIMEOUT : MOE_OK;
}

cudaError_t block_word(BlockWord *w) {
  static std::mutex mutex;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorNotSupported;
  char *seen = g_words_seen[dev].load(std::memory_order_acquire), *page = g_words.load(std::memory_order_acquire);
  if (!seen) {
    std::lock_guard<std::mutex> lock(mutex);
    page = g_words.load(std::memory_order_acquire);
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // this allocation is no part of any capture
    if ((e = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return e;
    if (!page) {
      void *p = nullptr;
      e = cudaHostAlloc(&p, kMaxDevices * kWordBytes, cudaHostAllocMapped | cudaHostAllocPortable);
      if (e == cudaSuccess) g_words.store(page = static_cast<char *>(memset(p, 0, kMaxDevices * kWordBytes)), std::memory_order_release);
    }
    void *p = nullptr;
    if (e == cudaSuccess) e = cudaHostGetDevicePointer(&p, page, 0);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    g_words_seen[dev].store(seen = static_cast<char *>(p), std::memory_order_release);
  }
  w->host = reinterpret_cast<uint32_t *>(page + dev * kWordBytes);
  w->dev = reinterpret_cast<uint32_t *>(seen + dev * kWordBytes);
  return cudaSuccess;
}
}  // namespace moe

extern "C" moe_status moe_debug_set_ring_spin_limit(uint64_t cycles) {
  if (cycles > kRingSpin / 10) return MOE_ERR_INVALID_ARGUMENT;
  g_ring_limit.store(cycles, std::memory_order_relaxed);
  return MOE_OK;
}

namespace moe {
moe_status norm_in_run(const void *x, int32_t x_dtype, int64_t x_stride, const void *weight, int32_t w_dtype, float eps,
                       int32_t unit_offset, void *h, int32_t h_dtype, int64_t h_stride, int32_t n_tokens, int32_t d_model,
                       void *stream, uint32_t *err) {
  if (n_tokens < 1 || d_model < 1 || !weight || !(eps >= 0.f) || unit_offset < 0 || unit_offset > 1 ||
      bad_rows(x, x_stride, d_model, n_tokens, x_dtype) || bad_rows(h, h_stride, d_model, n_tokens, h_dtype) ||
      bad_vec(weight, w_dtype) || misplaced(h, h_stride, h_dtype, x, x_stride, x_dtype, n_tokens))
    return MOE_ERR_INVALID_ARGUMENT;
  if (d_model > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if (const moe_status s = err ? MOE_OK : block_pending()) return s;
  NormFwd a{};
  a.res = x, a.res_ld = x_stride, a.res_bf16 = x_dtype == MOE_BF16;
  a.next_w = weight, a.w_bf16 = w_dtype == MOE_BF16, a.next_eps = eps, a.w_off = static_cast<float>(unit_offset);
  a.h = h, a.h_ld = h_stride, a.h_bf16 = h_dtype == MOE_BF16;
  a.d = d_model, a.inv_d = 1.f / d_model;
  VecRule v(d_model);
  v.row(x, x_stride, a.res_bf16), v.row(h, h_stride, a.h_bf16), v.row(weight, 0, a.w_bf16);
  return launch_fwd(a, n_tokens, v.v, static_cast<cudaStream_t>(stream), err);
}

moe_status norm_out_run(const moe_norm_out_args *p, void *stream, uint32_t *err) {
  if (!p || p->struct_size != sizeof(moe_norm_out_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model;
  if (n < 1 || d < 1 || bad_rows(p->o, p->o_stride, d, n, p->o_dtype) ||
      bad_rows(p->residual, p->res_stride, d, n, p->res_dtype) ||
      bad_rows(p->res_out, p->res_out_stride, d, n, p->res_out_dtype) || p->unit_offset < 0 || p->unit_offset > 1 ||
      (p->weight && (bad_vec(p->weight, p->w_dtype) || !(p->eps >= 0.f))) || (p->next_weight != nullptr) != (p->h != nullptr) ||
      (p->h && (bad_rows(p->h, p->h_stride, d, n, p->h_dtype) || bad_vec(p->next_weight, p->w_dtype) || !(p->next_eps >= 0.f))) ||
      p->h == p->res_out ||
      misplaced(p->res_out, p->res_out_stride, p->res_out_dtype, p->residual, p->res_stride, p->res_dtype, n) ||
      misplaced(p->res_out, p->res_out_stride, p->res_out_dtype, p->o, p->o_stride, p->o_dtype, n) ||
      misplaced(p->h, p->h_stride, p->h_dtype, p->o, p->o_stride, p->o_dtype, n))
    return MOE_ERR_INVALID_ARGUMENT;
  const moe_status gs = check_gate(p->gate, p->gate_kind, p->gate_act, p->gate_dtype, p->gate_stride, d, n);
  if (gs != MOE_OK) return gs;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if (const moe_status s = err ? MOE_OK : block_pending()) return s;
  NormFwd a{};
  a.o = p->o, a.o_ld = p->o_stride, a.o_bf16 = p->o_dtype == MOE_BF16;
  a.res = p->residual, a.res_ld = p->res_stride, a.res_bf16 = p->res_dtype == MOE_BF16;
  a.w = p->weight, a.w_bf16 = p->w_dtype == MOE_BF16, a.eps = p->eps, a.w_off = static_cast<float>(p->unit_offset);
  a.gate = p->gate, a.gate_kind = p->gate_kind, a.gate_act = p->gate_act, a.gate_ld = p->gate_stride;
  a.gate_bf16 = p->gate_dtype == MOE_BF16;
  a.scale = p->scale;
  a.res_out = p->res_out, a.out_ld = p->res_out_stride, a.out_bf16 = p->res_out_dtype == MOE_BF16;
  a.next_w = p->next_weight, a.next_eps = p->next_eps;
  a.h = p->h, a.h_ld = p->h_stride, a.h_bf16 = p->h_dtype == MOE_BF16;
  a.d = d, a.inv_d = 1.f / d;
  VecRule v(d);
  v.row(a.o, a.o_ld, a.o_bf16), v.row(a.res, a.res_ld, a.res_bf16), v.row(a.res_out, a.out_ld, a.out_bf16);
  v.row(a.h, a.h_ld, a.h_bf16), v.row(a.w, 0, a.w_bf16), v.row(a.next_w, 0, a.w_bf16);
  if (a.gate_kind == MOE_GATE_FULL) v.row(a.gate, a.gate_ld, a.gate_bf16);
  if (a.gate_kind == MOE_GATE_CHANNEL) v.row(a.gate, 0, a.gate_bf16);
  return launch_fwd(a, n, v.v, static_cast<cudaStream_t>(stream), err);
}
}  // namespace moe

extern "C" moe_status moe_norm_in(const void *x, int32_t x_dtype, int64_t x_stride, const void *weight, int32_t w_dtype,
                                  float eps, int32_t unit_offset, void *h, int32_t h_dtype, int64_t h_stride,
                                  int32_t n_tokens, int32_t d_model, void *stream) {
  return norm_in_run(x, x_dtype, x_stride, weight, w_dtype, eps, unit_offset, h, h_dtype, h_stride, n_tokens, d_model, stream, nullptr);
}

extern "C" moe_status moe_norm_out(const moe_norm_out_args *p, void *stream) { return norm_out_run(p, stream, nullptr); }

// Two sums of a row of d values for every block that a backward grid can have.
extern "C" uint64_t moe_norm_workspace(int32_t n_tokens, int32_t d_model) {
  int nsm = 0;
  if (n_tokens < 1 || d_model < 1 || d_model > kNormMaxD || current_sm_count(&nsm) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  const int64_t most = static_cast<int64_t>(nsm) * (d_model >= 2048 ? 3 : kMostBlocksPerSm);
  return static_cast<uint64_t>(n_tokens < most ? n_tokens : most) * d_model * 8;
}

extern "C" moe_status moe_norm_in_backward(const moe_norm_in_bwd_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_norm_in_bwd_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model;
  if (n < 1 || d < 1 || bad_rows(p->x, p->x_stride, d, n, p->x_dtype) || bad_rows(p->dh, p->dh_stride, d, n, p->dh_dtype) ||
      bad_rows(p->dx, p->dx_stride, d, n, p->dx_dtype) || !p->weight || bad_vec(p->weight, p->w_dtype) ||
      (p->dres && bad_rows(p->dres, p->dres_stride, d, n, p->dres_dtype)) || (p->dweight && bad_vec(p->dweight, p->w_dtype)) ||
      p->unit_offset < 0 || p->unit_offset > 1 || !(p->eps >= 0.f) ||
      misplaced(p->dx, p->dx_stride, p->dx_dtype, p->dres, p->dres_stride, p->dres_dtype, n))
    return MOE_ERR_INVALID_ARGUMENT;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if (const moe_status s = block_pending()) return s;
  NormBwd a{};
  a.x = p->x, a.x_ld = p->x_stride, a.x_bf16 = p->x_dtype == MOE_BF16;
  a.dy = p->dh, a.dy_ld = p->dh_stride, a.dy_bf16 = p->dh_dtype == MOE_BF16;
  a.w = p->weight, a.w_bf16 = p->w_dtype == MOE_BF16, a.w_off = static_cast<float>(p->unit_offset), a.eps = p->eps;
  a.dres = p->dres, a.dres_ld = p->dres_stride, a.dres_bf16 = p->dres_dtype == MOE_BF16;
  a.dx = p->dx, a.dx_ld = p->dx_stride, a.dx_bf16 = p->dx_dtype == MOE_BF16;
  a.gate_kind = MOE_GATE_NONE, a.scale = 1.f, a.d = d, a.n = n, a.inv_d = 1.f / d;
  VecRule v(d);
  v.row(a.x, a.x_ld, a.x_bf16), v.row(a.dy, a.dy_ld, a.dy_bf16), v.row(a.dres, a.dres_ld, a.dres_bf16);
  v.row(a.dx, a.dx_ld, a.dx_bf16), v.row(a.w, 0, a.w_bf16);
  return run_bwd(a, v.v, p->dweight, a.w_bf16, nullptr, 0, p->workspace, p->workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_norm_out_backward(const moe_norm_out_bwd_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_norm_out_bwd_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model;
  if (n < 1 || d < 1 || bad_rows(p->o, p->o_stride, d, n, p->o_dtype) || bad_rows(p->dres, p->dres_stride, d, n, p->dres_dtype) ||
      bad_rows(p->d_o, p->do_stride, d, n, p->o_dtype) || (p->weight && bad_vec(p->weight, p->w_dtype)) ||
      (p->dweight && (!p->weight || bad_vec(p->dweight, p->w_dtype))) || p->unit_offset < 0 || p->unit_offset > 1 ||
      (p->weight && !(p->eps >= 0.f)) || (p->dgate && !p->gate))
    return MOE_ERR_INVALID_ARGUMENT;
  moe_status gs = check_gate(p->gate, p->gate_kind, p->gate_act, p->gate_dtype, p->gate_stride, d, n);
  if (gs == MOE_OK && p->dgate)
    gs = check_gate(p->dgate, p->gate_kind, p->gate_act, p->gate_dtype, p->dgate_stride, d, n);
  if (gs != MOE_OK) return gs;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if ((gs = block_pending()) != MOE_OK) return gs;
  NormBwd a{};
  a.x = p->o, a.x_ld = p->o_stride, a.x_bf16 = p->o_dtype == MOE_BF16;
  a.dy = p->dres, a.dy_ld = p->dres_stride, a.dy_bf16 = p->dres_dtype == MOE_BF16;
  a.w = p->weight, a.w_bf16 = p->w_dtype == MOE_BF16, a.w_off = static_cast<float>(p->unit_offset), a.eps = p->eps;
  a.gate = p->gate, a.gate_kind = p->gate_kind, a.gate_act = p->gate_act, a.gate_ld = p->gate_stride;
  a.gate_bf16 = p->gate_dtype == MOE_BF16;
  a.dx = p->d_o, a.dx_ld = p->do_stride, a.dx_bf16 = a.x_bf16;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (!channel) a.dgate = p->dgate, a.dgate_ld = p->dgate_stride;
  a.scale = p->scale, a.d = d, a.n = n, a.inv_d = 1.f / d;
  VecRule v(d);
  v.row(a.x, a.x_ld, a.x_bf16), v.row(a.dy, a.dy_ld, a.dy_bf16), v.row(a.dx, a.dx_ld, a.dx_bf16), v.row(a.w, 0, a.w_bf16);
  if (a.gate_kind == MOE_GATE_FULL) v.row(a.gate, a.gate_ld, a.gate_bf16), v.row(a.dgate, a.dgate_ld, a.gate_bf16);
  if (channel) v.row(a.gate, 0, a.gate_bf16);
  return run_bwd(a, v.v, p->dweight, a.w_bf16, channel ? p->dgate : nullptr, a.gate_bf16, p->workspace,
                 p->workspace_bytes, static_cast<cudaStream_t>(stream));
}
