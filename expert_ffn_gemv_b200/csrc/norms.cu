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
// Sums over columns are taken over the row's threads (shuffles, then the warps in order), sums over
// tokens (dw, the gradient of a channel gate) in two steps: every block of a grid that depends on the
// device alone adds its rows in order, k_colsum adds the blocks' partial rows in order.  No atomics:
// the same call gives the same bits.
#include <math.h>

#include "block.cuh"

namespace moe {
namespace {

constexpr int kNormMaxD = 8192;      // V * NCH * threads
constexpr int kNormMaxThreads = 256;

template <int V>
__device__ __forceinline__ void load_v(const void *p, int64_t i, int bf16, float (&v)[V]) {
  if (bf16) {
    const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p) + i;
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4 *>(b);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
      v[0] = __bfloat162float(*b);
    }
  } else {
    const float *f = static_cast<const float *>(p) + i;
    if constexpr (V == 8) {
      const float4 a = *reinterpret_cast<const float4 *>(f), c = *reinterpret_cast<const float4 *>(f + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = c.x; v[5] = c.y; v[6] = c.z; v[7] = c.w;
    } else {
      v[0] = *f;
    }
  }
}

// Stores v rounded to the destination's type and leaves in v the values as they are stored.
template <int V>
__device__ __forceinline__ void store_v(void *p, int64_t i, int bf16, float (&v)[V]) {
  if (bf16) {
    __nv_bfloat16 *b = static_cast<__nv_bfloat16 *>(p) + i;
    if constexpr (V == 8) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        const float2 f = __bfloat1622float2(h[k]);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
      *reinterpret_cast<uint4 *>(b) = *reinterpret_cast<const uint4 *>(h);
    } else {
      const __nv_bfloat16 h = __float2bfloat16_rn(v[0]);
      *b = h;
      v[0] = __bfloat162float(h);
    }
  } else {
    float *f = static_cast<float *>(p) + i;
    if constexpr (V == 8) {
      *reinterpret_cast<float4 *>(f) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *f = v[0];
    }
  }
}

// Sums of NV values over the block, in every thread; `red` holds 8 warps x NV and is used in turn
// with a second buffer (`red` flips), so one barrier a call is enough.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float *red) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < NV; ++k) red[warp * NV + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float s = red[k];
    for (int w = 1; w < warps; ++w) s += red[w * NV + k];
    v[k] = s;
  }
}

__device__ __forceinline__ float gate_value(float g, int act) {
  return act == MOE_GATE_SIGMOID ? 1.0f / (1.0f + __expf(-g)) : g;
}

struct NormFwd {
  const void *o, *res, *w, *gate, *next_w;
  void *res_out, *h;
  int64_t o_ld, res_ld, gate_ld, out_ld, h_ld;
  int o_bf16, res_bf16, out_bf16, w_bf16, gate_bf16, h_bf16;
  int gate_kind, gate_act, d;
  float eps, next_eps, scale, w_off;
};

// One block per token; thread t holds columns (c blockDim + t) V .. + V - 1, c < NCH.
template <int V, int NCH>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_fwd(const __grid_constant__ NormFwd a) {
  __shared__ float red[16];
  const int64_t t = blockIdx.x;
  const int d = a.d;
  float r[NCH][V];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i = (c * blockDim.x + threadIdx.x) * V;
    if (i < d)
      load_v<V>(a.res, t * a.res_ld + i, a.res_bf16, r[c]);
    else
#pragma unroll
      for (int k = 0; k < V; ++k) r[c][k] = 0.f;
  }
  if (a.o) {
    float o[NCH][V];
    float ss[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i = (c * blockDim.x + threadIdx.x) * V;
      if (i < d) load_v<V>(a.o, t * a.o_ld + i, a.o_bf16, o[c]);
    }
    float q = 1.f;
    if (a.w) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int i = (c * blockDim.x + threadIdx.x) * V;
        if (i < d)
#pragma unroll
          for (int k = 0; k < V; ++k) ss[0] = fmaf(o[c][k], o[c][k], ss[0]);
      }
      block_sum<1>(ss, red);
      q = rsqrtf(ss[0] / d + a.eps);
    }
    float gt = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      float g1[1];
      load_v<1>(a.gate, t * a.gate_ld, a.gate_bf16, g1);
      gt = gate_value(g1[0], a.gate_act);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i = (c * blockDim.x + threadIdx.x) * V;
      if (i >= d) continue;
      float w[V], g[V];
      if (a.w) load_v<V>(a.w, i, a.w_bf16, w);
      if (a.gate_kind >= MOE_GATE_CHANNEL && a.gate_kind != MOE_GATE_TOKEN)
        load_v<V>(a.gate, (a.gate_kind == MOE_GATE_FULL ? t * a.gate_ld : 0) + i, a.gate_bf16, g);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float u = a.w ? o[c][k] * q * (w[k] + a.w_off) : o[c][k];
        const float av = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL ? gate_value(g[k], a.gate_act) : gt;
        r[c][k] = fmaf(a.scale * av, u, r[c][k]);
      }
      store_v<V>(a.res_out, t * a.out_ld + i, a.out_bf16, r[c]);
    }
  }
  if (!a.h) return;
  float ss[1] = {0.f};
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < V; ++k) ss[0] = fmaf(r[c][k], r[c][k], ss[0]);
  block_sum<1>(ss, red + 8);
  const float p = rsqrtf(ss[0] / d + a.next_eps);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i = (c * blockDim.x + threadIdx.x) * V;
    if (i >= d) continue;
    float w[V];
    load_v<V>(a.next_w, i, a.w_bf16, w);
#pragma unroll
    for (int k = 0; k < V; ++k) r[c][k] = r[c][k] * p * (w[k] + a.w_off);
    store_v<V>(a.h, t * a.h_ld + i, a.h_bf16, r[c]);
  }
}

struct NormBwd {
  const void *x, *dy, *w, *gate, *dres;  // post norm: x = o, dy = dr'; input norm: x, dy = dh, dres
  void *dx, *dgate;
  float *dw_part, *dg_part;              // [blocks][d] sums over the block's rows, or NULL
  int64_t x_ld, dy_ld, gate_ld, dres_ld, dx_ld, dgate_ld;
  int x_bf16, dy_bf16, w_bf16, gate_bf16, dres_bf16, dx_bf16;
  int gate_kind, gate_act, d, n;
  float eps, scale, w_off;
};

// Persistent: block b takes rows b, b + grid, ...; the column sums stay in registers.
template <int V, int NCH>
__global__ void __launch_bounds__(kNormMaxThreads) k_norm_bwd(const __grid_constant__ NormBwd a) {
  __shared__ float red[2][24];
  const int d = a.d;
  float dw[NCH][V], dg[NCH][V];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[c][k] = dg[c][k] = 0.f;
  const bool by_element = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x) {
    float x[NCH][V], dy[NCH][V];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i = (c * blockDim.x + threadIdx.x) * V;
      if (i < d) {
        load_v<V>(a.x, t * a.x_ld + i, a.x_bf16, x[c]);
        load_v<V>(a.dy, t * a.dy_ld + i, a.dy_bf16, dy[c]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[c][k] = dy[c][k] = 0.f;
      }
    }
    float gt = 1.f, gs = 0.f;  // token gate: its value, its slope
    if (a.gate_kind == MOE_GATE_TOKEN) {
      float g1[1];
      load_v<1>(a.gate, t * a.gate_ld, a.gate_bf16, g1);
      gt = gate_value(g1[0], a.gate_act);
      gs = a.gate_act == MOE_GATE_SIGMOID ? gt * (1.f - gt) : 1.f;
    }
    // sums of x^2, of (dy a w) x and of dy x w (the token gate's gradient), without their common
    // factors s and q
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i = (c * blockDim.x + threadIdx.x) * V;
      if (i >= d) continue;
      float w[V], g[V];
      if (a.w) load_v<V>(a.w, i, a.w_bf16, w);
      if (by_element) load_v<V>(a.gate, (a.gate_kind == MOE_GATE_FULL ? t * a.gate_ld : 0) + i, a.gate_bf16, g);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float wk = a.w ? w[k] + a.w_off : 1.f;
        const float av = by_element ? gate_value(g[k], a.gate_act) : gt;
        const float e = dy[c][k] * x[c][k] * wk;
        s[0] = fmaf(x[c][k], x[c][k], s[0]);
        s[1] = fmaf(e, av, s[1]);
        s[2] += e;
      }
    }
    block_sum<3>(s, red[(t / gridDim.x) & 1]);
    const float q = a.w ? rsqrtf(s[0] / d + a.eps) : 1.f;
    const float m = a.w ? q * q * (s[1] / d) : 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && threadIdx.x == 0) {
      float v1[1] = {a.scale * gs * q * s[2]};
      store_v<1>(a.dgate, t * a.dgate_ld, a.gate_bf16, v1);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i = (c * blockDim.x + threadIdx.x) * V;
      if (i >= d) continue;
      float w[V], g[V], out[V];
      if (a.w) load_v<V>(a.w, i, a.w_bf16, w);
      if (by_element) load_v<V>(a.gate, (a.gate_kind == MOE_GATE_FULL ? t * a.gate_ld : 0) + i, a.gate_bf16, g);
      if (a.dres)
        load_v<V>(a.dres, t * a.dres_ld + i, a.dres_bf16, out);
      else
#pragma unroll
        for (int k = 0; k < V; ++k) out[k] = 0.f;
      float gg[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float wk = a.w ? w[k] + a.w_off : 1.f;
        const float av = by_element ? gate_value(g[k], a.gate_act) : gt;
        const float dz = a.scale * dy[c][k];
        out[k] = fmaf(q, dz * av * wk - a.scale * x[c][k] * m, out[k]);
        dw[c][k] = fmaf(dz * av, x[c][k] * q, dw[c][k]);
        const float slope = a.gate_act == MOE_GATE_SIGMOID ? av * (1.f - av) : 1.f;
        gg[k] = dz * x[c][k] * q * wk * slope;
        dg[c][k] += gg[k];
      }
      store_v<V>(a.dx, t * a.dx_ld + i, a.dx_bf16, out);
      if (a.gate_kind == MOE_GATE_FULL && a.dgate) store_v<V>(a.dgate, t * a.dgate_ld + i, a.gate_bf16, gg);
    }
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i = (c * blockDim.x + threadIdx.x) * V;
    if (i >= d) continue;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * d + i;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (a.dw_part) a.dw_part[at + k] = dw[c][k];
      if (a.dg_part) a.dg_part[at + k] = dg[c][k];
    }
  }
}

// out[i] = sum over rows of part[row][i], in row order within eight interleaved runs that are then
// added in order; blockIdx.y picks one of two sums.
struct ColSum {
  const float *part[2];
  void *out[2];
  int bf16[2];
  int rows, d;
};
__global__ void __launch_bounds__(256) k_colsum(ColSum a) {
  __shared__ float s[8][33];
  const int which = blockIdx.y, i = blockIdx.x * 32 + threadIdx.x;
  const float *part = a.part[which];
  float v = 0.f;
  if (i < a.d)
    for (int r = threadIdx.y; r < a.rows; r += 8) v += part[static_cast<int64_t>(r) * a.d + i];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && i < a.d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
    float o[1] = {v};
    store_v<1>(a.out[which], i, a.bf16[which], o);
  }
}

// Rows can be read 8 values at a time: every pointer and row stride a multiple of 16 bytes.
struct VecRule {
  bool ok;
  explicit VecRule(int d) : ok(d % 8 == 0) {}
  void row(const void *p, int64_t ld, int bf16) {
    if (p) ok = ok && aligned16(p) && (ld * (bf16 ? 2 : 4)) % 16 == 0;
  }
};

int norm_threads(int d, int v) {
  const int need = (d + v - 1) / v, t = (need + 31) / 32 * 32;
  return t < kNormMaxThreads ? t : kNormMaxThreads;
}

// Calls f with the instantiation that holds a row of d values.
template <typename F>
cudaError_t pick_norm(int d, bool vec, F f) {
  const int v = vec ? 8 : 1, threads = norm_threads(d, v), nch = (d + v * threads - 1) / (v * threads);
#define MOE_NORM_CASE(V, N) f(std::integral_constant<int, V>{}, std::integral_constant<int, N>{}, threads)
  if (vec)
    nch <= 1 ? MOE_NORM_CASE(8, 1) : nch <= 2 ? MOE_NORM_CASE(8, 2) : MOE_NORM_CASE(8, 4);
  else
    nch <= 1 ? MOE_NORM_CASE(1, 1) : nch <= 4 ? MOE_NORM_CASE(1, 4) : nch <= 8 ? MOE_NORM_CASE(1, 8)
                                   : nch <= 16 ? MOE_NORM_CASE(1, 16) : MOE_NORM_CASE(1, 32);
#undef MOE_NORM_CASE
  return cudaGetLastError();
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

moe_status launch_fwd(const NormFwd &a, int n, bool vec, cudaStream_t st) {
  const cudaError_t e = pick_norm(a.d, vec, [&](auto v, auto nch, int threads) {
    k_norm_fwd<decltype(v)::value, decltype(nch)::value><<<n, threads, 0, st>>>(a);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Blocks of the backward grid: enough to fill the device, no more than rows; the partial sums need
// one row of d values for each.
constexpr int kBwdBlocksPerSm = 2;
cudaError_t bwd_blocks(int n, int *blocks) {
  int nsm = 0;
  const cudaError_t e = current_sm_count(&nsm);
  *blocks = n < nsm * kBwdBlocksPerSm ? n : nsm * kBwdBlocksPerSm;
  return e;
}

moe_status run_bwd(NormBwd &a, bool vec, void *dw, int dw_bf16, void *dg, int dg_bf16, void *ws, uint64_t ws_bytes,
                   cudaStream_t st) {
  int blocks = 0;
  if (bwd_blocks(a.n, &blocks) != cudaSuccess) return MOE_ERR_CUDA;
  const int sums = (dw ? 1 : 0) + (dg ? 1 : 0);
  const uint64_t need = static_cast<uint64_t>(blocks) * a.d * 4;
  if (sums && (!ws || ws_bytes < need * sums || !aligned16(ws))) return MOE_ERR_INVALID_ARGUMENT;
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
  cudaError_t e = pick_norm(a.d, vec, [&](auto v, auto nch, int threads) {
    k_norm_bwd<decltype(v)::value, decltype(nch)::value><<<blocks, threads, 0, st>>>(a);
  });
  if (e == cudaSuccess && sums) {
    k_colsum<<<dim3((a.d + 31) / 32, sums), dim3(32, 8), 0, st>>>(c);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_norm_in(const void *x, int32_t x_dtype, int64_t x_stride, const void *weight, int32_t w_dtype,
                                  float eps, int32_t unit_offset, void *h, int32_t h_dtype, int64_t h_stride,
                                  int32_t n_tokens, int32_t d_model, void *stream) {
  if (n_tokens < 1 || d_model < 1 || !weight || !(eps >= 0.f) || unit_offset < 0 || unit_offset > 1 ||
      bad_rows(x, x_stride, d_model, n_tokens, x_dtype) || bad_rows(h, h_stride, d_model, n_tokens, h_dtype) ||
      bad_vec(weight, w_dtype))
    return MOE_ERR_INVALID_ARGUMENT;
  if (d_model > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  NormFwd a{};
  a.res = x, a.res_ld = x_stride, a.res_bf16 = x_dtype == MOE_BF16;
  a.next_w = weight, a.w_bf16 = w_dtype == MOE_BF16, a.next_eps = eps, a.w_off = static_cast<float>(unit_offset);
  a.h = h, a.h_ld = h_stride, a.h_bf16 = h_dtype == MOE_BF16;
  a.d = d_model;
  VecRule v(d_model);
  v.row(x, x_stride, a.res_bf16), v.row(h, h_stride, a.h_bf16), v.row(weight, 0, 0);
  return launch_fwd(a, n_tokens, v.ok, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_norm_out(const moe_norm_out_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_norm_out_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model;
  if (n < 1 || d < 1 || bad_rows(p->o, p->o_stride, d, n, p->o_dtype) ||
      bad_rows(p->residual, p->res_stride, d, n, p->res_dtype) ||
      bad_rows(p->res_out, p->res_out_stride, d, n, p->res_out_dtype) || p->unit_offset < 0 || p->unit_offset > 1 ||
      (p->weight && (bad_vec(p->weight, p->w_dtype) || !(p->eps >= 0.f))) || (p->next_weight != nullptr) != (p->h != nullptr) ||
      (p->h && (bad_rows(p->h, p->h_stride, d, n, p->h_dtype) || bad_vec(p->next_weight, p->w_dtype) || !(p->next_eps >= 0.f))))
    return MOE_ERR_INVALID_ARGUMENT;
  const moe_status gs = check_gate(p->gate, p->gate_kind, p->gate_act, p->gate_dtype, p->gate_stride, d, n);
  if (gs != MOE_OK) return gs;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
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
  a.d = d;
  VecRule v(d);
  v.row(a.o, a.o_ld, a.o_bf16), v.row(a.res, a.res_ld, a.res_bf16), v.row(a.res_out, a.out_ld, a.out_bf16);
  v.row(a.h, a.h_ld, a.h_bf16), v.row(a.w, 0, 0), v.row(a.next_w, 0, 0);
  if (a.gate_kind == MOE_GATE_FULL) v.row(a.gate, a.gate_ld, a.gate_bf16);
  if (a.gate_kind == MOE_GATE_CHANNEL) v.row(a.gate, 0, 0);
  return launch_fwd(a, n, v.ok, static_cast<cudaStream_t>(stream));
}

extern "C" uint64_t moe_norm_workspace(int32_t n_tokens, int32_t d_model) {
  int blocks = 0;
  if (n_tokens < 1 || d_model < 1 || d_model > kNormMaxD || bwd_blocks(n_tokens, &blocks) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return static_cast<uint64_t>(blocks) * d_model * 8;
}

extern "C" moe_status moe_norm_in_backward(const moe_norm_in_bwd_args *p, void *stream) {
  if (!p || p->struct_size != sizeof(moe_norm_in_bwd_args)) return MOE_ERR_INVALID_ARGUMENT;
  const int n = p->n_tokens, d = p->d_model;
  if (n < 1 || d < 1 || bad_rows(p->x, p->x_stride, d, n, p->x_dtype) || bad_rows(p->dh, p->dh_stride, d, n, p->dh_dtype) ||
      bad_rows(p->dx, p->dx_stride, d, n, p->dx_dtype) || !p->weight || bad_vec(p->weight, p->w_dtype) ||
      (p->dres && bad_rows(p->dres, p->dres_stride, d, n, p->dres_dtype)) || (p->dweight && bad_vec(p->dweight, p->w_dtype)) ||
      p->unit_offset < 0 || p->unit_offset > 1 || !(p->eps >= 0.f))
    return MOE_ERR_INVALID_ARGUMENT;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  NormBwd a{};
  a.x = p->x, a.x_ld = p->x_stride, a.x_bf16 = p->x_dtype == MOE_BF16;
  a.dy = p->dh, a.dy_ld = p->dh_stride, a.dy_bf16 = p->dh_dtype == MOE_BF16;
  a.w = p->weight, a.w_bf16 = p->w_dtype == MOE_BF16, a.w_off = static_cast<float>(p->unit_offset), a.eps = p->eps;
  a.dres = p->dres, a.dres_ld = p->dres_stride, a.dres_bf16 = p->dres_dtype == MOE_BF16;
  a.dx = p->dx, a.dx_ld = p->dx_stride, a.dx_bf16 = p->dx_dtype == MOE_BF16;
  a.gate_kind = MOE_GATE_NONE, a.scale = 1.f, a.d = d, a.n = n;
  VecRule v(d);
  v.row(a.x, a.x_ld, a.x_bf16), v.row(a.dy, a.dy_ld, a.dy_bf16), v.row(a.dres, a.dres_ld, a.dres_bf16);
  v.row(a.dx, a.dx_ld, a.dx_bf16), v.row(a.w, 0, 0);
  return run_bwd(a, v.ok, p->dweight, a.w_bf16, nullptr, 0, p->workspace, p->workspace_bytes,
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
  NormBwd a{};
  a.x = p->o, a.x_ld = p->o_stride, a.x_bf16 = p->o_dtype == MOE_BF16;
  a.dy = p->dres, a.dy_ld = p->dres_stride, a.dy_bf16 = p->dres_dtype == MOE_BF16;
  a.w = p->weight, a.w_bf16 = p->w_dtype == MOE_BF16, a.w_off = static_cast<float>(p->unit_offset), a.eps = p->eps;
  a.gate = p->gate, a.gate_kind = p->gate_kind, a.gate_act = p->gate_act, a.gate_ld = p->gate_stride;
  a.gate_bf16 = p->gate_dtype == MOE_BF16;
  a.dx = p->d_o, a.dx_ld = p->do_stride, a.dx_bf16 = a.x_bf16;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (!channel) a.dgate = p->dgate, a.dgate_ld = p->dgate_stride;
  a.scale = p->scale, a.d = d, a.n = n;
  VecRule v(d);
  v.row(a.x, a.x_ld, a.x_bf16), v.row(a.dy, a.dy_ld, a.dy_bf16), v.row(a.dx, a.dx_ld, a.dx_bf16), v.row(a.w, 0, 0);
  if (a.gate_kind == MOE_GATE_FULL) v.row(a.gate, a.gate_ld, a.gate_bf16), v.row(a.dgate, a.dgate_ld, a.gate_bf16);
  if (channel) v.row(a.gate, 0, 0);
  return run_bwd(a, v.ok, p->dweight, a.w_bf16, channel ? p->dgate : nullptr, a.gate_bf16, p->workspace,
                 p->workspace_bytes, static_cast<cudaStream_t>(stream));
}
