// The whole routed layer for a few tokens (1 to 16) in two launches.
//
//   few_router   l[t, e] = sum_h W_r[e, h] x[t, h], the keys (sigmoid(l) + b, or l for the
//                softmax router) and the scores, in 64 bits: two neighbouring keys of the
//                border between the k-th and the next expert can lie closer than an fp32
//                sum resolves, and at a few tokens the 64-bit sums cost nothing that shows.
//   few_layer    every CTA picks the top k itself (the keys are a few KB, so this is cheaper
//                than another launch), then claims work units from a counter:
//                first the gate/up rows  h[p, i] = act(W_gate x)_i (W_up x)_i  of every
//                (token, slot) pair p and of the shared expert, then the rows
//                y[t, r] = sum_j w[t, j] (W_down h[t, j])_r + shared + residual.
// The down units wait until every gate/up unit is done.  Units are claimed in order and a
// CTA finishes its claims in order, so the units waited for are always held by CTAs that
// are running and do not wait themselves: the wait ends however many CTAs are resident and
// whatever else runs on the GPU.  It is bounded in time all the same (MOE_FLAG_TIMEOUT).
// The router launch zeroes the counters, so the workspace needs no initial state.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kRouterThreads = 128;
constexpr int kRouterTokens = 4;  // tokens per pass over a router row

// order-preserving image of a key: larger key, larger integer; 0 is kept for "not selectable"
__device__ __forceinline__ uint64_t sortable(double key) {
  const uint64_t u = (uint64_t)__double_as_longlong(key);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <int XF>
__device__ __forceinline__ void load4(const void* base, size_t i, float (&v)[4]) {
  if (XF == MOE_X_F32) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i));
    v[0] = bf16_to_f32(u.x & 0xFFFFu), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = bf16_to_f32(u.y & 0xFFFFu), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
}

// One CTA per expert.
template <int XF>
__global__ void __launch_bounds__(kRouterThreads)
    few_router_kernel(const void* __restrict__ x, const float* __restrict__ W_r, const float* __restrict__ bias,
                      const uint8_t* __restrict__ mask, int T, int H, int E, int router, uint64_t* __restrict__ keys,
                      double* __restrict__ scores, uint32_t* __restrict__ counters, uint32_t* flags) {
  pdl_wait();
  pdl_trigger();
  __shared__ double part[kRouterThreads / 32][kRouterTokens];
  const int e = blockIdx.x, tid = threadIdx.x;
  if (e == 0 && tid < kFewCounters) counters[tid] = 0;
  const float* row = W_r + (size_t)e * H;
  for (int t0 = 0; t0 < T; t0 += kRouterTokens) {
    double acc[kRouterTokens] = {};
    for (int c = tid * 4; c < H; c += kRouterThreads * 4) {
      float w[4];
      load4<MOE_X_F32>(row, c, w);
#pragma unroll
      for (int j = 0; j < kRouterTokens; ++j) {
        if (t0 + j >= T) break;
        float v[4];
        load4<XF>(x, (size_t)(t0 + j) * H + c, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j] = fma((double)w[q], (double)v[q], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kRouterTokens; ++j) {
      if (t0 + j >= T) break;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], off);
      if (lane_id() == 0) part[warp_id()][j] = acc[j];
    }
    __syncthreads();
    const int t = t0 + tid;
    if (tid < kRouterTokens && t < T) {
      double l = 0.0;
#pragma unroll
      for (int w = 0; w < kRouterThreads / 32; ++w) l += part[w][tid];
      const bool finite = isfinite((float)l);
      if (!finite) raise_flag(flags, MOE_FLAG_NONFINITE_LOGIT);
      double score = l, key = l;
      if (router == MOE_ROUTER_SIGMOID_BIAS) {
        score = 1.0 / (1.0 + exp(-l));
        key = score + (bias ? (double)bias[e] : 0.0);
      }
      const bool open = finite && key == key && (mask == nullptr || mask[e] != 0);
      keys[(size_t)t * E + e] = open ? sortable(key) : 0;
      scores[(size_t)t * E + e] = score;
    }
    __syncthreads();
  }
}

struct FewArgs {
  int T, H, I, E, k, Is;  // Is = 0: no shared expert
  int router, act;
  float scale;
  const void* x;
  const void* residual;
  const void* W[3];   // gate, up, down of the routed experts
  const float* s[3];
  const void* Ws[3];  // and of the shared expert
  const float* ss[3];
  const uint64_t* keys;
  const double* scores;
  float* h;           // [T k, I] of the routed pairs, then [T, Is] of the shared expert
  uint32_t* counters; // [0] claimed units, [kFewDone] finished gate/up units
  int32_t* idx;
  float* w;
  void* y;
  uint32_t* flags;
};

// Top k of one token by one warp, from keys held PER_LANE to a lane (expert lane + 32 j):
// k rounds of a warp-wide maximum over the 64-bit keys, upper halves first, then lower
// halves, ties to the lower expert.
template <int PER_LANE>
__device__ __forceinline__ void few_topk(const FewArgs& a, int t, int* out_e, float* out_w, bool write) {
  const int lane = lane_id();
  uint64_t key[PER_LANE];
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < a.E ? a.keys[(size_t)t * a.E + e] : 0;
  }
  int mine = -1;
  for (int slot = 0; slot < a.k; ++slot) {
    uint64_t best = 0;
    int bj = 0;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j)
      if (key[j] > best) best = key[j], bj = j;
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32));
    const bool in = best != 0 && (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, in ? (uint32_t)best : 0u);
    const bool win = in && (uint32_t)best == lo;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, win ? (uint32_t)(lane + 32 * bj) : 0xFFFFFFFFu);
    if (e == 0xFFFFFFFFu) {
      if (write && lane == 0) raise_flag(a.flags, MOE_FLAG_TOO_FEW_ACTIVE);
      break;
    }
    if ((int)(e & 31u) == lane) {
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j)
        if (j == (int)(e >> 5)) key[j] = 0;
    }
    if (lane == slot) mine = (int)e;
  }
  // the chosen scores, renormalised (softmax: relative to the best logit, which the full
  // denominator cancels against)
  const double score = mine >= 0 ? a.scores[(size_t)t * a.E + mine] : 0.0;
  const double top = __shfl_sync(0xFFFFFFFFu, score, 0);
  const double v = mine < 0 ? 0.0 : (a.router == MOE_ROUTER_SIGMOID_BIAS ? score : exp(score - top));
  double total = v;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
  if (lane < a.k) {
    const float w = (mine >= 0 && total > 0.0) ? (float)(v / total * (double)a.scale) : 0.f;
    out_e[t * a.k + lane] = mine;
    out_w[t * a.k + lane] = w;
    if (write) {
      a.idx[t * a.k + lane] = mine;
      a.w[t * a.k + lane] = w;
    }
  }
}

// lane's share of sum_c W[c] v[c] over one stored row; lanes take 8 columns in turn
template <int WF, typename LoadV>
__device__ __forceinline__ float row_dot(const void* W, const float* s, size_t row, int K, LoadV load_v) {
  float acc = 0.f;
  for (int c = lane_id() * 8; c < K; c += 256) {
    float v[8], q[8];
    load_v(c, v);
    float scale = 1.f;
    if constexpr (WF == MOE_W_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + row * K + c);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      q[0] = a.x, q[1] = a.y, q[2] = a.z, q[3] = a.w, q[4] = b.x, q[5] = b.y, q[6] = b.z, q[7] = b.w;
    } else if constexpr (WF == MOE_W_BF16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + row * K + c));
      const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[2 * j] = bf16_to_f32(word[j] & 0xFFFFu);
        q[2 * j + 1] = __uint_as_float(word[j] & 0xFFFF0000u);
      }
    } else if constexpr (WF == MOE_W_INT8_ROW) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(W) + row * K + c));
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = (float)(int8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
    } else {
      constexpr int kShift = WF == MOE_W_INT4_B32 ? 5 : 7;
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(W) + (row * K + c) / 2));
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = (float)((int)(u << (28 - 4 * j)) >> 28);
      scale = __ldg(s + row * (K >> kShift) + (c >> kShift));
    }
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) d = fmaf(q[j], v[j], d);
    acc = fmaf(d, scale, acc);
  }
  if constexpr (WF == MOE_W_INT8_ROW) acc *= __ldg(s + row);
  return acc;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

constexpr int kFewThreads = 256;
constexpr int kFewRows = kFewThreads / 32;  // rows of a unit: one per warp

template <int WF, int XF>
__global__ void __launch_bounds__(kFewThreads) few_layer_kernel(const FewArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int pair_e[MOE_FEW_MAX_TOKENS * 32];
  __shared__ float pair_w[MOE_FEW_MAX_TOKENS * 32];
  __shared__ uint32_t ticket;
  __shared__ int dead;
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) dead = 0;
  for (int t = warp; t < a.T; t += kFewThreads / 32) {
    if (a.E <= 256) few_topk<8>(a, t, pair_e, pair_w, blockIdx.x == 0);
    else few_topk<32>(a, t, pair_e, pair_w, blockIdx.x == 0);
  }
  const int P = a.T * a.k;
  const uint32_t ub = (uint32_t)(a.I / kFewRows), us = (uint32_t)(a.Is / kFewRows), hb = (uint32_t)(a.H / kFewRows);
  const uint32_t n_up = P * ub + a.T * us, n_all = n_up + a.T * hb;
  float* hs = a.h + (size_t)P * a.I;
  bool ready = false;
  for (;;) {
    __syncthreads();
    if (threadIdx.x == 0) ticket = atomicAdd(&a.counters[0], 1u);
    __syncthreads();
    const uint32_t u = ticket;
    if (u >= n_all) break;
    if (u < n_up) {
      const bool shared = u >= P * ub;
      const int p = shared ? (int)((u - P * ub) / us) : (int)(u / ub);
      const int i = (shared ? (int)((u - P * ub) % us) : (int)(u % ub)) * kFewRows + warp;
      const int t = shared ? p : p / a.k;
      const int e = shared ? 0 : pair_e[p];
      const int cols = shared ? a.Is : a.I;
      if (e >= 0) {
        auto lv = [&](int c, float (&v)[8]) {
          float lo[4], hi[4];
          load4<XF>(a.x, (size_t)t * a.H + c, lo);
          load4<XF>(a.x, (size_t)t * a.H + c + 4, hi);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = lo[j], v[4 + j] = hi[j];
        };
        const size_t row = (size_t)e * cols + i;
        const float g = warp_sum(row_dot<WF>(shared ? a.Ws[0] : a.W[0], shared ? a.ss[0] : a.s[0], row, a.H, lv));
        const float v = warp_sum(row_dot<WF>(shared ? a.Ws[1] : a.W[1], shared ? a.ss[1] : a.s[1], row, a.H, lv));
        if (lane == 0)
          (shared ? hs : a.h)[(size_t)p * cols + i] = a.act == MOE_ACT_SILU ? silu_mul(g, v) : gelu_tanh_mul(g, v);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(&a.counters[kFewDone], 1u);
      }
      continue;
    }
    if (!ready) {
      if (threadIdx.x == 0) {
        const uint64_t t0 = global_timer_ns();
        while (*reinterpret_cast<volatile uint32_t*>(&a.counters[kFewDone]) < n_up) {
          if (global_timer_ns() - t0 > kWaitLimitNs) {
            dead = 1;
            raise_flag(a.flags, MOE_FLAG_TIMEOUT);
            break;
          }
        }
        __threadfence();
      }
      __syncthreads();
      if (dead) break;
      ready = true;
    }
    const int t = (int)((u - n_up) / hb), r = (int)((u - n_up) % hb) * kFewRows + warp;
    float y = 0.f;
    for (int j = 0; j <= a.k; ++j) {
      const bool shared = j == a.k;
      if (shared && a.Is == 0) break;
      const int p = shared ? t : t * a.k + j, e = shared ? 0 : pair_e[p], cols = shared ? a.Is : a.I;
      if (e < 0) continue;
      const float* h = (shared ? hs : a.h) + (size_t)p * cols;
      auto lv = [&](int c, float (&v)[8]) {
        const float4 lo = __ldcg(reinterpret_cast<const float4*>(h + c));
        const float4 hi = __ldcg(reinterpret_cast<const float4*>(h + c + 4));
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
      };
      const float o = warp_sum(row_dot<WF>(shared ? a.Ws[2] : a.W[2], shared ? a.ss[2] : a.s[2],
                                           (size_t)e * a.H + r, cols, lv));
      y += shared ? o : pair_w[p] * o;
    }
    if (lane == 0) {
      const size_t at = (size_t)t * a.H + r;
      if constexpr (XF == MOE_X_F32) {
        if (a.residual) y += static_cast<const float*>(a.residual)[at];
        static_cast<float*>(a.y)[at] = y;
      } else {
        if (a.residual) y += bf16_to_f32(static_cast<const uint16_t*>(a.residual)[at]);
        static_cast<uint16_t*>(a.y)[at] = f32_to_bf16(y);
      }
    }
  }
}

struct FewLayout {
  size_t keys, scores, h, total;
};
FewLayout few_layout(const moe_desc& d, int Is, int T) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FewLayout l;
  l.keys = up(kFewCounters * sizeof(uint32_t));
  l.scores = l.keys + up((size_t)T * d.E * 8);
  l.h = l.scores + up((size_t)T * d.E * 8);
  l.total = l.h + up(((size_t)T * d.k * d.I + (size_t)T * Is) * 4);
  return l;
}

template <int WF>
cudaError_t launch_layer(const moe_desc& d, const FewArgs& a, int num_sms, cudaStream_t s) {
  const dim3 grid(num_sms * 4), block(kFewThreads);
  return d.xfmt == MOE_X_F32 ? launch_k(few_layer_kernel<WF, MOE_X_F32>, grid, block, 0, s, a)
                             : launch_k(few_layer_kernel<WF, MOE_X_BF16>, grid, block, 0, s, a);
}

}  // namespace

size_t few_workspace_bytes(const moe_desc& d, const moe_shared_expert* sh, int T) {
  return few_layout(d, sh ? sh->I : 0, T).total;
}

cudaError_t launch_few_router(const moe_desc& d, const moe_shared_expert* sh, const void* x, int T, void* workspace,
                              uint32_t* flags, cudaStream_t s) {
  const FewLayout l = few_layout(d, sh ? sh->I : 0, T);
  char* ws = static_cast<char*>(workspace);
  auto kernel = d.xfmt == MOE_X_F32 ? few_router_kernel<MOE_X_F32> : few_router_kernel<MOE_X_BF16>;
  return launch_k(kernel, dim3(d.E), dim3(kRouterThreads), 0, s, x, d.W_r, d.b, d.expert_mask, T, d.H, d.E, d.router,
                  reinterpret_cast<uint64_t*>(ws + l.keys), reinterpret_cast<double*>(ws + l.scores),
                  reinterpret_cast<uint32_t*>(ws), flags);
}

cudaError_t launch_few_layer(const moe_desc& d, const moe_shared_expert* sh, const void* x, int T, int32_t* idx,
                             float* w, const void* residual, void* y, void* workspace, int num_sms, uint32_t* flags,
                             cudaStream_t s) {
  const FewLayout l = few_layout(d, sh ? sh->I : 0, T);
  char* ws = static_cast<char*>(workspace);
  FewArgs a = {};
  a.T = T, a.H = d.H, a.I = d.I, a.E = d.E, a.k = d.k, a.Is = sh ? sh->I : 0;
  a.router = d.router, a.act = d.act, a.scale = d.scale;
  a.x = x, a.residual = residual;
  a.W[0] = d.W_gate, a.W[1] = d.W_up, a.W[2] = d.W_down;
  a.s[0] = d.s_gate, a.s[1] = d.s_up, a.s[2] = d.s_down;
  if (sh) {
    a.Ws[0] = sh->W_gate, a.Ws[1] = sh->W_up, a.Ws[2] = sh->W_down;
    a.ss[0] = sh->s_gate, a.ss[1] = sh->s_up, a.ss[2] = sh->s_down;
  }
  a.keys = reinterpret_cast<const uint64_t*>(ws + l.keys);
  a.scores = reinterpret_cast<const double*>(ws + l.scores);
  a.h = reinterpret_cast<float*>(ws + l.h);
  a.counters = reinterpret_cast<uint32_t*>(ws);
  a.idx = idx, a.w = w, a.y = y, a.flags = flags;
  switch (d.wfmt) {
    case MOE_W_F32: return launch_layer<MOE_W_F32>(d, a, num_sms, s);
    case MOE_W_BF16: return launch_layer<MOE_W_BF16>(d, a, num_sms, s);
    case MOE_W_INT8_ROW: return launch_layer<MOE_W_INT8_ROW>(d, a, num_sms, s);
    case MOE_W_INT4_B32: return launch_layer<MOE_W_INT4_B32>(d, a, num_sms, s);
    default: return launch_layer<MOE_W_INT4_B128>(d, a, num_sms, s);
  }
}

}  // namespace moe
