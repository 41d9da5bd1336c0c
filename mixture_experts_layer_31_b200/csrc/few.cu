// The whole routed layer for a few tokens (1 to 16) in two launches.
//
//   few_router   l[t, e] = sum_h W_r[e, h] x[t, h], the keys (sigmoid(l) + b, or l for the
//                softmax router) and the scores, in 64 bits: two neighbouring keys of the
//                border between the k-th and the next expert can lie closer than an fp32
//                sum resolves, and at a few tokens the 64-bit sums cost nothing that shows.
//   the layer    every CTA picks the top k itself (the keys are a few KB, so this is cheaper
//                than another launch), then takes its share first of the gate/up rows
//                h[p, i] = act(W_gate x)_i (W_up x)_i  of every (token, slot) pair p and
//                of the shared expert, then of the rows
//                y[t, r] = sum_j w[t, j] (W_down h[t, j])_r + shared + residual.
// Two kernels have the second part: few_stream (bf16 tokens on bf16, int8 or int4 weights) deals its
// units out as lists, one per CTA, which another CTA may take over; few_layer (fp32 tokens or
// weights) claims them from a counter.  In both, what is waited for between the two parts is
// always held by CTAs that are running and do not wait themselves -- few_layer's claims are
// made and finished in order, few_stream's lists are started by their CTA or taken over -- so
// the wait ends however many CTAs are resident and whatever else runs on the GPU.  It is
// bounded in time all the same (MOE_FLAG_TIMEOUT).
// The router launch zeroes the counters, so the workspace needs no initial state.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "stream_dev.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kRouterThreads = 256;

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

// One CTA per kRouterExperts experts and TT tokens.  Its warps share out the columns; each keeps
// the sums of all its tokens so that a router weight is widened to 64 bits once for all of
// them: the conversions, not the 64-bit multiply-adds, are what this costs (a token for each
// warp instead took 20 us at 16 tokens x 2,304 columns x 256 experts).
constexpr int kRouterExperts = 2;

template <int XF, int TT>
__global__ void __launch_bounds__(kRouterThreads)
    few_router_kernel(const void* __restrict__ x, const float* __restrict__ W_r, const float* __restrict__ bias,
                      const uint8_t* __restrict__ mask, int T, int H, int E, int router, uint64_t* __restrict__ keys,
                      double* __restrict__ scores, uint32_t* __restrict__ counters, int8_t* __restrict__ digits, int int4,
                      float* __restrict__ units, uint32_t* flags) {
  pdl_wait();
  pdl_trigger();
  constexpr int kSums = kRouterExperts * TT, kRWarps = kRouterThreads / 32;
  __shared__ double part[kRWarps][kSums];
  const int e0 = blockIdx.x * kRouterExperts, t0 = blockIdx.y * TT, tid = threadIdx.x, w = warp_id(), lane = lane_id();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < kFewCounters; i += kRouterThreads) counters[i] = 0;
  if (e0 >= E) {
    // the CTAs past the experts: a token each, as digits for the integer products
    const int t = t0 + blockIdx.x - (E + kRouterExperts - 1) / kRouterExperts;
    if (t >= T) return;
    __shared__ float warps[kRouterThreads / 32];
    if constexpr (XF == MOE_X_BF16)
      stream::write_digits(static_cast<const uint16_t*>(x) + (size_t)t * H, H, int4, digits + (size_t)t * 4 * stream::digit_pitch(H),
                           units + t, warps);
    return;
  }
  const float* row[kRouterExperts];
#pragma unroll
  for (int i = 0; i < kRouterExperts; ++i) row[i] = W_r + (size_t)min(e0 + i, E - 1) * H;
  double acc[kSums] = {};
#pragma unroll 2
  for (int c = w * 128 + lane * 4; c < H; c += kRWarps * 128) {
    float v[kRouterExperts][4], u[TT][4];
#pragma unroll
    for (int i = 0; i < kRouterExperts; ++i) load4<MOE_X_F32>(row[i], c, v[i]);
#pragma unroll
    for (int j = 0; j < TT; ++j) load4<XF>(x, (size_t)min(t0 + j, T - 1) * H + c, u[j]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      double wd[kRouterExperts];
#pragma unroll
      for (int i = 0; i < kRouterExperts; ++i) wd[i] = (double)v[i][q];
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const double xd = (double)u[j][q];
#pragma unroll
        for (int i = 0; i < kRouterExperts; ++i) acc[j * kRouterExperts + i] = fma(wd[i], xd, acc[j * kRouterExperts + i]);
      }
    }
  }
  // sums over the lanes: halves of the values change sides until each lane has at most one
  int n = kSums, first = 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int k = 0; k < kSums / 2; ++k) {
        if (k >= n) break;
        const double give = up ? acc[k] : acc[k + n], keep = up ? acc[k + n] : acc[k];
        acc[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, off);
      }
      if (up) first += n;
    } else {
      acc[0] += __shfl_xor_sync(0xFFFFFFFFu, acc[0], off);
    }
  }
  part[w][first] = acc[0];  // lanes with the same value write the same sum
  __syncthreads();
  const int j = tid / kRouterExperts, e = e0 + tid % kRouterExperts, t = t0 + j;
  if (tid < kSums && t < T && e < E) {
    double l = 0.0;
#pragma unroll
    for (int i = 0; i < kRWarps; ++i) l += part[i][tid];
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
  const int8_t* digits;  // [T][4][digit_pitch(H)] and the tokens' units: quantised weights on the streaming path
  const float* units;
  const uint64_t* keys;
  const double* scores;
  float* h;           // [T k, I] of the routed pairs, then [T, Is] of the shared expert
  uint16_t* h2;       // the same in two bf16 planes (value and remainder) on the streaming path
  size_t plane;       // elements of a plane
  // int4 block scales come with the weights as boxes, per matrix, or are read where they
  // lie: [0] routed gate/up, [1] routed down, [2], [3] shared
  uint8_t boxed[4];
  int team, down_team;  // warps that share a gate/up unit, a down entry
  uint32_t* counters; // few_layer: claimed units, [kFewDone] finished gate/up units; few_stream: CTAs, lists
  int32_t* idx;
  float* w;
  void* y;
  uint32_t* flags;
};

// The k best experts of one token by one warp, from keys held PER_LANE to a lane (expert lane +
// 32 j): k rounds of a warp-wide maximum over the lanes' best keys, by their upper halves
// and, only where those are equal, the lower halves and then the expert's number.  Lane
// `slot` returns its expert, -1 where none is left.
template <int PER_LANE>
__device__ __forceinline__ int few_topk(const FewArgs& a, int t) {
  const int lane = lane_id();
  uint64_t key[PER_LANE];
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < a.E ? a.keys[(size_t)t * a.E + e] : 0;
  }
  int mine = -1;
  uint64_t best = 0;
  int bj = 0;
  auto find = [&] {
    best = 0;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j)
      if (key[j] > best) best = key[j], bj = j;
  };
  find();
  for (int slot = 0; slot < a.k; ++slot) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32));
    uint32_t who = __ballot_sync(0xFFFFFFFFu, best != 0 && (uint32_t)(best >> 32) == hi);
    if (who == 0) break;
    if (who & (who - 1)) {
      const bool in = (who >> lane) & 1u;
      const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, in ? (uint32_t)best : 0u);
      const bool win = in && (uint32_t)best == lo;
      const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, win ? (uint32_t)(lane + 32 * bj) : 0xFFFFFFFFu);
      who = 1u << (e & 31u);
    }
    const int from = __ffs(who) - 1;
    const int e = __shfl_sync(0xFFFFFFFFu, lane + 32 * bj, from);
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j)
        if (j == bj) key[j] = 0;
      find();
    }
    if (lane == slot) mine = e;
  }
  return mine;
}

__device__ __forceinline__ int few_topk(const FewArgs& a, int t) {
  return a.E <= 256 ? few_topk<8>(a, t) : few_topk<32>(a, t);
}

// The weight of lane `slot`'s expert: the chosen scores renormalised (softmax: relative to the
// best logit, which the full denominator cancels against).  The whole warp calls it.
__device__ __forceinline__ float few_weight(const FewArgs& a, int t, int e) {
  const double score = e >= 0 ? a.scores[(size_t)t * a.E + e] : 0.0;
  const double top = __shfl_sync(0xFFFFFFFFu, score, 0);
  const double v = e < 0 ? 0.0 : (a.router == MOE_ROUTER_SIGMOID_BIAS ? score : exp(score - top));
  double total = v;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
  return (e >= 0 && total > 0.0) ? (float)(v / total * (double)a.scale) : 0.f;
}

// one CTA writes the routing out
__device__ __forceinline__ void few_write_route(const FewArgs& a, int t, int e, float w) {
  if (lane_id() >= a.k) return;
  a.idx[t * a.k + lane_id()] = e;
  a.w[t * a.k + lane_id()] = w;
  if (e < 0) raise_flag(a.flags, MOE_FLAG_TOO_FEW_ACTIVE);
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
    const int e = few_topk(a, t);
    const float wt = few_weight(a, t, e);
    if (lane < a.k) pair_e[t * a.k + lane] = e, pair_w[t * a.k + lane] = wt;
    if (blockIdx.x == 0) few_write_route(a, t, e, wt);
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

// ------------------------------------------------------------------ the streaming kernel
//
// bf16 tokens on bf16, int8 or int4 weights.  One persistent CTA per SM, twelve equal warps.
// A gate/up unit is 16 rows of W_gate and the same 16 of W_up of one expert for up to 8 of its
// tokens: both projections of an output end up in one lane.  The unit's reduction is shared
// out over the warps box by box (16 rows x 128 bytes), so that a unit streams at the whole
// SM's rate; each warp copies its boxes into a ring of its own by TMA, several stages
// ahead and across units, and needs no other warp for that.  The warps' sums meet in shared
// memory; the warp whose share of the unit is smallest adds them up, applies the activation
// and stores h.  (One copying, one summing and ten multiplying warps measured worse: the
// summing warp, all latency, held up the rest.)
// Units are dealt out as lists, one per CTA.  Nothing makes the CTAs of a launch run at the same
// time (another launch of this kind may hold SMs and wait as well), so a CTA that is done
// with its list takes over those that no CTA has started on, and one that starts late and
// finds its list taken leaves: whoever waits at the barrier waits for CTAs that are running.
// After that barrier over the lists a CTA computes 16 rows of y for every chosen expert (and the
// shared one), one after the other, so the combine stays inside the CTA.  Down weights do not
// depend on h: the rings are full of them before the barrier opens.  h is handed over as
// bf16 value plus bf16 remainder (16 significant bits): the remainder takes token columns of
// the matrix instruction that would be empty, where a rounded h would add an error as large
// as y's own rounding.  What is summed together depends on the plan alone, so the same call
// gives the same bits.
//
// Measured, both launches among calls on other inputs (ranges: over several GPUs), with what the
// bytes alone need at the copy rate of 6.55 TB/s:
//   1 token   bf16, 2,304 wide, 256 experts of 2,048, 8 chosen, shared    55 us       39 us
//   4 tokens  int8, the same layer                                        97-99 us    69 us
//   16 tokens int8, the same layer, 160 experts active                   238-245 us  194 us
//   1 token   int4, 2,048 wide, 128 experts of 768, 8 chosen              26 us        4 us
//   16 tokens int4, the same layer                                       107-111 us   37 us
// The first three are bound by HBM behind some 15 us of router, plan, first loads and barrier; one
// int4 token by those alone.  Sixteen int4 tokens are bound by the instructions of the
// products (a box of 2 KB takes some 250 of them, at 0.43 per cycle and scheduler with three
// warps): gate and up 45 us, down 38, barrier and imbalance 10.

constexpr int kWarps = 12;
constexpr int kStreamThreads = 32 * kWarps;
constexpr int kMaxPairs = MOE_FEW_MAX_TOKENS * 32;
constexpr int kDownTokens = 4;  // tokens of a down tile: values in columns 0..3, remainders in 4..7
constexpr int kMaxStages = 4;

template <int WF>
struct Ring {
  using F = stream::Format<WF>;
  static constexpr bool kDigits = WF != MOE_W_BF16;       // gate/up products are integer ones
  // Codes are up to 128 times what they stand for in units of the row's largest weight: h is kept
  // smaller by a power of two, so that its products with codes overflow no sooner than h.
  static constexpr float kHScale = WF == MOE_W_BF16 ? 1.f : 1.f / 256.f;
  static constexpr int kUpTiles = kDigits ? 2 : 1;        // token tiles of a gate/up unit
  static constexpr int kUpTokens = kDigits ? kUpTiles * stream::kDigitTokens : 8;
  static constexpr int kStage = 2 * (stream::kBoxBytes + F::kScaleBox);  // gate and up box, or down boxes
  static constexpr int kDownBoxes = F::kInt4 ? 1 : 2;                    // of a stage (bounds the tokens loaded ahead)
  static constexpr int kStages = F::kScaleBoxes ? 3 : kMaxStages;
  static constexpr int kBytes = kWarps * kStages * kStage;
};

struct FewMaps {
  CUtensorMap w[3], ws[3];  // gate, up, down of the routed experts and of the shared one
  CUtensorMap s[3], ss[3];  // their int4 block-32 scales, where `boxed` says so
};

// A group of tokens of one expert, packed: expert (or kSharedEntry), first sorted pair (shared:
// first token), tokens.
constexpr uint32_t kSharedEntry = 1024;
__device__ __forceinline__ uint32_t pack_entry(uint32_t e, int start, int n) {
  return e | (uint32_t)start << 11 | (uint32_t)n << 21;
}
__device__ __forceinline__ uint32_t entry_e(uint32_t v) { return v & 2047u; }
__device__ __forceinline__ int entry_start(uint32_t v) { return (int)(v >> 11 & 1023u); }
__device__ __forceinline__ int entry_n(uint32_t v) { return (int)(v >> 21); }

struct StreamShared {
  uint64_t full[kWarps][kMaxStages];
  uint64_t rfull[kWarps][2], rempty[kWarps][2];  // by team: its warps' sums of a unit written / added up
  int n_up, n_down;              // entries
  int adopted;                   // a list taken over, -1 for none
  int taken, all;                // this CTA's list is another's; every CTA has started
  uint16_t lists[kFewLists];     // this CTA's lists
  float pair_w[kMaxPairs];
  uint16_t pair[kMaxPairs];      // valid pairs in expert order: pair | token << 9
  uint32_t up[kMaxPairs + 4], down[kMaxPairs + 4];  // entries: shared first / shared last
  union alignas(16) {            // read in pieces of 16 bytes
    float part[2][kWarps][2][16][8];           // [unit parity][warp][gate, up][row][token]
    struct {
      float y[kWarps][MOE_FEW_MAX_TOKENS][16];   // down: each warp's share of 16 rows
      uint32_t at[kMaxPairs + 4][kDownTokens];   // by down entry: where its tokens' h starts
    };
    struct {
      int e[kMaxPairs];                        // building the plan: by pair
      int by_rank[kMaxPairs];                  // in expert order: expert, -1 at the end
      int place[kMaxPairs];                    //   place among the expert's pairs << 16 | their number
    } plan;
  };
};

static_assert(offsetof(StreamShared, plan) % 16 == 0 && offsetof(StreamShared, part) % 16 == 0, "alignment");

__device__ __forceinline__ void few_wait(uint64_t* bar, uint32_t parity, bool& dead, uint32_t* flags) {
  if (dead) return;
  if (!mbar_wait(bar, parity)) {
    dead = true;
    raise_flag(flags, MOE_FLAG_TIMEOUT);
  }
}

// Entries of at most `most` tokens from the sorted pairs, appended from list[n] on by one warp.
__device__ __forceinline__ int list_entries(const StreamShared& sh, int P, int most, uint32_t* list, int n) {
  const int lane = lane_id();
  for (int r0 = 0; r0 < P; r0 += 32) {
    const int r = r0 + lane;
    const int e = r < P ? sh.plan.by_rank[r] : -1;
    const int at = e >= 0 ? sh.plan.place[r] >> 16 : 0, of = e >= 0 ? sh.plan.place[r] & 0xFFFF : 0;
    const bool head = e >= 0 && at % most == 0;
    const uint32_t heads = __ballot_sync(0xFFFFFFFFu, head);
    if (head) list[n + __popc(heads & ((1u << lane) - 1u))] = pack_entry((uint32_t)e, r, min(most, of - at));
    n += __popc(heads);
  }
  return n;
}

template <int WF>
__global__ void __launch_bounds__(kStreamThreads, 1)
    few_stream_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a) {
  using R = Ring<WF>;
  using F = stream::Format<WF>;
  constexpr int kUpTokens = R::kUpTokens;
  extern __shared__ uint8_t smem[];
  // the rings first, on 1,024 bytes (the swizzle's period)
  uint8_t* rings = smem + (((smem_u32(smem) + 1023u) & ~1023u) - smem_u32(smem));
  StreamShared& sh = *reinterpret_cast<StreamShared*>(rings + R::kBytes);
  const int w = warp_id(), lane = lane_id(), g = lane >> 2, c = lane & 3;
  uint8_t* ring = rings + w * R::kStages * R::kStage;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps; ++i)
      for (int j = 0; j < R::kStages; ++j) mbar_init(&sh.full[i][j], 1);
    for (int i = 0; i < kWarps / a.team; ++i)
      for (int j = 0; j < 2; ++j) {
        mbar_init(&sh.rfull[i][j], a.team);
        mbar_init(&sh.rempty[i][j], 1);
      }
    fence_mbar_init();
  }
  if (lane == 0 && w < 3) {
    prefetch_tmap(&maps.w[w]);
    if (a.Is) prefetch_tmap(&maps.ws[w]);
  }
  __syncthreads();
  const int P = a.T * a.k, grid = (int)gridDim.x;
  const int su = a.Is ? (a.T + kUpTokens - 1) / kUpTokens : 0, sd = a.Is ? (a.T + kDownTokens - 1) / kDownTokens : 0;
  const int sb = a.Is / 16, ub = a.I / 16, hb = a.H / 16;  // blocks of 16 rows
  const int boxes_h = (a.H + F::kBoxCols - 1) / F::kBoxCols;
  const int boxes_i = (a.I + F::kBoxCols - 1) / F::kBoxCols, boxes_s = (a.Is + F::kBoxCols - 1) / F::kBoxCols;
  const int steps_r = (boxes_i + R::kDownBoxes - 1) / R::kDownBoxes, steps_s = (boxes_s + R::kDownBoxes - 1) / R::kDownBoxes;
  bool dead = false;

  // Teams of warps take the units in turn: numbers team, team + teams, ... of the entries'
  // blocks of 16 rows (of the down entries, for every 16 rows of y).  Within a team the
  // boxes, one unit after the other, go round the warps.
  const int up_teams = kWarps / a.team, up_team = w / a.team, up_w = w % a.team;
  const int down_teams = kWarps / a.down_team, down_team = w / a.down_team, down_w = w % a.down_team;
  struct UpWalk {
    int n, entry, block, j;  // the team's n-th unit: entry and block of rows; box
  };
  int n_up = su, n_down = 0;  // entries; without the routed ones before the plan
  auto step_unit = [&](UpWalk& k) {
    ++k.n;
    k.block += grid * up_teams;
    for (int of; k.block >= (of = k.entry < su ? sb : ub); ++k.entry) k.block -= of;
  };
  auto first_unit = [&](int list, int j) {
    UpWalk k = {-1, 0, (list - grid) * up_teams + up_team, j};
    step_unit(k);
    return k;
  };
  auto seek_up = [&](UpWalk& k) {
    while (k.j >= boxes_h) {
      k.j -= boxes_h;
      step_unit(k);
    }
  };
  // The boxes of a team's down entries, one after the other, go round its warps too; the list's
  // blocks of y's rows follow one another.  Which entry and stage of it a warp's n-th stage is
  // takes two divisions, so a lane works it out for one stage of the next 32: those of
  // number n with n % 32 == lane.
  int per_blk = 0, down_blk = hb, n_stages = 0;  // a warp's stages of one block; the list's first block; its stages
  int entries_r = 0;                             // the team's routed entries; those of the shared expert follow
  uint32_t win = 0;                              // entry << 16 | stage of the entry
  int win_blk = 0;
  auto window = [&](int from) {
    if (n_stages == 0) return;
    const uint32_t n = (uint32_t)from + ((uint32_t)(lane - from) & 31u), q = n / (uint32_t)per_blk;
    int box = down_w + (int)(n - q * (uint32_t)per_blk) * a.down_team, x = 0, steps = steps_r;
    if (box >= entries_r * steps_r) box -= entries_r * steps_r, x = entries_r, steps = steps_s;
    const int of = box / steps;
    win = (uint32_t)(down_team + (x + of) * down_teams) << 16 | (uint32_t)(box - of * steps);
    win_blk = down_blk + (int)q * grid;
  };
  auto first_down = [&](int list) {
    auto of_team = [&](int n) { return n > down_team ? (n - down_team + down_teams - 1) / down_teams : 0; };
    const int entries = of_team(n_down);
    entries_r = of_team(n_down - sd);
    const int boxes = entries_r * steps_r + (entries - entries_r) * steps_s;
    per_blk = boxes > down_w ? (boxes - down_w + a.down_team - 1) / a.down_team : 0;
    down_blk = list;
    n_stages = list < hb ? per_blk * ((hb - list + grid - 1) / grid) : 0;
    window(0);
  };

  // copies run kStages ahead: `head` and `head_down` are the next to start
  int issued = 0, in_slot = 0;
  UpWalk head = first_unit((int)blockIdx.x, up_w);
  seek_up(head);
  int head_down = 0;
  auto issue = [&](bool down) {
    uint32_t v = 0;
    int blk = 0;
    if (down) v = __shfl_sync(0xFFFFFFFFu, win, head_down & 31), blk = __shfl_sync(0xFFFFFFFFu, win_blk, head_down & 31);
    if (lane == 0 && !dead) {
      uint8_t* stage = ring + in_slot * R::kStage;
      uint64_t* bar = &sh.full[w][in_slot];
      if (!down) {
        const bool shared = head.entry < su;
        const int row = head.block * 16 + (shared ? 0 : (int)entry_e(sh.up[head.entry]) * a.I);
        const bool boxed = F::kScaleBoxes && a.boxed[shared ? 2 : 0];
        const CUtensorMap* wm = shared ? maps.ws : maps.w;
        mbar_arrive_expect_tx(bar, 2 * (stream::kBoxBytes + (boxed ? F::kScaleBox : 0)));
        tma_load_2d(stage, wm, head.j * 128, row, bar);
        tma_load_2d(stage + stream::kBoxBytes, wm + 1, head.j * 128, row, bar);
        if (boxed) {
          const CUtensorMap* sm = shared ? maps.ss : maps.s;
          tma_load_2d(stage + 2 * stream::kBoxBytes, sm, head.j * 8, row, bar);
          tma_load_2d(stage + 2 * stream::kBoxBytes + F::kScaleBox, sm + 1, head.j * 8, row, bar);
        }
      } else {
        const uint32_t e = entry_e(sh.down[v >> 16]);
        const bool shared = e == kSharedEntry;
        const int row = blk * 16 + (shared ? 0 : (int)e * a.H);
        const int j = (int)(v & 0xFFFFu) * R::kDownBoxes;
        const int n = min((shared ? boxes_s : boxes_i) - j, R::kDownBoxes);
        const bool boxed = F::kScaleBoxes && a.boxed[shared ? 3 : 1];
        const CUtensorMap* wm = shared ? maps.ws + 2 : maps.w + 2;
        mbar_arrive_expect_tx(bar, n * (stream::kBoxBytes + (boxed ? F::kScaleBox : 0)));
        tma_load_2d(stage, wm, j * 128, row, bar);
        if (R::kDownBoxes > 1 && n > 1) tma_load_2d(stage + stream::kBoxBytes, wm, j * 128 + 128, row, bar);
        if (boxed) tma_load_2d(stage + 2 * stream::kBoxBytes, shared ? maps.ss + 2 : maps.s + 2, j * 8, row, bar);
      }
    }
    ++issued;
    in_slot = in_slot + 1 == R::kStages ? 0 : in_slot + 1;
  };
  auto issue_up = [&] {
    issue(false);
    head.j += a.team;
    seek_up(head);
  };
  auto issue_next = [&] {
    if (head.entry < n_up) {
      issue_up();
    } else if (head_down < n_stages) {
      issue(true);
      ++head_down;
    }
  };
  // The shared expert's units need no routing, and weights are nothing that the launch before this
  // one writes: their copies start before its end is waited for.  (Launches before that one
  // are over: it lets this one start only after its own wait.)
  while (issued < R::kStages && head.entry < n_up) issue_up();
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    atomicAdd(&a.counters[0], 1u);
    sh.taken = atomicExch(&a.counters[kFewOwner + blockIdx.x], 1u) != 0;
  }

  // the plan: routing, the pairs in expert order, entries of up to 8 (gate/up) and 4 (down) tokens
  for (int t = w; t < a.T; t += kWarps) {
    const int e = few_topk(a, t);
    if (lane < a.k) sh.plan.e[t * a.k + lane] = e;
  }
  __syncthreads();
  const int P4 = (P + 3) & ~3;
  if (threadIdx.x < P4 - P) sh.plan.e[P + threadIdx.x] = -1;  // past every pair
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += kStreamThreads) {
    const int e = sh.plan.e[p], mine = e < 0 ? 1024 : e;
    int before = 0, place = 0, of = 0;
#pragma unroll 2
    for (int q = 0; q < P4; q += 4) {
      const int4 f = *reinterpret_cast<const int4*>(&sh.plan.e[q]);
      const int v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        before += (uint32_t)v[i] < (uint32_t)mine;  // -1 lies past every expert
        const bool same = v[i] == e;
        of += same;
        place += same && q + i < p;
      }
    }
    const int rank = before + place;
    sh.pair[rank] = (uint16_t)(p | (p / a.k) << 9);
    sh.plan.by_rank[rank] = e;
    sh.plan.place[rank] = place << 16 | of;
  }
  __syncthreads();
  if (w == 0) {
    if (lane < su) sh.up[lane] = pack_entry(kSharedEntry, lane * kUpTokens, min(kUpTokens, a.T - lane * kUpTokens));
    const int n = list_entries(sh, P, kUpTokens, sh.up, su);
    if (lane == 0) sh.n_up = n;
  } else if (w == 1) {
    const int n = list_entries(sh, P, kDownTokens, sh.down, 0);
    if (lane < sd) sh.down[n + lane] = pack_entry(kSharedEntry, lane * kDownTokens, min(kDownTokens, a.T - lane * kDownTokens));
    if (lane == 0) sh.n_down = n + sd;
  } else if (w == 2 && lane == 0) {
    sh.all = *reinterpret_cast<volatile uint32_t*>(&a.counters[0]) >= (uint32_t)grid;
  }
  __syncthreads();
  n_up = sh.n_up;
  n_down = sh.n_down;
  // the usual case: every CTA has started, so no list will be left over, and the rings may run on
  // into the down weights
  const bool all = sh.all != 0;
  if (all) first_down((int)blockIdx.x);
  auto fill = [&](int have) {
#pragma unroll 1
    for (int i = have; i < R::kStages; ++i) issue_next();
  };
  if (!sh.taken) fill(issued);
  // this warp's tokens' experts, for the weights later (warp 0 will wait for the grid meanwhile, so
  // it comes last); then the plan's space becomes the units' sums
  const int my_t = kWarps - 1 - w;
  int my_e[2] = {-1, -1};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (my_t + i * kWarps < a.T && lane < a.k) my_e[i] = sh.plan.e[(my_t + i * kWarps) * a.k + lane];
  static_assert(MOE_FEW_MAX_TOKENS <= 2 * kWarps, "a warp has at most two tokens' weights");
  __syncthreads();

  int done = 0, out_slot = 0;                     // stages read
  uint32_t phase = 0;
  auto landed = [&] {
    few_wait(&sh.full[w][out_slot], phase, dead, a.flags);
    __syncwarp();
  };
  auto read = [&] {
    __syncwarp();
    ++done;
    if (++out_slot == R::kStages) out_slot = 0, phase ^= 1u;
    issue_next();
  };

  // ---------------------------------------------------------------- gate and up
  int n_lists = 0, events = 0;
  for (int list = sh.taken ? -1 : (int)blockIdx.x; list >= 0;) {
    using Sum = std::conditional_t<R::kDigits, stream::DigitSum<WF>, float>;
    Sum acc[2][R::kUpTiles][4] = {};
    UpWalk unit = first_unit(list, 0);  // the next to hand over
    // this warp's sums of the unit to shared memory; the warp whose turn it is adds them up
    auto hand_over = [&] {
      const int buf = events & 1, parity = (events >> 1) & 1;
      const int from = a.team == 1 ? 0 : unit.n * boxes_h % a.team;  // the warps that had boxes, in their order
      const int shares = min(boxes_h, a.team);
      few_wait(&sh.rempty[up_team][buf], parity ^ 1, dead, a.flags);
      if (shares == a.team || (up_w >= from ? up_w - from : up_w + a.team - from) < shares) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < R::kUpTiles; ++nt) {
            float(&p)[16][8] = sh.part[buf][w][mt];
            if constexpr (R::kDigits) {
              float r0, r8;
              stream::join_digits(acc[mt][nt], r0, r8);
              if ((c & 1) == 0) p[g][2 * nt + c / 2] = r0, p[g + 8][2 * nt + c / 2] = r8;
            } else {
              *reinterpret_cast<float2*>(&p[g][2 * c]) = make_float2(acc[mt][nt][0], acc[mt][nt][1]);
              *reinterpret_cast<float2*>(&p[g + 8][2 * c]) = make_float2(acc[mt][nt][2], acc[mt][nt][3]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[mt][nt][k] = 0;
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.rfull[up_team][buf]);
      if (a.team == 1 || unit.n % a.team == up_w) {
        const bool shared = unit.entry < su;
        const uint32_t en = sh.up[unit.entry];
        const int i0 = unit.block * 16 + g, start = entry_start(en), m = entry_n(en);
        // lane 4g + c holds rows g and g + 8 for tokens 2c and 2c + 1
        float scale[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
        if constexpr (WF == MOE_W_INT8_ROW) {
          const size_t row = (shared ? 0 : (size_t)entry_e(en) * a.I) + i0;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) scale[mt][r] = __ldg((shared ? a.ss[mt] : a.s[mt]) + row + 8 * r);
        }
        float unit_x[2] = {1.f, 1.f};
        size_t to[2];  // where the two tokens' h go
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = min(2 * c + i, m - 1);
          if constexpr (R::kDigits)
            unit_x[i] = a.units[shared ? start + j : sh.pair[start + j] >> 9] * (F::kInt4 ? 0.0625f : 1.f);
          to[i] = (shared ? (size_t)P * a.I + (size_t)(start + j) * a.Is : (size_t)(sh.pair[start + j] & 511) * a.I) + i0;
        }
        few_wait(&sh.rfull[up_team][buf], parity, dead, a.flags);
        float sum[2][4] = {};
        int s = from;
#pragma unroll 4
        for (int i = 0; i < shares; ++i, s = s + 1 == a.team ? 0 : s + 1) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float(&p)[16][8] = sh.part[buf][up_team * a.team + s][mt];
            const float2 r0 = *reinterpret_cast<const float2*>(&p[g][2 * c]), r8 = *reinterpret_cast<const float2*>(&p[g + 8][2 * c]);
            sum[mt][0] += r0.x, sum[mt][1] += r0.y, sum[mt][2] += r8.x, sum[mt][3] += r8.y;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.rempty[up_team][buf]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (2 * c + (k & 1) >= m) continue;
          const float gate = sum[0][k] * unit_x[k & 1] * scale[0][k >> 1], up = sum[1][k] * unit_x[k & 1] * scale[1][k >> 1];
          const float h = (a.act == MOE_ACT_SILU ? silu_mul(gate, up) : gelu_tanh_mul(gate, up)) * R::kHScale;
          const uint16_t hi = f32_to_bf16(h);
          const float rest = h - bf16_to_f32(hi);
          uint16_t* at = a.h2 + to[k & 1] + 8 * (k >> 1);
          at[0] = hi;
          at[a.plane] = isfinite(rest) ? f32_to_bf16(rest) : (uint16_t)0;
        }
      }
      ++events;
      step_unit(unit);
    };
    UpWalk at = first_unit(list, up_w);
    seek_up(at);
    // the lane's token columns: bf16, or a digit of each tile's token
    using Columns = std::conditional_t<R::kDigits, stream::Digits<WF>, stream::Bf16Columns<WF>>;
    Columns x[R::kUpTiles] = {}, x_next[R::kUpTiles] = {};
    const char* tok[R::kUpTiles] = {};  // of the unit at `at`
    int tiles = 1, tiles_next = 1;
    size_t row = 0;                     // int4: row of the block scales
    auto unit_of = [&] {
      const uint32_t en = sh.up[at.entry];
      const int m = entry_n(en);
      tiles_next = R::kDigits ? (m + stream::kDigitTokens - 1) / stream::kDigitTokens : 1;
#pragma unroll
      for (int nt = 0; nt < R::kUpTiles; ++nt) {
        // columns past the tokens are not used
        const int j = entry_start(en) + min(R::kDigits ? stream::kDigitTokens * nt + g / 4 : g, m - 1);
        const int t = at.entry < su ? j : sh.pair[j] >> 9;
        if constexpr (R::kDigits)
          tok[nt] = reinterpret_cast<const char*>(a.digits) + ((size_t)t * 4 + (g & 3)) * stream::digit_pitch(a.H);
        else
          tok[nt] = reinterpret_cast<const char*>(static_cast<const uint16_t*>(a.x) + (size_t)t * a.H);
      }
      if constexpr (F::kInt4) row = (at.entry < su ? 0 : (size_t)entry_e(en) * a.I) + at.block * 16 + g;
    };
    auto fetch = [&] {
#pragma unroll
      for (int nt = 0; nt < R::kUpTiles; ++nt) {
        if (nt >= tiles_next) break;
        if constexpr (R::kDigits)
          stream::load_digits<WF>(reinterpret_cast<const int8_t*>(tok[nt]) + at.j * F::kBoxCols, x_next[nt]);
        else
          stream::load_token<WF>(reinterpret_cast<const uint16_t*>(tok[nt]) + at.j * F::kBoxCols, a.H - at.j * F::kBoxCols,
                                 x_next[nt].v);
      }
    };
    if (at.entry < n_up) {
      unit_of();
      fetch();
    }
#pragma unroll 1
    for (;;) {
      const bool more = at.entry < n_up;
      while (more ? unit.n < at.n : unit.entry < n_up) hand_over();
      if (!more) break;
      tiles = tiles_next;
      x[0] = x_next[0];
#pragma unroll
      for (int nt = 1; nt < R::kUpTiles; ++nt)
        if (nt < tiles) x[nt] = x_next[nt];
      const uint32_t stage = smem_u32(ring + out_slot * R::kStage);
      stream::Scales sc[2];
      if constexpr (F::kInt4) {
        const bool shared = at.entry < su;
        const size_t pitch = (size_t)(a.H >> F::kScaleShift);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          sc[mt].box = stage + 2 * stream::kBoxBytes + mt * F::kScaleBox;
          sc[mt].in_box = a.boxed[shared ? 2 : 0];
          sc[mt].left = a.H - at.j * F::kBoxCols;
          if (!sc[mt].in_box) {
            sc[mt].s0 = (shared ? a.ss[mt] : a.s[mt]) + row * pitch + (at.j * F::kBoxCols >> F::kScaleShift);
            sc[mt].s8 = sc[mt].s0 + 8 * pitch;
          }
        }
      }
      at.j += a.team;
      if (at.j >= boxes_h) {
        seek_up(at);
        if (at.entry < n_up) unit_of();
      }
      if (at.entry < n_up) fetch();
      landed();
      if constexpr (R::kDigits) {
        stream::mac_box_digits<WF, 2, R::kUpTiles>(stage, tiles, x, sc, acc);
      } else {
        float(&sums)[2][4] = reinterpret_cast<float(&)[2][4]>(acc);
        stream::mac_box<WF, 2>(stage, x[0].v, sc, sums);
      }
      read();
    }
    if (threadIdx.x == 0) sh.lists[n_lists] = (uint16_t)list;
    ++n_lists;
    list = -1;
    if (!all) {
      if (threadIdx.x == 0) {
        int b = 0;
        while (b < grid && (*reinterpret_cast<volatile uint32_t*>(&a.counters[kFewOwner + b]) != 0 ||
                            atomicExch(&a.counters[kFewOwner + b], 1u) != 0))
          ++b;
        if (b < grid) atomicAdd(&a.counters[kFewTakenOver], 1u);
        sh.adopted = b < grid ? b : -1;
      }
      __syncthreads();
      list = sh.adopted;
      __syncthreads();
      if (list >= 0) {
        head = first_unit(list, up_w);
        seek_up(head);
        fill(0);
      }
    }
  }
  // ---------------------------------------------------------------- every h is stored
  __syncthreads();
  if (n_lists == 0) {
    // taken over: the copies that were started have to land first
    for (; done < issued; ++done) {
      mbar_wait(&sh.full[w][out_slot], phase);
      if (++out_slot == R::kStages) out_slot = 0, phase ^= 1u;
    }
    return;
  }
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&a.counters[kFewDone], (uint32_t)n_lists);
  }
  // while the grid finishes: the weights, empty sums, and where the down entries' tokens lie
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = my_t + i * kWarps;
    if (t >= a.T) break;
    const float wt = few_weight(a, t, my_e[i]);
    if (lane < a.k) sh.pair_w[t * a.k + lane] = wt;
    bool first = blockIdx.x == 0;  // the owner of the first list writes the routing out
    for (int j = 1; j < n_lists; ++j) first |= sh.lists[j] == 0;
    if (first) few_write_route(a, t, my_e[i], wt);
  }
  for (int i = lane; i < a.T * 16; i += 32) (&sh.y[w][0][0])[i] = 0.f;
  for (int i = threadIdx.x; i < n_down * kDownTokens; i += kStreamThreads) {
    const uint32_t en = sh.down[i / kDownTokens];
    const int j = entry_start(en) + min(i % kDownTokens, entry_n(en) - 1);  // columns past the tokens are not used
    sh.at[i / kDownTokens][i % kDownTokens] =
        entry_e(en) == kSharedEntry ? (uint32_t)P * a.I + (uint32_t)j * a.Is : (uint32_t)(sh.pair[j] & 511) * a.I;
  }
  if (threadIdx.x == 0) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(&a.counters[kFewDone]) : "memory");
      if (v >= (uint32_t)grid) break;
      if (dead || global_timer_ns() - t0 > kWaitLimitNs) {
        if (!dead) raise_flag(a.flags, MOE_FLAG_TIMEOUT);
        dead = true;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();

  // ---------------------------------------------------------------- down and combine
  constexpr int DB = R::kDownBoxes;
  uint4 x[DB][F::kLoads];
  // the warp's next stage: of which entry and where in it; the entry's reduction length, the lane's
  // token (value or remainder)
  uint32_t stage_at = 0, en = 0;
  int K = 0;
  const uint16_t* const h_lane = a.h2 + (g < 4 ? 0 : a.plane);
  float s_row = 1.f;      // int8: scale of the row whose sums the lane will hold
  const float* s0 = nullptr;  // int4, scales not copied: block scales of row g
  bool boxed = false;
  auto fetch = [&](int n) {
    stage_at = __shfl_sync(0xFFFFFFFFu, win, n & 31);
    const int blk = __shfl_sync(0xFFFFFFFFu, win_blk, n & 31);
    en = sh.down[stage_at >> 16];
    const bool shared = entry_e(en) == kSharedEntry;
    K = shared ? a.Is : a.I;
    boxed = F::kScaleBoxes && a.boxed[shared ? 3 : 1];
    const int c0 = (int)(stage_at & 0xFFFFu) * DB * F::kBoxCols, left = K - c0;
    const uint16_t* tok = h_lane + (sh.at[stage_at >> 16][g & 3] + c0);
#pragma unroll
    for (int d = 0; d < DB; ++d)
      if (d == 0 || left > d * F::kBoxCols)
        stream::load_token<WF>(tok + d * F::kBoxCols, left - d * F::kBoxCols, x[d]);
    if constexpr (WF == MOE_W_INT8_ROW) {
      const int row = (shared ? 0 : (int)entry_e(en) * a.H) + blk * 16 + g;
      s_row = __ldg((shared ? a.ss[2] : a.s[2]) + row + (c < 2 ? 0 : 8));
    }
    if constexpr (F::kInt4) {
      if (!boxed) {
        const size_t row = (shared ? 0 : (size_t)entry_e(en) * a.H) + blk * 16 + g;
        s0 = (shared ? a.ss[2] : a.s[2]) + row * (size_t)(K >> F::kScaleShift);
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < n_lists; ++i) {
    if (!all || i > 0) {
      first_down(sh.lists[i]);
      head_down = 0;
      fill(0);
    }
    if (n_stages > 0) fetch(0);
    int n = 0;
    for (int blk = sh.lists[i]; blk < hb; blk += grid) {
      float acc[1][4] = {};
#pragma unroll 1
      for (int r = 0; r < per_blk; ++r) {
        const uint32_t stage = smem_u32(ring + out_slot * R::kStage);
        const int c0 = (int)(stage_at & 0xFFFFu) * DB * F::kBoxCols, left = K - c0;
        stream::Scales sc[DB][1];
        if constexpr (F::kInt4) {
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            sc[d][0].box = stage + 2 * stream::kBoxBytes + d * F::kScaleBox;
            sc[d][0].in_box = boxed;
            sc[d][0].left = left - d * F::kBoxCols;
            if (!boxed) {
              sc[d][0].s0 = s0 + (c0 + d * F::kBoxCols >> F::kScaleShift);
              sc[d][0].s8 = sc[d][0].s0 + 8 * (size_t)(K >> F::kScaleShift);
            }
          }
        }
        landed();
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          if (d > 0 && left <= d * F::kBoxCols) break;
          stream::mac_box<WF, 1>(stage + d * stream::kBoxBytes, x[d], sc[d], acc);
        }
        // the next stage's tokens, of the same entry or of the next
        const uint32_t now = en, x_now = stage_at >> 16;
        const float s_now = s_row;
        if ((++n & 15) == 0) window(n);
        if (n < n_stages) fetch(n);
        read();
        if (r + 1 < per_blk && stage_at >> 16 == x_now) continue;
        // the entry's sums, weighted, to this warp's share of y
        const bool shared = entry_e(now) == kSharedEntry;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = acc[0][k] + __shfl_xor_sync(0xFFFFFFFFu, acc[0][k], 2);
          acc[0][k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 2 * (c & 1) + k;
          if (j >= entry_n(now)) continue;
          const int p = sh.pair[shared ? 0 : entry_start(now) + j];
          const int to = shared ? entry_start(now) + j : p >> 9;
          const float wt = (shared ? 1.f : sh.pair_w[p & 511]) * s_now * (1.f / R::kHScale);
          sh.y[w][to][c < 2 ? g : g + 8] += wt * (c < 2 ? v[k] : v[2 + k]);
        }
        __syncwarp();
      }
      __syncthreads();
      for (int i = threadIdx.x; i < a.T * 16; i += kStreamThreads) {
        const int t = i >> 4, r = i & 15;
        const size_t to = (size_t)t * a.H + blk * 16 + r;
        float y = 0.f;
#pragma unroll
        for (int s = 0; s < kWarps; ++s) {
          y += sh.y[s][t][r];
          sh.y[s][t][r] = 0.f;
        }
        if (a.residual) y += bf16_to_f32(static_cast<const uint16_t*>(a.residual)[to]);
        static_cast<uint16_t*>(a.y)[to] = f32_to_bf16(y);
      }
      __syncthreads();
    }
  }
  // after a wait that ran out: leave only when the copies have landed
  if (dead) {
    for (; done < issued; ++done) {
      mbar_wait(&sh.full[w][out_slot], phase);
      if (++out_slot == R::kStages) out_slot = 0, phase ^= 1u;
    }
  }
}

// bf16 tokens on quantised weights: the gate/up products are integer ones
bool few_digits(const moe_desc& d) { return d.xfmt == MOE_X_BF16 && d.wfmt >= MOE_W_INT8_ROW; }

struct FewLayout {
  size_t keys, scores, digits, units, h, total;
};
FewLayout few_layout(const moe_desc& d, int Is, int T) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FewLayout l;
  l.keys = up(kFewCounters * sizeof(uint32_t));
  l.scores = l.keys + up((size_t)T * d.E * 8);
  l.digits = l.scores + up((size_t)T * d.E * 8);
  l.units = l.digits + (few_digits(d) ? up((size_t)T * 4 * stream::digit_pitch(d.H)) : 0);
  l.h = l.units + up((size_t)T * 4);
  l.total = l.h + up(((size_t)T * d.k * d.I + (size_t)T * Is) * 4);
  return l;
}

template <int WF>
cudaError_t weight_maps(CUtensorMap* w, CUtensorMap* sc, const void* W, const float* s, uint64_t rows, int K, bool boxed) {
  using F = stream::Format<WF>;
  const uint64_t bytes = (uint64_t)K * F::kBits / 8;
  cudaError_t e = make_tmap(w, W, CU_TENSOR_MAP_DATA_TYPE_UINT8, bytes, rows, bytes, 128, stream::kBoxRows,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess && boxed)
    e = make_tmap(sc, s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (uint64_t)(K / 32), rows, (uint64_t)(K / 32) * 4, 8,
                  stream::kBoxRows, CU_TENSOR_MAP_SWIZZLE_NONE);
  return e;
}

template <int WF>
cudaError_t launch_stream(FewArgs a, int num_sms, cudaStream_t s) {
  constexpr size_t smem = 1024 + sizeof(StreamShared) + (size_t)Ring<WF>::kBytes;
  static_assert(smem <= 232448, "the rings do not fit in shared memory");
  // Sharing a unit out costs each warp some hundred instructions of hand-over, which counts where
  // instructions bound the stream; where the units are few, smaller teams leave warps without
  // work in the last round.  Measured by events after a flush of L2 (teams of 12, 3, 1): 1 token bf16
  // 68, 68, 70 us and int4 33, 31, 41 us; 4 tokens int8 129, 117, 128 us; 16 tokens int8 298, 242,
  // 251 us and int4 135, 109, 121 us.  Down teams of 12, 3, 1: 1 token bf16 68, 70, 70 us, 16 tokens
  // int8 250, 242, 242 us, all others within 1%.
  // The tokens' experts are not known here: expect them to differ.
  const int touched = std::min(a.T * a.k, a.E);
  a.team = (int64_t)touched * (a.I / 16) >= 4LL * 4 * num_sms ? 3 : kWarps;
  a.down_team = touched >= 2 * kWarps ? 3 : kWarps;
  FewMaps m;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
    const int rows = i < 2 ? a.I : a.H, K = i < 2 ? a.H : a.I;
    e = weight_maps<WF>(&m.w[i], &m.s[i], a.W[i], a.s[i], (uint64_t)a.E * rows, K, a.boxed[i / 2]);
    if (e == cudaSuccess && a.Is)
      e = weight_maps<WF>(&m.ws[i], &m.ss[i], a.Ws[i], a.ss[i], (uint64_t)(i < 2 ? a.Is : a.H), i < 2 ? a.H : a.Is,
                          a.boxed[2 + i / 2]);
  }
  static std::atomic<bool> allowed[64];
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(few_stream_kernel<WF>), smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_k_after(few_stream_kernel<WF>, dim3(std::min(num_sms, kFewLists)), dim3(kStreamThreads), smem, s, m, a);
}

// The scales of a [rows, K] int4 block-32 matrix can be copied by TMA: rows of whole 16-byte
// pieces, on 16 bytes.
bool boxed_scales(int wfmt, const float* s, int K) {
  return wfmt == MOE_W_INT4_B32 && (reinterpret_cast<uintptr_t>(s) % 16) == 0 && K % 128 == 0;
}

template <int WF>
cudaError_t launch_layer(const moe_desc& d, const FewArgs& a, int num_sms, cudaStream_t s) {
  if constexpr (WF != MOE_W_F32)
    if (d.xfmt == MOE_X_BF16) return launch_stream<WF>(a, num_sms, s);
  const dim3 grid(num_sms * 4), block(kFewThreads);
  if (d.xfmt == MOE_X_F32) return launch_k_after(few_layer_kernel<WF, MOE_X_F32>, grid, block, 0, s, a);
  if constexpr (WF == MOE_W_F32) return launch_k_after(few_layer_kernel<WF, MOE_X_BF16>, grid, block, 0, s, a);
  return cudaErrorInvalidValue;  // not reached
}

}  // namespace

size_t few_workspace_bytes(const moe_desc& d, const moe_shared_expert* sh, int T) {
  return few_layout(d, sh ? sh->I : 0, T).total;
}

cudaError_t launch_few_router(const moe_desc& d, const moe_shared_expert* sh, const void* x, int T, void* workspace,
                              uint32_t* flags, cudaStream_t s) {
  const FewLayout l = few_layout(d, sh ? sh->I : 0, T);
  char* ws = static_cast<char*>(workspace);
  auto go = [&](auto kernel, int tokens) {
    const dim3 grid((d.E + kRouterExperts - 1) / kRouterExperts + (few_digits(d) ? std::min(T, tokens) : 0), (T + tokens - 1) / tokens);
    return launch_k(kernel, grid, dim3(kRouterThreads), 0, s, x, d.W_r, d.b, d.expert_mask, T, d.H, d.E, d.router,
                    reinterpret_cast<uint64_t*>(ws + l.keys), reinterpret_cast<double*>(ws + l.scores),
                    reinterpret_cast<uint32_t*>(ws), reinterpret_cast<int8_t*>(ws + l.digits),
                    (int)(d.wfmt != MOE_W_INT8_ROW), reinterpret_cast<float*>(ws + l.units), flags);
  };
  if (d.xfmt == MOE_X_F32)
    return T == 1 ? go(few_router_kernel<MOE_X_F32, 1>, 1)
                  : (T <= 4 ? go(few_router_kernel<MOE_X_F32, 4>, 4) : go(few_router_kernel<MOE_X_F32, 8>, 8));
  return T == 1 ? go(few_router_kernel<MOE_X_BF16, 1>, 1)
                : (T <= 4 ? go(few_router_kernel<MOE_X_BF16, 4>, 4) : go(few_router_kernel<MOE_X_BF16, 8>, 8));
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
  a.h2 = reinterpret_cast<uint16_t*>(ws + l.h);
  a.plane = (size_t)T * (d.k * (size_t)d.I + a.Is);
  a.boxed[0] = boxed_scales(d.wfmt, d.s_gate, d.H) && boxed_scales(d.wfmt, d.s_up, d.H);
  a.boxed[1] = boxed_scales(d.wfmt, d.s_down, d.I);
  if (sh) {
    a.boxed[2] = boxed_scales(d.wfmt, sh->s_gate, d.H) && boxed_scales(d.wfmt, sh->s_up, d.H);
    a.boxed[3] = boxed_scales(d.wfmt, sh->s_down, sh->I);
  }
  a.digits = reinterpret_cast<const int8_t*>(ws + l.digits);
  a.units = reinterpret_cast<const float*>(ws + l.units);
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
