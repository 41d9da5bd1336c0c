// The dense product in fp32 multiply-adds for a few tokens, where tokens or weights are fp32:
// a warp takes R rows of W, its lanes 8 columns in turn, for TT tokens at a time.  The
// weights' way from HBM bounds it; R rows share a token's columns, without which the
// tokens' way from L1 would (16 tokens: 512 bytes of tokens for 32 of weights).  Measured,
// 2,304 x 2,304 fp32 (3.2 us at the copy rate): 1 token 12 us, 5 tokens 13, 16 tokens 25, where the
// tensor cores' three launches take 31.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "linear.h"

namespace moe {
namespace {

constexpr int kThreads = 128;

// R rows of W, or R / 2 rows of W and the same of W_up
template <int WF, int XF, int R, int TT, bool GATED>
__global__ void __launch_bounds__(kThreads) linear_rows_kernel(const __grid_constant__ LinearArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kOut = GATED ? R / 2 : R;
  const int lane = lane_id();
  const int n0 = (blockIdx.x * (kThreads / 32) + warp_id()) * kOut;
  if (n0 >= a.N) return;
  for (int m0 = 0; m0 < a.M; m0 += TT) {
    float acc[R][TT] = {};
    for (int c = lane * 8; c < a.K; c += 256) {
      float w[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int side = GATED ? r & 1 : 0;
        weights8<WF>(a.W[side], a.s[side], (size_t)min(n0 + (GATED ? r >> 1 : r), a.N - 1), c, a.K, w[r]);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float x[8];
        token8<XF>(a.x, (size_t)min(m0 + t, a.M - 1) * a.ldx + c, c + 4 < a.K, x);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[r][t] = fmaf(w[r][j], x[j], acc[r][t]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc[r][t] += __shfl_xor_sync(0xFFFFFFFFu, acc[r][t], off);
    // lane o finishes output o / TT of token o % TT
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int o = 0; o < kOut; ++o)
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (lane == o * TT + t) v = acc[GATED ? 2 * o : o][t], u = GATED ? acc[2 * o + (R > 1)][t] : 0.f;
    const int n = n0 + lane / TT, m = m0 + lane % TT;
    if (lane < kOut * TT && n < a.N && m < a.M) linear_finish(a, WF == MOE_W_INT8_ROW, m, n, v, u);
  }
}

template <int WF, int XF>
cudaError_t launch(const LinearArgs& a, int num_sms, cudaStream_t s) {
  const bool gated = a.W[1] != nullptr;
  auto go = [&](auto kernel, int out) {
    const int per = kThreads / 32 * out;
    return launch_k(kernel, dim3((a.N + per - 1) / per), dim3(kThreads), 0, s, a);
  };
  // four rows a warp where they leave 16 warps for every SM
  const bool four = a.N >= 16 * 4 * num_sms;
  if (a.M == 1) {
    if (gated) return go(linear_rows_kernel<WF, XF, 2, 1, true>, 1);
    return four ? go(linear_rows_kernel<WF, XF, 4, 1, false>, 4) : go(linear_rows_kernel<WF, XF, 1, 1, false>, 1);
  }
  if (gated) return go(linear_rows_kernel<WF, XF, 4, 8, true>, 2);
  return four ? go(linear_rows_kernel<WF, XF, 4, 8, false>, 4) : go(linear_rows_kernel<WF, XF, 2, 8, false>, 2);
}

template <int WF>
cudaError_t launch(const moe_linear_desc& d, const LinearArgs& a, int num_sms, cudaStream_t s) {
  if (d.xfmt == MOE_X_F32) return launch<WF, MOE_X_F32>(a, num_sms, s);
  if constexpr (WF == MOE_W_F32) return launch<WF, MOE_X_BF16>(a, num_sms, s);
  return cudaErrorInvalidValue;  // not reached: bf16 tokens on other weights stream
}

}  // namespace

cudaError_t launch_linear_rows(const moe_linear_desc& d, const LinearArgs& a, int num_sms, cudaStream_t s) {
  switch (d.wfmt) {
    case MOE_W_F32: return launch<MOE_W_F32>(d, a, num_sms, s);
    case MOE_W_BF16: return launch<MOE_W_BF16>(d, a, num_sms, s);
    case MOE_W_INT8_ROW: return launch<MOE_W_INT8_ROW>(d, a, num_sms, s);
    case MOE_W_INT4_B32: return launch<MOE_W_INT4_B32>(d, a, num_sms, s);
    default: return launch<MOE_W_INT4_B128>(d, a, num_sms, s);
  }
}

}  // namespace moe
