// Dense matrix product with its epilogue fused:
//   v = s * (W x) + b,   y = act(v) [* v_up] + residual,
// in fp32 with one rounding to y's format.  Weights in the layer's storage formats.
//
// A CTA computes 64 tokens x 64 outputs from 16-column slices of x and W held in shared
// memory as fp32 (weights decoded on the way in), 4 x 4 sums per thread.
#include "common.cuh"
#include "internal.h"
#include "linear.h"

namespace moe {
namespace {

constexpr int kTile = 64;
constexpr int kSlice = 16;

// four stored weights of row r from column c on (c a multiple of 4)
template <int WF>
__device__ __forceinline__ void weights4(const void* W, const float* s, size_t r, int c, int K, float (&v)[4]) {
  if constexpr (WF == MOE_W_F32) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(W) + r * K + c));
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else if constexpr (WF == MOE_W_BF16) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(W) + r * K + c));
    v[0] = bf16_to_f32(u.x & 0xFFFFu), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = bf16_to_f32(u.y & 0xFFFFu), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else if constexpr (WF == MOE_W_INT8_ROW) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(W) + r * K + c));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(u >> (8 * j));
  } else {
    constexpr int kShift = WF == MOE_W_INT4_B32 ? 5 : 7;
    const uint32_t u = __ldg(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(W) + (r * K + c) / 2));
    const float scale = __ldg(s + r * (K >> kShift) + (c >> kShift));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)((int)(u << (28 - 4 * j)) >> 28) * scale;
  }
}

template <int WF, int XF, bool GATED>
__global__ void __launch_bounds__(256) linear_simt_kernel(const LinearArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int G = GATED ? 2 : 1;
  __shared__ float xs[kSlice][kTile + 4];
  __shared__ float ws[G][kSlice][kTile + 4];
  const int tid = threadIdx.x;
  const int n0 = blockIdx.x * kTile, m0 = blockIdx.y * kTile;
  const int tn = (tid & 15) * 4, tm = (tid >> 4) * 4;
  float acc[G][4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kSlice) {
    const int r = tid >> 2, c = (tid & 3) * 4;
    float v[4] = {};
    if (m0 + r < a.M && k0 + c < a.K) {
      const size_t at = (size_t)(m0 + r) * a.ldx + k0 + c;
      if constexpr (XF == MOE_X_F32) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + at));
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + at));
        v[0] = bf16_to_f32(u.x & 0xFFFFu), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
        v[2] = bf16_to_f32(u.y & 0xFFFFu), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) xs[c + j][r] = v[j];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float q[4] = {};
      if (n0 + r < a.N && k0 + c < a.K) weights4<WF>(a.W[g], a.s[g], (size_t)(n0 + r), k0 + c, a.K, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) ws[g][c + j][r] = q[j];
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kSlice; ++kk) {
      const float4 xv = *reinterpret_cast<const float4*>(&xs[kk][tm]);
      const float xa[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float4 wv = *reinterpret_cast<const float4*>(&ws[g][kk][tn]);
        const float wa[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[g][i][j] = fmaf(xa[i], wa[j], acc[g][i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + tn + j;
    if (n >= a.N) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + tm + i;
      if (m >= a.M) break;
      linear_finish(a, WF == MOE_W_INT8_ROW, m, n, acc[0][i][j], acc[G - 1][i][j]);
    }
  }
}

template <int WF>
cudaError_t launch_simt(const moe_linear_desc& d, const LinearArgs& a, cudaStream_t s) {
  const dim3 grid((a.N + kTile - 1) / kTile, (a.M + kTile - 1) / kTile), block(256);
  if (d.xfmt == MOE_X_F32)
    return a.W[1] ? launch_k(linear_simt_kernel<WF, MOE_X_F32, true>, grid, block, 0, s, a)
                  : launch_k(linear_simt_kernel<WF, MOE_X_F32, false>, grid, block, 0, s, a);
  return a.W[1] ? launch_k(linear_simt_kernel<WF, MOE_X_BF16, true>, grid, block, 0, s, a)
                : launch_k(linear_simt_kernel<WF, MOE_X_BF16, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_linear_simt(const moe_linear_desc& d, const LinearArgs& a, cudaStream_t s) {
  switch (d.wfmt) {
    case MOE_W_F32: return launch_simt<MOE_W_F32>(d, a, s);
    case MOE_W_BF16: return launch_simt<MOE_W_BF16>(d, a, s);
    case MOE_W_INT8_ROW: return launch_simt<MOE_W_INT8_ROW>(d, a, s);
    case MOE_W_INT4_B32: return launch_simt<MOE_W_INT4_B32>(d, a, s);
    default: return launch_simt<MOE_W_INT4_B128>(d, a, s);
  }
}

}  // namespace moe
