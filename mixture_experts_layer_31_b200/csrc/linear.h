// Shared by the kernels of the dense product (moe_linear).
#pragma once
#include "common.cuh"

namespace moe {

struct LinearArgs {
  int M, N, K;
  int act, yfmt;
  const void* x;
  long long ldx;
  const void* W[2];  // W, W_up (NULL: not gated)
  const float* s[2];
  const float* b[2];
  const void* residual;
  long long ldr;
  void* y;
  long long ldy;
};

// Up to this many bf16 tokens the weights stream through warp-wide matrix instructions; beyond, the
// tensor cores take them, quantised ones after a pass that widens them.  The stream costs more
// for every tile of 8 tokens, the more so the more weights there are; the tensor cores have a
// fixed cost of some 17 us (two launches, few units) and the widening pass.  Measured, stream and
// tensor cores, in us:
//   bf16   9216 x 2304, 32 tokens 17, 20;  2304 x 18432, 24 tokens 30, 29, 32 tokens 34, 24
//   int8   9216 x 2304, 64 tokens 29, 37;  2304 x (9216 + 9216), 48 tokens 49, 52, 64 tokens 62, 54
//   int4   2304 x (9216 + 9216), 40 tokens 46, 52;  2048 x 4999, 32 tokens 15, 23, 48 tokens 25, 23;
//          9216 x 2304, 48 tokens 25, 36, 64 tokens 40, 38
// Ten more shapes from 1024 x 1024 to 768 x 16384 and 16384 x 1024 (by events after a flush of L2, 4 us
// more than the above): the rule takes the faster form or one within 15% on square ones; short or long
// reductions cross over sooner.  The worst: 768 x 16384, bf16 32 tokens 25, 17, int8 48 tokens 37, 27,
// int4 40 tokens 41, 23; 16384 x 1024, bf16 32 tokens 31, 23, int8 64 tokens 47, 31, int4 48 tokens 62, 30.
inline int linear_stream_tokens(const moe_linear_desc& d) {
  const bool large = (int64_t)d.N * d.K * (d.W_up ? 2 : 1) > 32 << 20;
  if (d.wfmt == MOE_W_INT8_ROW) return large ? 48 : 64;
  if (d.wfmt == MOE_W_BF16) return large ? 24 : 32;
  return d.K > 4096 ? 48 : 40;
}

__device__ __forceinline__ float linear_act(float v, int act) {
  if (act == MOE_ACT_SILU) return silu_mul(v, 1.f);
  if (act == MOE_ACT_GELU_TANH) return gelu_tanh_mul(v, 1.f);
  return v;
}

// y[m, n] from the sums of W (v) and W_up (u): row scales of int8 weights, bias, activation,
// gate, residual, one rounding.  The residual's element is read before y's is written.
__device__ __forceinline__ void linear_finish(const LinearArgs& a, bool row_scales, int m, int n, float v, float u) {
  if (row_scales) v *= __ldg(a.s[0] + n);
  if (a.b[0]) v += __ldg(a.b[0] + n);
  float y = linear_act(v, a.act);
  if (a.W[1]) {
    if (row_scales) u *= __ldg(a.s[1] + n);
    if (a.b[1]) u += __ldg(a.b[1] + n);
    y *= u;
  }
  if (a.yfmt == MOE_X_F32) {
    if (a.residual) y += static_cast<const float*>(a.residual)[(size_t)m * a.ldr + n];
    static_cast<float*>(a.y)[(size_t)m * a.ldy + n] = y;
  } else {
    if (a.residual) y += bf16_to_f32(static_cast<const uint16_t*>(a.residual)[(size_t)m * a.ldr + n]);
    static_cast<uint16_t*>(a.y)[(size_t)m * a.ldy + n] = f32_to_bf16(y);
  }
}

// 8 stored weights of row r from column c on (c a multiple of 8, or of 4 with 4 columns left)
template <int WF>
__device__ __forceinline__ void weights8(const void* W, const float* s, size_t r, int c, int K, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if constexpr (WF == MOE_W_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + r * K + c);
    const float4 a = __ldg(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    if (c + 4 < K) {
      const float4 b = __ldg(p + 1);
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else if constexpr (WF == MOE_W_BF16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + r * K + c));
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_to_f32(word[j] & 0xFFFFu), v[2 * j + 1] = __uint_as_float(word[j] & 0xFFFF0000u);
  } else if constexpr (WF == MOE_W_INT8_ROW) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(W) + r * K + c));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
  } else {
    constexpr int kShift = WF == MOE_W_INT4_B32 ? 5 : 7;
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(W) + (r * K + c) / 2));
    const float scale = __ldg(s + r * (K >> kShift) + (c >> kShift));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((int)(u << (28 - 4 * j)) >> 28) * scale;
  }
}

// 8 columns of a token
template <int XF>
__device__ __forceinline__ void token8(const void* x, size_t at, bool all, float (&v)[8]) {
  if constexpr (XF == MOE_X_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(p), b = all ? __ldg(p + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_to_f32(word[j] & 0xFFFFu), v[2 * j + 1] = __uint_as_float(word[j] & 0xFFFF0000u);
  }
}

bool linear_stream_ok(const moe_linear_desc& d, int M);
bool linear_stream_digits(const moe_linear_desc& d, int M);        // the tokens are taken as digits
bool linear_stream_digits_first(const moe_linear_desc& d, int M);  // which a launch before it makes
size_t linear_stream_workspace(const moe_linear_desc& d, int M);
cudaError_t launch_linear_digits(const moe_linear_desc& d, const LinearArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_linear_stream(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, uint32_t* flags,
                                 cudaStream_t s);
// fp32 tokens or weights: up to this many tokens a warp computes rows of W in fp32
constexpr int kLinearRowTokens = 16;
cudaError_t launch_linear_rows(const moe_linear_desc& d, const LinearArgs& a, int num_sms, cudaStream_t s);
// beyond that, tensor cores: quantised and fp32 weights and fp32 tokens are first widened into bf16
// (parts) in the workspace, by one launch; where linear_tc_split() a last launch adds up the
// parts of the reduction
bool linear_tc_ok(const moe_linear_desc& d, int M);
size_t linear_tc_workspace(const moe_linear_desc& d, int M);
bool linear_tc_split(const moe_linear_desc& d, int M);
bool linear_tc_layouts(const moe_linear_desc& d);  // a launch that lays operands out comes first
cudaError_t launch_linear_layouts(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, cudaStream_t s);
cudaError_t launch_linear_tc(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, uint32_t* flags,
                             cudaStream_t s);
cudaError_t launch_linear_sum(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, cudaStream_t s);

}  // namespace moe
