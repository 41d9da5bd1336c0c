// The dense product for a few tokens (up to 64): a stream of stored weights through warp-wide
// matrix instructions (stream_dev.cuh).
//
// What bounds it is the weights' way from HBM.  A CTA takes units of 16 rows of W (32 where there
// are rows enough, or 16 of W and the same 16 of W_up), and its twelve warps share the
// reduction box by box (16 rows x 128 bytes), each with a ring of its own that TMA fills
// stages ahead, across units.  Their sums meet in shared memory, where bias, activation,
// gate and residual are applied.  A few tokens meet quantised weights as digits, made by every
// CTA for itself where they are small, else by a launch before this one, in both cases
// while the first weights are already on their way; beyond that every weight is widened
// once for all tokens.  The tokens' columns come from L1 and L2.
//
// Measured, 8 tokens, bf16, 9,216 columns, 2,304 outputs: 14.4 us cold for 42 MB, 45% of the copy rate
// (6.5 us): the launch, the first loads' latency and the last sums are as long as the stream.
// One token, int8, 2,304 columns, 9,216 gated outputs: 17 us with its digits made in place, again
// 42 MB.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "linear.h"
#include "stream_dev.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxStages = 4;
constexpr int kSmem = 232448;

struct StreamMaps {
  CUtensorMap w[2], s[2];  // W and W_up; their int4 block-32 scales, where `boxed`
};

struct StreamLinear {
  LinearArgs l;
  int boxed;
  const int8_t* digits;  // [M][4][digit_pitch(K)], and the tokens' units
  const float* units;
  int local;             // the digits are made here
};

// one token per CTA
__global__ void __launch_bounds__(256) linear_digits_kernel(const __grid_constant__ LinearArgs a, int int4, int8_t* digits,
                                                            float* units) {
  pdl_wait();
  pdl_trigger();
  __shared__ float warps[8];
  const int t = blockIdx.x;
  stream::write_digits(static_cast<const uint16_t*>(a.x) + (size_t)t * a.ldx, a.K, int4,
                       digits + (size_t)t * 4 * stream::digit_pitch(a.K), units + t, warps);
}

// NT: tiles of 8 tokens; DIG: of 2 tokens as digits
constexpr int kLocal = 16384;  // bytes of digits that a CTA makes for itself

template <int WF, int MT, int NT, bool DIG>
struct Plan {
  using F = stream::Format<WF>;
  static constexpr int kDigits = DIG && NT == 1 ? kLocal + 256 : 0;
  static constexpr int kStage = MT * (stream::kBoxBytes + F::kScaleBox);
  static constexpr int kStride = (kStage + 1023) / 1024 * 1024;
  static constexpr int kPart = kWarps * MT * NT * 32 * 16;  // bytes of the warps' sums
  static constexpr int kFit = (kSmem - 1024 - 512 - kPart - kDigits) / (kWarps * kStride);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kBytes = 1024 + kWarps * kStages * kStride + kPart + 512 + kDigits;
  static_assert(kStages >= 2 && kWarps * kMaxStages * 8 <= 512, "shared memory");
};

template <int WF, int MT, int NT, bool DIG>
__global__ void __launch_bounds__(kThreads, 1)
    linear_stream_kernel(const __grid_constant__ StreamMaps maps, const __grid_constant__ StreamLinear p, uint32_t* flags) {
  using P = Plan<WF, MT, NT, DIG>;
  using F = stream::Format<WF>;
  extern __shared__ uint8_t smem[];
  uint8_t* rings = smem + (((smem_u32(smem) + 1023u) & ~1023u) - smem_u32(smem));
  float* part = reinterpret_cast<float*>(rings + kWarps * P::kStages * P::kStride);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(part) + P::kPart);
  const LinearArgs& a = p.l;
  const int w = warp_id(), lane = lane_id(), g = lane >> 2, c = lane & 3;
  uint8_t* ring = rings + w * P::kStages * P::kStride;
  uint64_t* bars = full + w * kMaxStages;
  if (lane == 0) {
    for (int i = 0; i < P::kStages; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
    if (w == 0) prefetch_tmap(&maps.w[0]);
  }
  __syncwarp();

  const bool gated = a.W[1] != nullptr;
  const int rows = gated ? 16 : 16 * MT;  // output columns of a unit
  const int units = (a.N + rows - 1) / rows, boxes = (a.K + F::kBoxCols - 1) / F::kBoxCols, grid = (int)gridDim.x;
  const int ntiles = DIG ? (a.M + stream::kDigitTokens - 1) / stream::kDigitTokens : (a.M + 7) / 8;
  bool dead = false;

  struct Walk {
    int u, j;
  };
  auto seek = [&](Walk& k) {
    while (k.j >= boxes) k.j -= boxes, k.u += grid;
  };
  int issued = 0, in_slot = 0, done = 0, out_slot = 0;
  uint32_t phase = 0;
  Walk head = {(int)blockIdx.x, w};
  seek(head);
  auto issue = [&] {
    if (head.u >= units) return;
    if (lane == 0 && !dead) {
      uint8_t* stage = ring + in_slot * P::kStride;
      uint64_t* bar = &bars[in_slot];
      mbar_arrive_expect_tx(bar, MT * (stream::kBoxBytes + (p.boxed ? F::kScaleBox : 0)));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int m = gated ? mt : 0, row = head.u * rows + (gated ? 0 : 16 * mt);
        tma_load_2d(stage + mt * stream::kBoxBytes, &maps.w[m], head.j * 128, row, bar);
        if (F::kScaleBoxes && p.boxed)
          tma_load_2d(stage + MT * stream::kBoxBytes + mt * F::kScaleBox, &maps.s[m], head.j * 8, row, bar);
      }
    }
    ++issued;
    in_slot = in_slot + 1 == P::kStages ? 0 : in_slot + 1;
    head.j += kWarps;
    seek(head);
  };
  // The digits' launch writes no weights, so their copies start before its end is waited for; the
  // launches before that one are over, as it lets this one start only after its own wait.
  const bool after = DIG && !p.local;
  if (!after) pdl_wait();
  for (int i = 0; i < P::kStages; ++i) issue();
  if (after) pdl_wait();
  pdl_trigger();

  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  Walk at = {(int)blockIdx.x, w};
  seek(at);
  using Sum = std::conditional_t<DIG, stream::DigitSum<WF>, float>;
  stream::Digits<WF> dx[DIG ? NT : 1] = {}, dx_next[DIG ? NT : 1] = {};
  const int8_t* drow[DIG ? NT : 1];
  const float* units_x = p.units;
  auto fetch_digits = [&] {
#pragma unroll
    for (int nt = 0; nt < (DIG ? NT : 1); ++nt)
      if (nt < ntiles) stream::load_digits<WF>(drow[nt] + at.j * F::kBoxCols, dx_next[nt]);
  };
  if constexpr (DIG) {
    const int8_t* digits = p.digits;
    if constexpr (P::kDigits > 0) {
      uint8_t* here = reinterpret_cast<uint8_t*>(full) + 512;  // after the barriers
      if (p.local) {
        units_x = reinterpret_cast<float*>(here + kLocal);
        for (int t = 0; t < a.M; ++t)
          stream::write_digits(x + (size_t)t * a.ldx, a.K, F::kInt4,
                               reinterpret_cast<int8_t*>(here) + (size_t)t * 4 * stream::digit_pitch(a.K),
                               reinterpret_cast<float*>(here + kLocal) + t, reinterpret_cast<float*>(here + kLocal + 64));
        digits = reinterpret_cast<const int8_t*>(here);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      drow[nt] = digits + ((size_t)min(stream::kDigitTokens * nt + g / 4, a.M - 1) * 4 + (g & 3)) * stream::digit_pitch(a.K);
    if (at.u < units) fetch_digits();
  }
  uint4 x_next[F::kLoads];
  const uint16_t* tok = x + (size_t)min(g, a.M - 1) * a.ldx;  // columns past the tokens are not used
  if (!DIG && NT == 1 && at.u < units)
    stream::load_token<WF>(tok + at.j * F::kBoxCols, a.K - at.j * F::kBoxCols, x_next);
  for (int u = (int)blockIdx.x; u < units; u += grid) {
    Sum acc[MT][NT][4] = {};
#pragma unroll 1
    while (at.u == u) {
      const int c0 = at.j * F::kBoxCols, left = a.K - c0;
      const uint32_t stage = smem_u32(ring + out_slot * P::kStride);
      stream::Scales sc[MT];
      if constexpr (F::kInt4) {
        const size_t pitch = (size_t)(a.K >> F::kScaleShift);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // rows past the last are zero weights: any scale that can be read does
          const int r = u * rows + (gated ? 0 : 16 * mt) + g;
          const float* s = a.s[gated ? mt : 0] + (c0 >> F::kScaleShift);
          sc[mt].box = stage + MT * stream::kBoxBytes + mt * F::kScaleBox;
          sc[mt].in_box = p.boxed;
          sc[mt].left = left;
          if (!p.boxed) {
            sc[mt].s0 = s + (size_t)min(r, a.N - 1) * pitch;
            sc[mt].s8 = s + (size_t)min(r + 8, a.N - 1) * pitch;
          }
        }
      }
      uint4 x_now[F::kLoads];
      if constexpr (DIG) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (nt < ntiles) dx[nt] = dx_next[nt];
      } else if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < F::kLoads; ++i) x_now[i] = x_next[i];
      }
      at.j += kWarps;
      seek(at);
      if constexpr (DIG) {
        if (at.u < units) fetch_digits();
      } else if (NT == 1 && at.u < units) {
        stream::load_token<WF>(tok + at.j * F::kBoxCols, a.K - at.j * F::kBoxCols, x_next);
      }
      if (!dead && !mbar_wait(&bars[out_slot], phase)) {
        dead = true;
        raise_flag(flags, MOE_FLAG_TIMEOUT);
      }
      __syncwarp();
      if constexpr (DIG) {
        stream::mac_box_digits<WF, MT, NT>(stage, ntiles, dx, sc, acc);
      } else if constexpr (NT == 1) {
        float(&acc1)[MT][4] = reinterpret_cast<float(&)[MT][4]>(acc);
        stream::mac_box<WF, MT>(stage, x_now, sc, acc1);
      } else {
        auto load = [&](int nt, int i) {
          const int col = F::kInt4 ? 32 * i + 8 * c : (F::kBoxCols / 4) * c + 8 * i;
          const uint16_t* t = x + (size_t)min(nt * 8 + g, a.M - 1) * a.ldx + c0;
          return col < left ? *reinterpret_cast<const uint4*>(t + col) : make_uint4(0, 0, 0, 0);
        };
        stream::mac_box_tiles<WF, MT, NT>(stage, load, sc, acc);
      }
      __syncwarp();
      ++done;
      if (++out_slot == P::kStages) out_slot = 0, phase ^= 1u;
      issue();
    }
    // to shared memory as [warp][mt][nt][row][token]
    constexpr int kToks = DIG ? stream::kDigitTokens : 8;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt >= ntiles) break;
        float* t = part + ((w * MT + mt) * NT + nt) * 16 * kToks;
        if constexpr (DIG) {
          float r0, r8;
          stream::join_digits(acc[mt][nt], r0, r8);
          if ((c & 1) == 0) t[g * kToks + c / 2] = r0, t[(g + 8) * kToks + c / 2] = r8;
        } else {
          *reinterpret_cast<float2*>(t + g * kToks + 2 * c) = make_float2(acc[mt][nt][0], acc[mt][nt][1]);
          *reinterpret_cast<float2*>(t + (g + 8) * kToks + 2 * c) = make_float2(acc[mt][nt][2], acc[mt][nt][3]);
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * a.M; i += kThreads) {
      const int r = i % rows, m = i / rows, n = u * rows + r;
      if (n >= a.N) continue;
      const int mt = gated ? 0 : r >> 4;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kWarps; ++s) {
        const float* f = part + (((s * MT + mt) * NT + m / kToks) * 16 + (r & 15)) * kToks + m % kToks;
        v[0] += f[0];
        if (gated) v[1] += f[NT * 16 * kToks];
      }
      if constexpr (DIG) {
        const float unit = units_x[m] * (F::kInt4 ? 0.0625f : 1.f);
        v[0] *= unit, v[1] *= unit;
      }
      linear_finish(a, WF == MOE_W_INT8_ROW, m, n, v[0], v[1]);
    }
    __syncthreads();
  }
  // after a wait that ran out: leave only when the copies have landed
  if (dead) {
    for (; done < issued; ++done) {
      mbar_wait(&bars[out_slot], phase);
      if (++out_slot == P::kStages) out_slot = 0, phase ^= 1u;
    }
  }
}

// one or two tokens whose digits fit beside the rings
bool digits_local(const moe_linear_desc& d, int M) {
  return M <= stream::kDigitTokens && M * 4 * stream::digit_pitch(d.K) <= kLocal;
}

struct DigitLayout {
  size_t units, total;
};
DigitLayout digit_layout(const moe_linear_desc& d, int M) {
  DigitLayout l = {0, 0};
  if (!linear_stream_digits(d, M) || digits_local(d, M)) return l;
  l.units = (size_t)M * 4 * stream::digit_pitch(d.K);  // a multiple of 256
  l.total = l.units + 256;
  return l;
}

template <int WF, int MT, int NT, bool DIG>
cudaError_t launch(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, uint32_t* flags,
                   cudaStream_t s) {
  using P = Plan<WF, MT, NT, DIG>;
  using F = stream::Format<WF>;
  StreamMaps m;
  char* ws = static_cast<char*>(workspace);
  StreamLinear p = {a, 0, reinterpret_cast<const int8_t*>(ws), reinterpret_cast<const float*>(ws + digit_layout(d, a.M).units), 0};
  p.local = DIG && digits_local(d, a.M);
  const bool gated = d.W_up != nullptr;
  p.boxed = F::kScaleBoxes && d.K % 128 == 0 && reinterpret_cast<uintptr_t>(d.s) % 16 == 0 &&
            (!gated || reinterpret_cast<uintptr_t>(d.s_up) % 16 == 0);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < (gated ? 2 : 1) && e == cudaSuccess; ++i) {
    const uint64_t bytes = (uint64_t)d.K * F::kBits / 8;
    e = make_tmap(&m.w[i], a.W[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, bytes, (uint64_t)d.N, bytes, 128, stream::kBoxRows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess && p.boxed)
      e = make_tmap(&m.s[i], a.s[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (uint64_t)(d.K / 32), (uint64_t)d.N,
                    (uint64_t)(d.K / 32) * 4, 8, stream::kBoxRows, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  auto kernel = linear_stream_kernel<WF, MT, NT, DIG>;
  static std::atomic<bool> allowed[64];
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(kernel), P::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const int rows = gated ? 16 : 16 * MT, units = (d.N + rows - 1) / rows;
  const dim3 grid(std::min(units, num_sms)), block(kThreads);
  return DIG && !p.local ? launch_k_after(kernel, grid, block, P::kBytes, s, m, p, flags)
                         : launch_k(kernel, grid, block, P::kBytes, s, m, p, flags);
}

template <int WF>
cudaError_t launch(const moe_linear_desc& d, const LinearArgs& a, void* ws, int num_sms, uint32_t* flags, cudaStream_t s) {
  // two tiles of rows halve what a box costs in token columns, where they leave work for every SM
  const bool two = d.W_up != nullptr || d.N >= 2 * 32 * num_sms;
  if constexpr (WF != MOE_W_BF16) {
    if (a.M <= 2)
      return two ? launch<WF, 2, 1, true>(d, a, ws, num_sms, flags, s) : launch<WF, 1, 1, true>(d, a, ws, num_sms, flags, s);
    if constexpr (WF == MOE_W_INT8_ROW) {
      if (a.M <= 8)
        return two ? launch<WF, 2, 4, true>(d, a, ws, num_sms, flags, s) : launch<WF, 1, 4, true>(d, a, ws, num_sms, flags, s);
    }
  }
  if constexpr (WF != MOE_W_INT8_ROW) {
    if (a.M <= 8)
      return two ? launch<WF, 2, 1, false>(d, a, ws, num_sms, flags, s) : launch<WF, 1, 1, false>(d, a, ws, num_sms, flags, s);
  }
  auto run = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    return two ? launch<WF, 2, NT, false>(d, a, ws, num_sms, flags, s) : launch<WF, 1, NT, false>(d, a, ws, num_sms, flags, s);
  };
  using std::integral_constant;
  if (a.M <= 16) return run(integral_constant<int, 2>());
  if (a.M <= 24) return run(integral_constant<int, 3>());
  if (a.M <= 32) return run(integral_constant<int, 4>());
  if constexpr (WF != MOE_W_BF16) {
    if (a.M <= 40) return run(integral_constant<int, 5>());
    if (a.M <= 48) return run(integral_constant<int, 6>());
  }
  if constexpr (WF == MOE_W_INT8_ROW)
    if (a.M <= 64) return run(integral_constant<int, 8>());
  return cudaErrorInvalidValue;  // not reached: linear_stream_tokens()
}

}  // namespace

bool linear_stream_ok(const moe_linear_desc& d, int M) {
  return d.xfmt == MOE_X_BF16 && d.wfmt != MOE_W_F32 && M <= linear_stream_tokens(d);
}

bool linear_stream_digits(const moe_linear_desc& d, int M) {
  // int4 sums of more than one tile are fp32 by digit, more than the registers hold
  return linear_stream_ok(d, M) && d.wfmt != MOE_W_BF16 && M <= (d.wfmt == MOE_W_INT8_ROW ? 8 : stream::kDigitTokens);
}

bool linear_stream_digits_first(const moe_linear_desc& d, int M) { return linear_stream_digits(d, M) && !digits_local(d, M); }

size_t linear_stream_workspace(const moe_linear_desc& d, int M) { return digit_layout(d, M).total; }

cudaError_t launch_linear_digits(const moe_linear_desc& d, const LinearArgs& a, void* workspace, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  return launch_k(linear_digits_kernel, dim3(a.M), dim3(256), 0, s, a, (int)(d.wfmt != MOE_W_INT8_ROW),
                  reinterpret_cast<int8_t*>(ws), reinterpret_cast<float*>(ws + digit_layout(d, a.M).units));
}

cudaError_t launch_linear_stream(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, uint32_t* flags,
                                 cudaStream_t s) {
  switch (d.wfmt) {
    case MOE_W_BF16: return launch<MOE_W_BF16>(d, a, workspace, num_sms, flags, s);
    case MOE_W_INT8_ROW: return launch<MOE_W_INT8_ROW>(d, a, workspace, num_sms, flags, s);
    case MOE_W_INT4_B32: return launch<MOE_W_INT4_B32>(d, a, workspace, num_sms, flags, s);
    default: return launch<MOE_W_INT4_B128>(d, a, workspace, num_sms, flags, s);
  }
}

}  // namespace moe
