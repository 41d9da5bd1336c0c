// The dense product for a few tokens (up to 64): a stream of stored weights through warp-wide
// matrix instructions (stream_dev.cuh).
//
// What bounds it is the weights' way from HBM.  A CTA takes units of 16 rows of W (32 where there
// are rows enough, or 16 of W and the same 16 of W_up), and its twelve warps share the
// reduction box by box (16 rows x 128 bytes), each with a ring of its own that TMA fills
// stages ahead, across units.  Their sums meet in shared memory, where bias, activation,
// gate and residual are applied.  Every weight is widened once for all tokens; the tokens'
// columns come from L1 and L2.
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
};

template <int WF, int MT, int NT>
struct Plan {
  using F = stream::Format<WF>;
  static constexpr int kStage = MT * (stream::kBoxBytes + F::kScaleBox);
  static constexpr int kStride = (kStage + 1023) / 1024 * 1024;
  static constexpr int kPart = kWarps * MT * NT * 32 * 16;  // bytes of the warps' sums
  static constexpr int kFit = (kSmem - 1024 - 512 - kPart) / (kWarps * kStride);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kBytes = 1024 + kWarps * kStages * kStride + kPart + 512;
  static_assert(kStages >= 2 && kWarps * kMaxStages * 8 <= 512, "shared memory");
};

template <int WF, int MT, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_stream_kernel(const __grid_constant__ StreamMaps maps, const __grid_constant__ StreamLinear p, uint32_t* flags) {
  using P = Plan<WF, MT, NT>;
  using F = stream::Format<WF>;
  extern __shared__ uint8_t smem[];
  uint8_t* rings = smem + (((smem_u32(smem) + 1023u) & ~1023u) - smem_u32(smem));
  float4* part = reinterpret_cast<float4*>(rings + kWarps * P::kStages * P::kStride);  // [warp][mt][nt][lane]
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
  pdl_wait();
  pdl_trigger();

  const bool gated = a.W[1] != nullptr;
  const int rows = gated ? 16 : 16 * MT;  // output columns of a unit
  const int units = (a.N + rows - 1) / rows, boxes = (a.K + F::kBoxCols - 1) / F::kBoxCols, grid = (int)gridDim.x;
  const int ntiles = (a.M + 7) / 8;
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
  for (int i = 0; i < P::kStages; ++i) issue();

  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  Walk at = {(int)blockIdx.x, w};
  seek(at);
  uint4 x_next[F::kLoads];
  const uint16_t* tok = x + (size_t)min(g, a.M - 1) * a.ldx;  // columns past the tokens are not used
  if (NT == 1 && at.u < units) stream::load_token<WF>(tok + at.j * F::kBoxCols, a.K - at.j * F::kBoxCols, x_next);
  for (int u = (int)blockIdx.x; u < units; u += grid) {
    float acc[MT][NT][4] = {};
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
          sc[mt].s0 = s + (size_t)min(r, a.N - 1) * pitch;
          sc[mt].s8 = s + (size_t)min(r + 8, a.N - 1) * pitch;
        }
      }
      uint4 x_now[F::kLoads];
      if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < F::kLoads; ++i) x_now[i] = x_next[i];
      }
      at.j += kWarps;
      seek(at);
      if (NT == 1 && at.u < units) stream::load_token<WF>(tok + at.j * F::kBoxCols, a.K - at.j * F::kBoxCols, x_next);
      if (!dead && !mbar_wait(&bars[out_slot], phase)) {
        dead = true;
        raise_flag(flags, MOE_FLAG_TIMEOUT);
      }
      __syncwarp();
      if constexpr (NT == 1) {
        float(&acc1)[MT][4] = reinterpret_cast<float(&)[MT][4]>(acc);
        stream::mac_box<WF, MT>(stage, x_now, sc, acc1);
      } else {
        auto load = [&](int nt, int i) {
          const int col = F::kInt4 ? 32 * i + 8 * c : (F::kBoxCols / 4) * c + 8 * i;
          const uint16_t* t = x + (size_t)min(nt * 8 + g, a.M - 1) * a.ldx + c0;
          return col < left ? *reinterpret_cast<const uint4*>(t + col) : make_uint4(0, 0, 0, 0);
        };
        stream::mac_box_tiles<WF, MT, NT>(stage, ntiles, load, sc, acc);
      }
      __syncwarp();
      ++done;
      if (++out_slot == P::kStages) out_slot = 0, phase ^= 1u;
      issue();
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt < ntiles)
          part[((w * MT + mt) * NT + nt) * 32 + lane] = make_float4(acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]);
    __syncthreads();
    // lane 4g + c of a tile holds rows g and g + 8 for tokens 2c and 2c + 1
    for (int i = threadIdx.x; i < rows * a.M; i += kThreads) {
      const int r = i % rows, m = i / rows, n = u * rows + r;
      if (n >= a.N) continue;
      const int mt = gated ? 0 : r >> 4, at_lane = (r & 7) * 4 + (m & 7) / 2, k = ((r >> 3) & 1) * 2 + (m & 1);
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kWarps; ++s) {
        const float* f = reinterpret_cast<const float*>(&part[((s * MT + mt) * NT + m / 8) * 32 + at_lane]);
        v[0] += f[k];
        if (gated) v[1] += f[NT * 32 * 4 + k];
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

template <int WF, int MT, int NT>
cudaError_t launch(const moe_linear_desc& d, const LinearArgs& a, int num_sms, uint32_t* flags, cudaStream_t s) {
  using P = Plan<WF, MT, NT>;
  using F = stream::Format<WF>;
  StreamMaps m;
  StreamLinear p = {a, 0};
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
  auto kernel = linear_stream_kernel<WF, MT, NT>;
  static std::atomic<bool> allowed[64];
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(kernel), P::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const int rows = gated ? 16 : 16 * MT, units = (d.N + rows - 1) / rows;
  return launch_k(kernel, dim3(std::min(units, num_sms)), dim3(kThreads), P::kBytes, s, m, p, flags);
}

template <int WF>
cudaError_t launch(const moe_linear_desc& d, const LinearArgs& a, int num_sms, uint32_t* flags, cudaStream_t s) {
  // two tiles of rows halve what a box costs in token columns, where they leave work for every SM
  const bool two = d.W_up != nullptr || d.N >= 2 * 32 * num_sms;
  if (a.M <= 8) return two ? launch<WF, 2, 1>(d, a, num_sms, flags, s) : launch<WF, 1, 1>(d, a, num_sms, flags, s);
  if (a.M <= 16) return two ? launch<WF, 2, 2>(d, a, num_sms, flags, s) : launch<WF, 1, 2>(d, a, num_sms, flags, s);
  if (a.M <= 32) return two ? launch<WF, 2, 4>(d, a, num_sms, flags, s) : launch<WF, 1, 4>(d, a, num_sms, flags, s);
  return two ? launch<WF, 2, 8>(d, a, num_sms, flags, s) : launch<WF, 1, 8>(d, a, num_sms, flags, s);
}

}  // namespace

bool linear_stream_ok(const moe_linear_desc& d, int M) {
  return d.xfmt == MOE_X_BF16 && d.wfmt != MOE_W_F32 && M <= linear_stream_tokens(d.wfmt);
}

cudaError_t launch_linear_stream(const moe_linear_desc& d, const LinearArgs& a, int num_sms, uint32_t* flags, cudaStream_t s) {
  switch (d.wfmt) {
    case MOE_W_BF16: return launch<MOE_W_BF16>(d, a, num_sms, flags, s);
    case MOE_W_INT8_ROW: return launch<MOE_W_INT8_ROW>(d, a, num_sms, flags, s);
    case MOE_W_INT4_B32: return launch<MOE_W_INT4_B32>(d, a, num_sms, flags, s);
    default: return launch<MOE_W_INT4_B128>(d, a, num_sms, flags, s);
  }
}

}  // namespace moe
