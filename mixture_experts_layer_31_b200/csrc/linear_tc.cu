// The dense product for many tokens on the 5th-generation tensor cores.
//
// y [M, N] = act(x W^T + b) ...: tokens are the rows of the matrix instruction, outputs its
// columns.  A pair of CTAs (cta_group::2) computes 256 tokens x 256 columns: each CTA holds 128
// tokens and 128 rows of W per 64-column stage, 32 KB where a CTA of its own would load
// 48 KB for the same instructions -- what an SM can take from L2 is the bound that a single
// CTA's 128 x 256 tile meets first.  Gated, one CTA's rows of W are gate rows and the other's
// the up rows with the same numbers, so that both of an output's projections end up in the
// TMEM lane of its token.
//
// Roles in each CTA of the persistent pair:
//   warp 0       TMA: its 128 tokens and its 128 rows of W, signalled to the leader's barrier
//   warp 1       (leader) tcgen05.mma for both CTAs; commits free the stages of both
//   warp 2       TMEM
//   warps 4..11  epilogue from TMEM, two groups of 128 lanes: one accumulator is drained while
//                the next tile is multiplied into the other
// Where the tiles are fewer than the pairs, the reduction is split; the splits' fp32 sums are
// added in order by a second launch with the same epilogue.
// fp32 operands go through the same instructions in three bf16 parts, x = h + m + l with 8
// significant bits each, exactly: the products of parts that matter to 24 bits (six of two
// fp32 operands, three where one is exact in bf16) are summed, the small ones first; what is
// left out is below 2^-23 of each product.  That is six times the operations of a bf16
// product and still several times the rate of fp32 multiply-adds.  An infinity has the parts
// (inf, 0, 0), and infinity times another operand's zero or negative part is NaN where the product
// is infinite: sums of parts that come out NaN are formed again in fp32 from the operands themselves.
// The tensor core's own additions cut off: over 2,304 columns in one accumulator the result
// came out 2 x 10^-6 too small (of its mean magnitude), over 9,216 columns 4 x 10^-6.  Where the
// output is fp32, the accumulator is therefore drained every kSegment stages and the drained
// sums are added in fp32 registers, rounded to nearest: 7 x 10^-7 off, as a chain of fp32
// multiply-adds is.  A bf16 output's own rounding is a thousand times that.
// Quantised weights are widened to bf16 in the workspace first: int8 codes exactly, with the row
// scale left for the epilogue, int4 as q s rounded once where y is bf16 (half a step of bf16 per
// weight, as the routed layer's tensor-core path has it: measured against 64 bits 2.2 x 10^-3
// where y's own rounding alone leaves 1.7 x 10^-3), in two parts where two such projections are
// multiplied (one part left 2.7 x 10^-3), in three parts where y is fp32.
// The pass reads 1 byte per weight of int8, 0.5 and the scales of int4, 4 of fp32, and writes 2 for
// each part (fp32 and int4 for fp32 outputs: 6); the product reads the parts again.  Where they
// fit L2 (126 MB) with the rest, most of that stays there; larger matrices go through HBM
// twice more: 229 tokens, 6,272 columns, 12,694 gated outputs, int4 in two parts, 637 MB each way
// are the larger part of 320 us.
//
// Measured: 4,096 tokens, 2,304 columns, 9,216 gated outputs, bf16, one launch by itself under the
// profiler 219 to 250 us over several GPUs (up to 1,586 TFLOP/s, 97% of the rate of a large
// library product; the tensor pipe is busy 81% of the cycles on all of them) and 287 to 298 us
// among other calls, where the power limit lowers the clock; 1,999 tokens, 9,216 columns,
// 2,304 outputs, int8, 66 to 74 us by itself behind a widening pass of 13, both together 88 to
// 90 us among other calls; 2,048 tokens, 2,304 x 2,304, fp32, 117 us.  L2 is at half its rate
// meanwhile.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "linear.h"
#include "stream_dev.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kRows = 128;  // tokens, and rows of W, per CTA and stage
constexpr int kK = 64;      // columns per stage: one 128-byte swizzle row of bf16
constexpr int kHalf = kRows * kK * 2;
constexpr int kStage = 2 * kHalf;
constexpr int kStages = 6;
constexpr int kTileN = 256;  // columns of the pair's accumulator
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kTurn = 32 * 17 * 4;  // a warp's 32 x 16 results, turned from a row a lane to a row at a time
constexpr int kSmem = 1024 + kStages * kStage + 512 + kEpiWarps * kTurn;

struct TcArgs {
  LinearArgs l;
  int row_scales;       // int8: the epilogue scales the sums
  int mt, nt, splits;   // tiles of 256 tokens, of 256 (gated: 128) outputs; parts of the reduction
  int ksteps, segment;  // columns steps of the reduction; of one accumulator
  int xparts, wparts;   // bf16 parts of x and of W, whose rows follow one another: 1, 3 of an fp32 operand, 2 of int4
  int xfmt, wfmt;       // of the operands as they are stored
  int again;            // products of parts: sums that are NaN are formed again
  int vec;              // y and residual rows in 16-byte pieces
  float* partial;       // splits > 1: [splits][1 or 2][M][np]
  int np;               // N rounded up to 16
};

// the products of parts, least first: (part of x, part of W)
struct Parts {
  int x, w;
};
__device__ __forceinline__ int products(int xp, int wp) { return xp == 1 ? wp : (wp == 1 ? xp : 6); }
__device__ __forceinline__ Parts product(int xp, int wp, int i) {
  if (wp == 1) return Parts{xp - 1 - i, 0};
  if (xp == 1) return Parts{0, wp - 1 - i};
  // (2, 0) (0, 2) (1, 1) (1, 0) (0, 1) (0, 0)
  return Parts{(0x001102 >> (4 * i)) & 15, (0x010120 >> (4 * i)) & 15};
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the shared address of the leader CTA's copy of a variable
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// 2-D tile into this CTA's shared memory, completing on a barrier of the pair
__device__ __forceinline__ void tma_load_pair(void* dst, const void* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs when the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}

struct Tile {
  int m, n, split;
};
// tokens fastest within groups of 8 token tiles, so that the tiles in flight share x and W in L2
__device__ __forceinline__ Tile tile_of(const TcArgs& a, int t) {
  Tile r;
  r.split = t % a.splits;
  t /= a.splits;
  const int group = 8 * a.nt, g = t / group, in = t - g * group;
  const int size = min(8, a.mt - g * 8);
  r.m = g * 8 + in % size;
  r.n = in / size;
  return r;
}

// Columns c, c + step, ... (8 from each on) of the product of token m and row n of W (side 0) or W_up, in
// fp32 multiply-adds; int8 codes without their row's scale, as the accumulators have them.
__device__ __noinline__ float sum_again(const TcArgs& a, int side, int m, int n, int c, int step) {
  const LinearArgs& l = a.l;
  float acc = 0.f;
#pragma unroll 2
  for (; c < l.K && acc == acc; c += step) {  // a NaN stays one
    float w[8], x[8];
    switch (a.wfmt) {
      case MOE_W_F32: weights8<MOE_W_F32>(l.W[side], l.s[side], n, c, l.K, w); break;
      case MOE_W_BF16: weights8<MOE_W_BF16>(l.W[side], l.s[side], n, c, l.K, w); break;
      case MOE_W_INT8_ROW: weights8<MOE_W_INT8_ROW>(l.W[side], l.s[side], n, c, l.K, w); break;
      case MOE_W_INT4_B32: weights8<MOE_W_INT4_B32>(l.W[side], l.s[side], n, c, l.K, w); break;
      default: weights8<MOE_W_INT4_B128>(l.W[side], l.s[side], n, c, l.K, w);
    }
    const size_t at = (size_t)m * l.ldx + c;
    if (a.xfmt == MOE_X_F32) token8<MOE_X_F32>(l.x, at, c + 4 < l.K, x);
    else token8<MOE_X_BF16>(l.x, at, true, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = fmaf(w[j], x[j], acc);
  }
  return acc;
}

// The NaNs among 16 columns of the warp's 32 tokens again; the whole warp calls it.  Rare and slow:
// 1,999 tokens of 9,216 columns with an infinity each, 2,304 outputs, take 72 ms where finite ones
// take 0.5 (a token that holds a NaN itself is left as it is).
template <bool GATED>
__device__ __noinline__ void again16(const TcArgs& a, int m, int n0, uint32_t (&v)[16], uint32_t (&u)[16]) {
  const int lane = lane_id();
  uint32_t looked = 0, lost = 0;  // tokens looked through, and those of them that hold a NaN
#pragma unroll 1
  for (int i = 0; i < (GATED ? 32 : 16); ++i) {
    const int side = i >> 4, j = i & 15;
    const float now = __uint_as_float(side ? u[j] : v[j]);
    uint32_t who = __ballot_sync(0xFFFFFFFFu, now != now && m < a.l.M && n0 + j < a.l.N);
#pragma unroll 1
    for (; who; who &= who - 1) {
      const int r = __ffs(who) - 1, row = m - lane + r;
      if (!(looked >> r & 1u)) {
        bool nan = false;
        for (int c = lane; c < a.l.K; c += 32) {
          const size_t at = (size_t)row * a.l.ldx + c;
          const float x = a.xfmt == MOE_X_F32 ? static_cast<const float*>(a.l.x)[at]
                                              : bf16_to_f32(static_cast<const uint16_t*>(a.l.x)[at]);
          nan |= x != x;
        }
        looked |= 1u << r;
        lost |= (uint32_t)__any_sync(0xFFFFFFFFu, nan) << r;
      }
      if (lost >> r & 1u) continue;
      float sum = sum_again(a, side, row, n0 + j, 8 * lane, 256);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
      if (lane == r) (side ? u[j] : v[j]) = __float_as_uint(sum);
    }
  }
}

// The epilogue's code is kept short on purpose: a tile passes through it once, and its way into the
// instruction cache shows (with every activation inlined for every column it took 17 us before
// the first tile was stored, whatever the reduction's length).

// The activation of 16 sums: v / (1 + exp(-z)), z = v (SiLU) or twice the tanh-GELU's argument.  Far
// below zero the exponential is infinite and nothing may be left of v, however large: FAST
// multiplies v with a reciprocal that has gone to 0 by then.
template <bool FAST>
__device__ __forceinline__ void activate16(float (&v)[16], int act) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float z = act == MOE_ACT_SILU ? v[j] : 2.0f * gelu_tanh_z(v[j]);
    // FAST, for bf16 outputs: a few units in the last place of fp32
    if (FAST) v[j] *= __fdividef(1.0f, 1.0f + __expf(-z));
    else v[j] = v[j] / (1.0f + expf(-z));
  }
}

// 16 columns of the warp's 32 tokens, the lane's token m; the whole warp calls it
template <bool GATED>
__device__ __forceinline__ void output16(const TcArgs& a, int split, int m, int n0, const uint32_t (&v)[16],
                                         const uint32_t (&u)[16], float* turn) {
  const LinearArgs& l = a.l;
  if (a.splits > 1) {
    if (m >= l.M || n0 >= a.np) return;
    uint4* out = reinterpret_cast<uint4*>(a.partial + (((size_t)split * (GATED ? 2 : 1)) * l.M + m) * a.np + n0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      if (GATED) out[(size_t)l.M * a.np / 4 + j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
    }
    return;
  }
  const int last = l.N - 1 - n0;  // columns past the last one are computed with its scale and bias
  if (last < 0) return;
  float y[16], g[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] = __uint_as_float(v[j]);
    if (GATED) g[j] = __uint_as_float(u[j]);
  }
  if (a.row_scales) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      y[j] *= __ldg(l.s[0] + n0 + min(j, last));
      if (GATED) g[j] *= __ldg(l.s[1] + n0 + min(j, last));
    }
  }
  if (l.b[0]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] += __ldg(l.b[0] + n0 + min(j, last));
  }
  if (l.act != MOE_ACT_NONE) {
    if (l.yfmt == MOE_X_BF16) activate16<true>(y, l.act);
    else activate16<false>(y, l.act);
  }
  if constexpr (GATED) {
    if (l.b[1]) {
#pragma unroll
      for (int j = 0; j < 16; ++j) g[j] += __ldg(l.b[1] + n0 + min(j, last));
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] *= g[j];
  }
  if (!a.vec || last < 15) {
    // rows of y that 16-byte pieces do not fit: turned from a row a lane to two rows at a time, 16
    // columns each.  Pieces of sectors are what this costs: 1,172 x 1,472 -> 6,290, bf16, 48 us
    // where 6,288 columns take 29 (and 71 with the activation behind the turn).
    const int lane = lane_id(), c = lane & 15, first = m - lane + (lane >> 4);
#pragma unroll
    for (int j = 0; j < 16; ++j) turn[lane * 17 + j] = y[j];
    __syncwarp();
    if (c <= last) {
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += 16) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 2 * i, row = first + r;
          o[i] = turn[(r + (lane >> 4)) * 17 + c];
          if (l.residual && row < l.M) {
            const size_t at = (size_t)row * l.ldr + n0 + c;
            o[i] += l.yfmt == MOE_X_F32 ? static_cast<const float*>(l.residual)[at]
                                        : bf16_to_f32(static_cast<const uint16_t*>(l.residual)[at]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = first + r0 + 2 * i;
          if (row >= l.M) break;
          const size_t at = (size_t)row * l.ldy + n0 + c;
          if (l.yfmt == MOE_X_F32) static_cast<float*>(l.y)[at] = o[i];
          else static_cast<uint16_t*>(l.y)[at] = f32_to_bf16(o[i]);
        }
      }
    }
    __syncwarp();
    return;
  }
  if (m >= l.M) return;
  if (l.yfmt == MOE_X_BF16) {
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(l.y) + (size_t)m * l.ldy + n0);
    if (l.residual) {
      const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(l.residual) + (size_t)m * l.ldr + n0);
      const uint4 r0 = r[0], r1 = r[1];
      const uint32_t rr[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[2 * j] += bf16_to_f32(rr[j] & 0xFFFFu);
        y[2 * j + 1] += __uint_as_float(rr[j] & 0xFFFF0000u);
      }
    }
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  } else {
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(l.y) + (size_t)m * l.ldy + n0);
    const float* r = static_cast<const float*>(l.residual);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 o = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      if (r) {
        const float4 e = *reinterpret_cast<const float4*>(r + (size_t)m * l.ldr + n0 + 4 * j);
        o.x += e.x, o.y += e.y, o.z += e.z, o.w += e.w;
      }
      out[j] = o;
    }
  }
}
// one copy of it for a loop that is unrolled: eight copies' way into the instruction cache took
// longer than all the rest (37 us a tile)
template <bool GATED>
__device__ __noinline__ void output16_call(const TcArgs& a, int split, int m, int n0, const uint32_t (&v)[16],
                                           const uint32_t (&u)[16], float* turn) {
  output16<GATED>(a, split, m, n0, v, u, turn);
}

// SEG: the reduction goes through the accumulators in segments.  PARTS: products of parts, whose NaNs
// are formed again; kept out of the other products' kernels, where the code alone cost 1% (4,096
// tokens bf16 gated 287 -> 290 us).
template <bool GATED, bool SEG, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w0,
                     const __grid_constant__ CUtensorMap map_w1, const __grid_constant__ TcArgs a, uint32_t* flags) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStage);  // leader's: both CTAs' stage has landed
  uint64_t* empty = full + kStages;                                       // the MMAs have read the stage
  uint64_t* acc_full = empty + kStages;                                   // [2]
  uint64_t* acc_empty = acc_full + 2;                                     // [2] leader's: both CTAs have drained it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int w = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(rank && GATED ? &map_w1 : &map_w0);
  }
  if (w == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int tiles = a.mt * a.nt * a.splits, pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
  auto steps_of = [&](int split, int& k0) {
    k0 = (int)((long long)split * a.ksteps / a.splits);
    return (int)((long long)(split + 1) * a.ksteps / a.splits) - k0;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity, bool& dead) {
    if (dead) return;
    if (!mbar_wait(bar, parity)) {
      dead = true;
      raise_flag(flags, MOE_FLAG_TIMEOUT);
    }
  };

  if (w == 0) {
    if (lane == 0) {
      bool dead = false;
      uint32_t it = 0;
      const CUtensorMap* map_w = GATED && rank ? &map_w1 : &map_w0;
      for (int t = pair; t < tiles && !dead; t += pairs) {
        const Tile tl = tile_of(a, t);
        int k0;
        const int nk = steps_of(tl.split, k0), all = nk * products(a.xparts, a.wparts);
        const int seg = SEG ? a.segment : nk;
        const int row_x = tl.m * 2 * kRows + (int)rank * kRows;
        const int row_w = GATED ? tl.n * kRows : tl.n * 2 * kRows + (int)rank * kRows;
        // segment by segment the products of parts, each over the segment's columns
        int k = 0, i = 0, from = 0, to = min(seg, nk);
        Parts p = product(a.xparts, a.wparts, 0);
        for (int n = 0; n < all; ++n, ++it) {
          const int s = it % kStages;
          wait(&empty[s], ((it / kStages) & 1u) ^ 1u, dead);
          if (dead) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStage);
          const uint32_t bar = leader_addr(&full[s]);
          uint8_t* stage = smem + s * kStage;
          // a tile's last rows may be the next part's first: rows past M and N are not used
          tma_load_pair(stage, &map_x, (k0 + k) * kK, row_x + p.x * a.l.M, bar);
          tma_load_pair(stage + kHalf, map_w, (k0 + k) * kK, row_w + p.w * a.l.N, bar);
          if (++k == to) {
            if (++i == products(a.xparts, a.wparts)) i = 0, from = to, to = min(to + seg, nk);
            k = from;
            p = product(a.xparts, a.wparts, i);
          }
        }
      }
      // after a wait that ran out: the copies in flight end before the pair leaves
      if (dead && rank == 0)
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1u);
    }
  } else if (w == 1) {
    if (rank == 0 && lane == 0) {
      bool dead = false;
      uint32_t it = 0, n = 0;
      const uint32_t idesc = umma_idesc_bf16(2 * kRows, kTileN);
      for (int t = pair; t < tiles && !dead; t += pairs) {
        const Tile tl = tile_of(a, t);
        int k0;
        const int nk = steps_of(tl.split, k0), seg = SEG ? a.segment : nk, prods = products(a.xparts, a.wparts);
        for (int from = 0; from < nk && !dead; from += seg, ++n) {
          const int all = min(seg, nk - from) * prods;
          const uint32_t buf = n & 1u, d = tmem + buf * kTileN;
          wait(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, dead);
          tc_fence_after();
          for (int k = 0; k < all && !dead; ++k, ++it) {
            const int s = it % kStages;
            wait(&full[s], (it / kStages) & 1u, dead);
            if (dead) break;
            tc_fence_after();
            const uint32_t stage = smem_u32(smem + s * kStage);
#pragma unroll
            for (int j = 0; j < kK / 16; ++j)
              umma_pair(d, umma_desc_sw128(stage + 32 * j), umma_desc_sw128(stage + kHalf + 32 * j), idesc, (k | j) != 0);
            commit_pair(&empty[s]);
          }
          if (!dead) commit_pair(&acc_full[buf]);
        }
      }
    }
  } else if (w >= 4) {
    const int q = w & 3, group = (w - 4) >> 2;  // lane quarter; half of the columns
    constexpr int kCols = GATED ? kTileN / 4 : kTileN / 2;  // outputs of a group
    const int outs = GATED ? kRows : 2 * kRows;             // outputs of a tile
    bool dead = false;
    uint32_t n = 0;
    for (int t = pair; t < tiles && !dead; t += pairs) {
      const Tile tl = tile_of(a, t);
      const int m = tl.m * 2 * kRows + (int)rank * kRows + q * 32 + lane;
      const int c_first = tl.n * outs + group * kCols;
      const uint32_t column = tmem + ((uint32_t)(q * 32) << 16) + group * kCols;
      auto drain = [&](uint32_t buf) {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(leader_addr(&acc_empty[buf]));
      };
      auto filled = [&](uint32_t buf) {
        wait(&acc_full[buf], (n >> 1) & 1u, dead);
        dead = __any_sync(0xFFFFFFFFu, dead);
        tc_fence_after();
      };
      constexpr int kChunks = SEG ? kCols / 16 : 1, kSides = SEG && GATED ? 2 : 1;
      float sum[kSides][kChunks][16] = {};
      if constexpr (SEG) {
        int k0;
        const int nk = steps_of(tl.split, k0);
        for (int from = 0; from < nk && !dead; from += a.segment, ++n) {
          const uint32_t buf = n & 1u;
          filled(buf);
          if (dead) break;
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int side = 0; side < kSides; ++side) {
              uint32_t v[16];
              tmem_ld16(column + buf * kTileN + side * (kTileN / 2) + 16 * i, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                sum[side][i][j] += __uint_as_float(v[j]);
            }
          drain(buf);
        }
      }
      const uint32_t buf = n & 1u, at = column + buf * kTileN;
      if constexpr (!SEG) filled(buf);
      if (dead) break;
      constexpr int kUnroll = SEG ? kChunks : 1;  // sums in registers need their places known
#pragma unroll kUnroll
      for (int c = 0; c < kCols; c += 16) {
        uint32_t v[16], u[16];
        __syncwarp();
        if constexpr (SEG) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = __float_as_uint(sum[0][(c / 16) % kChunks][j]);
            if (GATED) u[j] = __float_as_uint(sum[kSides - 1][(c / 16) % kChunks][j]);
          }
        } else {
          tmem_ld16(at + c, v);
          if (GATED) tmem_ld16(at + kTileN / 2 + c, u);
          tmem_ld_wait();
        }
        if (PARTS && a.splits == 1) {
          float nan = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) nan += __uint_as_float(v[j]) + (GATED ? __uint_as_float(u[j]) : 0.f);
          if (__any_sync(0xFFFFFFFFu, nan != nan)) {
            uint32_t v2[16], u2[16];  // the call's own: v and u stay in registers
#pragma unroll
            for (int j = 0; j < 16; ++j) v2[j] = v[j], u2[j] = GATED ? u[j] : 0u;
            again16<GATED>(a, m, c_first + c, v2, u2);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = v2[j], u[j] = u2[j];
          }
        }
        float* turn = reinterpret_cast<float*>(smem + kStages * kStage + 512 + (w - 4) * kTurn);
        if constexpr (SEG) output16_call<GATED>(a, tl.split, m, c_first + c, v, u, turn);
        else output16<GATED>(a, tl.split, m, c_first + c, v, u, turn);
      }
      if constexpr (!SEG) {
        drain(buf);
        ++n;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();  // the peer's MMAs have read this CTA's shared memory, its drains this TMEM
  if (w == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// the splits' sums in order, then the epilogue
__global__ void __launch_bounds__(256) linear_sum_kernel(const __grid_constant__ TcArgs a) {
  pdl_wait();
  pdl_trigger();
  const LinearArgs& l = a.l;
  const int quads = a.np / 4, parts = l.W[1] ? 2 : 1;
  const size_t n = (size_t)l.M * quads;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
    const int m = (int)(i / quads), c = (int)(i - (size_t)m * quads) * 4;
    float v[4] = {}, u[4] = {};
    for (int s = 0; s < a.splits; ++s) {
      const float4 p = *reinterpret_cast<const float4*>(a.partial + ((size_t)s * parts * l.M + m) * a.np + c);
      v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
      if (parts == 2) {
        const float4 q = *reinterpret_cast<const float4*>(a.partial + (((size_t)s * 2 + 1) * l.M + m) * a.np + c);
        u[0] += q.x, u[1] += q.y, u[2] += q.z, u[3] += q.w;
      }
    }
    const float nan = v[0] + v[1] + v[2] + v[3] + u[0] + u[1] + u[2] + u[3];
    if (a.again && nan != nan) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (v[j] != v[j] && c + j < l.N) v[j] = sum_again(a, 0, m, c + j, 0, 8);
        if (u[j] != u[j] && c + j < l.N) u[j] = sum_again(a, 1, m, c + j, 0, 8);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < l.N) linear_finish(l, a.row_scales, m, c + j, v[j], u[j]);
  }
}

// x = h + m + l in bf16: h and m rounded to nearest, so that each rest has 8 significant bits
// less, exactly.  An infinity or NaN is its own h; a finite value that would round to infinity
// is cut instead.
__device__ __forceinline__ void split3(float x, uint16_t (&p)[3]) {
  p[0] = f32_to_bf16(x);
  if (isinf(bf16_to_f32(p[0])) && isfinite(x)) p[0] = (uint16_t)(__float_as_uint(x) >> 16);
  float r = x - bf16_to_f32(p[0]);
  if (!isfinite(r)) r = 0.f;
  p[1] = f32_to_bf16(r);
  p[2] = f32_to_bf16(r - bf16_to_f32(p[1]));
}

// The passes below take kItems pieces of 8 values per thread and step, their loads first: with one
// piece at a time the loads' latency was most of the time (9,216 x 2,304 int8: 20 us, so 13).
constexpr int kItems = 4;

// The code of column j of 8 int4 codes, times s: the code plus 2^23 + 8 is made by its bits, which
// takes no conversion.
__device__ __forceinline__ float int4_value(uint32_t codes, int j, float s) {
  const uint32_t v = (codes >> (4 * j) & 15u) ^ 0x4B000008u;
  return (__uint_as_float(v) - 8388616.f) * s;
}

// 8 values in PARTS bf16 parts, `plane` apart
template <int PARTS>
__device__ __forceinline__ void store_parts(const float (&v)[8], uint16_t* out, size_t plane) {
  if constexpr (PARTS == 3) {
    uint16_t p[8][3];
#pragma unroll
    for (int j = 0; j < 8; ++j) split3(v[j], p[j]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4*>(out + q * plane) =
          make_uint4(p[0][q] | (uint32_t)p[1][q] << 16, p[2][q] | (uint32_t)p[3][q] << 16, p[4][q] | (uint32_t)p[5][q] << 16,
                     p[6][q] | (uint32_t)p[7][q] << 16);
  } else {
    uint32_t h[4], m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      const float h0 = bf16_to_f32(h[j] & 0xFFFFu), h1 = __uint_as_float(h[j] & 0xFFFF0000u);
      if (PARTS == 2) m[j] = pack_bf16x2(isfinite(h0) ? v[2 * j] - h0 : 0.f, isfinite(h1) ? v[2 * j + 1] - h1 : 0.f);
    }
    *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1], h[2], h[3]);
    if (PARTS == 2) *reinterpret_cast<uint4*>(out + plane) = make_uint4(m[0], m[1], m[2], m[3]);
  }
}

// fp32 rows to their three parts, [3][rows][pitch], zero between cols and pitch.
__device__ __forceinline__ void split_rows(const float* __restrict__ W, long long ld, int rows, int cols, int pitch,
                                           uint16_t* __restrict__ out) {
  const int eights = pitch / 8;
  const size_t n = (size_t)rows * eights, plane = (size_t)rows * pitch;
  constexpr int kAtOnce = kItems / 2;
  for (size_t i0 = (size_t)blockIdx.x * 256 * kAtOnce + threadIdx.x; i0 < n; i0 += (size_t)gridDim.x * 256 * kAtOnce) {
    float v[kAtOnce][8];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const size_t i = i0 + 256 * k;
      const int r = (int)(n >> 32 ? i / (size_t)eights : (uint32_t)i / (uint32_t)eights);
      const int c = (int)(i - (size_t)r * eights) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
      if (i >= n || c >= cols) continue;
      const float4* p = reinterpret_cast<const float4*>(W + (size_t)r * ld + c);  // cols is a multiple of 4
      const float4 a = __ldg(p);
      v[k][0] = a.x, v[k][1] = a.y, v[k][2] = a.z, v[k][3] = a.w;
      if (c + 4 < cols) {
        const float4 b = __ldg(p + 1);
        v[k][4] = b.x, v[k][5] = b.y, v[k][6] = b.z, v[k][7] = b.w;
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const size_t i = i0 + 256 * k;
      if (i >= n) break;
      store_parts<3>(v[k], out + 8 * i, plane);  // pieces follow one another in a plane: row r, column c is piece i
    }
  }
}

// stored weights to bf16: int8 codes, or int4 codes times their block scales in fp32 in PARTS parts
template <int WF, int PARTS>
__device__ __forceinline__ void widen_values(const void* __restrict__ W, const float* __restrict__ s, size_t n8,
                                             uint16_t* __restrict__ out) {
  for (size_t i0 = (size_t)blockIdx.x * 256 * kItems + threadIdx.x; i0 < n8; i0 += (size_t)gridDim.x * 256 * kItems) {
    uint2 q[kItems] = {};
    float scale[kItems] = {};
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const size_t i = i0 + 256 * k;
      if (i >= n8) break;
      if constexpr (WF == MOE_W_INT8_ROW) {
        q[k] = __ldg(static_cast<const uint2*>(W) + i);
      } else {
        constexpr int kShift = WF == MOE_W_INT4_B32 ? 5 : 7;
        q[k].x = __ldg(static_cast<const uint32_t*>(W) + i);
        scale[k] = __ldg(s + ((8 * i) >> kShift));  // K is a multiple of the block: blocks do not cross rows
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const size_t i = i0 + 256 * k;
      if (i >= n8) break;
      if constexpr (WF == MOE_W_INT8_ROW) {
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w = h ? q[k].y : q[k].x, even = stream::widen_int8(w), odd = stream::widen_int8(w >> 8);
          o[2 * h] = __byte_perm(even, odd, 0x5410), o[2 * h + 1] = __byte_perm(even, odd, 0x7632);
        }
        *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = int4_value(q[k].x, j, scale[k]);
        store_parts<PARTS>(v, out + 8 * i, 8 * n8);
      }
    }
  }
}

// Everything a call has to lay out anew, by blockIdx.y, in one launch: W, W_up and fp32 tokens.
struct Layouts {
  const void* from[3];
  const float* s[3];
  uint16_t* to[3];
  int x, rows_w, rows_x, K, pitch;  // which one holds the tokens, -1 for none
  long long ldx;
};

template <int WF, int PARTS>
__global__ void __launch_bounds__(256) linear_layout_kernel(const __grid_constant__ Layouts p) {
  pdl_wait();
  pdl_trigger();
  const int j = blockIdx.y;
  if (j == p.x) split_rows(static_cast<const float*>(p.from[j]), p.ldx, p.rows_x, p.K, p.pitch, p.to[j]);
  else if constexpr (WF == MOE_W_F32) split_rows(static_cast<const float*>(p.from[j]), p.K, p.rows_w, p.K, p.pitch, p.to[j]);
  else widen_values<WF, PARTS>(p.from[j], p.s[j], (size_t)p.rows_w * p.K / 8, p.to[j]);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// fp32 outputs: 64-column steps that go through one accumulator at a time
constexpr int kSegment = 12;

struct TcLayout {
  int mt, nt, ksteps, segment, splits, pitch, np;
  int xparts, wparts;
  bool w_copy;                // the weights are read from the workspace
  size_t x, w[2], partial, total;  // offsets in the workspace
};
TcLayout tc_layout(const moe_linear_desc& d, int M) {
  TcLayout t;
  const bool gated = d.W_up != nullptr, int4 = d.wfmt == MOE_W_INT4_B32 || d.wfmt == MOE_W_INT4_B128;
  const int outs = gated ? kRows : 2 * kRows, sides = gated ? 2 : 1;
  t.xparts = d.xfmt == MOE_X_F32 ? 3 : 1;
  // an fp32 output keeps what a rounded q s would lose, and so, in part, does a product of two
  t.wparts = d.wfmt == MOE_W_F32 || (int4 && (d.xfmt == MOE_X_F32 || d.yfmt == MOE_X_F32)) ? 3 : (int4 && gated ? 2 : 1);
  t.mt = (M + 2 * kRows - 1) / (2 * kRows);
  t.nt = (d.N + outs - 1) / outs;
  t.ksteps = (d.K + kK - 1) / kK;
  t.pitch = (d.K + 7) / 8 * 8;
  t.np = (d.N + 15) / 16 * 16;
  // 74 pairs of SMs: split the reduction while the tiles leave half of them idle and a part
  // keeps 8 stages (the pipeline's fill) to work on
  const int steps = t.ksteps * (t.xparts == 1 ? t.wparts : (t.wparts == 1 ? t.xparts : 6));
  const long long tiles = (long long)t.mt * t.nt;
  t.splits = 1;
  if (tiles * 2 <= 74)
    t.splits = std::max(1, std::min({(int)(74 / tiles), steps / 8, t.ksteps, 16}));
  t.segment = d.yfmt == MOE_X_F32 ? kSegment : 0;
  t.w_copy = d.wfmt != MOE_W_BF16;
  const size_t wide = t.w_copy ? up256((size_t)t.wparts * d.N * t.pitch * 2) : 0;
  t.w[0] = 0;
  t.w[1] = wide;
  t.x = wide * sides;
  t.partial = t.x + (t.xparts == 3 ? up256((size_t)3 * M * t.pitch * 2) : 0);
  t.total = t.partial + (t.splits > 1 ? (size_t)t.splits * sides * M * t.np * 4 : 0);
  return t;
}

}  // namespace

bool linear_tc_ok(const moe_linear_desc& d, int M) {
  const bool f32 = d.xfmt == MOE_X_F32 || d.wfmt == MOE_W_F32;
  return M > (f32 ? kLinearRowTokens : linear_stream_tokens(d));
}

size_t linear_tc_workspace(const moe_linear_desc& d, int M) { return tc_layout(d, M).total; }

// The launches of one call follow one another closely: each may start while the one before it
// finishes, and waits for its end before it touches memory.
template <typename... KArgs, typename... Args>
static cudaError_t launch_next(bool first, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                               Args&&... args) {
  return first ? launch_k(kernel, grid, block, smem, s, static_cast<Args&&>(args)...)
               : launch_k_after(kernel, grid, block, smem, s, static_cast<Args&&>(args)...);
}

static dim3 grid_for(size_t items, int num_sms) {
  return dim3((unsigned)std::min<size_t>((items + 255) / 256, (size_t)num_sms * 8));
}

bool linear_tc_layouts(const moe_linear_desc& d) { return d.wfmt != MOE_W_BF16 || d.xfmt == MOE_X_F32; }

cudaError_t launch_linear_layouts(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, cudaStream_t s) {
  const TcLayout t = tc_layout(d, a.M);
  char* ws = static_cast<char*>(workspace);
  Layouts p = {};
  p.x = -1, p.rows_w = d.N, p.rows_x = a.M, p.K = d.K, p.pitch = t.pitch, p.ldx = a.ldx;
  int n = 0;
  size_t most = 0;
  auto add = [&](const void* from, const float* sc, size_t to, size_t rows) {
    p.from[n] = from, p.s[n] = sc, p.to[n] = reinterpret_cast<uint16_t*>(ws + to);
    most = std::max(most, rows * t.pitch);
    ++n;
  };
  for (int i = 0; t.w_copy && i < (d.W_up ? 2 : 1); ++i) add(a.W[i], a.s[i], t.w[i], (size_t)d.N);
  if (t.xparts == 3) {
    p.x = n;
    add(a.x, nullptr, t.x, (size_t)a.M);
  }
  const size_t blocks = (most / 8 + 256 * kItems - 1) / (256 * kItems);
  const dim3 grid((unsigned)std::min<size_t>(blocks, (size_t)num_sms * 8), n);
  auto go = [&](auto kernel) { return launch_k(kernel, grid, dim3(256), 0, s, p); };
  auto int4 = [&](auto format) {
    constexpr int WF = decltype(format)::value;
    return t.wparts == 1 ? go(linear_layout_kernel<WF, 1>) : (t.wparts == 2 ? go(linear_layout_kernel<WF, 2>) : go(linear_layout_kernel<WF, 3>));
  };
  switch (d.wfmt) {
    case MOE_W_INT8_ROW: return go(linear_layout_kernel<MOE_W_INT8_ROW, 1>);
    case MOE_W_INT4_B32: return int4(std::integral_constant<int, MOE_W_INT4_B32>());
    case MOE_W_INT4_B128: return int4(std::integral_constant<int, MOE_W_INT4_B128>());
    default: return go(linear_layout_kernel<MOE_W_F32, 3>);  // fp32 weights, or fp32 tokens alone
  }
}

static TcArgs tc_args(const moe_linear_desc& d, const LinearArgs& a, const TcLayout& t, void* workspace) {
  TcArgs p = {};
  p.l = a;
  p.row_scales = d.wfmt == MOE_W_INT8_ROW;
  p.mt = t.mt, p.nt = t.nt, p.splits = t.splits, p.ksteps = t.ksteps, p.segment = t.segment;
  p.xparts = t.xparts, p.wparts = t.wparts, p.np = t.np;
  p.xfmt = d.xfmt, p.wfmt = d.wfmt, p.again = t.xparts > 1 || t.wparts > 1;
  const int yb = d.yfmt == MOE_X_F32 ? 4 : 2;
  auto pieces = [&](const void* q, long long ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * yb % 16 == 0; };
  p.vec = pieces(a.y, a.ldy) && (!a.residual || pieces(a.residual, a.ldr));
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + t.partial);
  return p;
}

cudaError_t launch_linear_tc(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, uint32_t* flags,
                             cudaStream_t s) {
  const TcLayout t = tc_layout(d, a.M);
  const TcArgs p = tc_args(d, a, t, workspace);
  const bool gated = d.W_up != nullptr;
  char* ws = static_cast<char*>(workspace);
  CUtensorMap mx, mw[2];
  const void* x = t.xparts == 3 ? ws + t.x : a.x;
  cudaError_t e = make_tmap(&mx, x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)d.K, (uint64_t)a.M * t.xparts,
                            t.xparts == 3 ? (uint64_t)t.pitch * 2 : (uint64_t)a.ldx * 2, kK, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
  for (int i = 0; i < (gated ? 2 : 1) && e == cudaSuccess; ++i)
    e = make_tmap(&mw[i], t.w_copy ? ws + t.w[i] : a.W[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)d.K,
                  (uint64_t)d.N * t.wparts, t.wparts > 1 ? (uint64_t)t.pitch * 2 : (uint64_t)d.K * 2, kK, kRows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  if (!gated) mw[1] = mw[0];
  // a split that is one segment long needs no segments
  const bool seg = t.segment > 0 && (t.ksteps + t.splits - 1) / t.splits > t.segment;
  auto pick = [&](auto parts) {
    constexpr bool P = decltype(parts)::value;
    return gated ? (seg ? linear_tc_kernel<true, true, P> : linear_tc_kernel<true, false, P>)
                 : (seg ? linear_tc_kernel<false, true, P> : linear_tc_kernel<false, false, P>);
  };
  auto kernel = p.again ? pick(std::true_type()) : pick(std::false_type());
  static std::atomic<bool> allowed[8][64];
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, allowed[4 * p.again + 2 * seg + gated]);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)t.mt * t.nt * t.splits;
  const int pairs = (int)std::min<long long>(tiles, num_sms / 2);
  return launch_next(!linear_tc_layouts(d), kernel, dim3(2 * pairs), dim3(kThreads), kSmem, s, mx, mw[0], mw[1], p, flags);
}

bool linear_tc_split(const moe_linear_desc& d, int M) { return tc_layout(d, M).splits > 1; }

cudaError_t launch_linear_sum(const moe_linear_desc& d, const LinearArgs& a, void* workspace, int num_sms, cudaStream_t s) {
  const TcLayout t = tc_layout(d, a.M);
  return launch_next(false, linear_sum_kernel, grid_for((size_t)a.M * t.np / 4, num_sms), dim3(256), 0, s, tc_args(d, a, t, workspace));
}

}  // namespace moe
