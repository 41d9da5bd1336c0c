// Weight streaming on warp-wide matrix instructions: 16 stored weight rows from shared
// memory times a few columns (tokens) of bf16.
//
// At a few tokens every weight is used once or a few times, so the rate is set by how many
// weight bytes an SM can take in and by the instructions spent on each.  One m16n8k16
// instruction multiplies 256 weights with up to 8 tokens, where fp32 lanes would need 8 per
// token, and takes bf16 weights as they lie in memory: a dot product may visit its terms in
// any order as long as both operands agree, so a lane reads 16 consecutive bytes of a row
// and the same columns of the token, and no transposition is needed.  (The tensor cores'
// tcgen05 form wants 64 rows and 8 tokens at least and its operands in swizzled tiles; with
// the HBM stream as the bound there is nothing left for it to win here.)
// Quantised codes are widened exactly:
//   int8  q = (128 + low 7 bits) - (128 or 256 by the sign bit), both terms exact in bf16
//   int4  the code (q + 8) goes into the upper mantissa bits of 16: 16 + (q + 8) = q + 24;
//         an instruction with -24 in every place of the weights takes 24 x out again
// int8 rows are scaled in the caller's epilogue, int4 blocks here, in fp32.
//
// Widening takes more instructions than everything else.  Where a token can be prepared
// beforehand (mac_box_digits) the codes stay integers and the token becomes four signed
// digits of 8 bits,  x = 2^(e - 30) (d0 + 2^8 d1 + 2^16 d2 + 2^24 d3),  |x| < 2^e for the whole
// token, each digit a column of its own of an integer matrix instruction: sums are exact,
// and only the rounding of x to 2^(e - 31) (the 31st bit below the token's largest value; a
// bf16 value keeps all its bits down to 2^-22 of that) stands for the 8 bits of each bf16
// product.  Measured in the few-token layer: 4 tokens int8 117 us with widened codes and 108
// with digits, 16 tokens 255 and 240.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace stream {

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b + c, with c kept
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }

// one three-input logic instruction each: (v & mask) | bits, (v & mask) ^ bits
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}

// bytes 0 and 2 of w (int8) as a bf16 pair
__device__ __forceinline__ uint32_t widen_int8(uint32_t w) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;"
      : "=r"(r)
      : "r"(and_or(w, 0x007F007Fu, 0x43004300u)), "r"(and_or(w, 0x00800080u, 0xC300C300u)));
  return r;
}

constexpr uint32_t kMinus24 = 0xC1C0C1C0u;  // bf16 pair of -24

// columns j and j + 4 of the 8 int4 codes in w as a bf16 pair of q + 24
__device__ __forceinline__ uint32_t widen_int4(uint32_t w, int j) {
  const uint32_t v = j == 0 ? w << 3 : w >> (4 * j - 3);
  return and_xor(v, 0x00780078u, 0x41C041C0u);
}

// the same columns as a bf16 pair of q itself: (16 + low 3 bits) - (16 or 24 by the sign bit)
__device__ __forceinline__ uint32_t widen_int4_signed(uint32_t w, int j) {
  const uint32_t v = j == 0 ? w << 3 : w >> (4 * j - 3);
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;"
      : "=r"(r)
      : "r"(and_or(v, 0x00380038u, 0x41804180u)), "r"(and_or(v, 0x00400040u, 0xC180C180u)));
  return r;
}

template <int WF>
struct Format {
  static constexpr bool kInt4 = WF == MOE_W_INT4_B32 || WF == MOE_W_INT4_B128;
  static constexpr int kBits = WF == MOE_W_BF16 ? 16 : (WF == MOE_W_INT8_ROW ? 8 : 4);
  static constexpr int kScaleShift = WF == MOE_W_INT4_B128 ? 7 : 5;  // log2 of the int4 scale block
  static constexpr int kBoxCols = 128 * 8 / kBits;                   // columns of a box
  static constexpr int kLoads = kBoxCols / 32;                       // 16-byte token loads of a lane per box
  // int4 block 32: the 8 scales of a box's 16 rows come as a box of their own (block 128 has
  // two per row and box, less than TMA copies)
  static constexpr bool kScaleBoxes = WF == MOE_W_INT4_B32;
  static constexpr int kScaleBox = kScaleBoxes ? 16 * 32 : 0;
};

constexpr int kBoxRows = 16;
constexpr int kBoxBytes = kBoxRows * 128;  // 16 rows x 128 bytes

// Where the int4 block scales of one box's rows are.
struct Scales {
  uint32_t box;     // shared address of the scale box, where there is one (in_box)
  bool in_box;
  const float* s0;  // else those of the lane's rows g and g + 8, from the box's first column on
  const float* s8;
  int left;         // columns of the matrix from the box's first column on
};

// int4 block scales of the lane's rows g and g + 8 for the four units of half h of a box
template <int WF, bool BOXED>
__device__ __forceinline__ void load_block_scales(const Scales& sc, int h, float (&s0)[4], float (&s8)[4]) {
  using F = Format<WF>;
  if constexpr (BOXED) {
    const uint32_t at = sc.box + (lane_id() >> 2) * 32 + h * 16;
    const uint4 a = ld_shared_v4(at), b = ld_shared_v4(at + 256);
    s0[0] = __uint_as_float(a.x), s0[1] = __uint_as_float(a.y), s0[2] = __uint_as_float(a.z), s0[3] = __uint_as_float(a.w);
    s8[0] = __uint_as_float(b.x), s8[1] = __uint_as_float(b.y), s8[2] = __uint_as_float(b.z), s8[3] = __uint_as_float(b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // boxes reach past the end of a reduction that is no multiple of theirs: zero weights
      const int col = 128 * h + 32 * i;
      const bool in = col < sc.left;
      s0[i] = in ? __ldg(sc.s0 + (col >> F::kScaleShift)) : 0.f;
      s8[i] = in ? __ldg(sc.s8 + (col >> F::kScaleShift)) : 0.f;
    }
  }
}

// The columns of the lane's token for one box; `tok` points at the box's first column, `left`
// columns follow there.  Past the end of a reduction that is no multiple of a box the
// weights read as zero, and so must the token.
template <int WF>
__device__ __forceinline__ void load_token(const uint16_t* tok, int left, uint4 (&x)[Format<WF>::kLoads]) {
  using F = Format<WF>;
  const int c = lane_id() & 3;
  // int4: word c of each unit; else the lane's 32 bytes of the box, units 2c and 2c + 1
  const int first = F::kInt4 ? 8 * c : (F::kBoxCols / 4) * c;
  constexpr int kNext = F::kInt4 ? 32 : 8;
  if (left >= F::kBoxCols) {
#pragma unroll
    for (int i = 0; i < F::kLoads; ++i) x[i] = *reinterpret_cast<const uint4*>(tok + first + kNext * i);
  } else {
#pragma unroll
    for (int i = 0; i < F::kLoads; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (first + kNext * i < left) x[i] = *reinterpret_cast<const uint4*>(tok + first + kNext * i);
    }
  }
}

// acc[mt] += box mt (16 rows x 128 bytes at `boxes` + mt kBoxBytes) times the token columns x.
// The weights lie as TMA puts them: the 16-byte unit u of row r at unit u ^ (r & 7).  Lane
// 4g + c works on rows g and g + 8.  A quad reads units {0, 2, 4, 6}, then {1, 3, 5, 7} of a row
// (lane c: 2c and 2c + 1), so that the two rows of an eight-lane phase fall into different
// banks; int4 lanes read word c of each unit.
template <int WF, int MT, bool BOXED>
__device__ __forceinline__ void mac_box_as(uint32_t boxes, const uint4 (&x)[Format<WF>::kLoads], const Scales (&sc)[MT],
                                           float (&acc)[MT][4]) {
  using F = Format<WF>;
  const int g = lane_id() >> 2, c = lane_id() & 3;
  const uint32_t row = boxes + g * 128;
  if constexpr (WF == MOE_W_BF16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = row + (((2 * c + h) ^ g) << 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 a = ld_shared_v4(at + mt * kBoxBytes), b = ld_shared_v4(at + mt * kBoxBytes + 1024);
        mma16816(acc[mt], a.x, b.x, a.y, b.y, x[h].x, x[h].y);
        mma16816(acc[mt], a.z, b.z, a.w, b.w, x[h].z, x[h].w);
      }
    }
  } else if constexpr (WF == MOE_W_INT8_ROW) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = row + (((2 * c + h) ^ g) << 4);
      uint32_t t[4][2];  // token pairs in the order the widening leaves the codes in: (0, 2), (1, 3)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = x[2 * h + (i >> 1)];
        const uint32_t lo = (i & 1) ? v.z : v.x, hi = (i & 1) ? v.w : v.y;
        t[i][0] = __byte_perm(lo, hi, 0x5410);
        t[i][1] = __byte_perm(lo, hi, 0x7632);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 av = ld_shared_v4(at + mt * kBoxBytes), bv = ld_shared_v4(at + mt * kBoxBytes + 1024);
        const uint32_t a[4] = {av.x, av.y, av.z, av.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma16816(acc[mt], widen_int8(a[i]), widen_int8(b[i]), widen_int8(a[i] >> 8), widen_int8(b[i] >> 8), t[i][0],
                   t[i][1]);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s0[MT][4], s8[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) load_block_scales<WF, BOXED>(sc[mt], h, s0[mt], s8[mt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = x[4 * h + i];
        const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
        const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(d, kMinus24, kMinus24, kMinus24, kMinus24, b0, b1);
        mma16816(d, kMinus24, kMinus24, kMinus24, kMinus24, b2, b3);
        const uint32_t at = row + (((4 * h + i) ^ g) << 4) + 4 * c;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t a = ld_shared_u32(at + mt * kBoxBytes), b = ld_shared_u32(at + mt * kBoxBytes + 1024);
          float q[4];
          mma16816(q, widen_int4(a, 0), widen_int4(b, 0), widen_int4(a, 1), widen_int4(b, 1), b0, b1, d);
          mma16816(q, widen_int4(a, 2), widen_int4(b, 2), widen_int4(a, 3), widen_int4(b, 3), b2, b3);
          acc[mt][0] = fmaf(q[0], s0[mt][i], acc[mt][0]);
          acc[mt][1] = fmaf(q[1], s0[mt][i], acc[mt][1]);
          acc[mt][2] = fmaf(q[2], s8[mt][i], acc[mt][2]);
          acc[mt][3] = fmaf(q[3], s8[mt][i], acc[mt][3]);
        }
      }
    }
  }
}

// Where the scales are is asked once per box, here: a branch in the loop over the units would keep
// the compiler from overlapping one unit's instructions with the next one's, and a unit is a
// chain of some 80 cycles.
template <int WF, int MT>
__device__ __forceinline__ void mac_box(uint32_t boxes, const uint4 (&x)[Format<WF>::kLoads], const Scales (&sc)[MT],
                                        float (&acc)[MT][4]) {
  if (Format<WF>::kScaleBoxes && sc[0].in_box) mac_box_as<WF, MT, Format<WF>::kScaleBoxes>(boxes, x, sc, acc);
  else mac_box_as<WF, MT, false>(boxes, x, sc, acc);
}

// The same for several tiles of 8 tokens: every code is widened once for all of them, int4 with its
// sign, as the products with -24 would be needed for every tile.  The token columns are loaded
// here, piece by piece: load(nt, i) is the i-th 16-byte piece of the lane's token of tile nt (in
// load_token's order).  No branch on the number of tiles keeps a later unit's loads back.
template <int WF, int MT, int NT, bool BOXED, typename Load>
__device__ __forceinline__ void mac_box_tiles_as(uint32_t boxes, Load load, const Scales (&sc)[MT],
                                                 float (&acc)[MT][NT][4]) {
  using F = Format<WF>;
  const int g = lane_id() >> 2, c = lane_id() & 3;
  const uint32_t row = boxes + g * 128;
  if constexpr (!F::kInt4) {
    constexpr int kHalf = F::kLoads / 2;  // pieces of half a box
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 x[NT][kHalf];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
          x[nt][i] = load(nt, h * kHalf + i);
      const uint32_t at = row + (((2 * c + h) ^ g) << 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 av = ld_shared_v4(at + mt * kBoxBytes), bv = ld_shared_v4(at + mt * kBoxBytes + 1024);
        if constexpr (WF == MOE_W_BF16) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(acc[mt][nt], av.x, bv.x, av.y, bv.y, x[nt][0].x, x[nt][0].y);
            mma16816(acc[mt][nt], av.z, bv.z, av.w, bv.w, x[nt][0].z, x[nt][0].w);
          }
        } else {
          const uint32_t a[4] = {av.x, av.y, av.z, av.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = widen_int8(a[i]), a1 = widen_int8(b[i]), a2 = widen_int8(a[i] >> 8), a3 = widen_int8(b[i] >> 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 v = x[nt][i >> 1];
              const uint32_t lo = (i & 1) ? v.z : v.x, hi = (i & 1) ? v.w : v.y;
              mma16816(acc[mt][nt], a0, a1, a2, a3, __byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
            }
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s0[MT][4], s8[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) load_block_scales<WF, BOXED>(sc[mt], h, s0[mt], s8[mt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 x[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          x[nt] = load(nt, 4 * h + i);
        const uint32_t at = row + (((4 * h + i) ^ g) << 4) + 4 * c;
        uint32_t wa[MT][4], wb[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t a = ld_shared_u32(at + mt * kBoxBytes), b = ld_shared_u32(at + mt * kBoxBytes + 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) wa[mt][k] = widen_int4_signed(a, k), wb[mt][k] = widen_int4_signed(b, k);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = __byte_perm(x[nt].x, x[nt].z, 0x5410), b1 = __byte_perm(x[nt].x, x[nt].z, 0x7632);
          const uint32_t b2 = __byte_perm(x[nt].y, x[nt].w, 0x5410), b3 = __byte_perm(x[nt].y, x[nt].w, 0x7632);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float q[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(q, wa[mt][0], wb[mt][0], wa[mt][1], wb[mt][1], b0, b1);
            mma16816(q, wa[mt][2], wb[mt][2], wa[mt][3], wb[mt][3], b2, b3);
            acc[mt][nt][0] = fmaf(q[0], s0[mt][i], acc[mt][nt][0]);
            acc[mt][nt][1] = fmaf(q[1], s0[mt][i], acc[mt][nt][1]);
            acc[mt][nt][2] = fmaf(q[2], s8[mt][i], acc[mt][nt][2]);
            acc[mt][nt][3] = fmaf(q[3], s8[mt][i], acc[mt][nt][3]);
          }
        }
      }
    }
  }
}

template <int WF, int MT, int NT, typename Load>
__device__ __forceinline__ void mac_box_tiles(uint32_t boxes, Load load, const Scales (&sc)[MT],
                                              float (&acc)[MT][NT][4]) {
  if (Format<WF>::kScaleBoxes && sc[0].in_box) mac_box_tiles_as<WF, MT, NT, Format<WF>::kScaleBoxes>(boxes, load, sc, acc);
  else mac_box_tiles_as<WF, MT, NT, false>(boxes, load, sc, acc);
}

// ---------------------------------------------------------------- tokens as digits

// d = a b + c, signed 8-bit integers, 32 columns of the reduction
__device__ __forceinline__ void imma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, int c0, int c1, int c2, int c3) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

constexpr int kDigitTokens = 2;  // of a tile: column 4 t + d is digit d of token t
// bytes of a digit's row: whole boxes, so that no load has to ask where the columns end (the
// weights past them read as zero)
__host__ __device__ inline int digit_pitch(int K) { return (K + 255) / 256 * 256; }

// A token's digits, [4][pitch], and what a unit of the lowest one stands for, by one block.
// int4: the even columns of each 8 come before the odd ones, as the codes are taken apart.
// A token with an infinity or NaN becomes NaN as a whole.
__device__ __forceinline__ void write_digits(const uint16_t* x, int K, bool int4, int8_t* out, float* unit, float* smem) {
  const int tid = threadIdx.x, threads = blockDim.x, pitch = digit_pitch(K);
  float m = 0.f;
  bool bad = false;
  for (int c = tid * 8; c < K; c += threads * 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + c));
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = fabsf(bf16_to_f32(word[j] & 0xFFFFu)), b = fabsf(__uint_as_float(word[j] & 0xFFFF0000u));
      m = fmaxf(m, fmaxf(a, b));
      bad |= !isfinite(a) || !isfinite(b);
    }
  }
  // magnitudes are ordered like their bits; a value that is not finite is above all
  uint32_t bits = bad ? 0x7F800000u : __float_as_uint(m);
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if (lane_id() == 0) smem[warp_id()] = __uint_as_float(bits);
  __syncthreads();
  for (int w = 0; w < threads / 32; ++w) bits = max(bits, __float_as_uint(smem[w]));
  const bool finite = bits < 0x7F800000u;
  const int e = max((int)(bits >> 23) - 126, -90);  // |x| < 2^e; what lies below 2^-121 is dropped
  const float scale = __uint_as_float((uint32_t)(127 + 30 - e) << 23);
  if (tid == 0) *unit = finite ? __uint_as_float((uint32_t)(127 - 30 + e) << 23) : __uint_as_float(0x7FC00000u);
  for (int c = tid * 8; c < pitch; c += threads * 8) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (c < K && finite) u = __ldg(reinterpret_cast<const uint4*>(x + c));
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
    uint32_t d[4][2] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = (j & 1) ? __uint_as_float(word[j >> 1] & 0xFFFF0000u) : bf16_to_f32(word[j >> 1] & 0xFFFFu);
      int v = __float2int_rn(f * scale);
      const int at = int4 ? (j >> 1) + 4 * (j & 1) : j;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int digit = (int)(int8_t)v;
        d[k][at >> 2] |= (uint32_t)(digit & 255) << (8 * (at & 3));
        v = (v - digit) >> 8;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint2*>(out + (size_t)k * pitch + c) = make_uint2(d[k][0], d[k][1]);
  }
  __syncthreads();
}

template <int WF>
struct Bf16Columns {
  uint4 v[Format<WF>::kLoads];
};

// The lane's digits for one box: 2 x 16 bytes (int8: units 2c and 2c + 1) or 8 x 8 bytes (int4: word
// c of each unit); `row` is the digit's row of the lane's token, from the box's first column on.
template <int WF>
struct Digits {
  uint32_t v[Format<WF>::kInt4 ? 16 : 8];
};
template <int WF>
__device__ __forceinline__ void load_digits(const int8_t* row, Digits<WF>& x) {
  const int c = lane_id() & 3;
  if constexpr (Format<WF>::kInt4) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint2 p = *reinterpret_cast<const uint2*>(row + 32 * u + 8 * c);
      x.v[2 * u] = p.x, x.v[2 * u + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 p = *reinterpret_cast<const uint4*>(row + 32 * c + 16 * h);
      x.v[4 * h] = p.x, x.v[4 * h + 1] = p.y, x.v[4 * h + 2] = p.z, x.v[4 * h + 3] = p.w;
    }
  }
}

// Sums by digit: int8 the whole reduction as integers (at most 2^14 a column, 65,536 columns),
// int4 in fp32 with the block scales applied, 16 times too large.
template <int WF>
using DigitSum = std::conditional_t<Format<WF>::kInt4, float, int>;

// acc[mt][nt] += box mt times the digits of tile nt < TILES
template <int WF, int MT, int NT, int TILES, bool BOXED>
__device__ __forceinline__ void mac_box_digits_as(uint32_t boxes, const Digits<WF> (&x)[NT], const Scales (&sc)[MT],
                                                  DigitSum<WF> (&acc)[MT][NT][4]) {
  using F = Format<WF>;
  const int g = lane_id() >> 2, c = lane_id() & 3;
  const uint32_t row = boxes + g * 128;
  if constexpr (!F::kInt4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = row + (((2 * c + h) ^ g) << 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 a = ld_shared_v4(at + mt * kBoxBytes), b = ld_shared_v4(at + mt * kBoxBytes + 1024);
#pragma unroll
        for (int nt = 0; nt < TILES; ++nt) {
          int(&d)[4] = acc[mt][nt];
          imma16832(d, a.x, b.x, a.y, b.y, x[nt].v[4 * h], x[nt].v[4 * h + 1], d[0], d[1], d[2], d[3]);
          imma16832(d, a.z, b.z, a.w, b.w, x[nt].v[4 * h + 2], x[nt].v[4 * h + 3], d[0], d[1], d[2], d[3]);
        }
      }
    }
  } else {
    // 2^23 + 2^22 as bits: added to an integer below 2^22 it makes the float 12582912 + the integer
    constexpr int kOne = 0x4B400000;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s0[MT][4], s8[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) load_block_scales<WF, BOXED>(sc[mt], h, s0[mt], s8[mt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = row + (((4 * h + i) ^ g) << 4) + 4 * c;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t a = ld_shared_u32(at + mt * kBoxBytes), b = ld_shared_u32(at + mt * kBoxBytes + 1024);
          // a code in the upper half of a byte is 16 times itself: low nibbles (even columns), high ones
          const uint32_t al = (a << 4) & 0xF0F0F0F0u, ah = a & 0xF0F0F0F0u;
          const uint32_t bl = (b << 4) & 0xF0F0F0F0u, bh = b & 0xF0F0F0F0u;
#pragma unroll
          for (int nt = 0; nt < TILES; ++nt) {
            int d[4];
            imma16832(d, al, bl, ah, bh, x[nt].v[8 * h + 2 * i], x[nt].v[8 * h + 2 * i + 1], kOne, kOne, kOne, kOne);
            acc[mt][nt][0] = fmaf(__int_as_float(d[0]) - 12582912.f, s0[mt][i], acc[mt][nt][0]);
            acc[mt][nt][1] = fmaf(__int_as_float(d[1]) - 12582912.f, s0[mt][i], acc[mt][nt][1]);
            acc[mt][nt][2] = fmaf(__int_as_float(d[2]) - 12582912.f, s8[mt][i], acc[mt][nt][2]);
            acc[mt][nt][3] = fmaf(__int_as_float(d[3]) - 12582912.f, s8[mt][i], acc[mt][nt][3]);
          }
        }
      }
    }
  }
}

// for ntiles tiles: one, or all of them (those without a token cost their instructions only)
template <int WF, int MT, int NT>
__device__ __forceinline__ void mac_box_digits(uint32_t boxes, int ntiles, const Digits<WF> (&x)[NT], const Scales (&sc)[MT],
                                               DigitSum<WF> (&acc)[MT][NT][4]) {
  constexpr bool kBoxes = Format<WF>::kScaleBoxes;
  if (kBoxes && sc[0].in_box) {
    if (ntiles == 1) mac_box_digits_as<WF, MT, NT, 1, kBoxes>(boxes, x, sc, acc);
    else mac_box_digits_as<WF, MT, NT, NT, kBoxes>(boxes, x, sc, acc);
  } else {
    if (ntiles == 1) mac_box_digits_as<WF, MT, NT, 1, false>(boxes, x, sc, acc);
    else mac_box_digits_as<WF, MT, NT, NT, false>(boxes, x, sc, acc);
  }
}

// The four digits of a token put together: rows g (r0) and g + 8 (r8) of token lane % 4 / 2, in both
// lanes of a pair.  To be multiplied by the token's unit (and int4 by 1/16).
template <typename T>
__device__ __forceinline__ void join_digits(const T (&acc)[4], float& r0, float& r8) {
  const bool high = lane_id() & 1;  // the lane's columns are digits 0 and 1, or 2 and 3
  const float w0 = high ? 65536.f : 1.f, w1 = high ? 16777216.f : 256.f;
  r0 = fmaf((float)acc[1], w1, (float)acc[0] * w0);
  r8 = fmaf((float)acc[3], w1, (float)acc[2] * w0);
  r0 += __shfl_xor_sync(0xFFFFFFFFu, r0, 1);
  r8 += __shfl_xor_sync(0xFFFFFFFFu, r8, 1);
}

}  // namespace stream
}  // namespace moe
