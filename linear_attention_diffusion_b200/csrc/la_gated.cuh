// Device building blocks of gated linear attention: 16-token tiles in shared
// memory, fragments of the warp-level matrix product, numbers split into bf16
// parts, and the decays of a block.
//
// Matrix products run as mma.sync m16n8k16 on bf16 with float32 sums. Two
// small products follow each other with an elementwise step between them (the
// decay), and one operand of nearly every product is a register result of the
// one before: the accumulator of S^T = sum v k^T is, register for register,
// the operand of q S, and the masked q k^T is that of P V. Kept in registers
// they need no trip through tensor memory, whose 128-row tiles would also do
// 8 times the work of a 16-token block's triangle. mma.sync measured 550
// TFLOP/s on a B200; a forward block (16 tokens of a head) takes 44 of them,
// half the time that its bytes take from HBM.
//
// A float32 number enters a product as a sum of bf16 parts: x = x0 + x1 + ...,
// each the rounding of what the earlier ones leave. Two parts keep 17 bits (a
// relative error of 2^-17 at most per number, 6e-7 in the mean square), three
// keep all 24. bf16 tensors are one part. What the kernels compute (states,
// decayed keys, masked weights) enters with two parts for bf16 tensors and
// three for float32 tensors; every sum is float32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "la_block_internal.h"

namespace la {
namespace gated {

template <int NP>
struct Io;
template <>
struct Io<1> {
  using T = __nv_bfloat16;
};
template <>
struct Io<3> {
  using T = float;
};

constexpr int kPlane = kGateBlock * 64;  // bytes of 16 tokens x 32 bf16
constexpr float kLog2e = 1.4426950408889634f;
// A gate whose decay 2^x is below the smallest float32 lets nothing through:
// it is kept apart from the sums of the others, where it would cost their
// precision (and -inf would give NaN).
constexpr float kStop = -150.0f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Byte offset of the 16-byte chunk `c` (8 bf16) of row `row` in a tile of 64-byte
// rows. The exclusive-or puts the eight rows that one 8x8 matrix load reads into
// eight different 16-byte bank groups.
__device__ __forceinline__ uint32_t tile_off(int row, int c) {
  return static_cast<uint32_t>(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two float32 numbers as kParts pairs of bf16.
template <int kParts>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&out)[kParts]) {
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    out[p] = pack2(x, y);
    if (p + 1 < kParts) {
      x -= lo_f(out[p]);
      y -= hi_f(out[p]);
    }
  }
}

// Offsets a lane uses for the matrix loads of any tile.
struct LaneOff {
  uint32_t a[2];  // rows of a 16x16 operand, columns 16 ks ..; transposed: two 8-column tiles
  uint32_t b[2];  // two 8-row tiles of a column operand, columns 16 ks ..
  __device__ __forceinline__ explicit LaneOff(int lane) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      a[ks] = tile_off(lane & 15, 2 * ks + (lane >> 4));
      b[ks] = tile_off((lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
    }
  }
};

// The four ways a 16-token tile enters a product, NP parts each.
//  rows: tokens are the product's rows, the head's 32 dimensions its depth (2 steps)
//  cols: tokens are the product's columns, the dimensions its depth; [ks]: regs 0,1 for
//        tokens 0-7, regs 2,3 for tokens 8-15
//  deep: tokens are the product's depth; [pair]: dimensions 16 pair .. + 15. As columns,
//        regs 0,1 are dimensions 0-7 and regs 2,3 dimensions 8-15 of the pair; as rows the
//        same registers in the order 0, 2, 1, 3.
template <int NP>
struct Frag {
  uint32_t r[NP][2][4];
  __device__ __forceinline__ void rows(uint32_t tile, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4(r[p][ks], tile + p * kPlane + o.a[ks]);
  }
  __device__ __forceinline__ void cols(uint32_t tile, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4(r[p][ks], tile + p * kPlane + o.b[ks]);
  }
  __device__ __forceinline__ void deep(uint32_t tile, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4_t(r[p][ks], tile + p * kPlane + o.a[ks]);
  }
};

// Products of parts that matter: the sum of the part numbers stays below the
// larger number of parts (what is left out is as small as what the parts leave).
constexpr __host__ __device__ bool pair_counts(int i, int j, int pa, int pb) {
  return i + j < (pa > pb ? pa : pb);
}

// s[2] (16 tokens x 16 tokens) = A (tokens as rows) B (tokens as columns), over the dimensions.
template <int NP>
__device__ __forceinline__ void token_product(float (&s)[2][4], const Frag<NP>& A,
                                              const Frag<NP>& B) {
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nt][i] = 0.0f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (pair_counts(i, j, NP, NP)) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma(s[nt], A.r[i][ks], B.r[j][ks][2 * nt], B.r[j][ks][2 * nt + 1]);
      }
}

// acc (16 tokens x 32) += W (16 x 16 weights, an accumulator) X (tokens as depth).
template <int NP, int NC>
__device__ __forceinline__ void weigh(float (&acc)[4][4], const float (&w)[2][4],
                                      const Frag<NP>& X) {
  uint32_t a[NC][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // rows lo / hi of columns 0-7, then of columns 8-15
    uint32_t t[NC];
    const int nt = i >> 1, h = (i & 1) * 2;
    split2<NC>(w[nt][h], w[nt][h + 1], t);
#pragma unroll
    for (int p = 0; p < NC; ++p) a[p][i] = t[p];
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (pair_counts(i, j, NC, NP)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma(acc[e], a[i], X.r[j][e >> 1][2 * (e & 1)], X.r[j][e >> 1][2 * (e & 1) + 1]);
      }
}

// A 32 x 32 float32 state held as accumulators: st[mt][nt] covers rows 16 mt ..,
// columns 8 nt ..; lane l holds rows l / 4 and l / 4 + 8, columns 2 (l % 4) and + 1.
struct State {
  float c[2][4][4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt][nt][i] = 0.0f;
  }
  // From / to the kernels' own layout: 256 float4, tile by tile, lane by lane.
  __device__ __forceinline__ void load(const float* p, int lane) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p) + (mt * 4 + nt) * 32 + lane);
        c[mt][nt][0] = v.x;
        c[mt][nt][1] = v.y;
        c[mt][nt][2] = v.z;
        c[mt][nt][3] = v.w;
      }
  }
  __device__ __forceinline__ void store(float* p, int lane) const {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        reinterpret_cast<float4*>(p)[(mt * 4 + nt) * 32 + lane] =
            make_float4(c[mt][nt][0], c[mt][nt][1], c[mt][nt][2], c[mt][nt][3]);
  }
  // Row-major [32][32] outside; kTransposed: this state's rows are its columns.
  template <bool kTransposed>
  static __device__ __forceinline__ int outer(int mt, int nt, int i, int lane) {
    const int m = mt * 16 + (lane >> 2) + (i >> 1) * 8, n = nt * 8 + (lane & 3) * 2 + (i & 1);
    return kTransposed ? n * 32 + m : m * 32 + n;
  }
  template <bool kTransposed>
  __device__ __forceinline__ void load_outer(const float* p, int lane) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt][nt][i] = p[outer<kTransposed>(mt, nt, i, lane)];
  }
  template <bool kTransposed>
  __device__ __forceinline__ void store_outer(float* p, int lane) const {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[outer<kTransposed>(mt, nt, i, lane)] = c[mt][nt][i];
  }

  // state = decay * state + sum over tokens of w A^T B; A gives the rows, B the columns.
  // w: the weights of tokens 2 (l % 4) + {0, 1, 8, 9}.
  template <int NP, int NC>
  __device__ __forceinline__ void update(float decay, const Frag<NP>& A, const Frag<NP>& B,
                                         const float (&w)[4]) {
    if (decay == 0.0f) {  // the same in all lanes: a stop drops the state whatever it holds
      zero();
    } else {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[mt][nt][i] *= decay;
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t a[NC][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int p = NP - 1; p >= 0; --p) {  // smallest part first: the sum is exact
          x += lo_f(A.r[p][mt][i]);
          y += hi_f(A.r[p][mt][i]);
        }
        uint32_t t[NC];
        split2<NC>(x * w[2 * (i & 1)], y * w[2 * (i & 1) + 1], t);
        const int at = ((i & 1) << 1) | (i >> 1);  // registers 0, 2, 1, 3
#pragma unroll
        for (int p = 0; p < NC; ++p) a[p][at] = t[p];
      }
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < NP; ++j)
            if (pair_counts(i, j, NC, NP))
              mma(c[mt][nt], a[i], B.r[j][nt >> 1][2 * (nt & 1)],
                  B.r[j][nt >> 1][2 * (nt & 1) + 1]);
    }
  }

  // acc (16 tokens x 32) += X (tokens as rows; depth = this state's columns) state^T.
  template <int NP, int NC>
  __device__ __forceinline__ void apply(float (&acc)[4][4], const Frag<NP>& X) const {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t b0[NC], b1[NC];
        const int h = 2 * (e & 1);
        split2<NC>(c[e >> 1][2 * ks][h], c[e >> 1][2 * ks][h + 1], b0);
        split2<NC>(c[e >> 1][2 * ks + 1][h], c[e >> 1][2 * ks + 1][h + 1], b1);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (pair_counts(i, j, NP, NC)) mma(acc[e], X.r[i][ks], b0[j], b1[j]);
      }
  }
  // The same, and acc_t += Y (depth = this state's rows) state, from the same parts:
  // an 8x8 tile turned over is the other product's operand.
  template <int NP, int NC>
  __device__ __forceinline__ void apply_both(float (&acc)[4][4], const Frag<NP>& X,
                                             float (&acc_t)[4][4], const Frag<NP>& Y) const {
#pragma unroll
    for (int e = 0; e < 4; ++e)      // 8 rows of the state
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {  // 16 columns of the state
        uint32_t b0[NC], b1[NC];
        const int h = 2 * (e & 1);
        split2<NC>(c[e >> 1][2 * ks][h], c[e >> 1][2 * ks][h + 1], b0);
        split2<NC>(c[e >> 1][2 * ks + 1][h], c[e >> 1][2 * ks + 1][h + 1], b1);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (pair_counts(i, j, NP, NC)) mma(acc[e], X.r[i][ks], b0[j], b1[j]);
      }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {  // 16 rows (depth) x 8 columns
        uint32_t b0[NC], b1[NC];
        split2<NC>(c[mt][nt][0], c[mt][nt][1], b0);
        split2<NC>(c[mt][nt][2], c[mt][nt][3], b1);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          b0[j] = transpose8(b0[j]);
          b1[j] = transpose8(b1[j]);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (pair_counts(i, j, NP, NC)) mma(acc_t[nt], Y.r[i][mt], b0[j], b1[j]);
      }
  }
  __device__ __forceinline__ float dot(const State& o) const {
    float s = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(c[mt][nt][i], o.c[mt][nt][i], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
  }
};

// Scale one row of an accumulator; a factor of zero drops it whatever it holds.
__device__ __forceinline__ void scale_row(float (&acc)[4][4], int h, float f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e][2 * h] = f == 0.0f ? 0.0f : acc[e][2 * h] * f;
    acc[e][2 * h + 1] = f == 0.0f ? 0.0f : acc[e][2 * h + 1] * f;
  }
}

// The decays of a block of 16 tokens. Lane l stands for token i = l % 16; c is the sum of
// log2 gates from the block's first token to token i (stops left out), kept as a float32
// and what its rounding left: a decay is the difference of two sums, and gates of -100
// would otherwise cost the small gates next to them 7 bits of their exponent.
struct Decay {
  float c, low;    // sum at token i: c + low
  float last, last_low;  // the same at the block's last token
  uint32_t stops;  // bit i: token i's gate lets nothing through
  __device__ __forceinline__ Decay(float g, int lane) {
    float x = g * kLog2e;
    const bool stop = x < kStop;
    stops = __ballot_sync(0xffffffffu, stop) & 0xffffu;
    if (stop) x = 0.0f;
    low = 0.0f;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, x, d, 16);
      const float yl = __shfl_up_sync(0xffffffffu, low, d, 16);
      if ((lane & 15) >= d) {
        const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);  // s + what it rounds off
        low += yl + (__fsub_rn(x, __fsub_rn(s, t)) + __fsub_rn(y, t));
        x = s;
      }
    }
    c = x;
    last = __shfl_sync(0xffffffffu, c, 15);
    last_low = __shfl_sync(0xffffffffu, low, 15);
  }
  // from the state before the block to token i
  __device__ __forceinline__ float head(int lane) const {
    return (stops & ((2u << (lane & 15)) - 1u)) ? 0.0f : exp2_fast(c);
  }
  // from token i to the block's end
  __device__ __forceinline__ float tail(int lane) const {
    return (stops >> ((lane & 15) + 1)) ? 0.0f : exp2_fast((last - c) + (last_low - low));
  }
  __device__ __forceinline__ float whole() const { return stops ? 0.0f : exp2_fast(last); }
  // of `x`, one value per token: the values of tokens 2 (l % 4) + {0, 1, 8, 9}
  static __device__ __forceinline__ void spread(float x, int lane, float (&out)[4]) {
    const int j = 2 * (lane & 3);
    out[0] = __shfl_sync(0xffffffffu, x, j);
    out[1] = __shfl_sync(0xffffffffu, x, j + 1);
    out[2] = __shfl_sync(0xffffffffu, x, j + 8);
    out[3] = __shfl_sync(0xffffffffu, x, j + 9);
  }
  // Decays of an accumulator of 16 x 16 tokens: l[h][x] belongs to row token l / 4 + 8 h
  // and column token 2 (l % 4) + {0, 1, 8, 9}; from the earlier to the later of the two,
  // rows the later ones (kRowsLater) or the earlier ones. Pairs in the other order, or with
  // a stop between them (the later token's own included), give 0.
  template <bool kRowsLater>
  __device__ __forceinline__ void between(int lane, float (&l)[2][4]) const {
    float cc[4], cl[4];
    spread(c, lane, cc);
    spread(low, lane, cl);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (lane >> 2) + 8 * h;
      const float cr = __shfl_sync(0xffffffffu, c, row);
      const float lr = __shfl_sync(0xffffffffu, low, row);
      int first, end;  // the column tokens that count
      if (kRowsLater) {
        const uint32_t before = stops & ((2u << row) - 1u);
        first = before != 0 ? 31 - __clz(before) : 0;
        end = row + 1;
      } else {
        const uint32_t after = stops & ~((2u << row) - 1u);
        first = row;
        end = after != 0 ? __ffs(after) - 1 : 16;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int col = 2 * (lane & 3) + (x & 1) + 8 * (x >> 1);
        const float d = (cr - cc[x]) + (lr - cl[x]);
        l[h][x] = (col >= first && col < end) ? exp2_fast(kRowsLater ? d : -d) : 0.0f;
      }
    }
  }
};

// Shared memory of one warp: kStages stages of NT tiles and two lines of 16 floats
// (the gates and one more value per token); float32 tiles arrive as they are and are
// split into three bf16 planes before use (the first NS of them).
template <int NP, int NT, int kStages, int NS = NT>
struct Smem {
  static constexpr int kTile = NP == 1 ? kPlane : kGateBlock * 128;
  static constexpr int kStage = NT * kTile + 128;
  static constexpr int kPlanes = NP == 1 ? 0 : NS * 3 * kPlane;
  static constexpr int kWarp = kStages * kStage + kPlanes;
};

// 16-byte chunk of a float32 tile (rows of 128 bytes); the exclusive-or keeps the
// 32-byte reads of the split free of bank conflicts.
__device__ __forceinline__ uint32_t tile_off_f32(int row, int c16) {
  return static_cast<uint32_t>(row * 128 + ((c16 ^ (row & 1)) << 4));
}

// Start the copy of tokens [n0, n0 + 16) of one head; rows at or past `N` become zero.
template <int NP>
__device__ __forceinline__ void load_tile(uint32_t dst, const typename Io<NP>::T* base,
                                          size_t stride, int n0, int N, int lane) {
  constexpr int kRow = NP == 1 ? 4 : 8;  // 16-byte chunks of a row
  constexpr int kElems = NP == 1 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < kRow / 2; ++i) {
    const int idx = lane + 32 * i, row = idx / kRow, c = idx % kRow;
    const bool in = n0 + row < N;
    const typename Io<NP>::T* src = base + (in ? static_cast<size_t>(n0 + row) * stride : 0) +
                                    c * kElems;
    cp16(dst + (NP == 1 ? tile_off(row, c) : tile_off_f32(row, c)), src, in ? 16 : 0);
  }
}

// float32 tile -> three bf16 planes.
__device__ __forceinline__ void split_tile(const uint8_t* src, uint8_t* planes, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int idx = lane + 32 * i, row = idx >> 2, c = idx & 3;
    const float4 a = *reinterpret_cast<const float4*>(src + tile_off_f32(row, 2 * c));
    const float4 b = *reinterpret_cast<const float4*>(src + tile_off_f32(row, 2 * c + 1));
    uint32_t w[4][3];
    split2<3>(a.x, a.y, w[0]);
    split2<3>(a.z, a.w, w[1]);
    split2<3>(b.x, b.y, w[2]);
    split2<3>(b.z, b.w, w[3]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(planes + p * kPlane + tile_off(row, c)) =
          make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
  }
}

// acc (16 tokens x 32, accumulators) through shared memory to rows of the tensor.
template <int NP>
__device__ __forceinline__ void store_tile(const float (&acc)[4][4], uint8_t* tile,
                                           typename Io<NP>::T* base, size_t stride, int n0, int N,
                                           int lane) {
  const int r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = r + 8 * h;
      if (NP == 1)
        *reinterpret_cast<uint32_t*>(tile + tile_off(row, e) + q * 4) =
            pack2(acc[e][2 * h], acc[e][2 * h + 1]);
      else
        *reinterpret_cast<float2*>(tile + tile_off_f32(row, 2 * e + (q >> 1)) + (q & 1) * 8) =
            make_float2(acc[e][2 * h], acc[e][2 * h + 1]);
    }
  __syncwarp();
  constexpr int kRow = NP == 1 ? 4 : 8;
  constexpr int kElems = NP == 1 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < kRow / 2; ++i) {
    const int idx = lane + 32 * i, row = idx / kRow, c = idx % kRow;
    const uint4 v = *reinterpret_cast<const uint4*>(
        tile + (NP == 1 ? tile_off(row, c) : tile_off_f32(row, c)));
    if (n0 + row < N)
      *reinterpret_cast<uint4*>(base + static_cast<size_t>(n0 + row) * stride + c * kElems) = v;
  }
}

// Sum over the 32 dimensions of acc * X, X the tile as it lies in shared memory
// (bf16 or float32): the values of tokens l / 4 and l / 4 + 8, in every lane of the four.
template <int NP>
__device__ __forceinline__ void row_dots(const float (&acc)[4][4], const uint8_t* tile, int lane,
                                         float (&out)[2]) {
  const int r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x, y;
      if (NP == 1) {
        const uint32_t v =
            *reinterpret_cast<const uint32_t*>(tile + tile_off(r + 8 * h, e) + q * 4);
        x = lo_f(v);
        y = hi_f(v);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(
            tile + tile_off_f32(r + 8 * h, 2 * e + (q >> 1)) + (q & 1) * 8);
        x = v.x;
        y = v.y;
      }
      s = fmaf(acc[e][2 * h], x, fmaf(acc[e][2 * h + 1], y, s));
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    out[h] = s;
  }
}

}  // namespace gated
}  // namespace la
