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
// TFLOP/s on a B200 (a product a scheduler every 4.4 ns, a result after 12.6 ns); a forward
// block (16 tokens of a head) takes 50 of them, half the time that its bytes take from HBM.
//
// A float32 number enters a product as a sum of bf16 parts: x = x0 + x1 + ...,
// each the rounding of what the earlier ones leave. Two parts keep 17 bits (a
// relative error of 2^-17 at most per number, 2.7e-6 in the mean square), three
// keep all 24. bf16 tensors are one part. What the kernels compute (states,
// decayed keys, masked weights) enters with two parts where only a bf16 output depends
// on it, with three where a float32 one does (the state, the gates' gradient) and for
// float32 tensors; every sum is float32. Two parts where a bf16 output follows: one output in
// 300 then rounds to the other neighbour (three parts: one in 4000), the error against 64 bits
// is 1.66e-3 of the 2-norm either way, the output's own rounding, and 32760 tokens of 70 heads
// take 213 us instead of 252, 8 x 509 tokens of 36 heads 19 instead of 25.
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
constexpr float kLog2e = 1.4426950408889634f;     // rounded, and
constexpr float kLog2eRest = 1.925963033500012e-8f;  // the rest of it
// A gate whose decay 2^x is below the smallest float32 lets nothing through:
// it is kept apart from the sums of the others, where it would cost their
// precision (and -inf would give NaN).
constexpr float kStop = -150.0f;
constexpr int kNan = 0x7fffffff;

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
// The store of the same layout: four 8x8 matrices, each lane one row's address.
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                      uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b: the first product of a sum, without zeroing registers for it.
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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

// Float `i` of shared memory at `addr`.
__device__ __forceinline__ float lds(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds2(uint32_t addr) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint4 lds4(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}
__device__ __forceinline__ void sts(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void sts2(uint32_t addr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void sts4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Packed bf16 arithmetic, each result rounded once.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t neg2(uint32_t a) {
  uint32_t d;
  asm("neg.bf16x2 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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
  // `plane`: bytes from one part of the tile to the next
  __device__ __forceinline__ void rows(uint32_t tile, int plane, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4(r[p][ks], tile + p * plane + o.a[ks]);
  }
  __device__ __forceinline__ void cols(uint32_t tile, int plane, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4(r[p][ks], tile + p * plane + o.b[ks]);
  }
  __device__ __forceinline__ void deep(uint32_t tile, int plane, const LaneOff& o) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ldsm4_t(r[p][ks], tile + p * plane + o.a[ks]);
  }
};

// Products of parts that matter: the sum of the part numbers stays below the
// larger number of parts (what is left out is as small as what the parts leave).
constexpr __host__ __device__ bool pair_counts(int i, int j, int pa, int pb) {
  return i + j < (pa > pb ? pa : pb);
}

// Products of parts go into two sums, the leading one (part 0 x part 0) and the rest, which
// are added at the end: the tensor cores cut a sum off after each step instead of rounding
// it, and six more steps on the leading sum would cost it as many half steps.
template <int kN>
__device__ __forceinline__ void zero(float (&c)[kN][4]) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
}
template <int kN>
__device__ __forceinline__ void add(float (&c)[kN][4], const float (&d)[kN][4]) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] += d[i][j];
}

// s[2] (16 tokens x 16 tokens) = A (tokens as rows) B (tokens as columns), over the dimensions.
template <int NP>
__device__ __forceinline__ void token_product(float (&s)[2][4], const Frag<NP>& A,
                                              const Frag<NP>& B) {
  float rest[2][4];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (pair_counts(i, j, NP, NP)) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint32_t b0 = B.r[j][ks][2 * nt], b1 = B.r[j][ks][2 * nt + 1];
            if (i + j == 0) {
              if (ks == 0)
                mma0(s[nt], A.r[i][ks], b0, b1);
              else
                mma(s[nt], A.r[i][ks], b0, b1);
            } else if (ks == 0 && i == 0 && j == 1) {
              mma0(rest[nt], A.r[i][ks], b0, b1);
            } else {
              mma(rest[nt], A.r[i][ks], b0, b1);
            }
          }
        }
  if (NP > 1) add(s, rest);
}

// acc (16 tokens x 32) += W (16 x 16 weights, an accumulator) X (tokens as depth). kZero:
// a quarter of W that is known to be 0 (2 nt + h), or -1.
template <int NP, int NC, int kZero>
__device__ __forceinline__ void weigh(float (&acc)[4][4], const float (&w)[2][4],
                                      const Frag<NP>& X) {
  uint32_t a[NC][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // rows lo / hi of columns 0-7, then of columns 8-15
    uint32_t t[NC];
    const int nt = i >> 1, h = (i & 1) * 2;
    if (i != kZero) split2<NC>(w[nt][h], w[nt][h + 1], t);
#pragma unroll
    for (int p = 0; p < NC; ++p) a[p][i] = i == kZero ? 0u : t[p];
  }
  float rest[4][4];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (pair_counts(i, j, NC, NP)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // four sums in turn: none waits for its own last step
          const uint32_t b0 = X.r[j][e >> 1][2 * (e & 1)], b1 = X.r[j][e >> 1][2 * (e & 1) + 1];
          if (NP == 1 || i + j == 0)
            mma(acc[e], a[i], b0, b1);
          else if (i == 0 && j == 1)
            mma0(rest[e], a[i], b0, b1);
          else
            mma(rest[e], a[i], b0, b1);
        }
      }
  if (NP > 1) add(acc, rest);
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
  // The same in shared memory.
  __device__ __forceinline__ void put(uint32_t at, int lane) const {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        sts4(at + ((mt * 4 + nt) * 32 + lane) * 16, __float_as_uint(c[mt][nt][0]),
             __float_as_uint(c[mt][nt][1]), __float_as_uint(c[mt][nt][2]),
             __float_as_uint(c[mt][nt][3]));
  }
  // state = decay * state + what put() left there; a decay of zero drops it whatever it holds.
  __device__ __forceinline__ void follow(uint32_t at, float decay, int lane) {
    if (decay == 0.0f) zero();
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const uint4 v = lds4(at + ((mt * 4 + nt) * 32 + lane) * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[mt][nt][i] = fmaf(c[mt][nt][i], decay, __uint_as_float(w[i]));
      }
  }
  __device__ __forceinline__ void spoil() {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt][nt][i] = __int_as_float(kNan);
  }
  __device__ __forceinline__ void add_scaled(const State& o, float f) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt][nt][i] = fmaf(o.c[mt][nt][i], f, c[mt][nt][i]);
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

  // state = decay * state + sum over the tokens of NB blocks of w A^T B; A gives the rows,
  // B the columns, w[b] the weights of tokens 2 (l % 4) + {0, 1, 8, 9} of block b.
  // The weighted numbers keep 24 bits (kParts = 3) or 17 (2).
  template <int NP, int NB, int kParts, bool kStops>
  __device__ __forceinline__ void update(float decay, const Frag<NP> (&A)[NB],
                                         const Frag<NP> (&B)[NB], const float (&w)[NB][4]) {
    constexpr int NC = NP == 1 && kParts == 3 ? 4 : kParts == 2 && NP == 1 ? 2 : 3;
    if (kStops && decay == 0.0f) zero();  // a stop drops the state whatever it holds
    uint32_t wp[NB][2][kParts];
    if (NP == 1) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        split2<kParts>(w[b][0], w[b][1], wp[b][0]);
        split2<kParts>(w[b][2], w[b][3], wp[b][1]);
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t a[NB][NC][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = ((i & 1) << 1) | (i >> 1);  // registers 0, 2, 1, 3
          if (NP == 1) {
            // w = w0 + w1 + w2 in bf16 parts: v w0 is exactly its rounding and one more bf16;
            // v w1 likewise, the latter with v w2 added. Packed arithmetic, five instructions
            // for two numbers where a float32 product split three ways takes fifteen. With two
            // parts v w1 is added to what the rounding of v w0 left.
            const uint32_t(&x)[kParts] = wp[b][i & 1];
            const uint32_t v = A[b].r[0][mt][i];
            const uint32_t p0 = mul2(v, x[0]), left = fma2(v, x[0], neg2(p0));
            a[b][0][at] = p0;
            if (NC == 4) {
              const uint32_t p2 = mul2(v, x[1]);
              a[b][1][at] = left;
              a[b][NC - 2][at] = p2;
              a[b][NC - 1][at] = fma2(v, x[kParts - 1], fma2(v, x[1], neg2(p2)));
            } else {
              a[b][1][at] = fma2(v, x[1], left);
            }
          } else {
            float f = 0.0f, g = 0.0f;
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) {  // smallest part first: the sum is exact
              f += lo_f(A[b].r[p][mt][i]);
              g += hi_f(A[b].r[p][mt][i]);
            }
            uint32_t t[NC];
            split2<NC>(f * w[b][2 * (i & 1)], g * w[b][2 * (i & 1) + 1], t);
#pragma unroll
            for (int p = 0; p < NC; ++p) a[b][p][at] = t[p];
          }
        }
      // the blocks' own sum by itself, so that the state is rounded once
      float own[4][4], rest[4][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < NP; ++j)
            if (pair_counts(i, j, NC, NP)) {
#pragma unroll
              for (int nt = 0; nt < 4; ++nt) {
                const uint32_t b0 = B[b].r[j][nt >> 1][2 * (nt & 1)],
                               b1 = B[b].r[j][nt >> 1][2 * (nt & 1) + 1];
                if (NP == 1 || i + j == 0) {
                  if (b == 0 && i == 0)
                    mma0(own[nt], a[b][i], b0, b1);
                  else
                    mma(own[nt], a[b][i], b0, b1);
                } else if (b == 0 && i == 0 && j == 1) {
                  mma0(rest[nt], a[b][i], b0, b1);
                } else {
                  mma(rest[nt], a[b][i], b0, b1);
                }
              }
            }
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[mt][nt][i] = fmaf(c[mt][nt][i], decay, NP > 1 ? own[nt][i] + rest[nt][i] : own[nt][i]);
    }
  }

  // acc[b] (16 tokens x 32) = X[b] (tokens as rows; depth = this state's columns) state^T,
  // the state in NC parts.
  template <int NP, int NC, int NB>
  __device__ __forceinline__ void apply(float (&acc)[NB][4][4], const Frag<NP> (&X)[NB]) const {
    float rest[NB][4][4];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {  // 16 columns of the state
      uint32_t b0[4][NC], b1[4][NC];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // 8 rows of the state
        const int h = 2 * (e & 1);
        split2<NC>(c[e >> 1][2 * ks][h], c[e >> 1][2 * ks][h + 1], b0[e]);
        split2<NC>(c[e >> 1][2 * ks + 1][h], c[e >> 1][2 * ks + 1][h + 1], b1[e]);
      }
      product<NP, NC, NB>(acc, rest, X, ks, b0, b1);
    }
    if (NP > 1) {
#pragma unroll
      for (int b = 0; b < NB; ++b) add(acc[b], rest[b]);
    }
  }
  // acc[b] = Y[b] (tokens as rows; depth = this state's rows) state: an 8x8 tile of the
  // state turned over is the operand.
  template <int NP, int NC, int NB>
  __device__ __forceinline__ void apply_turned(float (&acc)[NB][4][4],
                                               const Frag<NP> (&Y)[NB]) const {
    float rest[NB][4][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t b0[4][NC], b1[4][NC];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        split2<NC>(c[mt][nt][0], c[mt][nt][1], b0[nt]);
        split2<NC>(c[mt][nt][2], c[mt][nt][3], b1[nt]);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          b0[nt][j] = transpose8(b0[nt][j]);
          b1[nt][j] = transpose8(b1[nt][j]);
        }
      }
      product<NP, NC, NB>(acc, rest, Y, mt, b0, b1);
    }
    if (NP > 1) {
#pragma unroll
      for (int b = 0; b < NB; ++b) add(acc[b], rest[b]);
    }
  }
  // One step of depth 16 of the two above: 4 NB sums in turn.
  template <int NP, int NC, int NB>
  static __device__ __forceinline__ void product(float (&acc)[NB][4][4], float (&rest)[NB][4][4],
                                                 const Frag<NP> (&X)[NB], int ks,
                                                 const uint32_t (&b0)[4][NC],
                                                 const uint32_t (&b1)[4][NC]) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (pair_counts(i, j, NP, NC)) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool first = ks == 0 && i == 0;
              if (NP == 1 || i + j == 0) {
                if (first && j == 0)
                  mma0(acc[b][e], X[b].r[i][ks], b0[e][j], b1[e][j]);
                else
                  mma(acc[b][e], X[b].r[i][ks], b0[e][j], b1[e][j]);
              } else if (first && j == 1) {
                mma0(rest[b][e], X[b].r[i][ks], b0[e][j], b1[e][j]);
              } else {
                mma(rest[b][e], X[b].r[i][ks], b0[e][j], b1[e][j]);
              }
            }
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

// Scale one row of an accumulator; kStops: a factor of zero drops it whatever it holds.
template <bool kStops>
__device__ __forceinline__ void scale_row(float (&acc)[4][4], int h, float f) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int i = 2 * h; i < 2 * h + 2; ++i)
      acc[e][i] = kStops && f == 0.0f ? 0.0f : acc[e][i] * f;
}

// The decays of NB blocks of 16 tokens. Lane l stands for token l % (16 NB); c is the sum of
// log2 gates from its block's first token to it, stops left out.
//
// A decay is the difference of two such sums. Where a sum falls below kEasy (and always for
// float32 tensors) the sums carry what their rounding left in `low`, so that gates of -100 cost
// neither the small gates next to them nor what passes them low bits; above it the difference is good to
// 2^-18 (sums of gates that let the state grow, to 2^-24 of their size). Where a bf16 step is
// `hard`, for that or for a stop, it runs a second copy of the step's code that minds both, so
// that the ordinary one stays free of branches, one long stretch in which the scheduler can lay
// products beside the arithmetic around them.
template <int NP, int NB>
struct Decay {
  static constexpr float kEasy = NP == 1 ? -32.0f : 1.0f;
  float c, low;          // sum at the lane's token: c + low
  float last, last_low;  // the same at the last token of its block
  uint32_t stops;        // bit i: token i's gate lets nothing through
  bool hard;
  static __device__ __forceinline__ bool is_stop(float g) { return g * kLog2e < kStop; }
  static __device__ __forceinline__ uint32_t find_stops(float g) {
    const uint32_t found = __ballot_sync(0xffffffffu, is_stop(g));
    return NB == 1 ? found & 0xffffu : found;
  }
  __device__ __forceinline__ Decay(float g, uint32_t found, int lane) : stops(found) {
    float x = g * kLog2e;
    if (x < kStop) x = 0.0f;
    const float x0 = x;
    low = last_low = 0.0f;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, x, d, 16);
      if ((lane & 15) >= d) x += y;
    }
    c = x;
    const bool wide = NP > 1 || __any_sync(0xffffffffu, !(c >= kEasy));
    hard = wide || stops != 0;
    if (wide) {
      x = x0;
      if (x0 != 0.0f) low = fmaf(g, kLog2e, -x0) + g * kLog2eRest;
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
      last_low = __shfl_sync(0xffffffffu, low, 15, 16);
    }
    last = __shfl_sync(0xffffffffu, c, 15, 16);
  }
  // stops of the lane's own block
  __device__ __forceinline__ uint32_t own_stops(int lane) const {
    return NB == 1 ? stops : (stops >> (lane & 16)) & 0xffffu;
  }
  // 2^(x + rest)
  template <bool kLow>
  static __device__ __forceinline__ float power(float x, float rest) {
    const float f = exp2_fast(x);
    return kLow ? fmaf(f, rest * 0.6931471805599453f, f) : f;
  }
  // from the state before the lane's block to its token
  template <bool kStops, bool kLow>
  __device__ __forceinline__ float head(int lane) const {
    const float f = power<kLow>(c, low);
    return kStops && (own_stops(lane) & ((2u << (lane & 15)) - 1u)) ? 0.0f : f;
  }
  // from the lane's token to its block's end
  template <bool kStops, bool kLow>
  __device__ __forceinline__ float tail(int lane) const {
    const float f = exp2_fast(kLow ? (last - c) + (last_low - low) : last - c);
    return kStops && (own_stops(lane) >> ((lane & 15) + 1)) ? 0.0f : f;
  }
  // over the whole of the lane's block
  template <bool kStops, bool kLow>
  __device__ __forceinline__ float whole(int lane) const {
    return kStops && own_stops(lane) ? 0.0f : power<kLow>(last, last_low);
  }
  // of `x`, one value per token: the values of tokens 16 b + 2 (l % 4) + {0, 1, 8, 9}
  static __device__ __forceinline__ void spread(float x, int b, int lane, float (&out)[4]) {
    const int j = 16 * b + 2 * (lane & 3);
    out[0] = __shfl_sync(0xffffffffu, x, j);
    out[1] = __shfl_sync(0xffffffffu, x, j + 1);
    out[2] = __shfl_sync(0xffffffffu, x, j + 8);
    out[3] = __shfl_sync(0xffffffffu, x, j + 9);
  }
  // and of tokens 16 b + l / 4 + {0, 8}
  static __device__ __forceinline__ void spread_rows(float x, int b, int lane, float (&out)[2]) {
    out[0] = __shfl_sync(0xffffffffu, x, 16 * b + (lane >> 2));
    out[1] = __shfl_sync(0xffffffffu, x, 16 * b + (lane >> 2) + 8);
  }
  // Decays of an accumulator of 16 x 16 tokens of block b: l[h][x] belongs to row token
  // l / 4 + 8 h and column token 2 (l % 4) + {0, 1, 8, 9}; from the earlier to the later of
  // the two, rows the later ones (kRowsLater) or the earlier ones. Pairs in the other order,
  // or with a stop between them (the later token's own included), give 0. Of the four quarters
  // one is all zeros: columns 8-15 of rows 0-7, or rows 8-15 of columns 0-7.
  template <bool kRowsLater, bool kStops, bool kLow>
  __device__ __forceinline__ void within(int b, int lane, float (&l)[2][4]) const {
    float cc[4], cr[2], cl[4] = {0.0f, 0.0f, 0.0f, 0.0f}, lr[2] = {0.0f, 0.0f};
    spread(c, b, lane, cc);
    spread_rows(c, b, lane, cr);
    if (kLow) {
      spread(low, b, lane, cl);
      spread_rows(low, b, lane, lr);
    }
    const uint32_t st = (stops >> (16 * b)) & 0xffffu;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (lane >> 2) + 8 * h;
      int first = 0, end = 0;  // the column tokens that count
      if (kStops) {
        if (kRowsLater) {
          const uint32_t before = st & ((2u << row) - 1u);
          first = before != 0 ? 31 - __clz(before) : 0;
          end = row + 1;
        } else {
          const uint32_t after = st & ~((2u << row) - 1u);
          first = row;
          end = after != 0 ? __ffs(after) - 1 : 16;
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int col = 2 * (lane & 3) + (x & 1) + 8 * (x >> 1);
        const bool same = h == (x >> 1);  // a quarter on the diagonal
        if (!same && (h == 1) != kRowsLater) {
          l[h][x] = 0.0f;
          continue;
        }
        float d = kRowsLater ? cr[h] - cc[x] : cc[x] - cr[h];
        if (kLow) d += kRowsLater ? lr[h] - cl[x] : cl[x] - lr[h];
        if (kStops) {
          l[h][x] = col >= first && col < end ? exp2_fast(d) : 0.0f;
        } else {
          const float f = exp2_fast(d);
          l[h][x] = same && (kRowsLater ? col > row : col < row) ? 0.0f : f;
        }
      }
    }
  }
};

// w *= l; kStops: a factor of zero drops the number whatever it is.
template <bool kStops>
__device__ __forceinline__ void decay_by(float (&w)[2][4], const float (&l)[2][4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float& e = w[x >> 1][2 * h + (x & 1)];
      e = kStops && l[h][x] == 0.0f ? 0.0f : e * l[h][x];
    }
}

// Shared memory of one warp: kStages stages of NT tiles of NB blocks; float32 tiles arrive as
// they are and are split into three bf16 planes before use (the first NS of them).
template <int NP, int NB, int NT, int kStages, int NS = NT>
struct Smem {
  static constexpr int kTile = NB * (NP == 1 ? kPlane : kGateBlock * 128);
  static constexpr int kStage = NT * kTile + (NT == 4 ? 256 : 128);  // and a float or two per token
  static constexpr int kPart = NB * kPlane;  // one plane of one tile
  static constexpr int kPlanes = NP == 1 ? 0 : NS * 3 * kPart;
  static constexpr int kWarp = kStages * kStage + kPlanes;
};

// 16-byte chunk of a float32 tile (rows of 128 bytes); the exclusive-or keeps the
// 32-byte reads of the split free of bank conflicts.
__device__ __forceinline__ uint32_t tile_off_f32(int row, int c16) {
  return static_cast<uint32_t>(row * 128 + ((c16 ^ (row & 1)) << 4));
}

// The ring of stages that a warp fills from global memory while it works: NT tiles of NB
// blocks each, then the gates, then (NT = 4) one more float per token. A lane copies one
// 16-byte chunk of every eighth (bf16) or fourth (float32) row and keeps its own pointers,
// which move on by a step: computed afresh, the addresses took a third of all instructions.
template <int NP, int NB, int NT, int kStages, int NS, bool kBackwards, bool kExtra>
struct Ring {
  using T = typename Io<NP>::T;
  using M = Smem<NP, NB, NT, kStages, NS>;
  static constexpr int kStep = NB * kGateBlock;
  static constexpr int kChunks = NP == 1 ? 4 : 8;  // of a row
  static constexpr int kRows = 32 / kChunks;       // rows of one copy of the warp
  static constexpr int kCopies = kStep / kRows;
  static constexpr int kPitch = kRows * (NP == 1 ? 64 : 128);
  const char* src[NT];   // the lane's first chunk of the next step to copy
  const float *gate, *extra;
  int pitch, H;          // bytes of a token in the tensors; heads
  int left;              // tokens from the next step on; backwards: of it (the first may be short)
  int todo;              // steps still to copy
  uint32_t end, dst, cur;  // shared memory: past the ring, the lane's place in the next stage, the
                           // stage at hand

  // `heads`: each tensor at token 0 of the head; first: the first step's first token;
  // last: the segment's end.
  __device__ __forceinline__ Ring(uint32_t smem, const T* const (&heads)[NT], const float* G,
                                  int heads_per_token, const float* per_token, int first, int last,
                                  int steps, int lane) {
    H = heads_per_token;
    pitch = H * 32 * static_cast<int>(sizeof(T));
    const int row = lane / kChunks, c = lane % kChunks, i = lane & (kStep - 1);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      src[t] = reinterpret_cast<const char*>(heads[t]) + static_cast<size_t>(first + row) * pitch +
               c * 16;
    gate = G + static_cast<size_t>(first + i) * H;
    extra = kExtra ? per_token + first + i : nullptr;
    left = last - first;
    todo = steps;
    end = smem + kStages * M::kStage;
    dst = smem + (NP == 1 ? tile_off(row, c) : tile_off_f32(row, c));
    cur = smem - M::kStage;
  }
  // Start the copies of the next step (an empty group when there is none).
  __device__ __forceinline__ void issue(int lane) {
    if (todo > 0) {
      const int row = lane / kChunks, c = lane % kChunks, i = lane & (kStep - 1);
      const uint32_t line =
          dst + (NT * M::kTile + lane * 4 - (NP == 1 ? tile_off(row, c) : tile_off_f32(row, c)));
      const int down = kRows * pitch;
      if (left >= kStep) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const char* p = src[t];
#pragma unroll
          for (int k = 0; k < kCopies; ++k, p += down)
            cp16(dst + t * M::kTile + k * kPitch, p, 16);
        }
        cp4(line, gate, 4);
        if (kExtra) cp4(line + 128, extra, 4);
      } else {  // rows past the end become zero, and so do their gates
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < kCopies; ++k) {
            const bool in = row + k * kRows < left;
            cp16(dst + t * M::kTile + k * kPitch,
                 src[t] + (in ? k * static_cast<ptrdiff_t>(down) : -row * static_cast<ptrdiff_t>(pitch)),
                 in ? 16 : 0);
          }
        const bool in = i < left;
        cp4(line, in ? gate : gate - static_cast<ptrdiff_t>(i) * H, in ? 4 : 0);
        if (kExtra) cp4(line + 128, in ? extra : extra - i, in ? 4 : 0);
      }
      const ptrdiff_t move = static_cast<ptrdiff_t>(kBackwards ? -kStep : kStep) * pitch;
#pragma unroll
      for (int t = 0; t < NT; ++t) src[t] += move;
      gate += static_cast<ptrdiff_t>(kBackwards ? -kStep : kStep) * H;
      if (kExtra) extra += kBackwards ? -kStep : kStep;
      left = kBackwards ? kStep : left - kStep;  // only the segment's last step can be short
      --todo;
      dst += M::kStage;
      if (dst >= end) dst -= kStages * M::kStage;
    }
    cp_commit();
  }
  // The next stage, filled and seen by all lanes; the one before is free and filled anew.
  __device__ __forceinline__ uint32_t next(int lane) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(lane);
    cur += M::kStage;
    if (cur == end) cur -= kStages * M::kStage;
    return cur;
  }
};

// float32 tile -> three bf16 planes.
template <int NB>
__device__ __forceinline__ void split_tile(uint32_t src, uint32_t planes, int lane) {
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) {
    const int idx = lane + 32 * i, row = idx >> 2, c = idx & 3;
    const uint4 a = lds4(src + tile_off_f32(row, 2 * c));
    const uint4 b = lds4(src + tile_off_f32(row, 2 * c + 1));
    uint32_t w[4][3];
    split2<3>(__uint_as_float(a.x), __uint_as_float(a.y), w[0]);
    split2<3>(__uint_as_float(a.z), __uint_as_float(a.w), w[1]);
    split2<3>(__uint_as_float(b.x), __uint_as_float(b.y), w[2]);
    split2<3>(__uint_as_float(b.z), __uint_as_float(b.w), w[3]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      sts4(planes + p * NB * kPlane + tile_off(row, c), w[0][p], w[1][p], w[2][p], w[3][p]);
  }
}

// What is not finite and a stop in one step. A product adds up all tokens of its step, those
// behind a stop with a weight of zero, and zero times infinity is NaN. So a step with stops takes
// such tokens out: a gate that is no number becomes 0, a token's rows of two tiles zero. Both
// return the tokens' bits. What they should have spoiled, the outputs and states that no stop
// parts from them, is then set to NaN.
template <int NB>
__device__ __forceinline__ uint32_t take_out_gates(float& gate) {
  const bool odd = !(gate < __int_as_float(0x7f800000));
  const uint32_t found = __ballot_sync(0xffffffffu, odd);
  if (odd) gate = 0.0f;
  return NB == 1 ? found & 0xffffu : found;
}
// float32: also numbers so large that their first bf16 part is infinite.
template <int NP, int NB>
__device__ __forceinline__ uint32_t take_out(uint32_t t0, uint32_t t1, int lane) {
  const int token = lane & (NB * kGateBlock - 1);
  const uint32_t tile[2] = {t0, t1};
  uint32_t at[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    at[c] = NP == 1 ? tile_off(token, c) : tile_off_f32(token, c + (lane >> 4) * 4);
  bool bad = false;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = lds4(tile[t] + at[c]);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bad |= NP == 1 ? (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u
                       : (w[i] & 0x7fffffffu) >= 0x7f7f8000u;
    }
  uint32_t rows = __ballot_sync(0xffffffffu, bad);
  if (NB == 1) rows = (rows | rows >> 16) & 0xffffu;  // two lanes a token
  if (rows != 0) {
    if ((rows >> token) & 1u) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) sts4(tile[t] + at[c], 0u, 0u, 0u, 0u);
    }
    __syncwarp();
  }
  return rows;
}
// Whether one of the `bad` tokens reaches token i of the step forwards: from the last stop up to i on.
__device__ __forceinline__ float spoiled_from(uint32_t bad, uint32_t stops, int i) {
  const uint32_t upto = (2u << i) - 1u, before = stops & upto;
  const uint32_t from = before != 0 ? ~0u << (31 - __clz(before)) : ~0u;
  return (bad & upto & from) != 0 ? __int_as_float(kNan) : 0.0f;
}
// The same backwards: from i on, up to the next stop.
__device__ __forceinline__ float spoiled_to(uint32_t bad, uint32_t stops, int i) {
  const uint32_t later = ~((2u << i) - 1u), after = stops & later;
  const uint32_t upto = after != 0 ? (1u << (__ffs(after) - 1)) - 1u : ~0u;
  return (bad & (later | (1u << i)) & upto) != 0 ? __int_as_float(kNan) : 0.0f;
}
// And the state before the step.
__device__ __forceinline__ bool spoils_start(uint32_t bad, uint32_t stops) {
  return (bad & ((stops & (0u - stops)) - 1u)) != 0;
}
// Add 0 or NaN to the rows of block b, by a value per token.
template <int NP, int NB>
__device__ __forceinline__ void spoil_rows(float (&acc)[4][4], int b, float by_token, int lane) {
  float r[2];
  Decay<NP, NB>::spread_rows(by_token, b, lane, r);
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[e][i] += r[i >> 1];
}

// Rows of an output: an accumulator goes to a free tile in shared memory (put), and from there
// in 16-byte pieces, four or eight lanes a row, to the tensor (flush, after a __syncwarp).
template <int NP>
struct Out {
  static constexpr int kChunks = NP == 1 ? 4 : 8;  // of a row
  static constexpr int kRows = 32 / kChunks;       // rows the warp stores at once
  static constexpr int kRowBytes = NP == 1 ? 64 : 128;
  char* p;       // the lane's first piece of the next block
  int pitch;     // bytes of a token in the tensor
  uint32_t piece;
  __device__ __forceinline__ Out(void* o, size_t base, int heads, int n0, int lane) {
    using T = typename Io<NP>::T;
    pitch = heads * 32 * static_cast<int>(sizeof(T));
    const int row = lane / kChunks, c = lane % kChunks;
    p = reinterpret_cast<char*>(static_cast<T*>(o) + base) + static_cast<size_t>(n0 + row) * pitch +
        c * 16;
    piece = NP == 1 ? tile_off(row, c) : tile_off_f32(row, c);
  }
  static __device__ __forceinline__ void put(const float (&acc)[4][4], uint32_t tile,
                                             const LaneOff& off, int lane) {
    if (NP == 1) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        stsm4(tile + off.a[ks], pack2(acc[2 * ks][0], acc[2 * ks][1]),
              pack2(acc[2 * ks][2], acc[2 * ks][3]), pack2(acc[2 * ks + 1][0], acc[2 * ks + 1][1]),
              pack2(acc[2 * ks + 1][2], acc[2 * ks + 1][3]));
    } else {
      const int r = lane >> 2, q = lane & 3;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sts2(tile + tile_off_f32(r + 8 * h, 2 * e + (q >> 1)) + (q & 1) * 8, acc[e][2 * h],
               acc[e][2 * h + 1]);
    }
  }
  // `tokens` of the tile at hand, of which `rows` exist; moves on by `step` tokens.
  template <int kTokens, bool kWhole>
  __device__ __forceinline__ void flush(uint32_t tile, int rows, int step, int lane) {
    char* dst = p;
    const int down = kRows * pitch;
#pragma unroll
    for (int i = 0; i < kTokens / kRows; ++i, dst += down) {
      const uint4 v = lds4(tile + piece + i * kRows * kRowBytes);
      if (kWhole || lane / kChunks + i * kRows < rows) *reinterpret_cast<uint4*>(dst) = v;
    }
    p += static_cast<ptrdiff_t>(step) * pitch;
  }
};

// Sum over the 32 dimensions of acc * X for tokens l / 4 and l / 4 + 8, in every lane of the
// four: bf16 from X as an operand (its numbers lie where an accumulator's do), float32 from
// the tile as it lies in shared memory.
__device__ __forceinline__ void row_dots(const float (&acc)[4][4], const Frag<1>& X,
                                         float (&out)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = X.r[0][e >> 1][2 * (e & 1) + h];
      s = fmaf(acc[e][2 * h], lo_f(v), fmaf(acc[e][2 * h + 1], hi_f(v), s));
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    out[h] = s;
  }
}
__device__ __forceinline__ void row_dots_f32(const float (&acc)[4][4], uint32_t tile, int lane,
                                             float (&out)[2]) {
  const int r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 v = lds2(tile + tile_off_f32(r + 8 * h, 2 * e + (q >> 1)) + (q & 1) * 8);
      s = fmaf(acc[e][2 * h], __uint_as_float(v.x), fmaf(acc[e][2 * h + 1], __uint_as_float(v.y), s));
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    out[h] = s;
  }
}

}  // namespace gated
}  // namespace la
