// The end of one block and the start of the next, per token (row of C numbers):
//
//   u = f, or RMSNorm(f) w_post           norm after the block
//   h = x + alpha gate_b u                gated residual
//   y = norm(h) w_pre (1 + scale_b) + shift_b    norm (RMS or layer) before the next, modulated
//
// and its gradients. Bound by HBM: the forward reads x and f and writes h and y, the
// backward reads x, f, dh and dy and writes dx and df, each once; a row stays in
// registers from its load to its store, and the backward forms the norms' statistics
// again instead of keeping h. Statistics are float32, the variance from the
// differences to the mean (a second pass over the registers).
//
// The per-channel factors are combined once per CTA in shared memory (alpha gate w_post;
// w_pre (1 + scale); shift): read per row from global memory they would be more bytes
// than the row. So a CTA keeps to one batch element.
//
// Backward: a thread owns 16 columns of all its CTA's rows and sums the three
// column sums that the parameters' gradients need, sum dy n, sum dy and sum u dh, in
// registers; a second kernel adds the CTAs' partial sums in order. No atomics: the
// same bits every time.
//
// 16384 x 2240 in bf16 with gate and modulation: forward 53 us, 5.5 TB/s (the warps' next rows
// ahead in registers or in L2, or a CTA per row, measured slower: 58 to 71 us); backward 90 us,
// 4.9 TB/s, of which the column sums' second kernel is 8: three sums over a row, each its shuffles
// and a barrier, run beside the copies of the next row. Of the measured copy's rate, as many bytes
// of other widths take, forward: 84 to 86 % at 1152 to 2304 columns (float32 80 %), 62 to 66 % at
// 2560 to 4096 (76 to 82 %), 44 and 51 % at 5120 and 8192 (60 and 66 %). Backward: 74 to 81 % up to
// 2560 columns, 47 % at 2816, 62 to 70 % at 4096 to 8192; float32, whose rows are twice as long for
// a thread's registers, 53 % and 45 to 49 %.
#include "la_block_internal.h"
#include "la_common.cuh"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kVec = 8;  // columns a thread moves at once

// Eight numbers of an output row. Rows that are read or written once stream past L2 (loads and
// stores marked evict-first: 3 us less for the forward at 16384 x 2240).
__device__ __forceinline__ void store_cs(__nv_bfloat16* p, const float* x) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7])));
}
__device__ __forceinline__ void store_cs(float* p, const float* x) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }

};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

};

// A vector of C floats in shared memory: the first four of every eight columns, then the
// others, so that 16-byte reads of neighbouring threads meet different banks.
struct Line {
  float* p;
  int vecs;
  __device__ __forceinline__ void get(int v, float (&x)[8]) const {
    const float4 a = reinterpret_cast<const float4*>(p)[v];
    const float4 b = reinterpret_cast<const float4*>(p)[vecs + v];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void put(int v, const float (&x)[8]) const {
    reinterpret_cast<float4*>(p)[v] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[vecs + v] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Sums over the threads of a row: a warp's shuffles, then (kWarps > 1) one word per warp in
// shared memory, read back as whole lines (words of warps that a CTA lacks stay 0). `slot`
// alternates between two sets, so one barrier per sum is enough. Two sums go through the
// shuffles together: after the first step one half of the warp carries each.
constexpr int kScratch = 2 * 2 * 32;  // floats: slots x sums x warps

template <int kWarps>
__device__ __forceinline__ float across_warps(const float* s) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < (kWarps + 3) / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(s)[i];
    t += (v.x + v.y) + (v.z + v.w);
  }
  return t;
}
template <int kWarps>
__device__ __forceinline__ float row_sum(float x, float* scratch, int& slot) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  if (kWarps == 1) return x;
  float* s = scratch + slot;
  slot ^= 64;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  return across_warps<kWarps>(s);
}
template <int kWarps>
__device__ __forceinline__ void row_sum2(float& x, float& y, float* scratch, int& slot) {
  const bool low = (threadIdx.x & 16) == 0;
  float z = __shfl_xor_sync(0xffffffffu, low ? y : x, 16) + (low ? x : y);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
  if (kWarps == 1) {
    x = __shfl_sync(0xffffffffu, z, 0);
    y = __shfl_sync(0xffffffffu, z, 16);
    return;
  }
  float* s = scratch + slot;
  slot ^= 64;
  if ((threadIdx.x & 15) == 0) s[(low ? 0 : 32) + (threadIdx.x >> 5)] = z;
  __syncthreads();
  x = across_warps<kWarps>(s);
  y = across_warps<kWarps>(s + 32);
}

// Per-channel factors of batch element b: alpha gate w_post, w_pre (1 + scale), shift; eight
// columns a thread and turn, so that its loads are on their way together.
__device__ __forceinline__ void load8_or(const float* p, float fill, float (&x)[8]) {
  if (p != nullptr) {
    load8(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fill;
  }
}
template <bool kShift>
__device__ __forceinline__ void combine_params(const NormProblem& p, const NormParams& w, int b,
                                               const Line& l1, const Line& l2, const Line& l3) {
  const size_t bc = static_cast<size_t>(b) * p.C;
  for (int v = threadIdx.x; v < l1.vecs; v += blockDim.x) {
    const int c = v * kVec;
    float gate[8], post[8], pre[8], scale[8];
    load8_or(w.gate != nullptr ? w.gate + bc + c : nullptr, 1.0f, gate);
    load8_or(w.w_post != nullptr ? w.w_post + c : nullptr, 1.0f, post);
    load8_or(w.w_pre != nullptr ? w.w_pre + c : nullptr, 1.0f, pre);
    load8_or(w.mod_scale != nullptr ? w.mod_scale + bc + c : nullptr, 0.0f, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gate[i] = p.alpha * gate[i] * post[i];
      pre[i] *= 1.0f + scale[i];
    }
    l1.put(v, gate);
    l2.put(v, pre);
    if (kShift) {
      load8_or(w.mod_shift != nullptr ? w.mod_shift + bc + c : nullptr, 0.0f, scale);
      l3.put(v, scale);
    }
  }
}

// Forward: warps of a CTA take a row each (kOneWarp), or the whole CTA one row. KV: vectors
// of 8 columns per thread.
template <typename T, int KV, bool kOneWarp>
__global__ void __launch_bounds__(kOneWarp ? 128 : 1024)
norm_kernel(const NormProblem p, const T* x, const T* f, const NormParams w, T* h, T* y) {
  extern __shared__ __align__(16) float smem[];
  const int vecs = p.C / kVec, b = blockIdx.y;
  const Line l1 = {smem, vecs}, l2 = {smem + p.C, vecs}, l3 = {smem + 2 * p.C, vecs};
  float* scratch = smem + 3 * p.C;
  constexpr int kRowWarps = kOneWarp ? 1 : 32;
  for (int i = threadIdx.x; i < kScratch; i += blockDim.x) scratch[i] = 0.0f;
  combine_params<true>(p, w, b, l1, l2, l3);
  __syncthreads();
  const int width = kOneWarp ? 32 : blockDim.x;  // threads of a row
  const int t = kOneWarp ? threadIdx.x & 31 : threadIdx.x;
  const int per_cta = kOneWarp ? blockDim.x >> 5 : 1;
  const int first = blockIdx.x * per_cta + (kOneWarp ? threadIdx.x >> 5 : 0);
  const float inv = 1.0f / static_cast<float>(p.C);
  int slot = 0;
  for (int n = first; n < p.N; n += gridDim.x * per_cta) {
    const size_t row = (static_cast<size_t>(b) * p.N + n) * p.C;
    Raw<T> rx[KV], rf[KV];
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      rx[k].zero();
      rf[k].zero();
      if (v < vecs) {
        rx[k].load(x + row + v * kVec);
        if (f != nullptr) rf[k].load(f + row + v * kVec);
      }
    }
    float rstd_f = 1.0f;
    if (w.w_post != nullptr) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        float a[8];
        rf[k].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(a[i], a[i], s);
      }
      rstd_f = rsqrtf(fmaf(row_sum<kRowWarps>(s, scratch, slot), inv, p.eps));
    }
    float r[KV][8];
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      rx[k].get(r[k]);
      if (f != nullptr && v < vecs) {
        float a[8], m[8];
        rf[k].get(a);
        l1.get(v, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[k][i] = fmaf(a[i] * rstd_f, m[i], r[k][i]);
        if (h != nullptr) store_cs(h + row + v * kVec, r[k]);
      }
    }
    if (y == nullptr) continue;
    float mean = 0.0f;
    if (p.layer) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += r[k][i];
      mean = row_sum<kRowWarps>(s, scratch, slot) * inv;
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < KV; ++k)
      if (t + k * width < vecs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[k][i] -= mean;
          s = fmaf(r[k][i], r[k][i], s);
        }
      }
    const float rstd = rsqrtf(fmaf(row_sum<kRowWarps>(s, scratch, slot), inv, p.eps));
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      if (v < vecs) {
        float m[8], a[8];
        l2.get(v, m);
        l3.get(v, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaf(r[k][i] * rstd, m[i], a[i]);
        store_cs(y + row + v * kVec, a);
      }
    }
  }
}

// A backward thread owns two vectors of every row: the sums over a row cost each thread its
// shuffles and a barrier, which 16 columns pay for better than 8. The next row is on its way
// to shared memory meanwhile, every thread its own pieces, so nothing but the thread waits
// for them; in registers they would be 32 to 64 more of the 128 that a thread has, which do not
// hold all of a row's arithmetic as it is: bf16 spills 12 to 80 bytes, float32 24 to 236.
constexpr int kBackVecs = 2, kNarrow = 160, kWide = 512;
static_assert(kWide * kBackVecs * kVec == kNormMaxC, "the widest row");

// Shared memory as a 32-bit address.
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void widen(float4 a, float4 b, float (&x)[8]) {
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Backward of one batch element's rows; `part`: [B][CTAs][3][C] column sums (sum dy n, sum dy,
// sum u dh). kAll: f, dh and dy are all there (known to the compiler, the row's work is one
// stretch without branches).
template <typename T, int kThreads, bool kAll>
__global__ void __launch_bounds__(kThreads, kThreads == kWide ? 1 : 480 / kThreads)
norm_backward_kernel(const NormProblem p, const T* x, const T* f, const NormParams w, const T* dh,
                     const T* dy, T* dx, T* df, float* part) {
  constexpr int KV = kBackVecs, kRowWarps = kThreads / 32;
  extern __shared__ __align__(16) float smem[];
  const int vecs = p.C / kVec, b = blockIdx.y, t = threadIdx.x, width = blockDim.x;
  const Line l1 = {smem, vecs}, l2 = {smem + p.C, vecs};
  float* scratch = smem + 2 * p.C;
  sm100::pdl_trigger();
  const float inv = 1.0f / static_cast<float>(p.C);
  const bool has_f = kAll || f != nullptr, has_h = kAll || dh != nullptr;
  const bool has_y = kAll || dy != nullptr;
  const bool post = w.w_post != nullptr;
  int slot = 0;
  float sum_e[KV][8], sum_d[KV][8], sum_f[KV][8];
#pragma unroll
  for (int k = 0; k < KV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum_e[k][i] = sum_d[k][i] = sum_f[k][i] = 0.0f;

  // The thread's vectors t and t + width. Vectors past the row's end are worked on as zeros (their
  // pieces stay 0, and they borrow the first vector's factors) but neither loaded nor stored.
  // Byte offsets in a row, in the factors, and in the pieces of the next row:
  // [tensor][vector][16 bytes][thread].
  constexpr int kPieces = kVec * sizeof(T) / 16;
  const bool have[KV] = {t < vecs, t + width < vecs};
  const uint32_t base = sm100::smem_u32(smem);
  const uint32_t upper = vecs * 16, next = width * 16, line2 = p.C * 4;
  const uint32_t factor[KV] = {base + (have[0] ? t * 16 : 0), base + (have[1] ? (t + width) * 16 : 0)};
  const uint32_t ahead = base + (2 * p.C + kScratch) * 4 + t * 16;
  const size_t pitch = static_cast<size_t>(p.C) * sizeof(T);
  const size_t move = pitch * gridDim.x;
  size_t ofs = (static_cast<size_t>(b) * p.N + blockIdx.x) * pitch + t * kVec * sizeof(T);
  const uint32_t second = width * kVec * sizeof(T);
  auto fetch = [&](int n, size_t at) {
    if (n < p.N) {
      auto tensor = [&](int a, const T* src) {
        const char* q = reinterpret_cast<const char*>(src) + at;
#pragma unroll
        for (int k = 0; k < KV; ++k)
          if (have[k]) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               ahead + ((a * KV + k) * kPieces + i) * next),
                           "l"(q + k * second + i * 16)
                           : "memory");
          }
      };
      tensor(0, x);
      if (has_f) tensor(1, f);
      if (has_h) tensor(2, dh);
      if (has_y) tensor(3, dy);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < 4 * KV * kPieces; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(ahead + i * next), "r"(0) : "memory");
  auto take = [&](int a, int k, bool there, float (&out)[8]) {
    if (there) {
      const uint32_t at = ahead + (a * KV + k) * kPieces * next;
      const float4 v = lds4(at);
      if (sizeof(T) == 2) {
        Raw<__nv_bfloat16> r;
        r.u = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                         __float_as_uint(v.w));
        r.get(out);
      } else {
        widen(v, lds4(at + next), out);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = 0.0f;
    }
  };
  auto factors = [&](uint32_t line, int k, float (&m)[8]) {
    widen(lds4(factor[k] + line), lds4(factor[k] + line + upper), m);
  };
  fetch(blockIdx.x, ofs);  // on its way while the factors are combined
  for (int i = t; i < kScratch; i += width) scratch[i] = 0.0f;
  combine_params<false>(p, w, b, l1, l2, l2);
  __syncthreads();
  for (int n = blockIdx.x; n < p.N; n += gridDim.x, ofs += move) {
    float hx[KV][8], u[KV][8], g[KV][8], gy[KV][8];  // h, u / w_post, dh, dy
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      take(0, k, true, hx[k]);
      take(1, k, has_f, u[k]);
      take(2, k, has_h, g[k]);
      take(3, k, has_y, gy[k]);
    }
    fetch(n + gridDim.x, ofs + move);
    float rstd_f = 1.0f;
    if (post) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(u[k][i], u[k][i], s);
      rstd_f = rsqrtf(fmaf(row_sum<kRowWarps>(s, scratch, slot), inv, p.eps));
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] *= rstd_f;
    }
    if (has_f) {
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        float m[8];
        factors(0, k, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) hx[k][i] = fmaf(u[k][i], m[i], hx[k][i]);
      }
    }
    if (has_y) {
      float mean = 0.0f;
      if (p.layer) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < KV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s += hx[k][i];
        mean = row_sum<kRowWarps>(s, scratch, slot) * inv;
      }
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        const float centre = have[k] ? mean : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          hx[k][i] -= centre;
          s = fmaf(hx[k][i], hx[k][i], s);
        }
      }
      const float rstd = rsqrtf(fmaf(row_sum<kRowWarps>(s, scratch, slot), inv, p.eps));
      float along = 0.0f, off = 0.0f;  // the parts of t = dy w_pre (1 + scale) along n and 1
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        float m[8];
        factors(line2, k, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          hx[k][i] *= rstd;  // n
          sum_e[k][i] = fmaf(gy[k][i], hx[k][i], sum_e[k][i]);
          sum_d[k][i] += gy[k][i];
          gy[k][i] *= m[i];
          along = fmaf(gy[k][i], hx[k][i], along);
          off += gy[k][i];
        }
      }
      if (p.layer) {
        row_sum2<kRowWarps>(along, off, scratch, slot);
      } else {
        along = row_sum<kRowWarps>(along, scratch, slot);
        off = 0.0f;
      }
      along *= inv;
      off *= inv;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[k][i] = fmaf(rstd, gy[k][i] - fmaf(hx[k][i], along, off), g[k][i]);
    }
#pragma unroll
    for (int k = 0; k < KV; ++k)
      if (have[k])
        store_cs(reinterpret_cast<T*>(reinterpret_cast<char*>(dx) + ofs + k * second), g[k]);
    if (!has_f) continue;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      float m[8];
      factors(0, k, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum_f[k][i] = fmaf(u[k][i], g[k][i], sum_f[k][i]);
        g[k][i] *= m[i];
        s = fmaf(g[k][i], u[k][i], s);
      }
    }
    if (post) {
      const float part_u = row_sum<kRowWarps>(s, scratch, slot) * inv;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] = rstd_f * (g[k][i] - u[k][i] * part_u);
    }
#pragma unroll
    for (int k = 0; k < KV; ++k)
      if (have[k])
        store_cs(reinterpret_cast<T*>(reinterpret_cast<char*>(df) + ofs + k * second), g[k]);
  }
  float* out = part + (static_cast<size_t>(b) * gridDim.x + blockIdx.x) * 3 * p.C;
#pragma unroll
  for (int k = 0; k < KV; ++k) {
    const int v = t + k * width;
    if (have[k]) {
      store_row<8>(out + v * kVec, sum_e[k]);
      store_row<8>(out + p.C + v * kVec, sum_d[k]);
      store_row<8>(out + 2 * p.C + v * kVec, sum_f[k]);
    }
  }
}

// The parameters' gradients from the CTAs' column sums. blockIdx.y: which of the three sums.
// 32 columns a CTA, a warp's lanes one each; its warps share up to four batch elements at a
// time and add the partial sums of each, always in the same order. Two CTAs an SM, so that the
// three sums of 2240 columns are one wave.
constexpr int kColumnWarps = 16;
__global__ void __launch_bounds__(kColumnWarps * 32, 2)
norm_columns_kernel(const NormProblem p, const NormParams w, const NormGrads g, const float* part) {
  __shared__ float s[kColumnWarps][33];
  sm100::pdl_wait();
  const int which = blockIdx.y;
  float* per_b = which == 0 ? g.mod_scale : which == 1 ? g.mod_shift : g.gate;
  float* over_b = which == 0 ? g.w_pre : which == 1 ? nullptr : g.w_post;
  if (per_b == nullptr && over_b == nullptr) return;
  const int col = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  const int at_once = p.B >= 4 ? 4 : p.B >= 2 ? 2 : 1, share = kColumnWarps / at_once;  // warps
  const size_t pitch = static_cast<size_t>(3) * p.C;                          // a CTA's sums
  float total = 0.0f;
  for (int b0 = 0; b0 < p.B; b0 += at_once) {
    const int b = b0 + warp / share, first = warp % share;
    float t = 0.0f;
    if (c < p.C && b < p.B) {
      const float* at = part + (static_cast<size_t>(b) * p.ctas + first) * pitch +
                        static_cast<size_t>(which) * p.C + c;
#pragma unroll 8
      for (int i = first; i < p.ctas; i += share, at += share * pitch) t += __ldcg(at);
    }
    s[warp][col] = t;
    __syncthreads();
    // warp k adds up batch element b0 + k: its lane has the column's sum
    if (warp < at_once && b0 + warp < p.B && c < p.C) {
      float sum = 0.0f;
      for (int i = 0; i < share; ++i) sum += s[warp * share + i][col];
      const size_t bc = static_cast<size_t>(b0 + warp) * p.C + c;
      if (which == 0) {  // sum dy n
        if (per_b != nullptr) per_b[bc] = sum * (w.w_pre != nullptr ? w.w_pre[c] : 1.0f);
        if (w.mod_scale != nullptr) sum *= 1.0f + w.mod_scale[bc];
      } else if (which == 1) {  // sum dy
        per_b[bc] = sum;
      } else {  // sum u dh, u without its weight
        if (per_b != nullptr) per_b[bc] = sum * p.alpha * (w.w_post != nullptr ? w.w_post[c] : 1.0f);
        sum *= p.alpha * (w.gate != nullptr ? w.gate[bc] : 1.0f);
      }
      total += sum;
    }
    __syncthreads();
  }
  if (over_b == nullptr) return;
  if (warp < at_once) s[warp][col] = total;
  __syncthreads();
  if (warp == 0 && c < p.C) {
    float sum = 0.0f;
    for (int k = 0; k < at_once; ++k) sum += s[k][col];
    over_b[c] = sum;
  }
}

// `most`: what the widest row of the kernel takes, not the call's own bytes, which another
// thread's call could undo before the launch.
template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t most) {
  if (most <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(most));
}
constexpr size_t forward_smem(size_t C) { return (3 * C + kScratch) * sizeof(float); }
template <typename T>
constexpr size_t backward_smem(size_t C, size_t threads) {
  return (2 * C + kScratch) * sizeof(float) + 4 * threads * kBackVecs * kVec * sizeof(T);
}

constexpr long long kSms = 148;

template <typename T, int KV, bool kOneWarp>
cudaError_t run_forward(const NormProblem& p, int threads, const void* x, const void* f,
                        const NormParams& w, void* h, void* y, cudaStream_t s) {
  const size_t smem = forward_smem(p.C);
  auto kernel = norm_kernel<T, KV, kOneWarp>;
  cudaError_t e = allow_smem(kernel, forward_smem(kOneWarp ? KV * kVec * 32 : kNormMaxC));
  if (e != cudaSuccess) return e;
  int resident = 0;  // a CTA for every place on the GPU: each then walks its rows
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  const long long rows = kOneWarp ? (p.N + threads / 32 - 1) / (threads / 32) : p.N;
  long long ctas = (kSms * (resident > 0 ? resident : 1) + p.B - 1) / p.B;
  if (ctas > rows) ctas = rows;
  kernel<<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(p.B)), threads, smem, s>>>(
      p, static_cast<const T*>(x), static_cast<const T*>(f), w, static_cast<T*>(h),
      static_cast<T*>(y));
  return cudaGetLastError();
}

// A warp takes a row of up to 9 vectors per lane (2304 columns) where the rows fill the GPU;
// few or long rows get whole CTAs, a vector per thread. bf16, a warp and a CTA a row: 2240 columns,
// 154 rows 4.9 and 3.8 us, 600 rows 6.5 and 6.9, 1184 rows 8.0 and 8.9, 9600 rows 34 and 41; 1152
// columns, 154 rows 3.6 and 2.9, 1184 rows 5.5 and 6.7 (float32 7.0 and 8.0). Wider rows have the
// second form alone.
template <typename T>
cudaError_t forward(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                    void* h, void* y, cudaStream_t s) {
  const int vecs = p.C / kVec;
  const long long rows = 1LL * p.B * p.N;
  if (vecs <= 32 || (vecs <= 32 * 9 && rows >= kSms * 8)) {
    const int kv = (vecs + 31) / 32;
#define LA_NORM_KV(KV) \
  if (kv <= KV) return run_forward<T, KV, true>(p, 128, x, f, w, h, y, s)
    LA_NORM_KV(1);
    LA_NORM_KV(2);
    LA_NORM_KV(3);
    LA_NORM_KV(5);
    LA_NORM_KV(7);
    LA_NORM_KV(9);
#undef LA_NORM_KV
  }
  return run_forward<T, 1, false>(p, (vecs + 31) / 32 * 32, x, f, w, h, y, s);
}

int backward_threads(int C) { return (C + kBackVecs * kVec * 32 - 1) / (kBackVecs * kVec * 32) * 32; }

template <typename T, int kThreads>
cudaError_t run_backward(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                         const void* dh, const void* dy, void* dx, void* df, float* ws,
                         cudaStream_t s) {
  const int threads = backward_threads(p.C);
  const size_t smem = backward_smem<T>(p.C, threads);
  auto kernel = f != nullptr && dh != nullptr && dy != nullptr
                    ? norm_backward_kernel<T, kThreads, true>
                    : norm_backward_kernel<T, kThreads, false>;
  const cudaError_t e = allow_smem(kernel, backward_smem<T>(kThreads * kBackVecs * kVec, kThreads));
  if (e != cudaSuccess) return e;
  kernel<<<dim3(static_cast<unsigned>(p.ctas), static_cast<unsigned>(p.B)), threads, smem, s>>>(
      p, static_cast<const T*>(x), static_cast<const T*>(f), w,
                      static_cast<const T*>(dh), static_cast<const T*>(dy), static_cast<T*>(dx),
                      static_cast<T*>(df), ws);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                     const void* dh, const void* dy, void* dx, void* df, float* ws,
                     cudaStream_t s) {
  const int threads = backward_threads(p.C);
  if (threads == 32) return run_backward<T, 32>(p, x, f, w, dh, dy, dx, df, ws, s);
  if (threads <= kNarrow) return run_backward<T, kNarrow>(p, x, f, w, dh, dy, dx, df, ws, s);
  return run_backward<T, kWide>(p, x, f, w, dh, dy, dx, df, ws, s);
}

}  // namespace

// CTAs of a batch element in the backward: enough warps for the GPU (by registers; above 2560
// columns one CTA an SM), but at least 8 rows each: at 8 rows of bf16 the partial column sums,
// written and read back, are a quarter of the rows' bytes, of float32 an eighth.
void norm_split(NormProblem& p) {
  const int threads = backward_threads(p.C);
  const long long per_sm = threads <= kNarrow ? 480 / threads : 1;
  long long ctas = p.B > 0 ? (kSms * per_sm + p.B - 1) / p.B : 1;
  const long long most = (p.N + 7) / 8;
  if (ctas > most) ctas = most;
  p.ctas = ctas < 1 ? 1 : static_cast<int>(ctas);
}

size_t norm_workspace_floats(const NormProblem& p) {
  return static_cast<size_t>(p.B) * p.ctas * 3 * p.C;
}

cudaError_t launch_norm(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                        void* h, void* y, cudaStream_t s) {
  return p.io == LA_IO_BF16 ? forward<__nv_bfloat16>(p, x, f, w, h, y, s)
                            : forward<float>(p, x, f, w, h, y, s);
}

cudaError_t launch_norm_backward(const NormProblem& p, const void* x, const void* f,
                                 const NormParams& w, const void* dh, const void* dy, void* dx,
                                 void* df, const NormGrads& g, float* ws, cudaStream_t s) {
  cudaError_t e = p.io == LA_IO_BF16
                      ? backward<__nv_bfloat16>(p, x, f, w, dh, dy, dx, df, ws, s)
                      : backward<float>(p, x, f, w, dh, dy, dx, df, ws, s);
  if (e != cudaSuccess) return e;
  if (g.gate == nullptr && g.w_post == nullptr && g.w_pre == nullptr && g.mod_scale == nullptr &&
      g.mod_shift == nullptr)
    return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.C + 31) / 32), 3);
  cfg.blockDim = dim3(kColumnWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];  // its CTAs may be in place before the sums are done
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_columns_kernel, p, w, g, static_cast<const float*>(ws));
}

}  // namespace la
