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
// Backward: a thread owns 8 columns (16 in rows over 2560) of all its CTA's rows and sums the three
// column sums that the parameters' gradients need, sum dy n, sum dy and sum u dh, in
// registers; a second kernel adds the CTAs' partial sums in order. No atomics: the
// same bits every time.
#include "la_block_internal.h"
#include "la_common.cuh"

namespace la {
namespace {

constexpr int kVec = 8;  // columns a thread moves at once

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
  __device__ __forceinline__ float& at(int c) const {
    return p[((c >> 2) & 1) * 4 * vecs + (c >> 3) * 4 + (c & 3)];
  }
};

// Sums over the threads of a row: a warp's shuffles, then (kOneWarp = false) one word per
// warp. `slot` alternates between two sets, so one barrier per sum is enough.
template <bool kOneWarp, int kN>
__device__ __forceinline__ void row_sum(float (&x)[kN], float* scratch, int& slot) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
  if (kOneWarp) return;
  float* s = scratch + slot * 64;
  slot ^= 1;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i * 32 + (threadIdx.x >> 5)] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float t = 0.0f;
    for (int w = 0; w < warps; ++w) t += s[i * 32 + w];
    x[i] = t;
  }
}

// Per-channel factors of batch element b: alpha gate w_post, w_pre (1 + scale), shift.
__device__ __forceinline__ void combine_params(const NormProblem& p, const NormParams& w, int b,
                                               const Line& l1, const Line& l2, const Line* l3) {
  const size_t bc = static_cast<size_t>(b) * p.C;
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    float m = p.alpha;
    if (w.gate != nullptr) m *= w.gate[bc + c];
    if (w.w_post != nullptr) m *= w.w_post[c];
    l1.at(c) = m;
    m = w.w_pre != nullptr ? w.w_pre[c] : 1.0f;
    if (w.mod_scale != nullptr) m *= 1.0f + w.mod_scale[bc + c];
    l2.at(c) = m;
    if (l3 != nullptr) l3->at(c) = w.mod_shift != nullptr ? w.mod_shift[bc + c] : 0.0f;
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
  combine_params(p, w, b, l1, l2, &l3);
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
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        float a[8];
        rf[k].get(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(a[i], a[i], s[0]);
      }
      row_sum<kOneWarp>(s, scratch, slot);
      rstd_f = rsqrtf(fmaf(s[0], inv, p.eps));
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
        if (h != nullptr) store_row<8>(h + row + v * kVec, r[k]);
      }
    }
    if (y == nullptr) continue;
    float mean = 0.0f;
    if (p.layer) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += r[k][i];
      row_sum<kOneWarp>(s, scratch, slot);
      mean = s[0] * inv;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < KV; ++k)
      if (t + k * width < vecs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[k][i] -= mean;
          s[0] = fmaf(r[k][i], r[k][i], s[0]);
        }
      }
    row_sum<kOneWarp>(s, scratch, slot);
    const float rstd = rsqrtf(fmaf(s[0], inv, p.eps));
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      if (v < vecs) {
        float m[8], a[8];
        l2.get(v, m);
        l3.get(v, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaf(r[k][i] * rstd, m[i], a[i]);
        store_row<8>(y + row + v * kVec, a);
      }
    }
  }
}

// Threads of a backward CTA with one and with two vectors each: the most that leaves a thread
// the registers for its column sums and the next row.
constexpr int kOneThreads = 320, kTwoThreads = 512;
static_assert(kTwoThreads * 2 * kVec == kNormMaxC, "the widest row");

// Backward of one batch element's rows; `part`: [B][CTAs][3][C] column sums (sum dy n, sum dy,
// sum u dh).
template <typename T, int KV, bool kOneWarp>
__global__ void __launch_bounds__(KV == 1 ? kOneThreads : kTwoThreads, KV == 1 ? 2 : 1)
norm_backward_kernel(const NormProblem p, const T* x, const T* f, const NormParams w, const T* dh,
                     const T* dy, T* dx, T* df, float* part) {
  extern __shared__ __align__(16) float smem[];
  const int vecs = p.C / kVec, b = blockIdx.y, t = threadIdx.x, width = blockDim.x;
  const Line l1 = {smem, vecs}, l2 = {smem + p.C, vecs};
  float* scratch = smem + 2 * p.C;
  combine_params(p, w, b, l1, l2, nullptr);
  __syncthreads();
  const float inv = 1.0f / static_cast<float>(p.C);
  int slot = 0;
  float sum_e[KV][8], sum_d[KV][8], sum_f[KV][8];
#pragma unroll
  for (int k = 0; k < KV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum_e[k][i] = sum_d[k][i] = sum_f[k][i] = 0.0f;

  Raw<T> rx[KV], rf[KV], rh[KV], ry[KV];
  auto load = [&](int n) {
    const size_t row = (static_cast<size_t>(b) * p.N + n) * p.C;
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      rx[k].zero();
      rf[k].zero();
      rh[k].zero();
      ry[k].zero();
      if (n < p.N && v < vecs) {
        rx[k].load(x + row + v * kVec);
        if (f != nullptr) rf[k].load(f + row + v * kVec);
        if (dh != nullptr) rh[k].load(dh + row + v * kVec);
        if (dy != nullptr) ry[k].load(dy + row + v * kVec);
      }
    }
  };
  constexpr bool kAhead = KV == 1;  // registers for the next row too
  if (kAhead) load(blockIdx.x);
  for (int n = blockIdx.x; n < p.N; n += gridDim.x) {
    const size_t row = (static_cast<size_t>(b) * p.N + n) * p.C;
    if (!kAhead) load(n);
    float hx[KV][8], u[KV][8], g[KV][8], gy[KV][8];  // h, u / w_post, dh, dy
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      rx[k].get(hx[k]);
      rf[k].get(u[k]);
      rh[k].get(g[k]);
      ry[k].get(gy[k]);
    }
    if (kAhead) load(n + gridDim.x);  // the next row is on its way while this one is worked on
    float rstd_f = 1.0f;
    if (w.w_post != nullptr) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(u[k][i], u[k][i], s[0]);
      row_sum<kOneWarp>(s, scratch, slot);
      rstd_f = rsqrtf(fmaf(s[0], inv, p.eps));
    }
    if (f != nullptr) {
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        const int v = t + k * width;
        if (v < vecs) {
          float m[8];
          l1.get(v, m);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[k][i] *= rstd_f;
            hx[k][i] = fmaf(u[k][i], m[i], hx[k][i]);
          }
        }
      }
    }
    if (dy != nullptr) {
      float mean = 0.0f;
      if (p.layer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < KV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += hx[k][i];
        row_sum<kOneWarp>(s, scratch, slot);
        mean = s[0] * inv;
      }
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < KV; ++k)
        if (t + k * width < vecs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            hx[k][i] -= mean;
            s[0] = fmaf(hx[k][i], hx[k][i], s[0]);
          }
        }
      row_sum<kOneWarp>(s, scratch, slot);
      const float rstd = rsqrtf(fmaf(s[0], inv, p.eps));
      float s2[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        const int v = t + k * width;
        if (v < vecs) {
          float m[8];
          l2.get(v, m);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            hx[k][i] *= rstd;  // n
            sum_e[k][i] = fmaf(gy[k][i], hx[k][i], sum_e[k][i]);
            sum_d[k][i] += gy[k][i];
            gy[k][i] *= m[i];
            s2[0] = fmaf(gy[k][i], hx[k][i], s2[0]);
            s2[1] += gy[k][i];
          }
        }
      }
      row_sum<kOneWarp>(s2, scratch, slot);
      const float along = s2[0] * inv, off = p.layer ? s2[1] * inv : 0.0f;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[k][i] = fmaf(rstd, gy[k][i] - fmaf(hx[k][i], along, off), g[k][i]);
    }
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      if (v < vecs) store_row<8>(dx + row + v * kVec, g[k]);
    }
    if (f == nullptr) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      if (v < vecs) {
        float m[8];
        l1.get(v, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum_f[k][i] = fmaf(u[k][i], g[k][i], sum_f[k][i]);
          g[k][i] *= m[i];
          s[0] = fmaf(g[k][i], u[k][i], s[0]);
        }
      }
    }
    if (w.w_post != nullptr) {
      row_sum<kOneWarp>(s, scratch, slot);
      const float along = s[0] * inv;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] = rstd_f * (g[k][i] - u[k][i] * along);
    }
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const int v = t + k * width;
      if (v < vecs) store_row<8>(df + row + v * kVec, g[k]);
    }
  }
  float* out = part + (static_cast<size_t>(b) * gridDim.x + blockIdx.x) * 3 * p.C;
#pragma unroll
  for (int k = 0; k < KV; ++k) {
    const int v = t + k * width;
    if (v < vecs) {
      store_row<8>(out + v * kVec, sum_e[k]);
      store_row<8>(out + p.C + v * kVec, sum_d[k]);
      store_row<8>(out + 2 * p.C + v * kVec, sum_f[k]);
    }
  }
}

// The parameters' gradients from the CTAs' column sums. blockIdx.y: which of the three sums.
// 32 columns a CTA; 32 threads per column add the partial sums, always in the same order.
__global__ void __launch_bounds__(1024)
norm_columns_kernel(const NormProblem p, const NormParams w, const NormGrads g, const float* part) {
  __shared__ float s[32][33];
  const int which = blockIdx.y;
  float* per_b = which == 0 ? g.mod_scale : which == 1 ? g.mod_shift : g.gate;
  float* over_b = which == 0 ? g.w_pre : which == 1 ? nullptr : g.w_post;
  if (per_b == nullptr && over_b == nullptr) return;
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  float total = 0.0f;
  for (int b = 0; b < p.B; ++b) {
    float t = 0.0f;
    if (c < p.C)
      for (int i = lane; i < p.ctas; i += 32)
        t += part[((static_cast<size_t>(b) * p.ctas + i) * 3 + which) * p.C + c];
    s[lane][col] = t;
    __syncthreads();
    if (lane == 0 && c < p.C) {
      t = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) t += s[i][col];
      const size_t bc = static_cast<size_t>(b) * p.C + c;
      if (which == 0) {  // sum dy n
        if (per_b != nullptr) per_b[bc] = t * (w.w_pre != nullptr ? w.w_pre[c] : 1.0f);
        total = fmaf(t, w.mod_scale != nullptr ? 1.0f + w.mod_scale[bc] : 1.0f, total);
      } else if (which == 1) {  // sum dy
        per_b[bc] = t;
      } else {  // sum u dh, u without its weight
        if (per_b != nullptr) per_b[bc] = t * p.alpha * (w.w_post != nullptr ? w.w_post[c] : 1.0f);
        total = fmaf(t, p.alpha * (w.gate != nullptr ? w.gate[bc] : 1.0f), total);
      }
    }
    __syncthreads();
  }
  if (lane == 0 && c < p.C && over_b != nullptr) over_b[c] = total;
}

template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes));
}

constexpr long long kSms = 148;

template <typename T, int KV, bool kOneWarp>
cudaError_t run_forward(const NormProblem& p, int threads, const void* x, const void* f,
                        const NormParams& w, void* h, void* y, cudaStream_t s) {
  const size_t smem = (3 * static_cast<size_t>(p.C) + 128) * sizeof(float);
  auto kernel = norm_kernel<T, KV, kOneWarp>;
  cudaError_t e = allow_smem(kernel, smem);
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
// few or long rows get whole CTAs, a vector per thread.
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

template <typename T, int KV, bool kOneWarp>
cudaError_t run_backward(const NormProblem& p, int threads, const void* x, const void* f,
                         const NormParams& w, const void* dh, const void* dy, void* dx, void* df,
                         float* ws, cudaStream_t s) {
  const size_t smem = (2 * static_cast<size_t>(p.C) + 128) * sizeof(float);
  auto kernel = norm_backward_kernel<T, KV, kOneWarp>;
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(static_cast<unsigned>(p.ctas), static_cast<unsigned>(p.B)), threads, smem, s>>>(
      p, static_cast<const T*>(x), static_cast<const T*>(f), w, static_cast<const T*>(dh),
      static_cast<const T*>(dy), static_cast<T*>(dx), static_cast<T*>(df), ws);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                     const void* dh, const void* dy, void* dx, void* df, float* ws,
                     cudaStream_t s) {
  const int vecs = p.C / kVec, one = (vecs + 31) / 32 * 32, two = (vecs + 63) / 64 * 32;
  if (one == 32) return run_backward<T, 1, true>(p, 32, x, f, w, dh, dy, dx, df, ws, s);
  if (one <= kOneThreads)
    return run_backward<T, 1, false>(p, one, x, f, w, dh, dy, dx, df, ws, s);
  return run_backward<T, 2, false>(p, two, x, f, w, dh, dy, dx, df, ws, s);
}

}  // namespace

// CTAs of a batch element in the backward: enough warps for the GPU, but at least 8 rows each,
// so that the partial column sums stay a tenth of the traffic.
void norm_split(NormProblem& p) {
  int threads = (p.C / kVec + 31) / 32 * 32;
  if (threads > kOneThreads) threads = (p.C / kVec + 63) / 64 * 32;
  long long per_sm = 640 / (threads > 0 ? threads : 32);
  per_sm = per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm;
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
  norm_columns_kernel<<<dim3(static_cast<unsigned>((p.C + 31) / 32), 3), 1024, 0, s>>>(p, w, g, ws);
  return cudaGetLastError();
}

}  // namespace la
