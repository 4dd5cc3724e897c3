// Rotary positions: pairs of a head's first `rot` dimensions turn by
// position x rate, the rest pass through.
//
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = position * rate_k
//
// interleaved: pair k = dimensions (2 k, 2 k + 1); halves: (k, k + rot / 2). The
// inverse turns the other way (with the same m), which is the gradient.
//
// Reads and writes every number once: bound by HBM. The angle is formed and reduced
// in float64 (a float32 angle at position 10^6 is off by 0.03 rad), once per token
// and pair into a shared table that all heads of the token use, so the float64 work
// is 1 / heads of the pairs. A CTA owns a few tokens, about 32 KB of Q and K; with
// few tokens its heads are spread over more CTAs instead. Threads move 16 bytes (two
// 16-byte pieces, one of each half, in the halves layout) and have two such in flight,
// past L2 (each number is used once). Where a half is not made of whole 16-byte pieces,
// single numbers move.
//
// 16384 tokens of 140 heads of 32 in bf16, halves: 51 us, 5.7 TB/s (four pieces in flight and
// ordinary loads and stores: 60 us). Loading ahead of the table, or tables of more tokens,
// measured slower: the registers and the CTAs that they cost hide more than they.
#include "la_block_internal.h"
#include "la_common.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kFlight = 2;  // items in flight per thread
enum { kInterleaved = 0, kHalves = 1, kHalvesScalar = 2 };

// Division of numbers below 2^31 by a divisor the host knows, by the round-up method for invariant
// divisors (Granlund and Montgomery 1994): a high product and a shift (a number's place in the
// tensors takes two divisions, as many instructions as its rotation).
struct Divide {
  uint32_t d, m, shift;
  static Divide by(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return Divide{d, static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
  }
  __device__ __forceinline__ int operator()(int n) const {
    const uint32_t u = static_cast<uint32_t>(n);
    return static_cast<int>((static_cast<uint64_t>(__umulhi(m, u)) + u) >> shift);
  }
};

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
// The first `pairs` pairs of `turned`, the others as they were: a NaN would lose its bits on the
// way through float32. A float32 piece is no conversion.
__device__ __forceinline__ uint4 keep_bits(const uint4& turned, const uint4& was, int pairs, const float (&)[8]) {
  return make_uint4(turned.x, pairs > 1 ? turned.y : was.y, pairs > 2 ? turned.z : was.z,
                    pairs > 3 ? turned.w : was.w);
}
__device__ __forceinline__ uint4 keep_bits(const uint4& turned, const uint4&, int, const float (&)[4]) {
  return turned;
}
__device__ __forceinline__ void turn(float a, float b, float2 cs, float& x, float& y) {
  x = fmaf(a, cs.x, -b * cs.y);
  y = fmaf(a, cs.y, b * cs.x);
}

// Items of a head: what one thread moves at once.
template <typename T, int kLayout>
__host__ __device__ int items_of_head(int D, int rot) {
  constexpr int V = Vec<T>::kN;
  if (kLayout == kInterleaved) return D / V;
  if (kLayout == kHalves) return rot / (2 * V) + (D - rot) / V;
  return rot / 2 + (D - rot);
}

template <typename T, int kLayout>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const RotaryProblem p, int tokens, const Divide share, const Divide per_head,
              const T* q, const T* k, const int* pos, T* qo, T* ko) {
  constexpr int V = Vec<T>::kN;
  extern __shared__ float2 table[];  // [tokens][rot / 2]
  const int pairs = p.rot / 2;
  const long long row0 = static_cast<long long>(blockIdx.x) * tokens;
  const int here = static_cast<int>(min(static_cast<long long>(tokens), p.rows - row0));
  for (int i = threadIdx.x; i < here * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    const unsigned row = static_cast<unsigned>(row0) + t;  // below 2^31
    const int n = static_cast<int>(row % static_cast<unsigned>(p.N));
    const long long at = pos != nullptr ? static_cast<long long>(pos[p.pos_rows ? row : n])
                                        : static_cast<long long>(p.pos_offset) + n;
    const double kTurn = 6.283185307179586476925286766559;
    const double a = static_cast<double>(at) * p.rate[j];
    const double r = a - kTurn * rint(a * (1.0 / kTurn));
    float s, c;
    const float rf = static_cast<float>(r), rest = static_cast<float>(r - rf);
    sincosf(rf, &s, &c);
    const float m = static_cast<float>(p.mscale);
    const float c1 = fmaf(-s, rest, c) * m, s1 = fmaf(c, rest, s) * m;
    table[i] = make_float2(c1, p.inverse ? -s1 : s1);
  }
  __syncthreads();

  const int items = per_head.d, nq = p.H * items, per_token = nq + p.Hk * items;
  // this CTA's share of each token's items (the last CTA's may reach past them)
  const int first = blockIdx.y * share.d, total = here * static_cast<int>(share.d);
  for (int base = threadIdx.x; base < total; base += kThreads * kFlight) {
    const T* src[kFlight];
    T* dst[kFlight];
    int tok[kFlight], item[kFlight];
    uint4 u[kFlight], w[kFlight];
    T sa[kFlight], sb[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = base + f * kThreads;
      tok[f] = -1;
      const int t = share(i), x = first + i - t * static_cast<int>(share.d);
      if (i < total && x < per_token) {
        const bool is_q = x < nq;
        const int y = is_q ? x : x - nq;
        const int head = per_head(y);
        item[f] = y - head * items;
        tok[f] = t;
        const size_t ofs =
            (static_cast<size_t>(row0 + t) * (is_q ? p.H : p.Hk) + head) * p.D;
        src[f] = (is_q ? q : k) + ofs;
        dst[f] = (is_q ? qo : ko) + ofs;
        if (kLayout == kInterleaved) {
          u[f] = __ldcs(reinterpret_cast<const uint4*>(src[f] + item[f] * V));
        } else if (kLayout == kHalves) {
          const int turning = pairs / V;
          if (item[f] < turning) {
            u[f] = __ldcs(reinterpret_cast<const uint4*>(src[f] + item[f] * V));
            w[f] = __ldcs(reinterpret_cast<const uint4*>(src[f] + pairs + item[f] * V));
          } else {
            u[f] = __ldcs(reinterpret_cast<const uint4*>(src[f] + p.rot + (item[f] - turning) * V));
          }
        } else {
          if (item[f] < pairs) {
            sa[f] = src[f][item[f]];
            sb[f] = src[f][pairs + item[f]];
          } else {
            sa[f] = src[f][pairs + item[f]];  // rot + (item - pairs)
          }
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (tok[f] < 0) continue;
      const float2* cs = table + tok[f] * pairs;
      if (kLayout == kInterleaved) {
        const int j0 = item[f] * (V / 2);  // its first pair
        if (j0 < pairs) {
          float x[V];
          unpack(u[f], x);
#pragma unroll
          for (int j = 0; j < V / 2; ++j)
            if (j0 + j < pairs) {
              const float a = x[2 * j], b = x[2 * j + 1];
              turn(a, b, cs[j0 + j], x[2 * j], x[2 * j + 1]);
            }
          u[f] = keep_bits(pack(x), u[f], pairs - j0, x);
        }
        __stcs(reinterpret_cast<uint4*>(dst[f] + item[f] * V), u[f]);
      } else if (kLayout == kHalves) {
        const int turning = pairs / V;
        if (item[f] < turning) {
          float x[V], y[V];
          unpack(u[f], x);
          unpack(w[f], y);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float a = x[j], b = y[j];
            turn(a, b, cs[item[f] * V + j], x[j], y[j]);
          }
          __stcs(reinterpret_cast<uint4*>(dst[f] + item[f] * V), pack(x));
          __stcs(reinterpret_cast<uint4*>(dst[f] + pairs + item[f] * V), pack(y));
        } else {
          __stcs(reinterpret_cast<uint4*>(dst[f] + p.rot + (item[f] - turning) * V), u[f]);
        }
      } else {
        if (item[f] < pairs) {
          float x, y;
          turn(static_cast<float>(sa[f]), static_cast<float>(sb[f]), cs[item[f]], x, y);
          dst[f][item[f]] = static_cast<T>(x);
          dst[f][pairs + item[f]] = static_cast<T>(y);
        } else {
          dst[f][pairs + item[f]] = sa[f];
        }
      }
    }
  }
}

template <typename T, int kLayout>
cudaError_t launch(const RotaryProblem& p, const void* Q, const void* K, const int* pos, void* Qo,
                   void* Ko, cudaStream_t s) {
  const long long per_token = 1LL * (p.H + p.Hk) * items_of_head<T, kLayout>(p.D, p.rot);
  const long long bytes = 1LL * (p.H + p.Hk) * p.D * sizeof(T);
  long long tokens = 32768 / bytes;
  tokens = tokens < 1 ? 1 : tokens > 16 ? 16 : tokens;
  // at least two CTAs per SM: first fewer tokens each, then fewer heads
  const long long want = 2 * 148;
  while (tokens > 1 && (p.rows + tokens - 1) / tokens < want) tokens /= 2;
  const long long ctas = (p.rows + tokens - 1) / tokens;
  long long split = (want + ctas - 1) / ctas;
  const long long most = (per_token * tokens + kThreads - 1) / kThreads;
  split = split > most ? most : split;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const size_t smem = static_cast<size_t>(tokens) * (p.rot / 2) * sizeof(float2);
  const Divide share = Divide::by(static_cast<uint32_t>((per_token + split - 1) / split));
  const Divide per_head = Divide::by(static_cast<uint32_t>(items_of_head<T, kLayout>(p.D, p.rot)));
  rotary_kernel<T, kLayout>
      <<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(split)), kThreads, smem, s>>>(
          p, static_cast<int>(tokens), share, per_head, static_cast<const T*>(Q), static_cast<const T*>(K), pos,
          static_cast<T*>(Qo), static_cast<T*>(Ko));
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const RotaryProblem& p, const void* Q, const void* K, const int* pos, void* Qo,
                     void* Ko, cudaStream_t s) {
  if (!p.half) return launch<T, kInterleaved>(p, Q, K, pos, Qo, Ko, s);
  if ((p.rot / 2) % Vec<T>::kN == 0) return launch<T, kHalves>(p, Q, K, pos, Qo, Ko, s);
  return launch<T, kHalvesScalar>(p, Q, K, pos, Qo, Ko, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem& p, const void* Q, const void* K, const int* pos,
                          void* Qo, void* Ko, cudaStream_t s) {
  return p.io == LA_IO_BF16 ? dispatch<__nv_bfloat16>(p, Q, K, pos, Qo, Ko, s)
                            : dispatch<float>(p, Q, K, pos, Qo, Ko, s);
}

}  // namespace la
