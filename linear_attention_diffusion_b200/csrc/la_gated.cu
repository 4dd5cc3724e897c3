// Gated linear attention, forward and backward:
//
//   S_n = exp(g_n) S_{n-1} + k_n^T v_n,   o_n = scale q_n S_n
//
// per batch element and head, D = 32, S float32. The sequence is walked in blocks
// of 16 tokens. With c_i the sum of the log gates from the block's first token to
// token i and S the state before the block,
//
//   o_i = scale (exp(c_i) q_i S + sum_{j <= i} exp(c_i - c_j) (q_i . k_j) v_j)
//   S  <- exp(c_15) S + sum_j exp(c_15 - c_j) k_j^T v_j
//
// every exponent a sum of the gates between two tokens, so with gates <= 1 no
// factor exceeds 1 whatever the length. One warp owns a head's segment of the
// sequence, keeps S in registers from block to block and streams Q, K, V through a
// ring of asynchronous 16-byte copies of its own: no barrier between warps, and
// each of Q, K, V read once. Few heads do not fill the GPU, so the sequence is cut
// into segments: a first pass forms every segment's own state (it reads K and V
// once more), a second combines them in order, and the segments then run at once.
//
// Backward, with U_n = sum_{i >= n} (decay n to i) scale q_i^T dO_i, the gradient
// that reaches S_n:
//
//   dq_i = scale S_i dO_i,  dk_j = U_j v_j,  dv_j = k_j U_j,
//   dg_t = <exp(g_t) U_t, S_{t-1}> = dg_{t+1} + q_t . dq_t - k_t . dk_t
//
// dq is the forward with (q, k, v) = (dO, v, k); dk and dv come from one walk
// backwards that carries U. dg is summed backwards from the two walks' float32 row
// products, and set afresh to <U, S> every kGateAnchor tokens, where the first walk
// has left its S: rounding errors of the sum do not grow with the length.
#include "la_gated.cuh"

namespace la {
namespace gated {
namespace {

constexpr int kWarps = 4;  // warps of a CTA: neighbouring heads of one segment

struct Walk {
  const void *q, *k, *v, *w;  // operands; w: one more tile (see each kernel)
  const float* G;
  void *o, *o2;
  const float* init;     // external state at the walk's start, [B*H][32*32], or null
  float* final_;         // external state at the walk's end, or null
  const float* prefix;   // state at the start of each segment (nseg > 1), [B*H][nseg][1024]
  float* anchors;        // backward: S every kGateAnchor tokens, [B*H][anchors][1024]
  float* rows;           // backward: q . dq of every token, [B*H][N]
  float* dG;
  int anchor, nanchor;   // tokens between anchors; anchors per head
  GatedProblem p;
};

__device__ __forceinline__ size_t head_base(const GatedProblem& p, int bh) {
  return (static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H) * 32;
}

// One segment forwards. kBack = false: the forward itself, state rows = v's
// dimensions. kBack = true: dq from (q, k, v) = (dO, V, K) with w = Q; it also
// writes q . dq of every token and S at the anchors.
template <int NP, bool kBack, int kStages>
__global__ void __launch_bounds__(kWarps * 32, (kBack || NP == 3) ? 3 : 4)
walk_kernel(const Walk a) {
  using T = typename Io<NP>::T;
  constexpr int NC = NP == 1 ? 2 : 3;
  constexpr int NT = kBack ? 4 : 3;
  using M = Smem<NP, NT, kStages, 3>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const GatedProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int BH = p.B * p.H;
  if (unit >= static_cast<long long>(BH) * p.nseg) return;
  const int seg = static_cast<int>(unit / BH), bh = static_cast<int>(unit % BH);
  const int n_begin = seg * p.seg, n_end = min(p.N, n_begin + p.seg);
  const int nblk = (n_end - n_begin + kGateBlock - 1) / kGateBlock;
  const size_t stride = static_cast<size_t>(p.H) * 32;
  const size_t base = head_base(p, bh);
  const T* src[4] = {static_cast<const T*>(a.q) + base, static_cast<const T*>(a.k) + base,
                     static_cast<const T*>(a.v) + base,
                     kBack ? static_cast<const T*>(a.w) + base : nullptr};
  const float* G = a.G + static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
  uint8_t* smem = smem_all + warp * M::kWarp;
  uint8_t* planes = smem + kStages * M::kStage;
  const uint32_t smem_u = smem_addr(smem);

  auto issue = [&](int blk) {
    if (blk < nblk) {
      const uint32_t st = smem_u + (blk % kStages) * M::kStage;
      const int n0 = n_begin + blk * kGateBlock;
#pragma unroll
      for (int t = 0; t < NT; ++t) load_tile<NP>(st + t * M::kTile, src[t], stride, n0, n_end, lane);
      if (lane < 16) {
        const bool in = n0 + lane < n_end;
        cp4(st + NT * M::kTile + lane * 4, G + (in ? static_cast<size_t>(n0 + lane) * p.H : 0),
            in ? 4 : 0);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  State S;
  if (p.nseg > 1)
    S.load(a.prefix + (static_cast<size_t>(bh) * p.nseg + seg) * 1024, lane);
  else if (a.init != nullptr)
    S.template load_outer<!kBack>(a.init + static_cast<size_t>(bh) * 1024, lane);
  else
    S.zero();
  const LaneOff off(lane);
  const int r0 = lane >> 2;

  for (int blk = 0; blk < nblk; ++blk) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(blk + kStages - 1);  // into the stage that the block before has left
    uint8_t* st = smem + (blk % kStages) * M::kStage;
    const int n0 = n_begin + blk * kGateBlock;
    const float gate = *reinterpret_cast<const float*>(st + NT * M::kTile + (lane & 15) * 4);
    uint32_t tile[3];
    if (NP == 1) {
#pragma unroll
      for (int t = 0; t < 3; ++t) tile[t] = smem_addr(st) + t * M::kTile;
    } else {
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        split_tile(st + t * M::kTile, planes + t * 3 * kPlane, lane);
        tile[t] = smem_addr(planes) + t * 3 * kPlane;
      }
      __syncwarp();
    }
    if (kBack && (n0 % a.anchor) == 0)
      S.store(a.anchors + (static_cast<size_t>(bh) * a.nanchor + n0 / a.anchor) * 1024, lane);

    const Decay d(gate, lane);
    float acc[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[e][i] = 0.0f;
    float w[2][4];
    {
      Frag<NP> q, k;
      q.rows(tile[0], off);
      k.cols(tile[1], off);
      token_product(w, q, k);
      S.template apply<NP, NC>(acc, q);
    }
    {
      const float head = d.head(lane) * p.scale;
      float l[2][4];
      d.between<true>(lane, l);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        scale_row(acc, h, __shfl_sync(0xffffffffu, head, r0 + 8 * h));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float& e = w[x >> 1][2 * h + (x & 1)];
          e = l[h][x] == 0.0f ? 0.0f : e * (l[h][x] * p.scale);
        }
      }
    }
    Frag<NP> v;
    v.deep(tile[2], off);
    weigh<NP, NC>(acc, w, v);
    {
      float wt[4];
      Decay::spread(d.tail(lane), lane, wt);
      Frag<NP> k;
      k.deep(tile[1], off);
      S.template update<NP, NC>(d.whole(), v, k, wt);
    }
    if (kBack) {
      float dots[2];
      row_dots<NP>(acc, st + 3 * M::kTile, lane, dots);
      if ((lane & 3) == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (n0 + r0 + 8 * h < n_end)
            a.rows[static_cast<size_t>(bh) * p.N + n0 + r0 + 8 * h] = dots[h];
      }
    }
    __syncwarp();  // every lane is done with the first tile: the output passes through it
    store_tile<NP>(acc, st, static_cast<T*>(a.o) + base, stride, n0, n_end, lane);
  }
  cp_wait<0>();
  if (seg == p.nseg - 1) {
    if (!kBack && a.final_ != nullptr)
      S.template store_outer<true>(a.final_ + static_cast<size_t>(bh) * 1024, lane);
    if (kBack)  // the state after the last token: the anchor of the sequence's end
      S.store(a.anchors + (static_cast<size_t>(bh) * a.nanchor + a.nanchor - 1) * 1024, lane);
  }
}

// One segment backwards: dk and dv (o and o2), the log gates' gradient, and with
// a.final_ the gradient of the state before the first token. q, k, v as in the
// forward, w = dO. The carried state X (rows: k's dimensions, columns: v's) is the
// gradient that reaches the state at a block's end from later tokens.
template <int NP, int kStages>
__global__ void __launch_bounds__(kWarps * 32, NP == 3 ? 2 : 3) walk_back_kernel(const Walk a) {
  using T = typename Io<NP>::T;
  constexpr int NC = NP == 1 ? 2 : 3;
  constexpr int NT = 4;
  using M = Smem<NP, NT, kStages>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const GatedProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int BH = p.B * p.H;
  if (unit >= static_cast<long long>(BH) * p.nseg) return;
  const int seg = static_cast<int>(unit / BH), bh = static_cast<int>(unit % BH);
  const int n_begin = seg * p.seg, n_end = min(p.N, n_begin + p.seg);
  const int nblk = (n_end - n_begin + kGateBlock - 1) / kGateBlock;
  const size_t stride = static_cast<size_t>(p.H) * 32;
  const size_t base = head_base(p, bh);
  const T* src[4] = {static_cast<const T*>(a.k) + base, static_cast<const T*>(a.v) + base,
                     static_cast<const T*>(a.q) + base, static_cast<const T*>(a.w) + base};
  const size_t gbase = static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
  const float* rows = a.rows + static_cast<size_t>(bh) * p.N;
  uint8_t* smem = smem_all + warp * M::kWarp;
  uint8_t* planes = smem + kStages * M::kStage;
  const uint32_t smem_u = smem_addr(smem);

  auto issue = [&](int it) {  // it counts from the segment's last block
    if (it < nblk) {
      const uint32_t st = smem_u + (it % kStages) * M::kStage;
      const int n0 = n_begin + (nblk - 1 - it) * kGateBlock;
#pragma unroll
      for (int t = 0; t < NT; ++t) load_tile<NP>(st + t * M::kTile, src[t], stride, n0, n_end, lane);
      const int i = lane & 15;
      const bool in = n0 + i < n_end;
      cp4(st + NT * M::kTile + lane * 4,
          lane < 16 ? a.G + gbase + (in ? static_cast<size_t>(n0 + i) * p.H : 0)
                    : rows + (in ? n0 + i : 0),
          in ? 4 : 0);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  State X;
  if (p.nseg > 1)
    X.load(a.prefix + (static_cast<size_t>(bh) * p.nseg + seg) * 1024, lane);
  else if (a.init != nullptr)
    X.template load_outer<false>(a.init + static_cast<size_t>(bh) * 1024, lane);
  else
    X.zero();
  // dg just past the segment: <X, S> there. At the sequence's end S is the last anchor.
  const float* anchors = a.anchors + static_cast<size_t>(bh) * a.nanchor * 1024;
  float carry;
  {
    State S;
    S.load(anchors + static_cast<size_t>(seg == p.nseg - 1 ? a.nanchor - 1 : n_end / a.anchor) *
                         1024, lane);
    carry = X.dot(S);
  }
  const LaneOff off(lane);
  const int r0 = lane >> 2;

  for (int it = 0; it < nblk; ++it) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(it + kStages - 1);
    uint8_t* st = smem + (it % kStages) * M::kStage;
    const int n0 = n_begin + (nblk - 1 - it) * kGateBlock;
    const float gate = *reinterpret_cast<const float*>(st + NT * M::kTile + (lane & 15) * 4);
    const float rdot = *reinterpret_cast<const float*>(st + NT * M::kTile + 64 + (lane & 15) * 4);
    uint32_t tile[NT];
    if (NP == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t) tile[t] = smem_addr(st) + t * M::kTile;
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        split_tile(st + t * M::kTile, planes + t * 3 * kPlane, lane);
        tile[t] = smem_addr(planes) + t * 3 * kPlane;
      }
      __syncwarp();
    }
    const Decay d(gate, lane);
    float dk[4][4], dv[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) dk[e][i] = dv[e][i] = 0.0f;
    float wk[2][4], wv[2][4];  // rows: token j of k, v; columns: token i of q, dO
    {
      Frag<NP> v, k, c;
      v.rows(tile[1], off);
      k.rows(tile[0], off);
      X.template apply_both<NP, NC>(dk, v, dv, k);
      c.cols(tile[3], off);
      token_product(wk, v, c);  // v_j . dO_i
      c.cols(tile[2], off);
      token_product(wv, k, c);  // k_j . q_i
    }
    {
      const float tail = d.tail(lane);
      float l[2][4];
      d.between<false>(lane, l);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float tj = __shfl_sync(0xffffffffu, tail, r0 + 8 * h);
        scale_row(dk, h, tj);
        scale_row(dv, h, tj);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float f = l[h][x] * p.scale;
          float& ek = wk[x >> 1][2 * h + (x & 1)];
          float& ev = wv[x >> 1][2 * h + (x & 1)];
          ek = l[h][x] == 0.0f ? 0.0f : ek * f;
          ev = l[h][x] == 0.0f ? 0.0f : ev * f;
        }
      }
    }
    {
      float wt[4];
      Decay::spread(d.head(lane) * p.scale, lane, wt);
      Frag<NP> q, o;
      q.deep(tile[2], off);
      o.deep(tile[3], off);
      weigh<NP, NC>(dk, wk, q);
      weigh<NP, NC>(dv, wv, o);
      X.template update<NP, NC>(d.whole(), q, o, wt);
    }
    // dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t, summed from the block's end; a stop
    // passes no gradient and restarts the sum
    float dots[2];
    row_dots<NP>(dk, st, lane, dots);
    {
      const int i = lane & 15;
      const float lo = __shfl_sync(0xffffffffu, dots[0], (i & 7) * 4);
      const float hi = __shfl_sync(0xffffffffu, dots[1], (i & 7) * 4);
      float x = rdot - (i < 8 ? lo : hi);
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, x, s, 16);
        if (i + s < 16) x += y;
      }
      const uint32_t after = d.stops & ~((2u << i) - 1u);
      const int until = after != 0 ? __ffs(after) - 1 : 0;
      const float cut = __shfl_sync(0xffffffffu, x, until);
      float dg = after != 0 ? x - cut : carry + x;
      if ((d.stops >> i) & 1u) dg = 0.0f;
      if (lane < 16 && n0 + i < n_end) a.dG[gbase + static_cast<size_t>(n0 + i) * p.H] = dg;
      carry = __shfl_sync(0xffffffffu, dg, 0);
    }
    if (n0 % a.anchor == 0 && n0 > n_begin) {
      State S;
      S.load(anchors + static_cast<size_t>(n0 / a.anchor) * 1024, lane);
      carry = X.dot(S);
    }
    __syncwarp();
    store_tile<NP>(dk, st, static_cast<T*>(a.o) + base, stride, n0, n_end, lane);
    store_tile<NP>(dv, st + M::kTile, static_cast<T*>(a.o2) + base, stride, n0, n_end, lane);
  }
  cp_wait<0>();
  if (seg == 0 && a.final_ != nullptr)
    X.template store_outer<false>(a.final_ + static_cast<size_t>(bh) * 1024, lane);
}

// Every segment's own state from zero and its whole decay. Forward: S only, rows =
// v's dimensions. Backward: S and X = sum_i (decay from the segment's start to i)
// scale q_i^T dO_i, rows = k's (q's) dimensions. Segment s's S goes to slot s + 1 of
// `states` (it becomes the state at the start of s + 1), its X to slot s - 1 of `grads`.
template <int NP, bool kBack, int kStages>
__global__ void __launch_bounds__(kWarps * 32, NP == 3 ? 3 : 4)
segment_kernel(const GatedProblem p, const void* qv, const void* kv, const void* vv,
               const void* dov, const float* Gv, float* states, float* grads, float* decays) {
  using T = typename Io<NP>::T;
  constexpr int NC = NP == 1 ? 2 : 3;
  constexpr int NT = kBack ? 4 : 2;
  using M = Smem<NP, NT, kStages>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int BH = p.B * p.H;
  const int segs = kBack ? p.nseg : p.nseg - 1;  // nothing follows the last one forwards
  if (unit >= static_cast<long long>(BH) * segs) return;
  const int seg = static_cast<int>(unit / BH), bh = static_cast<int>(unit % BH);
  const int n_begin = seg * p.seg, n_end = min(p.N, n_begin + p.seg);
  const int nblk = (n_end - n_begin + kGateBlock - 1) / kGateBlock;
  const size_t stride = static_cast<size_t>(p.H) * 32;
  const size_t base = head_base(p, bh);
  const T* src[4] = {static_cast<const T*>(kBack ? kv : vv) + base,
                     static_cast<const T*>(kBack ? vv : kv) + base,
                     kBack ? static_cast<const T*>(qv) + base : nullptr,
                     kBack ? static_cast<const T*>(dov) + base : nullptr};
  const float* G = Gv + static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
  uint8_t* smem = smem_all + warp * M::kWarp;
  uint8_t* planes = smem + kStages * M::kStage;
  const uint32_t smem_u = smem_addr(smem);
  auto issue = [&](int blk) {
    if (blk < nblk) {
      const uint32_t st = smem_u + (blk % kStages) * M::kStage;
      const int n0 = n_begin + blk * kGateBlock;
#pragma unroll
      for (int t = 0; t < NT; ++t) load_tile<NP>(st + t * M::kTile, src[t], stride, n0, n_end, lane);
      if (lane < 16) {
        const bool in = n0 + lane < n_end;
        cp4(st + NT * M::kTile + lane * 4, G + (in ? static_cast<size_t>(n0 + lane) * p.H : 0),
            in ? 4 : 0);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  State S, X;
  S.zero();
  if (kBack) X.zero();
  float whole = 1.0f;
  const LaneOff off(lane);
  for (int blk = 0; blk < nblk; ++blk) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(blk + kStages - 1);
    const uint8_t* st = smem + (blk % kStages) * M::kStage;
    const float gate = *reinterpret_cast<const float*>(st + NT * M::kTile + (lane & 15) * 4);
    uint32_t tile[NT];
    if (NP == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t) tile[t] = smem_addr(st) + t * M::kTile;
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        split_tile(st + t * M::kTile, planes + t * 3 * kPlane, lane);
        tile[t] = smem_addr(planes) + t * 3 * kPlane;
      }
      __syncwarp();
    }
    const Decay d(gate, lane);
    float w[4];
    {
      Decay::spread(d.tail(lane), lane, w);
      Frag<NP> x, y;
      x.deep(tile[0], off);
      y.deep(tile[1], off);
      S.template update<NP, NC>(d.whole(), x, y, w);
    }
    if (kBack) {
      Decay::spread(d.head(lane) * (p.scale * whole), lane, w);
      Frag<NP> x, y;
      x.deep(tile[2], off);
      y.deep(tile[3], off);
      X.template update<NP, NC>(1.0f, x, y, w);
    }
    whole *= d.whole();
  }
  cp_wait<0>();
  const size_t slots = static_cast<size_t>(bh) * p.nseg;
  if (seg + 1 < p.nseg) S.store(states + (slots + seg + 1) * 1024, lane);
  if (kBack && seg > 0) X.store(grads + (slots + seg - 1) * 1024, lane);
  if (lane == 0) decays[slots + seg] = whole;
}

// Segments in order: slot s becomes the state at segment s's start (forwards), or the
// gradient at its end (backwards). One thread per four numbers of a head's state;
// blockIdx.y = 0: states, 1: gradients.
template <bool kTransposed>
__global__ void __launch_bounds__(256)
combine_kernel(int BH, int nseg, const float* decays, float* states, const float* s_init,
               float* grads, const float* x_init) {
  const int bh = blockIdx.x, f = threadIdx.x;
  const bool back = blockIdx.y == 1;
  float4* slot = reinterpret_cast<float4*>(back ? grads : states) +
                 static_cast<size_t>(bh) * nseg * 256 + f;
  const float* init = back ? x_init : s_init;
  const float* dec = decays + static_cast<size_t>(bh) * nseg;
  float4 run = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (init != nullptr) {
    const int mt = f >> 7, nt = (f >> 5) & 3, lane = f & 31;
    init += static_cast<size_t>(bh) * 1024;
    run.x = init[State::outer<kTransposed>(mt, nt, 0, lane)];
    run.y = init[State::outer<kTransposed>(mt, nt, 1, lane)];
    run.z = init[State::outer<kTransposed>(mt, nt, 2, lane)];
    run.w = init[State::outer<kTransposed>(mt, nt, 3, lane)];
  }
  // forwards: start of 0, then s = 1 .. with the decay of s - 1; backwards: end of the
  // last, then s = nseg - 2 .. 0 with the decay of s + 1
  slot[static_cast<size_t>(back ? nseg - 1 : 0) * 256] = run;
  constexpr int kAhead = 8;
  for (int s0 = 1; s0 < nseg; s0 += kAhead) {
    float4 t[kAhead];
    float m[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (s0 + k < nseg) {
        const int s = back ? nseg - 1 - (s0 + k) : s0 + k;
        t[k] = __ldcg(slot + static_cast<size_t>(s) * 256);
        m[k] = dec[back ? s + 1 : s - 1];
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (s0 + k < nseg) {
        const int s = back ? nseg - 1 - (s0 + k) : s0 + k;
        if (m[k] == 0.0f) run = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        run.x = fmaf(m[k], run.x, t[k].x);
        run.y = fmaf(m[k], run.y, t[k].y);
        run.z = fmaf(m[k], run.z, t[k].z);
        run.w = fmaf(m[k], run.w, t[k].w);
        slot[static_cast<size_t>(s) * 256] = run;
      }
  }
}

// A few tokens, one after another: one warp per head, the state in registers, eight
// rows of four columns per lane. Bound by the state's 8 KB read and written.
template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_f(float x) {
  return x;
}
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = lo_f(v.x);
  x[1] = hi_f(v.x);
  x[2] = lo_f(v.y);
  x[3] = hi_f(v.y);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}

template <typename T>
__global__ void __launch_bounds__(128)
step_kernel(const GatedProblem p, const T* Q, const T* K, const T* V, const float* G,
            const float* S_in, float* S_out, T* O) {
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.B) * p.H) return;
  const int bh = static_cast<int>(unit);
  const size_t base = head_base(p, bh);
  const size_t gbase = static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
  const int e4 = (lane & 7) * 4, dr = lane >> 3;
  float s[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (S_in != nullptr)
      load4(S_in + static_cast<size_t>(bh) * 1024 + (dr + 4 * i) * 32 + e4, s[i]);
    else
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
  }
  for (int n = 0; n < p.N; ++n) {
    const size_t at = base + static_cast<size_t>(n) * p.H * 32;
    const float g = G[gbase + static_cast<size_t>(n) * p.H] * kLog2e;
    const float a = g < kStop ? 0.0f : exp2_fast(g);
    const float k = to_f(K[at + lane]), q = to_f(Q[at + lane]) * p.scale;
    float v[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load4(V + at + e4, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float kd = __shfl_sync(0xffffffffu, k, dr + 4 * i);
      const float qd = __shfl_sync(0xffffffffu, q, dr + 4 * i);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // a stop drops the state whatever it holds
        s[i][x] = a == 0.0f ? kd * v[x] : fmaf(a, s[i][x], kd * v[x]);
        o[x] = fmaf(qd, s[i][x], o[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      o[x] += __shfl_xor_sync(0xffffffffu, o[x], 8);
      o[x] += __shfl_xor_sync(0xffffffffu, o[x], 16);
    }
    if (dr == 0) store4(O + at + e4, o);
  }
  if (S_out != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      store4(S_out + static_cast<size_t>(bh) * 1024 + (dr + 4 * i) * 32 + e4, s[i]);
  }
}

template <typename Kernel>
cudaError_t allow_smem(Kernel k, int bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

unsigned grid_of(long long units) { return static_cast<unsigned>((units + kWarps - 1) / kWarps); }

template <int NP>
cudaError_t forward(const GatedProblem& p, const void* Q, const void* K, const void* V,
                    const float* G, const float* S_in, float* S_out, void* O, float* ws,
                    cudaStream_t s) {
  constexpr int kSegStages = NP == 1 ? 6 : 3, kStages = NP == 1 ? 4 : 2;
  const long long BH = 1LL * p.B * p.H;
  float* states = ws;
  float* decays = ws + BH * p.nseg * 1024;
  cudaError_t e;
  if (p.nseg > 1) {
    auto seg = segment_kernel<NP, false, kSegStages>;
    const int bytes = kWarps * Smem<NP, 2, kSegStages>::kWarp;
    if ((e = allow_smem(seg, bytes)) != cudaSuccess) return e;
    seg<<<grid_of(BH * (p.nseg - 1)), kWarps * 32, bytes, s>>>(p, Q, K, V, nullptr, G, states,
                                                              nullptr, decays);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    combine_kernel<true><<<dim3(static_cast<unsigned>(BH), 1), 256, 0, s>>>(
        static_cast<int>(BH), p.nseg, decays, states, S_in, nullptr, nullptr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  Walk a = {};
  a.q = Q;
  a.k = K;
  a.v = V;
  a.G = G;
  a.o = O;
  a.init = S_in;
  a.final_ = S_out;
  a.prefix = states;
  a.p = p;
  auto walk = walk_kernel<NP, false, kStages>;
  const int bytes = kWarps * Smem<NP, 3, kStages, 3>::kWarp;
  if ((e = allow_smem(walk, bytes)) != cudaSuccess) return e;
  walk<<<grid_of(BH * p.nseg), kWarps * 32, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int NP>
cudaError_t backward(const GatedProblem& p, const void* Q, const void* K, const void* V,
                     const float* G, const float* S_in, const void* dO, const float* dS_out,
                     void* dQ, void* dK, void* dV, float* dG, float* dS_in, float* ws,
                     cudaStream_t s) {
  constexpr int kStages = NP == 1 ? 4 : 2;
  const long long BH = 1LL * p.B * p.H;
  Walk a = {};
  a.anchor = p.seg < kGateAnchor ? p.seg : kGateAnchor;
  a.nanchor = (p.N + a.anchor - 1) / a.anchor + 1;
  float* states = ws;
  float* grads = states + BH * p.nseg * 1024;
  a.anchors = grads + BH * p.nseg * 1024;
  a.rows = a.anchors + BH * a.nanchor * 1024;
  float* decays = a.rows + (BH * p.N + 3) / 4 * 4;
  cudaError_t e;
  if (p.nseg > 1) {
    auto seg = segment_kernel<NP, true, kStages>;
    const int bytes = kWarps * Smem<NP, 4, kStages>::kWarp;
    if ((e = allow_smem(seg, bytes)) != cudaSuccess) return e;
    seg<<<grid_of(BH * p.nseg), kWarps * 32, bytes, s>>>(p, Q, K, V, dO, G, states, grads, decays);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    combine_kernel<false><<<dim3(static_cast<unsigned>(BH), 2), 256, 0, s>>>(
        static_cast<int>(BH), p.nseg, decays, states, S_in, grads, dS_out);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  a.G = G;
  a.p = p;
  a.q = dO;
  a.k = V;
  a.v = K;
  a.w = Q;
  a.o = dQ;
  a.init = S_in;
  a.prefix = states;
  auto walk = walk_kernel<NP, true, NP == 1 ? 3 : 2>;
  int bytes = kWarps * Smem<NP, 4, NP == 1 ? 3 : 2, 3>::kWarp;
  if ((e = allow_smem(walk, bytes)) != cudaSuccess) return e;
  walk<<<grid_of(BH * p.nseg), kWarps * 32, bytes, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  a.q = Q;
  a.k = K;
  a.v = V;
  a.w = dO;
  a.o = dK;
  a.o2 = dV;
  a.init = dS_out;
  a.final_ = dS_in;
  a.prefix = grads;
  a.dG = dG;
  auto back = walk_back_kernel<NP, kStages>;
  bytes = kWarps * Smem<NP, 4, kStages>::kWarp;
  if ((e = allow_smem(back, bytes)) != cudaSuccess) return e;
  back<<<grid_of(BH * p.nseg), kWarps * 32, bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gated

// Segments: as many as fill one wave of warps (16 on each of 148 SMs), none below 64
// tokens, where a warp's start and the extra states would cost more than they give.
// The backward's segments are multiples of its anchors' distance.
void gated_split(GatedProblem& p, bool backward) {
  const long long BH = 1LL * p.B * p.H;
  const long long warps = 148LL * (backward ? 12 : 16);
  long long n = BH > 0 ? warps / BH : 1;
  if (n < 1) n = 1;
  long long seg = (p.N + n - 1) / n;
  if (seg < 64) seg = 64;
  long long unit = kGateBlock;
  if (backward) unit = seg <= 64 ? 64 : seg <= 128 ? 128 : kGateAnchor;
  seg = (seg + unit - 1) / unit * unit;
  p.seg = static_cast<int>(seg);
  p.nseg = p.N > 0 ? static_cast<int>((p.N + seg - 1) / seg) : 1;
}

size_t gated_workspace_floats(const GatedProblem& p, bool backward) {
  const size_t BH = static_cast<size_t>(p.B) * p.H;
  const size_t states = BH * p.nseg * 1024, decays = BH * p.nseg;
  if (!backward) return p.nseg > 1 ? states + decays : 0;
  const int anchor = p.seg < kGateAnchor ? p.seg : kGateAnchor;
  const size_t nanchor = static_cast<size_t>((p.N + anchor - 1) / anchor) + 1;
  return 2 * states + BH * nanchor * 1024 + (BH * p.N + 3) / 4 * 4 + decays;
}

cudaError_t launch_gated(const GatedProblem& p, const void* Q, const void* K, const void* V,
                         const float* G, const float* S_in, float* S_out, void* O, float* ws,
                         cudaStream_t s) {
  using namespace gated;
  if (p.N <= kGateStepTokens) {
    const unsigned grid = static_cast<unsigned>((1LL * p.B * p.H + 3) / 4);
    if (p.io == LA_IO_BF16) {
      using T = __nv_bfloat16;
      step_kernel<T><<<grid, 128, 0, s>>>(p, static_cast<const T*>(Q), static_cast<const T*>(K),
                                          static_cast<const T*>(V), G, S_in, S_out,
                                          static_cast<T*>(O));
    } else {
      step_kernel<float><<<grid, 128, 0, s>>>(
          p, static_cast<const float*>(Q), static_cast<const float*>(K),
          static_cast<const float*>(V), G, S_in, S_out, static_cast<float*>(O));
    }
    return cudaGetLastError();
  }
  return p.io == LA_IO_BF16 ? forward<1>(p, Q, K, V, G, S_in, S_out, O, ws, s)
                            : forward<3>(p, Q, K, V, G, S_in, S_out, O, ws, s);
}

cudaError_t launch_gated_backward(const GatedProblem& p, const void* Q, const void* K,
                                  const void* V, const float* G, const float* S_in,
                                  const void* dO, const float* dS_out, void* dQ, void* dK,
                                  void* dV, float* dG, float* dS_in, float* ws, cudaStream_t s) {
  using namespace gated;
  return p.io == LA_IO_BF16
             ? backward<1>(p, Q, K, V, G, S_in, dO, dS_out, dQ, dK, dV, dG, dS_in, ws, s)
             : backward<3>(p, Q, K, V, G, S_in, dO, dS_out, dQ, dK, dV, dG, dS_in, ws, s);
}

}  // namespace la
