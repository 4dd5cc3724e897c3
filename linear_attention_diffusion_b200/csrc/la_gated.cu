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
// once more), a second combines them in order, and the segments then run at once. Where four
// segments a row are enough, one CTA takes a row and does all three in one launch.
//
// What bounds it, at 16384 tokens of 70 heads in bf16 (294 MB that it cannot do without,
// 46 us; 109 us a call with the last state, 107 without): the first pass reads 147 MB in 42 us
// (34 without the last state, see segment_pass), of which a copy of its pattern takes 30; the
// walk moves 294 MB in 68 us, the pattern alone 57. Neither the tensor cores (50 products a
// block of the walk, 26 us), nor the schedulers (390 instructions a block, 23 us) nor HBM is full:
// with 8 to 12 warps an SM, as many as the registers allow, products and the arithmetic
// between them overlap only in part. More warps with fewer registers spill, and blocks of 16
// instead of two at a time trade registers for instructions: both measured the same or slower.
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
// has left its S: rounding errors of the sum do not grow with the length. At the size above
// the four launches take 76, 6, 98 and 143 us by themselves; the walk backwards issues 114 products
// and 760 instructions a block, together 108 us if nothing overlapped.
#include "la_gated.cuh"
#include "la_sm100.cuh"

namespace la {
namespace gated {
namespace {

// Warps of a CTA: neighbouring heads of one segment. Float32 warps need 22 to 29 KB of shared
// memory each; pairs of them pack the SM better than fours.
template <int NP>
constexpr int kWarps = NP == 1 ? 4 : 2;

template <bool k>
struct Const {
  static constexpr bool value = k;
};
// The copies of a step's code. kStops: there may be stops, and with them something to take out;
// kLow: sums of gates carry what their rounding left; kRagged: rows past the end are minded.
template <bool kStops_, bool kLow_, bool kRagged_>
struct Mode {
  static constexpr bool kStops = kStops_, kLow = kLow_, kRagged = kRagged_;
};
// A step's decays: formed here for float32, and where a gate may have been taken out, else known.
template <int NP, int NB, bool kStops, typename Known>
__device__ __forceinline__ Decay<NP, NB> decays(const Known& known, float gate, uint32_t stops,
                                                int lane) {
  if constexpr (NP == 1) {
    if (kStops && stops != 0) return Decay<NP, NB>(gate, stops, lane);
    return known;
  } else {
    return Decay<NP, NB>(gate, stops, lane);
  }
}
// Two copies each: bf16 one without any of the three and one with all; float32 one for steps
// with stops and one for the others, told apart by a vote, which the compiler knows to be the
// same for the whole warp (3 x 2003 tokens of 36 heads: 68 us; by the stops' bits, and with
// their masks in the common copy too, 75 us).
template <int NP, int NB, typename Step>
__device__ __forceinline__ void run_step(float gate, bool ragged, int lane, const Step& step) {
  if constexpr (NP == 1) {
    const uint32_t stops = Decay<NP, NB>::find_stops(gate);
    const Decay<NP, NB> d(gate, stops, lane);
    if (d.hard || ragged)
      step(Mode<true, true, true>(), d, stops);
    else
      step(Mode<false, false, false>(), d, 0u);
  } else {
    if (__any_sync(0xffffffffu, Decay<NP, NB>::is_stop(gate)))
      step(Mode<true, true, true>(), 0, Decay<NP, NB>::find_stops(gate));
    else
      step(Mode<false, true, true>(), 0, 0u);
  }
}

struct Walk {
  const void *q, *k, *v, *w;  // operands; w: one more tile (see each kernel)
  const float* G;
  void *o, *o2;
  const float* init;     // external state at the walk's start, [B*H][32*32], or null
  float* final_;         // external state at the walk's end, or null
  const float* prefix;   // state at the start of each segment (nseg > 1), [B*H][nseg][1024]
  float* anchors;        // backward: S every `anchor` tokens of a segment and at the row's
                         // end, [B*H][nseg * per_seg + 1][1024]
  float* rows;           // backward: q . dq of every token, [B*H][N]
  float* dG;
  int anchor, per_seg;   // tokens between anchors; anchors of a segment
  GatedProblem p;
};

// A warp's place: head bh, tokens [n_begin, n_end), walked in `iters` steps of 16 NB.
template <int NB>
struct Place {
  int bh, seg, n_begin, n_end, iters;
  size_t base, gbase;  // of the head's first token, in heads' rows and in G
  __device__ __forceinline__ Place(const GatedProblem& p, long long unit) {
    const int BH = p.B * p.H;
    seg = static_cast<int>(unit / BH);
    bh = static_cast<int>(unit % BH);
    n_begin = seg * p.seg;
    n_end = min(p.N, n_begin + p.seg);
    iters = (n_end - n_begin + NB * kGateBlock - 1) / (NB * kGateBlock);
    gbase = static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
    base = gbase * 32;
  }
};

// Two bf16 blocks a step share one split of the state and one update, and fill the 32 lanes
// with gates; float32 planes would not fit twice in shared memory beside enough warps.
template <int NP>
constexpr int kBlocks = NP == 1 ? 2 : 1;
// Parts of what the kernels compute: two for a bf16 output, three for what ends in float32
// (the gate's gradient is a difference of row sums) and for float32 tensors.
constexpr __host__ __device__ int parts(int NP, bool precise) { return NP == 1 && !precise ? 2 : 3; }

// Products of one block row (16 tokens) with the tiles of its step, decayed and summed onto
// `acc`. kLater: the row's tokens are the later ones of each pair (forward), else the earlier
// ones (backward). rowf: the row block's operand; colt / deept: shared-memory tiles whose
// tokens are the columns, and the depth of the second product.
template <int NP, int NB, int NC, bool kLater, bool kStops, bool kLow>
__device__ __forceinline__ void block_row(float (&acc)[4][4], int b, const Frag<NP>& rowf,
                                          uint32_t colt, uint32_t deept, int plane,
                                          const LaneOff& off, const Decay<NP, NB>& d, float head,
                                          float tail, float scale, int lane) {
#pragma unroll
  for (int o = 0; o < NB; ++o) {  // the other block
    if (kLater ? o > b : o < b) continue;
    float w[2][4];
    {
      Frag<NP> c;
      c.cols(colt + o * kPlane, plane, off);
      token_product(w, rowf, c);
    }
    float l[2][4];
    if (o == b) {
      d.template within<kLater, kStops, kLow>(b, lane, l);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x) l[h][x] *= scale;
    } else {
      float r[2], c[4];
      Decay<NP, NB>::spread_rows((kLater ? head : tail) * scale, b, lane, r);
      Decay<NP, NB>::spread(kLater ? tail : head, o, lane, c);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x) l[h][x] = r[h] * c[x];
    }
    decay_by<kStops>(w, l);
    Frag<NP> v;
    v.deep(deept + o * kPlane, plane, off);
    if (o == b)
      weigh<NP, NC, kLater ? 2 : 1>(acc, w, v);
    else
      weigh<NP, NC, -1>(acc, w, v);
  }
}

// One segment forwards. kBack = false: the forward itself, state rows = v's
// dimensions. kBack = true: dq from (q, k, v) = (dO, V, K) with w = Q; it also
// writes q . dq of every token and S at the anchors.
// kExact: the state's own update keeps 24 bits, for a state that goes out in float32 or stands
// behind a float32 gradient; else 17, as many as a bf16 output can show.
// `smem`: the warp's shared memory; start(S) sets the state at the segment's start, once the
// first copies are on their way; S is left as it is at the segment's end.
template <int NP, bool kBack, bool kExact, int kStages, typename Start>
__device__ __forceinline__ void walk_pass(const Walk& a, const Place<kBlocks<NP>>& at, uint32_t smem,
                                          int lane, State& S, const Start& start) {
  using T = typename Io<NP>::T;
  constexpr int NB = kBlocks<NP>, NT = kBack ? 4 : 3, NC = parts(NP, kBack);
  constexpr int kStep = NB * kGateBlock;
  using M = Smem<NP, NB, NT, kStages, 3>;
  const GatedProblem& p = a.p;
  const T* heads[NT];
  heads[0] = static_cast<const T*>(a.q) + at.base;
  heads[1] = static_cast<const T*>(a.k) + at.base;
  heads[2] = static_cast<const T*>(a.v) + at.base;
  if (kBack) heads[NT - 1] = static_cast<const T*>(a.w) + at.base;
  const uint32_t planes = smem + kStages * M::kStage;
  Ring<NP, NB, NT, kStages, 3, false, false> ring(smem, heads, a.G + at.gbase, p.H, nullptr,
                                                  at.n_begin, at.n_end, at.iters, lane);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ring.issue(lane);
  Out<NP> out(a.o, at.base, p.H, at.n_begin, lane);
  start(S);
  float* anchors = nullptr;
  if (kBack)
    anchors = a.anchors + (static_cast<size_t>(at.bh) * (p.nseg * a.per_seg + 1) +
                           static_cast<size_t>(at.seg) * a.per_seg) * 1024;
  const LaneOff off(lane);
  const int r0 = lane >> 2;

  int n0 = at.n_begin;
  for (int it = 0; it < at.iters; ++it, n0 += kStep) {
    const uint32_t st = ring.next(lane);
    float gate = lds(st + NT * M::kTile + lane * 4);
    if (kBack && (n0 - at.n_begin) % a.anchor == 0)
      S.store(anchors + static_cast<size_t>((n0 - at.n_begin) / a.anchor) * 1024, lane);
    uint32_t tile[3];
    const int plane = NP == 1 ? 0 : M::kPart;
#pragma unroll
    for (int t = 0; t < 3; ++t) tile[t] = NP == 1 ? st + t * M::kTile : planes + t * 3 * M::kPart;
    const int left = at.n_end - n0;
    auto step = [&](auto mode, auto known, uint32_t stops) {
      constexpr bool kStops = decltype(mode)::kStops, kLow = decltype(mode)::kLow;
      constexpr bool kRagged = decltype(mode)::kRagged;
      uint32_t bad = 0;
      if (kStops && stops != 0)
        bad = take_out_gates<NB>(gate) | take_out<NP, NB>(st + M::kTile, st + 2 * M::kTile, lane);
      if (NP > 1) {
#pragma unroll
        for (int t = 0; t < 3; ++t) split_tile<NB>(st + t * M::kTile, tile[t], lane);
        __syncwarp();
      }
      const Decay<NP, NB> d = decays<NP, NB, kStops>(known, gate, stops, lane);
      const float head = d.template head<kStops, kLow>(lane), tail = d.template tail<kStops, kLow>(lane);
      const float whole = d.template whole<kStops, kLow>(lane);
      // decays of the step's blocks, from its start and to its end
      const float w0 = __shfl_sync(0xffffffffu, whole, 0);
      const float w1 = NB == 1 ? 1.0f : __shfl_sync(0xffffffffu, whole, 16);
      const float from_start = (NB == 2 && lane >= 16 ? head * w0 : head) * p.scale;
      const float to_end = NB == 2 && lane < 16 ? tail * w1 : tail;
      float acc[NB][4][4];
      {
        Frag<NP> q[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) q[b].rows(tile[0] + b * kPlane, plane, off);
        S.template apply<NP, NC, NB>(acc, q);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float r[2];
          Decay<NP, NB>::spread_rows(from_start, b, lane, r);
          scale_row<kStops>(acc[b], 0, r[0]);
          scale_row<kStops>(acc[b], 1, r[1]);
          block_row<NP, NB, NC, true, kStops, kLow>(acc[b], b, q[b], tile[1], tile[2], plane, off,
                                                    d, head, tail, p.scale, lane);
          if (kStops && bad != 0)
            spoil_rows<NP, NB>(acc[b], b, spoiled_from(bad, stops, lane & (kStep - 1)), lane);
        }
      }
      {
        float wt[NB][4];
        Frag<NP> v[NB], k[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          Decay<NP, NB>::spread(to_end, b, lane, wt[b]);
          v[b].deep(tile[2] + b * kPlane, plane, off);
          k[b].deep(tile[1] + b * kPlane, plane, off);
        }
        S.template update<NP, NB, kExact ? 3 : 2, kStops>(w0 * w1, v, k, wt);
        if (kStops && bad != 0 && spoiled_from(bad, stops, kStep - 1) != 0.0f) S.spoil();
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (kBack) {
          float dots[2];
          const uint32_t w = st + 3 * M::kTile + b * M::kTile / NB;
          if constexpr (NP == 1) {
            Frag<1> x;
            x.rows(w, 0, off);
            row_dots(acc[b], x, dots);
          } else {
            row_dots_f32(acc[b], w, lane, dots);
          }
          if ((lane & 3) == 0) {
            float* r = a.rows + static_cast<size_t>(at.bh) * p.N + n0 + b * kGateBlock + r0;
            if (!kRagged || r0 + b * kGateBlock < left) r[0] = dots[0];
            if (!kRagged || r0 + b * kGateBlock + 8 < left) r[8] = dots[1];
          }
        }
      }
      __syncwarp();  // every lane is done with the first tile: the output passes through it
#pragma unroll
      for (int b = 0; b < NB; ++b) Out<NP>::put(acc[b], st + b * M::kTile / NB, off, lane);
      __syncwarp();
      out.template flush<kStep, !kRagged>(st, left, kStep, lane);
    };
    run_step<NP, NB>(gate, left < kStep, lane, step);
  }
  cp_wait<0>();
  if (kBack && at.seg == p.nseg - 1)  // the state after the last token: the anchor of the row's end
    S.store(anchors + static_cast<size_t>(a.per_seg) * 1024, lane);
}

template <int NP, bool kBack, bool kExact, int kStages>
__global__ void __launch_bounds__(kWarps<NP> * 32, kBack ? (NP == 1 ? 2 : 4) : NP == 1 ? 3 : 5)
walk_kernel(const Walk a) {
  extern __shared__ __align__(128) uint8_t smem_all[];
  const GatedProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps<NP> + warp;
  if (unit >= static_cast<long long>(p.B) * p.H * p.nseg) return;
  const Place<kBlocks<NP>> at(p, unit);
  State S;
  walk_pass<NP, kBack, kExact, kStages>(
      a, at, smem_addr(smem_all) + warp * Smem<NP, kBlocks<NP>, kBack ? 4 : 3, kStages, 3>::kWarp,
      lane, S, [&](State& s) {
        sm100::pdl_trigger();
        sm100::pdl_wait();  // the inputs were there before; the states come from the kernel before
        if (p.nseg > 1)
          s.load(a.prefix + (static_cast<size_t>(at.bh) * p.nseg + at.seg) * 1024, lane);
        else if (a.init != nullptr)
          s.template load_outer<!kBack>(a.init + static_cast<size_t>(at.bh) * 1024, lane);
        else
          s.zero();
      });
  if (!kBack && a.final_ != nullptr && at.seg == p.nseg - 1)
    S.template store_outer<true>(a.final_ + static_cast<size_t>(at.bh) * 1024, lane);
}

// One segment backwards: dk and dv (o and o2), the log gates' gradient, and with
// a.final_ the gradient of the state before the first token. q, k, v as in the
// forward, w = dO. The carried state X (rows: k's dimensions, columns: v's) is the
// gradient that reaches the state at a step's end from later tokens.
template <int NP, int kStages>
__global__ void __launch_bounds__(kWarps<NP> * 32, NP == 1 ? 2 : 3)
walk_back_kernel(const Walk a) {
  using T = typename Io<NP>::T;
  constexpr int NB = kBlocks<NP>, NT = 4, NK = parts(NP, true), NV = parts(NP, false);
  constexpr int kStep = NB * kGateBlock;
  using M = Smem<NP, NB, NT, kStages>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const GatedProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps<NP> + warp;
  if (unit >= static_cast<long long>(p.B) * p.H * p.nseg) return;
  const Place<NB> at(p, unit);
  const T* const heads[NT] = {static_cast<const T*>(a.k) + at.base, static_cast<const T*>(a.v) + at.base,
                              static_cast<const T*>(a.q) + at.base, static_cast<const T*>(a.w) + at.base};
  const uint32_t smem = smem_addr(smem_all) + warp * M::kWarp;
  const uint32_t planes = smem + kStages * M::kStage;
  sm100::pdl_wait();  // rows, anchors and states come from the kernels before
  int n0 = at.n_begin + (at.iters - 1) * kStep;  // the last step comes first
  Ring<NP, NB, NT, kStages, NT, true, true> ring(smem, heads, a.G + at.gbase, p.H,
                                                 a.rows + static_cast<size_t>(at.bh) * p.N, n0,
                                                 at.n_end, at.iters, lane);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ring.issue(lane);
  Out<NP> out_k(a.o, at.base, p.H, n0, lane), out_v(a.o2, at.base, p.H, n0, lane);

  State X;
  if (p.nseg > 1)
    X.load(a.prefix + (static_cast<size_t>(at.bh) * p.nseg + at.seg) * 1024, lane);
  else if (a.init != nullptr)
    X.template load_outer<false>(a.init + static_cast<size_t>(at.bh) * 1024, lane);
  else
    X.zero();
  // dg just past the segment: <X, S> there, S the first anchor of the next one (or the row's
  // end). Then `carry` is dg of the token after the step at hand.
  const float* anchors = a.anchors + (static_cast<size_t>(at.bh) * (p.nseg * a.per_seg + 1) +
                                      static_cast<size_t>(at.seg) * a.per_seg) * 1024;
  float carry;
  {
    State S;
    S.load(anchors + static_cast<size_t>(a.per_seg) * 1024, lane);
    carry = X.dot(S);
  }
  const LaneOff off(lane);

  for (int it = 0; it < at.iters; ++it, n0 -= kStep) {
    const uint32_t st = ring.next(lane);
    float gate = lds(st + NT * M::kTile + lane * 4);
    const float rdot = lds(st + NT * M::kTile + 128 + lane * 4);
    uint32_t tile[NT];
    const int plane = NP == 1 ? 0 : M::kPart;
#pragma unroll
    for (int t = 0; t < NT; ++t) tile[t] = NP == 1 ? st + t * M::kTile : planes + t * 3 * M::kPart;
    const int left = at.n_end - n0;
    auto step = [&](auto mode, auto known, uint32_t stops) {
      constexpr bool kStops = decltype(mode)::kStops, kLow = decltype(mode)::kLow;
      constexpr bool kRagged = decltype(mode)::kRagged;
      uint32_t bad = 0;
      if (kStops && stops != 0)
        bad = take_out_gates<NB>(gate) | take_out<NP, NB>(st + 2 * M::kTile, st + 3 * M::kTile, lane);
      if (NP > 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) split_tile<NB>(st + t * M::kTile, tile[t], lane);
        __syncwarp();
      }
      const Decay<NP, NB> d = decays<NP, NB, kStops>(known, gate, stops, lane);
      const float head = d.template head<kStops, kLow>(lane), tail = d.template tail<kStops, kLow>(lane);
      const float whole = d.template whole<kStops, kLow>(lane);
      const float w0 = __shfl_sync(0xffffffffu, whole, 0);
      const float w1 = NB == 1 ? 1.0f : __shfl_sync(0xffffffffu, whole, 16);
      const float to_end = NB == 2 && lane < 16 ? tail * w1 : tail;
      const float from_start = (NB == 2 && lane >= 16 ? head * w0 : head) * p.scale;
      float kdots[NB][2];
      // dk (which = 0): rows v, columns dO, summed over q; dv: rows k, columns q, summed over
      // dO. dk passes through v's tile, which is done with, dv then through k's.
      auto side = [&](auto second) {
        constexpr int which = decltype(second)::value;
        float acc[NB][4][4];
        Frag<NP> x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) x[b].rows(tile[1 - which] + b * kPlane, plane, off);
        if (which == 0)
          X.template apply<NP, NK, NB>(acc, x);
        else
          X.template apply_turned<NP, NV, NB>(acc, x);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float r[2];
          Decay<NP, NB>::spread_rows(to_end, b, lane, r);
          scale_row<kStops>(acc[b], 0, r[0]);
          scale_row<kStops>(acc[b], 1, r[1]);
          block_row<NP, NB, which == 0 ? NK : NV, false, kStops, kLow>(
              acc[b], b, x[b], tile[3 - which], tile[2 + which], plane, off, d, head, tail, p.scale,
              lane);
          if (kStops && bad != 0)
            spoil_rows<NP, NB>(acc[b], b, spoiled_to(bad, stops, lane & (kStep - 1)), lane);
        }
        if (which == 0) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if constexpr (NP == 1) {
              Frag<1> k;
              k.rows(tile[0] + b * kPlane, 0, off);
              row_dots(acc[b], k, kdots[b]);
            } else {
              row_dots_f32(acc[b], st + b * M::kTile / NB, lane, kdots[b]);
            }
          }
        }
        const uint32_t pass = st + (1 - which) * M::kTile;
        __syncwarp();
#pragma unroll
        for (int b = 0; b < NB; ++b) Out<NP>::put(acc[b], pass + b * M::kTile / NB, off, lane);
        __syncwarp();
        (which == 0 ? out_k : out_v).template flush<kStep, !kRagged>(pass, left, -kStep, lane);
      };
      side(Const<false>());
      side(Const<true>());
      {
        float wt[NB][4];
        Frag<NP> q[NB], o[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          Decay<NP, NB>::spread(from_start, b, lane, wt[b]);
          q[b].deep(tile[2] + b * kPlane, plane, off);
          o[b].deep(tile[3] + b * kPlane, plane, off);
        }
        X.template update<NP, NB, 3, kStops>(w0 * w1, q, o, wt);
        if (kStops && bad != 0 && spoils_start(bad, stops)) X.spoil();
      }
      // dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t, summed from the step's end, or from the next
      // stop, which passes no gradient
      const int i = lane & (kStep - 1);
      float own = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = __shfl_sync(0xffffffffu, kdots[b][h], (i & 7) * 4);
          if ((i >> 3) == 2 * b + h) own = y;
        }
      float x = rdot - own;
      const uint32_t after = kStops ? stops & ~((2u << i) - 1u) : 0u;
      const int end = after != 0 ? __ffs(after) - 1 : kStep;
#pragma unroll
      for (int s = 1; s < kStep; s <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, x, s, kStep);
        if (i + s < end) x += y;
      }
      float dg = after != 0 ? x : carry + x;
      if (kStops && ((stops >> i) & 1u)) dg = 0.0f;
      if (lane < kStep && (!kRagged || i < left))
        a.dG[at.gbase + static_cast<size_t>(n0 + i) * p.H] = dg;
      carry = __shfl_sync(0xffffffffu, dg, 0);
    };
    run_step<NP, NB>(gate, left < kStep, lane, step);
    if ((n0 - at.n_begin) % a.anchor == 0 && it + 1 < at.iters) {
      State S;
      S.load(anchors + static_cast<size_t>((n0 - at.n_begin) / a.anchor) * 1024, lane);
      carry = X.dot(S);
    }
  }
  cp_wait<0>();
  if (at.seg == 0 && a.final_ != nullptr)
    X.template store_outer<false>(a.final_ + static_cast<size_t>(at.bh) * 1024, lane);
}

// Every segment's own state from zero and its whole decay. Forward: S only, rows =
// v's dimensions. Backward: S and X = sum_i (decay from the segment's start to i)
// scale q_i^T dO_i, rows = k's (q's) dimensions. Segment s's S goes to slot s + 1 of
// `states` (it becomes the state at the start of s + 1; the last one is the end of the row),
// its X to slot s - 1 of `grads`. It walks a segment from its end: what it reads last, the
// segments' first tokens, the walk reads first, while it is still in L2. Once the decay to
// the segment's end has become 0, no earlier token has a part in S.
// kExact as in the walk: 16384 tokens of 70 heads take 42 us, with 17 bits (a forward whose last
// state nobody asks for) 34 us.
template <int NP, bool kBack, bool kExact, int kStages>
__device__ __forceinline__ void segment_pass(const GatedProblem& p, const Place<kBlocks<NP>>& at,
                                             const void* qv, const void* kv, const void* vv,
                                             const void* dov, const float* Gv, uint32_t smem,
                                             int lane, State& S, State& X, float& total) {
  using T = typename Io<NP>::T;
  constexpr int NB = kBlocks<NP>, NT = kBack ? 4 : 2;
  constexpr int kStep = NB * kGateBlock;
  using M = Smem<NP, NB, NT, kStages>;
  const T* heads[NT];
  heads[0] = static_cast<const T*>(kBack ? kv : vv) + at.base;
  heads[1] = static_cast<const T*>(kBack ? vv : kv) + at.base;
  if (kBack) {
    heads[NT - 2] = static_cast<const T*>(qv) + at.base;
    heads[NT - 1] = static_cast<const T*>(dov) + at.base;
  }
  const uint32_t planes = smem + kStages * M::kStage;
  Ring<NP, NB, NT, kStages, NT, true, false> ring(smem, heads, Gv + at.gbase, p.H, nullptr,
                                                  at.n_begin + (at.iters - 1) * kStep, at.n_end,
                                                  at.iters, lane);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ring.issue(lane);
  S.zero();
  if (kBack) X.zero();
  total = 1.0f;
  const LaneOff off(lane);
  for (int it = 0; it < at.iters; ++it) {
    const uint32_t st = ring.next(lane);
    float gate = lds(st + NT * M::kTile + lane * 4);
    uint32_t tile[NT];
    const int plane = NP == 1 ? 0 : M::kPart;
#pragma unroll
    for (int t = 0; t < NT; ++t) tile[t] = NP == 1 ? st + t * M::kTile : planes + t * 3 * M::kPart;
    auto step = [&](auto mode, auto known, uint32_t stops) {
      constexpr bool kStops = decltype(mode)::kStops, kLow = decltype(mode)::kLow;
      uint32_t bad = 0, bad_x = 0;
      if (kStops && stops != 0) {
        const uint32_t gates = take_out_gates<NB>(gate);
        bad = gates | take_out<NP, NB>(st, st + M::kTile, lane);
        if (kBack)
          bad_x = gates | take_out<NP, NB>(st + (NT - 2) * M::kTile, st + (NT - 1) * M::kTile, lane);
      }
      if (NP > 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) split_tile<NB>(st + t * M::kTile, tile[t], lane);
        __syncwarp();
      }
      const Decay<NP, NB> d = decays<NP, NB, kStops>(known, gate, stops, lane);
      const float whole = d.template whole<kStops, kLow>(lane);
      const float w0 = __shfl_sync(0xffffffffu, whole, 0);
      const float w1 = NB == 1 ? 1.0f : __shfl_sync(0xffffffffu, whole, 16);
      float w[NB][4];
      if (!kBack || total != 0.0f) {
        const float tail = d.template tail<kStops, kLow>(lane);
        const float to_end = (NB == 2 && lane < 16 ? tail * w1 : tail) * total;
        Frag<NP> x[NB], y[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          Decay<NP, NB>::spread(to_end, b, lane, w[b]);
          x[b].deep(tile[0] + b * kPlane, plane, off);
          y[b].deep(tile[1] + b * kPlane, plane, off);
        }
        S.template update<NP, NB, kExact ? 3 : 2, false>(1.0f, x, y, w);
        if (kStops && bad != 0 && spoiled_from(bad, stops, kStep - 1) != 0.0f) S.spoil();
      }
      if (kBack) {
        const float head = d.template head<kStops, kLow>(lane);
        const float from_start = (NB == 2 && lane >= 16 ? head * w0 : head) * p.scale;
        Frag<NP> x[NB], y[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          Decay<NP, NB>::spread(from_start, b, lane, w[b]);
          x[b].deep(tile[NT - 2] + b * kPlane, plane, off);
          y[b].deep(tile[NT - 1] + b * kPlane, plane, off);
        }
        X.template update<NP, NB, 3, kStops>(w0 * w1, x, y, w);
        if (kStops && bad_x != 0 && spoils_start(bad_x, stops)) X.spoil();
      }
      // a stop on either side of a gate that is no number leaves 0, not NaN
      total = total == 0.0f || w0 * w1 == 0.0f ? 0.0f : total * (w0 * w1);
    };
    run_step<NP, NB>(gate, false, lane, step);
    if (!kBack && total == 0.0f) break;
  }
  cp_wait<0>();
  __syncwarp();  // the stages are free
}

template <int NP, bool kBack, bool kExact, int kStages>
__global__ void __launch_bounds__(kWarps<NP> * 32, kBack ? (NP == 1 ? 2 : 4) : NP == 1 ? 4 : 5)
segment_kernel(const GatedProblem p, int segs, const void* qv, const void* kv, const void* vv,
               const void* dov, const float* Gv, float* states, float* last_states, float* grads,
               float* decays) {
  extern __shared__ __align__(128) uint8_t smem_all[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps<NP> + warp;
  if (unit >= static_cast<long long>(p.B) * p.H * segs) return;
  const Place<kBlocks<NP>> at(p, unit);
  sm100::pdl_trigger();
  State S, X;
  float total;
  segment_pass<NP, kBack, kExact, kStages>(
      p, at, qv, kv, vv, dov, Gv,
      smem_addr(smem_all) + warp * Smem<NP, kBlocks<NP>, kBack ? 4 : 2, kStages>::kWarp, lane, S, X,
      total);
  const size_t slots = static_cast<size_t>(at.bh) * p.nseg;
  if (at.seg + 1 < p.nseg)
    S.store(states + (slots + at.seg + 1) * 1024, lane);
  else if (!kBack)
    S.store(last_states + static_cast<size_t>(at.bh) * 1024, lane);
  if (kBack && at.seg > 0) X.store(grads + (slots + at.seg - 1) * 1024, lane);
  if (lane == 0) decays[slots + at.seg] = total;
}

// A whole row in one CTA: its warps take the segments of one head, leave the segments' own
// states in shared memory, and each adds up those before its own. K and V come from L2 the
// second time, and nothing of a second or third launch is left. 8 x 509 tokens of 36 heads in
// bf16 take 19.3 us in a graph, three launches 23.9; two warps instead of four took 1.28 times as
// long, six 1.03 times.
constexpr int kRowWarps = 4;
template <int NP>
struct RowSmem {
  static constexpr int kStages = 2;
  using M = Smem<NP, kBlocks<NP>, 3, kStages, 3>;  // the walk's; the first pass needs less
  static_assert(Smem<NP, kBlocks<NP>, 2, kStages>::kWarp <= M::kWarp, "the first pass's ring fits");
  static constexpr int kState = 4096 + 16;  // and the segment's decay
  static constexpr int kWarp = M::kWarp + kState;
};

template <int NP>
__global__ void __launch_bounds__(kRowWarps * 32, NP == 1 ? 3 : 2) row_kernel(const Walk a) {
  using R = RowSmem<NP>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const GatedProblem& p = a.p;
  const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
  const long long BH = static_cast<long long>(p.B) * p.H;
  const Place<kBlocks<NP>> at(p, seg * BH + blockIdx.x);
  const uint32_t smem = smem_addr(smem_all) + seg * R::M::kWarp;
  const uint32_t states = smem_addr(smem_all) + p.nseg * R::M::kWarp;  // [nseg] states, then decays
  const uint32_t decays = states + p.nseg * 4096;
  const float* init = a.init != nullptr ? a.init + static_cast<size_t>(at.bh) * 1024 : nullptr;
  State S, first;
  float total;
  segment_pass<NP, false, true, R::kStages>(p, at, nullptr, a.k, a.v, nullptr, a.G, smem, lane, S, first,
                                      total);
  first.zero();
  if (seg == 0 && init != nullptr) {  // read by this warp alone, before the last one writes
    first.template load_outer<true>(init, lane);
    if (total != 0.0f) S.add_scaled(first, total);
  }
  S.put(states + seg * 4096, lane);
  if (lane == 0) sts(decays + seg * 4, __float_as_uint(total));
  walk_pass<NP, false, NP == 3, R::kStages>(a, at, smem, lane, S, [&](State& s) {
    __syncthreads();
    s = first;  // of segment 0; the others' starts from zero
    for (int i = 0; i < seg; ++i) s.follow(states + i * 4096, lds(decays + i * 4), lane);
    if (a.final_ != nullptr && seg == p.nseg - 1) {
      State end = s;
      end.follow(states + seg * 4096, seg == 0 ? 0.0f : total, lane);
      end.template store_outer<true>(a.final_ + static_cast<size_t>(at.bh) * 1024, lane);
    }
  });
}

// Segments in order: slot s becomes the state at segment s's start (forwards), or the
// gradient at its end (backwards). One thread per four numbers of a head's state, 64 threads
// a CTA so that few heads still spread over the SMs (5 us for 25 segments of 70 heads, the
// latency of three rounds of loads); blockIdx.z = 0: states, 1: gradients.
// With s_final the states go on over the last segment, whose own state is in `tail_state`.
template <bool kTransposed>
__global__ void __launch_bounds__(64)
combine_kernel(int nseg, const float* decays, float* states, const float* s_init, float* grads,
               const float* x_init, const float* tail_state, float* s_final) {
  const int bh = blockIdx.x, f = blockIdx.y * 64 + threadIdx.x;
  const bool back = blockIdx.z == 1;
  sm100::pdl_trigger();
  sm100::pdl_wait();
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
  if (s_final != nullptr) {
    const float m = dec[nseg - 1];
    const float4 t = __ldcg(reinterpret_cast<const float4*>(tail_state) +
                            static_cast<size_t>(bh) * 256 + f);
    if (m == 0.0f) run = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int mt = f >> 7, nt = (f >> 5) & 3, lane = f & 31;
    s_final += static_cast<size_t>(bh) * 1024;
    s_final[State::outer<kTransposed>(mt, nt, 0, lane)] = fmaf(m, run.x, t.x);
    s_final[State::outer<kTransposed>(mt, nt, 1, lane)] = fmaf(m, run.y, t.y);
    s_final[State::outer<kTransposed>(mt, nt, 2, lane)] = fmaf(m, run.z, t.z);
    s_final[State::outer<kTransposed>(mt, nt, 3, lane)] = fmaf(m, run.w, t.w);
  }
}

// A few tokens, one after another: one warp per head, the state in registers, eight
// rows of four columns per lane. Bound by the state's 8 KB read and written.
// 64 one-token requests of 70 heads: 8.6 us for 37 MB; eight CTAs an SM, one wave.
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
__global__ void __launch_bounds__(128, 8)
step_kernel(const GatedProblem p, const T* Q, const T* K, const T* V, const float* G,
            const float* S_in, float* S_out, T* O) {
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.B) * p.H) return;
  const int bh = static_cast<int>(unit);
  const size_t gbase = static_cast<size_t>(bh / p.H) * p.N * p.H + bh % p.H;
  const size_t base = gbase * 32;
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
    const float g = G[gbase + static_cast<size_t>(n) * p.H], g2 = g * kLog2e;
    const float a = g2 < kStop ? 0.0f
                               : Decay<1, 1>::template power<true>(g2, fmaf(g, kLog2e, -g2) + g * kLog2eRest);
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

// Shared memory of a launch, and the most that any call of the kernel takes: its limit is set to
// that, never to the call's own, which another thread's call could undo before the launch.
struct SmemBytes {
  int bytes, most;
  SmemBytes(int fixed) : bytes(fixed), most(fixed) {}
  SmemBytes(int b, int m) : bytes(b), most(m) {}
};

// Launch a kernel with its shared memory. chained: it may start while the kernel before it on
// the stream, one of this call's own, still runs, and waits for it itself (pdl_wait).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, SmemBytes smem, bool chained,
                   cudaStream_t s, Args... args) {
  if (smem.most > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem.most);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem.bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <int NP>
dim3 grid_of(long long units) {
  return dim3(static_cast<unsigned>((units + kWarps<NP> - 1) / kWarps<NP>));
}

template <int NP>
cudaError_t forward(const GatedProblem& p, const void* Q, const void* K, const void* V,
                    const float* G, const float* S_in, float* S_out, void* O, float* ws,
                    cudaStream_t s) {
  constexpr int NB = kBlocks<NP>, kSegStages = 3, kStages = NP == 1 ? 3 : 2;
  const long long BH = 1LL * p.B * p.H;
  cudaError_t e;
  Walk a = {};
  a.q = Q;
  a.k = K;
  a.v = V;
  a.G = G;
  a.o = O;
  a.init = S_in;
  a.p = p;
  if (p.whole_row) {
    a.final_ = S_out;
    return launch(row_kernel<NP>, dim3(static_cast<unsigned>(BH)), p.nseg * 32,
                  {p.nseg * RowSmem<NP>::kWarp, kRowWarps * RowSmem<NP>::kWarp}, false, s, a);
  }
  float* states = ws;
  if (p.nseg > 1) {
    float* last_states = states + BH * p.nseg * 1024;
    float* decays = last_states + BH * 1024;
    const int segs = S_out != nullptr ? p.nseg : p.nseg - 1;
    auto first_pass = segment_kernel<NP, false, true, kSegStages>;
    if constexpr (NP == 1) {
      if (S_out == nullptr) first_pass = segment_kernel<NP, false, false, kSegStages>;
    }
    e = launch(first_pass, grid_of<NP>(BH * segs), kWarps<NP> * 32,
               kWarps<NP> * Smem<NP, NB, 2, kSegStages>::kWarp, false, s, p, segs, Q, K, V, nullptr,
               G, states, last_states, nullptr, decays);
    if (e != cudaSuccess) return e;
    e = launch(combine_kernel<true>, dim3(static_cast<unsigned>(BH), 4, 1), 64, 0, true, s, p.nseg,
               decays, states, S_in, nullptr, nullptr, last_states, S_out);
    if (e != cudaSuccess) return e;
  }
  a.final_ = p.nseg > 1 ? nullptr : S_out;
  a.prefix = states;
  auto walk = walk_kernel<NP, false, true, kStages>;
  if constexpr (NP == 1) {
    if (a.final_ == nullptr) walk = walk_kernel<NP, false, false, kStages>;
  }
  return launch(walk, grid_of<NP>(BH * p.nseg), kWarps<NP> * 32,
                kWarps<NP> * Smem<NP, NB, 3, kStages, 3>::kWarp, p.nseg > 1, s, a);
}

// Anchors of a segment: at its start and every kGateAnchor tokens after it.
int gated_anchors(const GatedProblem& p) { return (p.seg + kGateAnchor - 1) / kGateAnchor; }

template <int NP>
cudaError_t backward(const GatedProblem& p, const void* Q, const void* K, const void* V,
                     const float* G, const float* S_in, const void* dO, const float* dS_out,
                     void* dQ, void* dK, void* dV, float* dG, float* dS_in, float* ws,
                     cudaStream_t s) {
  constexpr int NB = kBlocks<NP>, kStages = NP == 1 ? 3 : 2;
  const long long BH = 1LL * p.B * p.H;
  Walk a = {};
  a.anchor = kGateAnchor;
  a.per_seg = gated_anchors(p);
  float* states = ws;
  float* grads = states + BH * p.nseg * 1024;
  a.anchors = grads + BH * p.nseg * 1024;
  a.rows = a.anchors + BH * (1LL * p.nseg * a.per_seg + 1) * 1024;
  float* decays = a.rows + (BH * p.N + 3) / 4 * 4;
  const int threads = kWarps<NP> * 32, smem = kWarps<NP> * Smem<NP, NB, 4, kStages>::kWarp;
  const dim3 grid = grid_of<NP>(BH * p.nseg);
  cudaError_t e;
  if (p.nseg > 1) {
    e = launch(segment_kernel<NP, true, true, kStages>, grid, threads, smem, false, s, p, p.nseg, Q, K, V,
               dO, G, states, nullptr, grads, decays);
    if (e != cudaSuccess) return e;
    e = launch(combine_kernel<false>, dim3(static_cast<unsigned>(BH), 4, 2), 64, 0, true, s, p.nseg,
               decays, states, S_in, grads, dS_out, nullptr, nullptr);
    if (e != cudaSuccess) return e;
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
  e = launch(walk_kernel<NP, true, true, kStages>, grid, threads,
             kWarps<NP> * Smem<NP, NB, 4, kStages, 3>::kWarp, p.nseg > 1, s, a);
  if (e != cudaSuccess) return e;
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
  return launch(walk_back_kernel<NP, kStages>, grid, threads, smem, true, s, a);
}

}  // namespace
}  // namespace gated

// Segments of a row. Cutting costs a second reading of K and V (and Q and dO backwards) and
// two launches more, so heads that fill half the GPU by themselves are not cut. 2500 tokens of 900
// heads, bf16: 155 us whole, 197 cut in two (880 heads: 152 and 172, 1700 heads: 253 and 326),
// backwards 544 and 699; 1500 tokens of 760 heads, float32: 254 and 274, backwards 692 and 753.
// Otherwise:
//  - as many segments as give every warp's place on 148 SMs one, by registers (bf16: 168 a
//    thread forwards, 255 backwards) or shared memory (float32). 16384 tokens of 70 heads, bf16:
//    109 us, with twice the segments 118 us.
//  - float32 is bound by its many products, and its warps, more of them, level out better in
//    four waves: 289 us against 291 us there, 742 against 852 us backwards.
//  - no segment so short that its start and its state cost more than its work: 64 tokens
//    (1024 tokens of 36 heads: 11.8 us, with 32 tokens 13.1 us), 96 for much float32 work (1024
//    tokens of 140 heads: 46.6 us, with 64 tokens 49.2 us); where little is to be done at all, the
//    time is one warp's, and 32 tokens are best (256 tokens of 36 heads: 7.0 us, with 64 tokens
//    8.9 us), up to a number of segments whose combination would take longer (4000 tokens of 4
//    heads, float32 backwards: 39 us with 125 segments, 62 us with 32).
//
// Forwards, a CTA takes a whole row where its four warps are enough: short rows, or rows of
// so many heads that they would not be cut much finer. In one launch against three, bf16: 256
// tokens of 70 heads 6.8 and 7.9 us (512 tokens: 12.3 and 11.1), 1024 tokens of 140 heads 21.9
// and 23.5 us (2048: 39.5 and 37.1), 2000 tokens of 630 heads 140 and 145 us (4096 of 280: 128
// and 114). float32, whose warps are fewer: 1024 tokens of 280 heads 68 and 78 us (of 140: 47 and
// 46), 64 tokens 8.2 and 9.9 us; more heads than one wave of CTAs: 172 and 163 us (630 heads).
void gated_split(GatedProblem& p, bool backward) {
  const long long BH = 1LL * p.B * p.H, work = BH * p.N;
  const bool bf16 = p.io == LA_IO_BF16;
  const long long per_sm = bf16 ? (backward ? 8 : 12) : (backward ? 6 : 10);
  const bool little = work < (!bf16 ? 60000 : backward ? 40000 : 20000);
  const int most = !bf16 ? 128 : backward ? 64 : 32;
  long long n = BH > 0 ? 148 * per_sm / BH : 1;
  if (n < 1) n = 1;
  if (!bf16 && n > 1) n *= 4;
  if (little && n > most) n = most;
  long long seg = (p.N + n - 1) / n;
  const long long least = little ? 32 : !bf16 && work >= 96000 ? 96 : 64;
  if (seg < least) seg = least;
  seg = (seg + 31) / 32 * 32;
  p.seg = static_cast<int>(seg);
  p.nseg = p.N > 0 ? static_cast<int>((p.N + seg - 1) / seg) : 1;
  p.whole_row = !backward && n > 1 && p.N > 0 &&
                (bf16 ? p.N <= 256 || (BH >= 128 && p.N <= 1024) || (BH >= 256 && p.N <= 2048)
                      : BH <= 296 && (p.N <= 128 || (BH >= 200 && p.N <= 2048)));
  if (p.whole_row) {
    seg = ((p.N + gated::kRowWarps - 1) / gated::kRowWarps + 31) / 32 * 32;
    p.seg = static_cast<int>(seg);
    p.nseg = static_cast<int>((p.N + seg - 1) / seg);
  }
}

size_t gated_workspace_floats(const GatedProblem& p, bool backward) {
  const size_t BH = static_cast<size_t>(p.B) * p.H;
  const size_t states = BH * p.nseg * 1024, decays = BH * p.nseg;
  if (!backward) return p.nseg > 1 && !p.whole_row ? states + BH * 1024 + decays : 0;
  const size_t anchors = BH * (static_cast<size_t>(p.nseg) * gated::gated_anchors(p) + 1) * 1024;
  return 2 * states + anchors + (BH * p.N + 3) / 4 * 4 + decays;
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
