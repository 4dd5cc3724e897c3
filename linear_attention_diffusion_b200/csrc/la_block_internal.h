// Internal interface between the C-ABI layer of the block operators
// (la_block_api.cu) and their kernels: gated linear attention, rotary
// positions, the gated residual with the norms around it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "la.h"

namespace la {

// Gated linear attention (la_gated.cu, la_gated.cuh).
struct GatedProblem {
  int B, N, H;
  int io;       // 0 bf16, 1 float32
  float scale;  // applied to the queries
  int seg;      // tokens of one warp's segment, a multiple of 32
  int nseg;     // segments per (batch element, head)
  bool whole_row;  // forwards: a CTA takes all segments of a head in one launch
};
constexpr int kGateBlock = 16;      // tokens of one tensor-core block
constexpr int kGateStepTokens = 4;  // up to here tokens are walked one by one (4 tokens of 70 heads:
                                    // 3.8 us, as a block 4.1 us; 8 tokens: 6.0 us)
constexpr int kGateAnchor = 256;    // tokens between two stored states of the backward

void gated_split(GatedProblem& p, bool backward);
size_t gated_workspace_floats(const GatedProblem& p, bool backward);
cudaError_t launch_gated(const GatedProblem& p, const void* Q, const void* K, const void* V,
                         const float* G, const float* S_in, float* S_out, void* O, float* ws,
                         cudaStream_t s);
cudaError_t launch_gated_backward(const GatedProblem& p, const void* Q, const void* K,
                                  const void* V, const float* G, const float* S_in,
                                  const void* dO, const float* dS_out, void* dQ, void* dK,
                                  void* dV, float* dG, float* dS_in, float* ws, cudaStream_t s);

// Rotary positions (la_rotary.cu).
constexpr int kRotaryMaxD = 256;
struct RotaryProblem {
  long long rows;    // tokens over the whole batch
  int N, H, Hk, D, rot;
  int io, half, inverse;
  int pos_rows;      // positions are [B, N] (1) or [N] (0)
  int pos_offset;    // position of token 0 when there are no positions
  double mscale;
  double rate[kRotaryMaxD / 2];  // radians per position of each pair
};
cudaError_t launch_rotary(const RotaryProblem& p, const void* Q, const void* K, const int* pos,
                          void* Qo, void* Ko, cudaStream_t s);

// Gated residual with the norms around it (la_norm.cu).
constexpr int kNormMaxC = 8192;
struct NormProblem {
  int B, N, C;
  int io, layer;   // layer: subtract the mean
  float eps, alpha;
  int ctas;        // backward: CTAs (and partial column sums) of a batch element
};
struct NormParams {  // [B, C] or [C] float32, or null
  const float *gate, *w_post, *w_pre, *mod_scale, *mod_shift;
};
struct NormGrads {
  float *gate, *w_post, *w_pre, *mod_scale, *mod_shift;
};
void norm_split(NormProblem& p);
size_t norm_workspace_floats(const NormProblem& p);
cudaError_t launch_norm(const NormProblem& p, const void* x, const void* f, const NormParams& w,
                        void* h, void* y, cudaStream_t s);
cudaError_t launch_norm_backward(const NormProblem& p, const void* x, const void* f,
                                 const NormParams& w, const void* dh, const void* dy, void* dx,
                                 void* df, const NormGrads& g, float* ws, cudaStream_t s);

}  // namespace la
