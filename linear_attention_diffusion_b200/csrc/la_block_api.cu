// C-ABI layer of the block operators of include/la.h: gated linear attention,
// rotary positions, the gated residual with its norms.
#include <cmath>
#include <cstdint>

#include "la.h"
#include "la_block_internal.h"
#include "la_internal.h"

using namespace la;
using namespace la::detail;

namespace {

#define LA_TRY(expr)              \
  do {                            \
    const la_status st_ = (expr); \
    if (st_ != LA_OK) return st_; \
  } while (0)

struct Buffer {
  const void* p;
  size_t n;
  const char* name;
};

// Outputs must not overlap each other or an input.
template <size_t kOut, size_t kIn>
la_status check_apart(const Buffer (&outs)[kOut], const Buffer (&ins)[kIn]) {
  for (size_t i = 0; i < kOut; ++i) {
    for (size_t j = i + 1; j < kOut; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return fail(LA_ERR_INVALID_ARG, "%s and %s overlap", outs[i].name, outs[j].name);
    for (size_t j = 0; j < kIn; ++j)
      if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
        return fail(LA_ERR_INVALID_ARG, "%s and %s overlap", outs[i].name, ins[j].name);
  }
  return LA_OK;
}

la_status check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return LA_OK;
  if (ws == nullptr) return fail(LA_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
  LA_TRY(check_ptr(ws, "workspace", true));
  if (ws_bytes < need)
    return fail(LA_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  return LA_OK;
}

la_status make_gated(const la_gated_shape* s, bool backward, GatedProblem& p) {
  if (s == nullptr) return fail(LA_ERR_INVALID_ARG, "shape is NULL");
  if (s->B < 0 || s->N < 0 || s->H < 0)
    return fail(LA_ERR_INVALID_ARG, "negative size B=%d N=%d H=%d", s->B, s->N, s->H);
  if (s->D != kD) return fail(LA_ERR_UNSUPPORTED, "head width D=%d (only 32 is built)", s->D);
  if (s->io_dtype != LA_IO_BF16 && s->io_dtype != LA_IO_F32)
    return fail(LA_ERR_INVALID_ARG, "io_dtype=%d", s->io_dtype);
  if (!std::isfinite(s->scale)) return fail(LA_ERR_INVALID_ARG, "scale must be finite");
  if (s->B > 65535 || s->H > 65535 || 1LL * s->B * s->H > (1LL << 24) || s->N > (1 << 30))
    return fail(LA_ERR_UNSUPPORTED, "B=%d, H=%d or N=%d too large", s->B, s->H, s->N);
  if (1.0 * s->B * s->N * s->H >= 1.0 * (1LL << 35))
    return fail(LA_ERR_UNSUPPORTED, "tensor too large");
  p.B = s->B;
  p.N = s->N;
  p.H = s->H;
  p.io = s->io_dtype;
  p.scale = s->scale;
  gated_split(p, backward);
  return LA_OK;
}

size_t gated_need(const GatedProblem& p, bool backward) {
  if (p.B == 0 || p.H == 0 || p.N == 0) return 0;
  if (!backward && p.N <= kGateStepTokens) return 0;
  return align256(gated_workspace_floats(p, backward) * sizeof(float));
}

// dst = src, or zero without src (an empty sequence passes its state on).
la_status pass_on(float* dst, const float* src, size_t bytes, cudaStream_t st) {
  if (dst == nullptr || dst == src) return LA_OK;
  const cudaError_t e = src != nullptr
                            ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st)
                            : cudaMemsetAsync(dst, 0, bytes, st);
  return e == cudaSuccess ? LA_OK : cuda_fail(e, "state of an empty sequence");
}

la_status make_norm(const la_norm_shape* s, NormProblem& p) {
  if (s == nullptr) return fail(LA_ERR_INVALID_ARG, "shape is NULL");
  if (s->B < 0 || s->N < 0) return fail(LA_ERR_INVALID_ARG, "negative size B=%d N=%d", s->B, s->N);
  if (s->C < 8 || s->C % 8 != 0 || s->C > kNormMaxC)
    return fail(LA_ERR_UNSUPPORTED, "width C=%d (a multiple of 8 in [8, %d])", s->C, kNormMaxC);
  if (s->io_dtype != LA_IO_BF16 && s->io_dtype != LA_IO_F32)
    return fail(LA_ERR_INVALID_ARG, "io_dtype=%d", s->io_dtype);
  if (s->norm != 0 && s->norm != 1) return fail(LA_ERR_INVALID_ARG, "norm=%d", s->norm);
  if (!(std::isfinite(s->eps) && s->eps >= 0.0f))
    return fail(LA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!std::isfinite(s->alpha)) return fail(LA_ERR_INVALID_ARG, "alpha must be finite");
  if (s->B > 65535 || s->N > (1 << 30) || 1.0 * s->B * s->N * s->C >= 1.0 * (1LL << 40))
    return fail(LA_ERR_UNSUPPORTED, "tensor too large");
  p = NormProblem{s->B, s->N, s->C, s->io_dtype, s->norm, s->eps, s->alpha, 1};
  norm_split(p);
  return LA_OK;
}

la_status check_param(const float* w, const char* name) { return check_ptr(w, name, w != nullptr); }

}  // namespace

extern "C" {

size_t la_gated_workspace_bytes(const la_gated_shape* shape, int backward) {
  GatedProblem p;
  if (make_gated(shape, backward != 0, p) != LA_OK) return 0;
  const size_t n = gated_need(p, backward != 0);
  return n == 0 ? 256 : n;
}

int la_gated_launches(const la_gated_shape* shape, int backward) {
  GatedProblem p;
  if (make_gated(shape, backward != 0, p) != LA_OK) return 0;
  if (p.B == 0 || p.H == 0 || p.N == 0) return 0;
  const bool cut = p.nseg > 1 && !p.whole_row;  // segments' states and their combination first
  if (backward) return cut ? 4 : 2;
  return cut && p.N > kGateStepTokens ? 3 : 1;
}

la_status la_gated_attention(const la_gated_shape* shape, const void* Q, const void* K,
                             const void* V, const float* G, const float* S_in, float* S_out,
                             void* O, void* ws, size_t ws_bytes, la_stream stream) {
  GatedProblem p;
  LA_TRY(make_gated(shape, false, p));
  const bool any_state = p.B > 0 && p.H > 0, any = any_state && p.N > 0;
  LA_TRY(check_ptr(Q, "Q", any));
  LA_TRY(check_ptr(K, "K", any));
  LA_TRY(check_ptr(V, "V", any));
  LA_TRY(check_ptr(G, "G", any));
  LA_TRY(check_ptr(O, "O", any));
  LA_TRY(check_ptr(S_in, "S_in", any_state && S_in != nullptr));
  LA_TRY(check_ptr(S_out, "S_out", any_state && S_out != nullptr));
  const size_t need = gated_need(p, false);
  LA_TRY(check_workspace(ws, ws_bytes, need));
  const size_t rows = static_cast<size_t>(p.B) * p.N * p.H;
  const size_t nx = rows * kD * (p.io == LA_IO_BF16 ? 2 : 4), ng = rows * 4;
  const size_t ns = static_cast<size_t>(p.B) * p.H * kD * kD * 4;
  const Buffer ins[] = {{Q, nx, "Q"}, {K, nx, "K"}, {V, nx, "V"}, {G, ng, "G"}, {ws, need, "the workspace"},
                        {S_in == S_out ? nullptr : S_in, ns, "S_in"}};
  const Buffer outs[] = {{O, nx, "O"}, {S_out, ns, "S_out"}};
  LA_TRY(check_apart(outs, ins));
  if (overlap(ws, need, S_in, ns))
    return fail(LA_ERR_INVALID_ARG, "S_in and the workspace overlap");
  if (!any_state) return LA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!any) return pass_on(S_out, S_in, ns, st);
  const cudaError_t e =
      launch_gated(p, Q, K, V, G, S_in, S_out, O, static_cast<float*>(ws), st);
  if (e != cudaSuccess) return cuda_fail(e, "gated attention");
  return LA_OK;
}

la_status la_gated_attention_backward(const la_gated_shape* shape, const void* Q, const void* K,
                                      const void* V, const float* G, const float* S_in,
                                      const void* dO, const float* dS_out, void* dQ, void* dK,
                                      void* dV, float* dG, float* dS_in, void* ws,
                                      size_t ws_bytes, la_stream stream) {
  GatedProblem p;
  LA_TRY(make_gated(shape, true, p));
  const bool any_state = p.B > 0 && p.H > 0, any = any_state && p.N > 0;
  LA_TRY(check_ptr(Q, "Q", any));
  LA_TRY(check_ptr(K, "K", any));
  LA_TRY(check_ptr(V, "V", any));
  LA_TRY(check_ptr(G, "G", any));
  LA_TRY(check_ptr(dO, "dO", any));
  LA_TRY(check_ptr(dQ, "dQ", any));
  LA_TRY(check_ptr(dK, "dK", any));
  LA_TRY(check_ptr(dV, "dV", any));
  LA_TRY(check_ptr(dG, "dG", any));
  LA_TRY(check_ptr(S_in, "S_in", any_state && S_in != nullptr));
  LA_TRY(check_ptr(dS_out, "dS_out", any_state && dS_out != nullptr));
  LA_TRY(check_ptr(dS_in, "dS_in", any_state && dS_in != nullptr));
  const size_t need = gated_need(p, true);
  LA_TRY(check_workspace(ws, ws_bytes, need));
  const size_t rows = static_cast<size_t>(p.B) * p.N * p.H;
  const size_t nx = rows * kD * (p.io == LA_IO_BF16 ? 2 : 4), ng = rows * 4;
  const size_t ns = static_cast<size_t>(p.B) * p.H * kD * kD * 4;
  const Buffer ins[] = {{Q, nx, "Q"}, {K, nx, "K"}, {V, nx, "V"}, {G, ng, "G"},
                        {S_in, ns, "S_in"}, {dO, nx, "dO"}, {dS_out, ns, "dS_out"}};
  const Buffer outs[] = {{dQ, nx, "dQ"}, {dK, nx, "dK"}, {dV, nx, "dV"}, {dG, ng, "dG"},
                         {dS_in, ns, "dS_in"}, {ws, need, "the workspace"}};
  LA_TRY(check_apart(outs, ins));
  if (!any_state) return LA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!any) return pass_on(dS_in, dS_out, ns, st);
  const cudaError_t e = launch_gated_backward(p, Q, K, V, G, S_in, dO, dS_out, dQ, dK, dV, dG,
                                              dS_in, static_cast<float*>(ws), st);
  if (e != cudaSuccess) return cuda_fail(e, "gated attention backward");
  return LA_OK;
}

la_status la_rotary(const la_rotary_shape* shape, const void* Q, const void* K,
                    const int* positions, void* Qo, void* Ko, la_stream stream) {
  if (shape == nullptr) return fail(LA_ERR_INVALID_ARG, "shape is NULL");
  const la_rotary_shape& s = *shape;
  if (s.B < 0 || s.N < 0 || s.H < 0 || s.Hk < 0)
    return fail(LA_ERR_INVALID_ARG, "negative size B=%d N=%d H=%d Hk=%d", s.B, s.N, s.H, s.Hk);
  if (s.D < 8 || s.D % 8 != 0 || s.D > kRotaryMaxD)
    return fail(LA_ERR_UNSUPPORTED, "head width D=%d (a multiple of 8 in [8, %d])", s.D, kRotaryMaxD);
  if (s.rot < 0 || s.rot > s.D || s.rot % 2 != 0)
    return fail(LA_ERR_INVALID_ARG, "rot=%d (even, at most D=%d)", s.rot, s.D);
  if (s.io_dtype != LA_IO_BF16 && s.io_dtype != LA_IO_F32)
    return fail(LA_ERR_INVALID_ARG, "io_dtype=%d", s.io_dtype);
  if ((s.half | s.inverse | s.pos_rows) & ~1)
    return fail(LA_ERR_INVALID_ARG, "half=%d, inverse=%d, pos_rows=%d (0 or 1)", s.half, s.inverse,
                s.pos_rows);
  if (s.scaling < 0 || s.scaling > 3) return fail(LA_ERR_INVALID_ARG, "scaling=%d", s.scaling);
  if (s.pos_offset < 0 || 1LL * s.pos_offset + s.N > 0x7fffffffLL)
    return fail(LA_ERR_INVALID_ARG, "pos_offset=%d", s.pos_offset);
  if (!(std::isfinite(s.base) && s.base > 1.0))
    return fail(LA_ERR_INVALID_ARG, "base must be finite and > 1");
  if (!std::isfinite(s.mscale)) return fail(LA_ERR_INVALID_ARG, "mscale must be finite");
  if (s.scaling != 0 && !(std::isfinite(s.factor) && s.factor >= 1.0))
    return fail(LA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (s.scaling == 3 && !(std::isfinite(s.original_length) && s.original_length > 0.0 &&
                          std::isfinite(s.slow) && std::isfinite(s.fast) && s.slow >= 0.0 &&
                          s.slow < s.fast))
    return fail(LA_ERR_INVALID_ARG, "original_length > 0 and 0 <= slow < fast are needed");
  const double rows = 1.0 * s.B * s.N;
  if (rows * s.D * (1.0 * s.H + s.Hk) >= 1.0 * (1LL << 40) || rows >= 1.0 * (1LL << 31) ||
      (1LL * s.H + s.Hk) * s.D >= (1LL << 24))
    return fail(LA_ERR_UNSUPPORTED, "tensor too large");
  const bool any_q = rows > 0 && s.H > 0, any_k = rows > 0 && s.Hk > 0;
  const size_t e = s.io_dtype == LA_IO_BF16 ? 2 : 4;
  const size_t nr = static_cast<size_t>(s.B) * s.N;
  const size_t nq = nr * s.H * s.D * e, nk = nr * s.Hk * s.D * e;
  const size_t np = (s.pos_rows ? nr : static_cast<size_t>(s.N)) * 4;
  LA_TRY(check_ptr(Q, "Q", any_q));
  LA_TRY(check_ptr(Qo, "Qo", any_q));
  LA_TRY(check_ptr(K, "K", any_k));
  LA_TRY(check_ptr(Ko, "Ko", any_k));
  if ((any_q || any_k) && (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
    return fail(LA_ERR_INVALID_ARG, "positions are not 4-byte aligned");
  const Buffer ins[] = {{Q == Qo ? nullptr : Q, nq, "Q"}, {K == Ko ? nullptr : K, nk, "K"},
                        {positions, np, "positions"}};
  const Buffer outs[] = {{Qo, nq, "Qo"}, {Ko, nk, "Ko"}};
  if (any_q || any_k) LA_TRY(check_apart(outs, ins));
  if (!any_q && !any_k) return LA_OK;
  RotaryProblem p = {};
  p.rows = static_cast<long long>(nr);
  p.N = s.N;
  p.H = s.H;
  p.Hk = s.Hk;
  p.D = s.D;
  p.rot = s.rot;
  p.io = s.io_dtype;
  p.half = s.half;
  p.inverse = s.inverse;
  p.pos_rows = s.pos_rows;
  p.pos_offset = s.pos_offset;
  p.mscale = s.mscale;
  double base = s.base;
  if (s.scaling == 2 && s.rot > 2) base *= std::pow(s.factor, 1.0 * s.rot / (s.rot - 2));
  for (int k = 0; k < s.rot / 2; ++k) {
    double f = std::pow(base, -2.0 * k / s.rot);
    if (s.scaling == 1) f /= s.factor;
    if (s.scaling == 3) {
      const double turns = s.original_length * f / 6.283185307179586476925286766559;
      const double w = std::fmin(1.0, std::fmax(0.0, (turns - s.slow) / (s.fast - s.slow)));
      f *= w + (1.0 - w) / s.factor;
    }
    p.rate[k] = f;
  }
  const cudaError_t err =
      launch_rotary(p, Q, K, positions, Qo, Ko, reinterpret_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err, "rotary");
  return LA_OK;
}

la_status la_gate_residual_norm(const la_norm_shape* shape, const void* x, const void* f,
                                const float* gate, const float* w_post, const float* w_pre,
                                const float* mod_scale, const float* mod_shift, void* h, void* y,
                                la_stream stream) {
  NormProblem p;
  LA_TRY(make_norm(shape, p));
  const bool any = p.B > 0 && p.N > 0;
  if (f == nullptr && any && (gate != nullptr || w_post != nullptr || h != nullptr))
    return fail(LA_ERR_INVALID_ARG, "without f there is no gate, w_post or h");
  if (any && h == nullptr && y == nullptr) return fail(LA_ERR_INVALID_ARG, "h and y are both NULL");
  LA_TRY(check_ptr(x, "x", any));
  LA_TRY(check_ptr(f, "f", any && f != nullptr));
  LA_TRY(check_ptr(h, "h", any && h != nullptr));
  LA_TRY(check_ptr(y, "y", any && y != nullptr));
  LA_TRY(check_param(gate, "gate"));
  LA_TRY(check_param(w_post, "w_post"));
  LA_TRY(check_param(w_pre, "w_pre"));
  LA_TRY(check_param(mod_scale, "mod_scale"));
  LA_TRY(check_param(mod_shift, "mod_shift"));
  if (!any) return LA_OK;
  const size_t n = static_cast<size_t>(p.B) * p.N * p.C * (p.io == LA_IO_BF16 ? 2 : 4);
  const size_t nc = static_cast<size_t>(p.C) * 4, nb = nc * p.B;
  const Buffer params[] = {{gate, nb, "gate"}, {w_post, nc, "w_post"}, {w_pre, nc, "w_pre"},
                           {mod_scale, nb, "mod_scale"}, {mod_shift, nb, "mod_shift"}};
  const Buffer outs[] = {{h, n, "h"}, {y, n, "y"}};
  LA_TRY(check_apart(outs, params));
  for (const Buffer& o : outs)  // x or f itself, but no part of it
    for (const void* in : {x, f})
      if (o.p != in && overlap(o.p, n, in, n))
        return fail(LA_ERR_INVALID_ARG, "%s overlaps x or f without being it", o.name);
  const cudaError_t e = launch_norm(p, x, f, NormParams{gate, w_post, w_pre, mod_scale, mod_shift},
                                    h, y, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gated residual norm");
  return LA_OK;
}

size_t la_norm_workspace_bytes(const la_norm_shape* shape) {
  NormProblem p;
  if (make_norm(shape, p) != LA_OK) return 0;
  const size_t n = align256(norm_workspace_floats(p) * sizeof(float));
  return n == 0 ? 256 : n;
}

la_status la_gate_residual_norm_backward(const la_norm_shape* shape, const void* x, const void* f,
                                         const float* gate, const float* w_post,
                                         const float* w_pre, const float* mod_scale,
                                         const void* dh, const void* dy, void* dx, void* df,
                                         float* dgate, float* dw_post, float* dw_pre,
                                         float* dmod_scale, float* dmod_shift, void* ws,
                                         size_t ws_bytes, la_stream stream) {
  NormProblem p;
  LA_TRY(make_norm(shape, p));
  const bool any = p.B > 0 && p.N > 0;
  if (any) {
    if (f == nullptr && (gate != nullptr || w_post != nullptr || df != nullptr ||
                         dgate != nullptr || dw_post != nullptr))
      return fail(LA_ERR_INVALID_ARG, "without f there is no gate, w_post or gradient of them");
    if (f != nullptr && df == nullptr) return fail(LA_ERR_INVALID_ARG, "df is NULL");
    if (dh == nullptr && dy == nullptr)
      return fail(LA_ERR_INVALID_ARG, "dh and dy are both NULL");
  }
  LA_TRY(check_ptr(x, "x", any));
  LA_TRY(check_ptr(f, "f", any && f != nullptr));
  LA_TRY(check_ptr(dh, "dh", any && dh != nullptr));
  LA_TRY(check_ptr(dy, "dy", any && dy != nullptr));
  LA_TRY(check_ptr(dx, "dx", any));
  LA_TRY(check_ptr(df, "df", any && df != nullptr));
  LA_TRY(check_param(gate, "gate"));
  LA_TRY(check_param(w_post, "w_post"));
  LA_TRY(check_param(w_pre, "w_pre"));
  LA_TRY(check_param(mod_scale, "mod_scale"));
  LA_TRY(check_param(dgate, "dgate"));
  LA_TRY(check_param(dw_post, "dw_post"));
  LA_TRY(check_param(dw_pre, "dw_pre"));
  LA_TRY(check_param(dmod_scale, "dmod_scale"));
  LA_TRY(check_param(dmod_shift, "dmod_shift"));
  const size_t need = any ? align256(norm_workspace_floats(p) * sizeof(float)) : 0;
  LA_TRY(check_workspace(ws, ws_bytes, need));
  const size_t n = static_cast<size_t>(p.B) * p.N * p.C * (p.io == LA_IO_BF16 ? 2 : 4);
  const size_t nc = static_cast<size_t>(p.C) * 4, nb = nc * p.B;
  const Buffer ins[] = {{x, n, "x"}, {f, n, "f"}, {gate, nb, "gate"}, {w_post, nc, "w_post"},
                        {w_pre, nc, "w_pre"}, {mod_scale, nb, "mod_scale"}};
  const Buffer outs[] = {{dx, n, "dx"}, {df, n, "df"}, {dgate, nb, "dgate"},
                         {dw_post, nc, "dw_post"}, {dw_pre, nc, "dw_pre"},
                         {dmod_scale, nb, "dmod_scale"}, {dmod_shift, nb, "dmod_shift"},
                         {ws, need, "the workspace"}};
  LA_TRY(check_apart(outs, ins));
  for (const Buffer& o : outs)
    for (const void* in : {dh, dy})
      if (!((o.p == dx || o.p == df) && o.p == in) && overlap(o.p, o.n, in, n))
        return fail(LA_ERR_INVALID_ARG, "%s overlaps dh or dy without being it", o.name);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!any) {  // no rows: parameters that exist all the same get zeros
    const Buffer zero[] = {{dgate, nb, ""}, {dw_post, nc, ""}, {dw_pre, nc, ""},
                           {dmod_scale, nb, ""}, {dmod_shift, nb, ""}};
    for (const Buffer& z : zero)
      if (z.p != nullptr && z.n != 0) {
        const cudaError_t e = cudaMemsetAsync(const_cast<void*>(z.p), 0, z.n, st);
        if (e != cudaSuccess) return cuda_fail(e, "gated residual norm backward (no rows)");
      }
    return LA_OK;
  }
  const cudaError_t e = launch_norm_backward(
      p, x, f, NormParams{gate, w_post, w_pre, mod_scale, nullptr}, dh, dy, dx, df,
      NormGrads{dgate, dw_post, dw_pre, dmod_scale, dmod_shift}, static_cast<float*>(ws), st);
  if (e != cudaSuccess) return cuda_fail(e, "gated residual norm backward");
  return LA_OK;
}

}  // extern "C"
