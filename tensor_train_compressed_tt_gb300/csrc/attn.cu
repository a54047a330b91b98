// Attention with a sliding window and first tokens that stay visible: the C
// entry points and the choice of kernels.
#include <cmath>
#include <new>

#include "attn.h"
#include "attn_decode.cuh"
#include "attn_general.cuh"
#include "attn_seq.cuh"
#include "attn_tc_bwd.cuh"
#include "attn_tc_fwd.cuh"
#include "ttc.h"

namespace ttc {

cudaError_t read_and_clear_attn_status(DeviceStatus* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(DeviceStatus));
  if (e != cudaSuccess || out->code == 0) return e;
  DeviceStatus z{0, 0};
  return cudaMemcpyToSymbol(g_status, &z, sizeof(z));
}

cudaError_t attn_set_wait_limit(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}

cudaError_t attn_set_debug_skip(int site) {
  return cudaMemcpyToSymbol(g_debug_skip, &site, sizeof(site));
}

namespace {

size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

bool seqs_ok(const tt_attn_seqs* s) {
  if (!s || s->B < 0 || s->B > (1 << 20) || s->max_q < 0 || s->max_k < 0 ||
      s->max_q > kAttnMaxLen || s->max_k > kAttnMaxLen || s->Tq < 0 || s->Tk < 0 ||
      s->Tq > 0x7FFFFFFF || s->Tk > 0x7FFFFFFF)
    return false;
  const int32_t* a[4] = {s->q_begin, s->q_end, s->k_begin, s->k_end};
  for (int i = 0; i < 4; ++i)
    if (s->B > 0 && (!a[i] || !aligned_to(a[i], 4))) return false;
  return true;
}

// Fewest query rows of a sequence for the tensor-core backward.  Of fewer, most of
// a 128-row tile is empty, and the sums over queries are so short that a weight's
// rounding to bf16 shows in dv (up to 6.2e-2 of its root mean square; the general
// kernels keep the weights in fp32).  Time, 12 heads of 64, general against
// tensor cores: 8 sequences of 16: 14 and 17 us, 256 of 16: 149 and 100 us,
// 256 of 32: 186 and 102 us, 256 of 48: 470 and 105 us.
constexpr int kTcBwdRows = 32;

AttnArgs make_args(const AttnPlan& P, const tt_attn_seqs* s) {
  AttnArgs a = {};
  a.B = s->B;
  a.heads = P.heads;
  a.kv = P.kv;
  a.group = P.heads / P.kv;
  a.dim = P.dim;
  a.left = P.left;
  a.right = P.right;
  a.sinks = P.sinks;
  a.scale = P.scale;
  a.max_q = s->max_q;
  a.max_k = s->max_k;
  a.Tq = s->Tq;
  a.Tk = s->Tk;
  a.q_begin = s->q_begin;
  a.q_end = s->q_end;
  a.k_begin = s->k_begin;
  a.k_end = s->k_end;
  return a;
}

// Workspace of a pass.  Forward: partial results of keys split over CTAs.  Backward: delta, then the partial sums of key tiles in pieces.
size_t delta_bytes(const AttnPlan& P, const tt_attn_seqs* s) {
  return al256((size_t)P.heads * (size_t)s->Tq * sizeof(float));
}
size_t attn_ws(const AttnPlan& P, const tt_attn_seqs* s, bool backward) {
  return backward ? delta_bytes(P, s) + al256(bwd_parts_bytes(P, s)) : al256(decode_bytes(P, s));
}

tt_status from_cuda(cudaError_t e) {
  if (e == cudaErrorInvalidConfiguration) return TT_ERR_UNSUPPORTED;  // more blocks than a grid has
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace
}  // namespace ttc

using namespace ttc;

extern "C" {

tt_status tt_attn_plan(const tt_attn_desc* desc, tt_plan_t** out) {
  if (!out) return TT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || desc->heads < 1 || desc->heads > 1024 || desc->kv_heads < 1 ||
      desc->heads % desc->kv_heads || desc->dim < 1 || desc->sinks < 0 || desc->flags ||
      !std::isfinite(desc->scale))
    return TT_ERR_INVALID_ARG;
  if (desc->act != TT_DT_F32 && desc->act != TT_DT_BF16 && desc->act != TT_DT_E4M3)
    return TT_ERR_INVALID_ARG;
  if (desc->act == TT_DT_E4M3 || desc->dim > 256) return TT_ERR_UNSUPPORTED;
  tt_plan_s* p = new (std::nothrow) tt_plan_s();
  if (!p) return TT_ERR_INVALID_ARG;
  p->kind = 5;
  AttnPlan& P = p->attn;
  P.heads = desc->heads;
  P.kv = desc->kv_heads;
  P.dim = desc->dim;
  // a bound beyond the longest sequence hides nothing
  P.left = desc->left < 0 || desc->left > kAttnMaxLen ? -1 : desc->left;
  P.right = desc->right < 0 || desc->right > kAttnMaxLen ? -1 : desc->right;
  P.sinks = desc->sinks > kAttnMaxLen ? kAttnMaxLen : desc->sinks;
  P.scale = desc->scale == 0.f ? 1.f / std::sqrt((float)desc->dim) : desc->scale;
  P.act = desc->act;
  *out = p;
  return TT_OK;
}

tt_status tt_attn_workspace_size(const tt_plan_t* plan, const tt_attn_seqs* seqs, int backward,
                                 size_t* bytes) {
  if (!plan || plan->kind != 5 || !bytes || !seqs_ok(seqs)) return TT_ERR_INVALID_ARG;
  *bytes = attn_ws(plan->attn, seqs, backward != 0);
  return TT_OK;
}

tt_status tt_attn_forward(const tt_plan_t* plan, const tt_attn_seqs* seqs, const tt_heads* q,
                          const tt_heads* k, const tt_heads* v, const tt_heads* o, float* lse,
                          void* ws, size_t ws_bytes, void* stream) {
  if (!plan || plan->kind != 5 || !seqs_ok(seqs)) return TT_ERR_INVALID_ARG;
  const AttnPlan& P = plan->attn;
  AttnArgs a = make_args(P, seqs);
  if (!heads_ok(q, a.Tq, P.act, &a.q) || !heads_ok(k, a.Tk, P.act, &a.k) ||
      !heads_ok(v, a.Tk, P.act, &a.v) || !heads_ok(o, a.Tq, P.act, &a.o) || !aligned_to(lse, 4))
    return TT_ERR_INVALID_ARG;
  const size_t need = attn_ws(P, seqs, false);
  if (need && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return TT_ERR_WORKSPACE;
  a.lse = lse;
  if (a.B == 0 || a.max_q == 0) return TT_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhFwd, st);
  const bool few = decode_shape(P, seqs) && decode_takes(a, P.act);
  const cudaError_t e = few                   ? decode(P, seqs, a, ws, st)
                        : P.act == TT_DT_F32 ? general_pass<float>(a, 0, st)
                        : tc_fwd_takes(a)    ? tc_fwd(a, st)
                                             : general_pass<__nv_bfloat16>(a, 0, st);
  prof_end(kPhFwd, st);
  return from_cuda(e);
}

tt_status tt_attn_backward(const tt_plan_t* plan, const tt_attn_seqs* seqs, const tt_heads* q,
                           const tt_heads* k, const tt_heads* v, const tt_heads* o,
                           const float* lse, const tt_heads* dout, const tt_heads* dq,
                           const tt_heads* dk, const tt_heads* dv, void* ws, size_t ws_bytes,
                           void* stream) {
  if (!plan || plan->kind != 5 || !seqs_ok(seqs)) return TT_ERR_INVALID_ARG;
  const AttnPlan& P = plan->attn;
  AttnArgs a = make_args(P, seqs);
  if (!heads_ok(q, a.Tq, P.act, &a.q) || !heads_ok(k, a.Tk, P.act, &a.k) ||
      !heads_ok(v, a.Tk, P.act, &a.v) || !heads_ok(o, a.Tq, P.act, &a.o) ||
      !heads_ok(dout, a.Tq, P.act, &a.dout) || !heads_ok(dq, a.Tq, P.act, &a.dq) ||
      !heads_ok(dk, a.Tk, P.act, &a.dk) || !heads_ok(dv, a.Tk, P.act, &a.dv) ||
      !aligned_to(lse, 4) || (a.Tq > 0 && !lse))
    return TT_ERR_INVALID_ARG;
  const size_t need = attn_ws(P, seqs, true);
  if (need && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return TT_ERR_WORKSPACE;
  a.lse_in = lse;
  a.delta = static_cast<float*>(ws);
  if (a.B == 0) return TT_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhBwd, st);
  cudaError_t e = cudaSuccess;
  const bool tc = P.act == TT_DT_BF16 && tc_bwd_takes(a) && a.max_q >= kTcBwdRows;
  if (tc)
    e = tc_bwd(P, seqs, a, reinterpret_cast<float*>(static_cast<char*>(ws) + delta_bytes(P, seqs)),
               st);
  for (int pass = 1; pass <= 2 && !tc && e == cudaSuccess; ++pass)
    e = P.act == TT_DT_BF16 ? general_pass<__nv_bfloat16>(a, pass, st)
                            : general_pass<float>(a, pass, st);
  prof_end(kPhBwd, st);
  return from_cuda(e);
}

}  // extern "C"
