// Sequences and masks of the attention kernels.
#pragma once

#include "attn.h"
#include "tc_ptx.cuh"

namespace ttc {
namespace {

// 2^x by the exponential unit alone (results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One sequence: its first query and key row and their counts.
struct Seq {
  int64_t q0, k0;
  int lq, lk;
  __device__ int off() const { return lk - lq; }  // position of query row 0
};

// False, and recorded in the status word (by the threads that tell), for a
// sequence outside the buffers or the caller's bounds.
__device__ __forceinline__ bool load_seq(const AttnArgs& p, int b, Seq* s, bool tell) {
  const int64_t q0 = p.q_begin[b], q1 = p.q_end[b], k0 = p.k_begin[b], k1 = p.k_end[b];
  if (q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk || q1 - q0 > p.max_q ||
      k1 - k0 > p.max_k) {
    if (tell) record_error(TT_ERR_DEVICE, 64);
    return false;
  }
  s->q0 = q0;
  s->k0 = k0;
  s->lq = (int)(q1 - q0);
  s->lk = (int)(k1 - k0);
  return true;
}

__device__ __forceinline__ bool visible(const AttnArgs& p, int i, int j) {
  return (p.right < 0 || j <= i + p.right) && (p.left < 0 || j >= i - p.left || j < p.sinks);
}

// The keys that some query at a position in [i0, i1] sees: [0, a1) and
// [b0, b1), the first empty when the second starts inside the first tokens.
struct KeySpan {
  int a1, b0, b1;
};
__device__ __forceinline__ KeySpan key_span(const AttnArgs& p, int lk, int i0, int i1) {
  int hi = p.right < 0 ? lk : min(lk, i1 + p.right + 1);
  if (hi < 0) hi = 0;
  int lo = p.left < 0 ? 0 : max(0, i0 - p.left);
  if (lo > hi) lo = hi;
  KeySpan s;
  s.a1 = min(p.sinks, lo);
  s.b0 = lo;
  s.b1 = hi;
  if (s.a1 == lo) s.a1 = 0, s.b0 = 0;
  return s;
}

// The query rows [t0, t1) that see some key of [j0, j1].
struct RowSpan {
  int t0, t1;
};
__device__ __forceinline__ RowSpan row_span(const AttnArgs& p, const Seq& s, int j0, int j1) {
  const int off = s.off();
  const int lo = p.right < 0 ? off : max(off, j0 - p.right);
  const int hi = (p.left < 0 || j0 < p.sinks) ? s.lk - 1 : min(s.lk - 1, j1 + p.left);
  RowSpan r;
  r.t0 = max(0, lo - off);
  r.t1 = max(r.t0, hi - off + 1);
  return r;
}

}  // namespace
}  // namespace ttc
