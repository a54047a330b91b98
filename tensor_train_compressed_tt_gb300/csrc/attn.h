// Tensors of heads, and what the translation unit of windowed attention shares.
#pragma once

#include "ttc_internal.h"

namespace ttc {

// A tensor of heads on the device: element (t, h, c) at p[t row + h head + c].
struct Heads {
  void* p = nullptr;
  int64_t row = 0, head = 0;
  template <typename T>
  __host__ __device__ T* at(int64_t t, int h) const {
    return static_cast<T*>(p) + t * row + h * head;
  }
};

inline bool aligned_to(const void* p, size_t n) {
  return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

// A tensor that the call reads or writes when it has rows.
inline bool heads_ok(const tt_heads* h, int64_t rows, int act, Heads* out) {
  if (!h || h->row < 0 || h->head < 0 || !aligned_to(h->p, act == TT_DT_F32 ? 4 : 2)) return false;
  if (rows > 0 && !h->p) return false;
  out->p = h->p;
  out->row = h->row;
  out->head = h->head;
  return true;
}

struct AttnArgs {
  int B, heads, kv, group, dim;
  int left, right, sinks;  // left, right < 0: unbounded; none above kAttnMaxLen
  float scale;
  int max_q, max_k;
  int64_t Tq, Tk;
  const int32_t *q_begin, *q_end, *k_begin, *k_end;
  Heads q, k, v, o, dout, dq, dk, dv;
  const float* lse_in;
  float* lse;
  float* delta;  // (heads, Tq): sum over the channels of o dout
};

// Longest sequence: position arithmetic (position + bound + tile) stays in 32 bits.
constexpr int kAttnMaxLen = 1 << 29;

}  // namespace ttc
