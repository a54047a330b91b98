// Dropout from a counter-based generator: which elements stay is computed from a
// seed and the element's index wherever it is needed, and stored nowhere.
//
// The generator is Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// 2011).  Key: the seed.  Counter: the index of a group of eight elements (48
// bits), the site (16) and the offset (64).  Its four words give eight elements 16
// bits each, lower halves first; an element stays when its bits are not below the
// cut.  16 bits resolve a probability to 2^-17, far below what a training run can
// tell apart, and halve the generator's time, which is what a pass over bf16 values
// has little of: a call is 20 wide multiplications, 20 exclusive ors and the round keys.
#pragma once

#include "rows.cuh"

namespace ttc {
namespace {

struct DropArgs {
  const int64_t* rng;  // device: seed, offset
  uint32_t cut;        // bits below it drop an element, as the upper half of a word
  bool all;            // every element is dropped
  uint32_t site;
  float scale;         // of the elements that stay
};

// The generator's state, read once a thread.
struct DropKey {
  uint32_t seed0, seed1, off0, off1;
  __device__ void read(const DropArgs& d) {
    const uint64_t s = (uint64_t)d.rng[0], o = (uint64_t)d.rng[1];
    seed0 = (uint32_t)s, seed1 = (uint32_t)(s >> 32);
    off0 = (uint32_t)o, off1 = (uint32_t)(o >> 32);
  }
  // The words of n groups: side by side they share the round keys.
  template <int N>
  __device__ __forceinline__ void words(const int64_t (&group)[N], uint32_t site,
                                        uint4 (&x)[N]) const {
#pragma unroll
    for (int g = 0; g < N; ++g)
      x[g] = make_uint4((uint32_t)group[g], (uint32_t)(group[g] >> 32) + (site << 16), off0, off1);
    uint32_t k0 = seed0, k1 = seed1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
      for (int g = 0; g < N; ++g) {
        const uint64_t a = (uint64_t)x[g].x * 0xD2511F53u, b = (uint64_t)x[g].z * 0xCD9E8D57u;
        x[g] = make_uint4((uint32_t)(b >> 32) ^ x[g].y ^ k0, (uint32_t)b,
                          (uint32_t)(a >> 32) ^ x[g].w ^ k1, (uint32_t)a);
      }
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
  }
};

// Two elements by the halves of one word, the lower one first.
__device__ __forceinline__ void drop2(uint32_t w, const DropArgs& d, float* f) {
  const float2 t = __fmul2_rn(make_float2(f[0], f[1]), make_float2(d.scale, d.scale));
  f[0] = w << 16 >= d.cut && !d.all ? t.x : 0.f;
  // the lower half adds less than a step of the cut
  f[1] = w >= d.cut && !d.all ? t.y : 0.f;
}

// VEC elements from index i on (a multiple of VEC) by the words of their group.
template <int VEC>
__device__ __forceinline__ void drop(const uint4& w, const DropArgs& d, int64_t i, float* f) {
  if (VEC == 8) {
    drop2(w.x, d, f);
    drop2(w.y, d, f + 2);
    drop2(w.z, d, f + 4);
    drop2(w.w, d, f + 6);
  } else if (VEC == 4) {
    const bool second = i & 4;
    drop2(second ? w.z : w.x, d, f);
    drop2(second ? w.w : w.y, d, f + 2);
  } else {
    const uint32_t a = i & 4 ? (i & 2 ? w.w : w.z) : (i & 2 ? w.y : w.x);
    f[0] = (i & 1 ? a : a << 16) >= d.cut && !d.all ? f[0] * d.scale : 0.f;
  }
}
template <int VEC>
__device__ __forceinline__ void drop(const DropKey& key, const DropArgs& d, int64_t i, float* f) {
  const int64_t group[1] = {i >> 3};
  uint4 w[1];
  key.words(group, d.site, w);
  drop<VEC>(w[0], d, i, f);
}

}  // namespace

// The arguments of a pass (false for a state that is missing or misaligned).
inline bool drop_args(const DropPlan& P, const int64_t* rng, DropArgs* d) {
  if (!rng || !aligned_to(rng, 8)) return false;
  d->rng = rng;
  d->cut = P.cut << 16;
  d->all = P.cut == 65536;
  d->site = P.site;
  d->scale = P.cut < 65536 ? 65536.f / (float)(65536 - P.cut) : 0.f;
  return true;
}

}  // namespace ttc
