// Dropout from a counter-based generator: which elements stay is computed from a
// seed and the element's index wherever it is needed, and stored nowhere.
//
// The generator is Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// 2011).  Key: the seed.  Counter: the index of a group of eight elements (48
// bits), the site (16) and the offset (64).  Its four words give eight elements 16
// bits each, lower halves first; an element stays when its bits are not below the
// cut.  16 bits resolve a probability to 2^-17, far below what a training run can
// tell apart, and halve the generator's time, which is what a pass over bf16 values
// has little of: a call is 20 wide multiplications and some 60 instructions.
#pragma once

#include "rows.cuh"

namespace ttc {
namespace {

struct DropArgs {
  const int64_t* rng;  // device: seed, offset
  uint32_t cut;        // 0 .. 65536: bits below it drop an element
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
  __device__ uint4 words(uint64_t group, uint32_t site) const {
    uint4 x = make_uint4((uint32_t)group, (uint32_t)(group >> 32) + (site << 16), off0, off1);
    uint32_t k0 = seed0, k1 = seed1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t a = (uint64_t)x.x * 0xD2511F53u, b = (uint64_t)x.z * 0xCD9E8D57u;
      x = make_uint4((uint32_t)(b >> 32) ^ x.y ^ k0, (uint32_t)b,
                     (uint32_t)(a >> 32) ^ x.w ^ k1, (uint32_t)a);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    return x;
  }
};

// Two elements by the halves of one word.
__device__ __forceinline__ void drop2(uint32_t w, const DropArgs& d, float* f) {
  f[0] = (w & 0xFFFFu) >= d.cut ? f[0] * d.scale : 0.f;
  f[1] = (w >> 16) >= d.cut ? f[1] * d.scale : 0.f;
}

// VEC elements from index i on (a multiple of VEC).
template <int VEC>
__device__ __forceinline__ void drop(const DropKey& key, const DropArgs& d, int64_t i, float* f) {
  const uint4 w = key.words((uint64_t)i >> 3, d.site);
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
    f[0] = (i & 1 ? a >> 16 : a & 0xFFFFu) >= d.cut ? f[0] * d.scale : 0.f;
  }
}

}  // namespace

// The arguments of a pass (false for a state that is missing or misaligned).
inline bool drop_args(const DropPlan& P, const int64_t* rng, DropArgs* d) {
  if (!rng || !aligned_to(rng, 8)) return false;
  d->rng = rng;
  d->cut = P.cut;
  d->site = P.site;
  d->scale = P.cut < 65536 ? 65536.f / (float)(65536 - P.cut) : 0.f;
  return true;
}

}  // namespace ttc
