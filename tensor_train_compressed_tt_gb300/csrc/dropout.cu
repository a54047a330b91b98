// Dropout of a dense tensor, with an optional residual sum: the same kernel is its
// own backward pass (of the gradient, without the residual).
//
// Bound by HBM: two or three values of traffic an element against some ten
// instructions of the generator.
#include <cmath>
#include <new>

#include "dropout.cuh"
#include "ttc.h"
#include "ttc_internal.h"

namespace ttc {
namespace {

constexpr int kThreads = 256;

// A thread takes kSide groups of eight elements a block's width apart, then the grid's
// next ones, which are loaded while the generator works on the current ones.  One group
// at a time had 16 KB of loads in flight an SM in bf16: 32768 x 4096 102 us against 85.
// In f32 a group is twice the bytes and one is enough: 4095 x 1023 with a residual 9.0 us
// against 10.3.
template <typename T>
constexpr int side_by_side = sizeof(T) == 2 ? 2 : 1;

template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) drop_kernel(int64_t n, const T* x, const T* res, T* y,
                                                        DropArgs d) {
  constexpr int kSide = side_by_side<T>;
  pdl_wait();
  pdl_trigger();
  DropKey key;
  key.read(d);
  const int64_t step = (int64_t)gridDim.x * kThreads * kSide, groups = n >> 3;
  int64_t first = (int64_t)blockIdx.x * kThreads * kSide + threadIdx.x;
  using R = Raw<T, 8>;
  R rx[kSide], rr[RES ? kSide : 1];
  auto fetch = [&](int64_t g) {
#pragma unroll
    for (int k = 0; k < kSide; ++k)
      if (g + k * kThreads < groups) {
        rx[k] = *reinterpret_cast<const R*>(x + 8 * (g + k * kThreads));
        if constexpr (RES) rr[k] = *reinterpret_cast<const R*>(res + 8 * (g + k * kThreads));
      }
  };
  fetch(first);
  for (; first < groups; first += step) {
    float f[kSide][8], r[RES ? kSide : 1][8];
    int64_t group[kSide];
#pragma unroll
    for (int k = 0; k < kSide; ++k) {
      rx[k].get(f[k]);
      if constexpr (RES) rr[k].get(r[k]);
      group[k] = first + k * kThreads;
    }
    if (first + step < groups) fetch(first + step);
    uint4 w[kSide];
    key.words(group, d.site, w);
#pragma unroll
    for (int k = 0; k < kSide; ++k) {
      drop<8>(w[k], d, 0, f[k]);
      if constexpr (RES) add<8>(f[k], r[k], f[k]);
      R o;
      o.set(f[k]);
      if (group[k] < groups) *reinterpret_cast<R*>(y + 8 * group[k]) = o;
    }
  }
  // the last elements, fewer than eight
  if (blockIdx.x == 0 && threadIdx.x < (n & 7)) {
    const int64_t i = (groups << 3) + threadIdx.x;
    float f, r = 0.f;
    reinterpret_cast<const Raw<T, 1>*>(x)[i].get(&f);
    if (RES) reinterpret_cast<const Raw<T, 1>*>(res)[i].get(&r);
    drop<1>(key, d, i, &f);
    f += r;
    reinterpret_cast<Raw<T, 1>*>(y)[i].set(&f);
  }
}

template <typename T>
cudaError_t drop_go(int64_t n, const void* x, const void* res, void* y, const DropArgs& d,
                    cudaStream_t st) {
  constexpr int kSide = side_by_side<T>;
  const int64_t need = ((n >> 3) + kThreads * kSide - 1) / (kThreads * kSide);
  const int64_t most = (int64_t)device_sms() * 8;
  const dim3 grid((unsigned)(need < 1 ? 1 : need < most ? need : most));
  const T *tx = static_cast<const T*>(x), *tr = static_cast<const T*>(res);
  return res ? launch_ex(drop_kernel<T, true>, grid, dim3(kThreads), 0, st, false, n, tx, tr,
                         static_cast<T*>(y), d)
             : launch_ex(drop_kernel<T, false>, grid, dim3(kThreads), 0, st, false, n, tx, tr,
                         static_cast<T*>(y), d);
}

}  // namespace
}  // namespace ttc

using namespace ttc;

extern "C" {

tt_status tt_dropout_plan(const tt_dropout_desc* desc, tt_plan_t** out) {
  if (!out) return TT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || !(desc->p >= 0.f) || !(desc->p <= 1.f) || desc->site < 0 || desc->site > 0xFFFF)
    return TT_ERR_INVALID_ARG;
  if (desc->act != TT_DT_F32 && desc->act != TT_DT_BF16 && desc->act != TT_DT_E4M3)
    return TT_ERR_INVALID_ARG;
  if (desc->act == TT_DT_E4M3) return TT_ERR_UNSUPPORTED;
  tt_plan_s* p = new (std::nothrow) tt_plan_s();
  if (!p) return TT_ERR_INVALID_ARG;
  p->kind = 7;
  p->drop.cut = (uint32_t)std::floor((double)desc->p * 65536. + 0.5);
  p->drop.site = (uint32_t)desc->site;
  p->drop.act = desc->act;
  *out = p;
  return TT_OK;
}

tt_status tt_dropout(const tt_plan_t* plan, int64_t n, const int64_t* rng, const void* x,
                     const void* res, void* y, void* stream) {
  if (!plan || plan->kind != 7 || n < 0 || n >= (int64_t)1 << 48) return TT_ERR_INVALID_ARG;
  if (n == 0) return TT_OK;
  DropArgs d;
  if (!x || !y || !aligned_to(x, 16) || !aligned_to(res, 16) || !aligned_to(y, 16) ||
      !drop_args(plan->drop, rng, &d))
    return TT_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  const cudaError_t e = plan->drop.act == TT_DT_BF16
                            ? drop_go<__nv_bfloat16>(n, x, res, y, d, st)
                            : drop_go<float>(n, x, res, y, d, st);
  prof_end(kPhElem, st);
  count_launches(1);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // extern "C"
