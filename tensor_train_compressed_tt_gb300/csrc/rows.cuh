// Rows of activations in registers: vector loads and stores, weights read through
// L1, and the sum of the blocks' shares of two weight gradients in block order.
// Shared by the kernels between the TT layers.
#pragma once

#include <cuda_bf16.h>

#include "attn.h"
#include "tc_ptx.cuh"

namespace ttc {
namespace {

// ---- vector loads and stores -------------------------------------------------
// VEC consecutive elements of type T as they lie in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 v;
  __device__ void get(float* f) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
  __device__ void set(const float* f) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Raw<float, 8> {
  float4 v[2];
  __device__ void get(float* f) const {
    f[0] = v[0].x, f[1] = v[0].y, f[2] = v[0].z, f[3] = v[0].w;
    f[4] = v[1].x, f[5] = v[1].y, f[6] = v[1].z, f[7] = v[1].w;
  }
  __device__ void set(const float* f) {
    v[0] = make_float4(f[0], f[1], f[2], f[3]);
    v[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ void get(float* f) const { f[0] = v.x, f[1] = v.y; }
  __device__ void set(const float* f) { v = make_float2(f[0], f[1]); }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ void get(float* f) const { f[0] = v; }
  __device__ void set(const float* f) { v = f[0]; }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 v;
  __device__ void get(float* f) const {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // a bf16 is the upper half of its f32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float* f) {
    v = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float* f) {
    v = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7]));
  }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ void get(float* f) const {
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xFFFF0000u);
  }
  __device__ void set(const float* f) { v = pack_bf16(f[0], f[1]); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ void get(float* f) const { f[0] = __bfloat162float(v); }
  __device__ void set(const float* f) { v = __float2bfloat16_rn(f[0]); }
};

// VEC values of gamma or beta (`other` where there is none).  Four in one load
// when the array is 16-byte aligned: a warp's loads then cover whole lines of
// the L1, which holds the array for every row but the first.
template <int VEC>
__device__ __forceinline__ void weights_at(const float* w, int j, float other, bool aligned,
                                           float* f) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = other;
  } else if (VEC >= 4 && aligned) {
#pragma unroll
    for (int i = 0; i + 3 < VEC; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + j + i));
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __ldg(w + j + i);
  }
}

// VEC values at once, two an instruction where they come in pairs.
template <int VEC>
__device__ __forceinline__ void add_up(float2& sum, const float* v) {  // sum += v
  if (VEC == 1) sum.x += v[0];
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2) sum = __fadd2_rn(sum, make_float2(v[i], v[i + 1]));
}
template <int VEC>
__device__ __forceinline__ void mul_up(float2& sum, const float* a, const float* b) {  // += a b
  if (VEC == 1) sum.x = fmaf(a[0], b[0], sum.x);
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2)
    sum = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), sum);
}
template <int VEC>
__device__ __forceinline__ void add(const float* a, const float* b, float* o) {  // o = a + b
  if (VEC == 1) o[0] = a[0] + b[0];
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2) {
    const float2 t = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    o[i] = t.x, o[i + 1] = t.y;
  }
}
template <int VEC>
__device__ __forceinline__ void mul(const float* a, const float* b, float* o) {  // o = a b
  if (VEC == 1) o[0] = a[0] * b[0];
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2) {
    const float2 t = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    o[i] = t.x, o[i + 1] = t.y;
  }
}
template <int VEC>
__device__ __forceinline__ void fma(const float* a, const float* b, const float* c,
                                    float* o) {  // o = a b + c
  if (VEC == 1) o[0] = fmaf(a[0], b[0], c[0]);
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2) {
    const float2 t = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]),
                                make_float2(c[i], c[i + 1]));
    o[i] = t.x, o[i + 1] = t.y;
  }
}
template <int VEC>
__device__ __forceinline__ void fill(float x, float* o) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = x;
}

// 16 bytes to shared memory, awaited with cp.async.wait_group.
__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(su32(to)), "l"(from) : "memory");
}

// dgamma[j] or dbeta[j] from its sum
__device__ __forceinline__ void put_sum(float* out, int j, float v, int accumulate) {
  if (out) out[j] = accumulate ? out[j] + v : v;
}

// Sums of partial rows of 2 N values (a share of two weight gradients each) in row
// order: 32 columns a block, 32 row slices side by side, then the slices in order.
__global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float* parts, int nparts, int N, float* dgamma, float* dbeta,
                     int accumulate) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (col < 2 * N)
    for (int r = slice; r < nparts; r += 32) v += parts[(size_t)r * 2 * N + col];
  acc[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && col < 2 * N) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += acc[k][lane];
    if (col < N)
      put_sum(dgamma, col, t, accumulate);
    else
      put_sum(dbeta, col - N, t, accumulate);
  }
}

}  // namespace
}  // namespace ttc
