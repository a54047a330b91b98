// Layer normalisation with a residual sum in front of it: forward, and
// backward with the reduction of the weight gradients.
//
// Both passes are bound by HBM: a row is read once, kept in registers (up to
// 16384 values across 1 to 32 warps), and written once.  Measured in bf16 (of the
// 6.8 TB/s that a copy reaches): forward with a residual 16384 x 768 19.8 us, 5.1
// TB/s; forward 32768 x 4096 105.5 us, 5.1 TB/s; f32 16384 x 4096 84 us, 6.4 TB/s
// (bf16 has twice the values a byte: 57 % of the issue slots, barriers in the
// rest); backward 16384 x 768 26 us, 3.9 TB/s, of which the sum of the partials 4;
// f32 4095 x 1023, whose values load one by one, 18.4 us, 2.7 TB/s.  16 x 64 takes
// 6.4 us a call, all of it the host's.  The variance is
// taken from the centred values in a second pass over the registers, so a
// large mean costs no accuracy.  The backward's sums over tokens (dgamma,
// dbeta) accumulate in registers over the rows a group of warps owns, each
// block leaves one partial row in the workspace, and a second kernel adds the
// partials in block order: no atomics, the same bits every time.
#include <cuda_bf16.h>

#include <cmath>
#include <new>

#include "tc_ptx.cuh"
#include "ttc.h"
#include "ttc_internal.h"

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

// The barrier of one group of W warps among the block's groups.
template <int W, int GROUPS>
__device__ __forceinline__ void group_sync(int group) {
  if (GROUPS == 1)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory");
}

// Sums of two values over the G = 32 W threads of a group, in a fixed order;
// every thread gets them.  `slot` alternates between shared rows so that one
// barrier a call is enough.
template <int W, int GROUPS>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 (*red)[32], int slot,
                                             int group) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (W == 1) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[slot][warp] = make_float2(a, b);
  group_sync<W, GROUPS>(group);
  float2 t = red[slot][group * W + (lane & (W - 1))];  // every W lanes hold the W shares
#pragma unroll
  for (int o = W / 2; o; o >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
  }
  return t;
}
// Of one value, by a block that is one group.
template <int W>
__device__ __forceinline__ float group_sum(float v, float2 (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[slot][warp].x = v;
  __syncthreads();
  v = red[slot][lane & (W - 1)].x;
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct NormFwdArgs {
  int64_t T;
  int N;
  float eps, n;  // n: N as a float; sums are divided, so that equal values have their own mean
  const void* x;
  const void* res;
  const float* gamma;
  const float* beta;
  void* sum;
  void* y;
  float2* stats;
  int gamma16, beta16;  // 16-byte aligned
};

struct NormBwdArgs {
  int64_t T;
  int N;
  float n;
  const void* s;
  const void* dy;
  const void* dsum;
  const float* gamma;
  const float2* stats;
  void* dx;
  float* parts;   // [gridDim.x][2 N]: this block's share of dgamma, then of dbeta
  float* dgamma;  // written directly when the grid is one block (parts unused)
  float* dbeta;
  int accumulate;
  int gamma16;  // 16-byte aligned
};

constexpr int kRowWarps = 8;  // rows side by side in a block when a warp holds a row

// A group of W warps holds ROWS rows of up to 32 W VEC CH values; groups stride
// over the rows, loading the next ones while the current ones are worked on.
template <typename T, int VEC, int CH, int W, bool RES, int ROWS>
__global__ void __launch_bounds__(W == 1 ? 32 * kRowWarps : 32 * W)
    norm_fwd_kernel(NormFwdArgs p) {
  using R = Raw<T, VEC>;
  constexpr int G = 32 * W;
  __shared__ float2 red[2][32];
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int per_block = W == 1 ? kRowWarps : 1;
  const int64_t step = (int64_t)gridDim.x * per_block;
  int64_t row = (int64_t)blockIdx.x * per_block + (W == 1 ? threadIdx.x >> 5 : 0);
  const int N = p.N;
  R rx[ROWS][CH], rr[ROWS][CH];
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](int k, int64_t r) {
    const T* x = static_cast<const T*>(p.x) + r * N;
    const T* s = static_cast<const T*>(p.res) + r * N;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * G + tid) * VEC;
      if (j < N) {
        rx[k][c] = *reinterpret_cast<const R*>(x + j);
        if (RES) rr[k][c] = *reinterpret_cast<const R*>(s + j);
      }
    }
  };
  // the sum of every row's share over the group
  auto sums = [&](float (&part)[ROWS], int slot) {
    if (ROWS == 2) {
      const float2 t = group_sum2<W, 1>(part[0], part[ROWS - 1], red, slot, 0);
      part[0] = t.x;
      part[ROWS - 1] = t.y;
    } else {
      part[0] = group_sum<W>(part[0], red, slot);
    }
  };
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if (row + k * step < p.T) fetch(k, row + k * step);
  for (; row < p.T; row += ROWS * step) {
    float v[ROWS][CH * VEC], part[ROWS], mean[ROWS], rstd[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int j = (c * G + tid) * VEC;
        if (j < N) {
          float* u = v[k] + c * VEC;
          rx[k][c].get(u);
          if (RES) {
            float a[VEC];
            rr[k][c].get(a);
            add<VEC>(u, a, u);
          }
          add_up<VEC>(sum, u);
        }
      }
      part[k] = sum.x + sum.y;
      const int64_t next = row + (ROWS + k) * step;
      if (next < p.T) fetch(k, next);
    }
    sums(part, 0);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      mean[k] = part[k] / p.n;
      float2 sum = make_float2(0.f, 0.f);
      float shift[VEC], d[VEC];
      fill<VEC>(-mean[k], shift);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((c * G + tid) * VEC < N) {
          add<VEC>(v[k] + c * VEC, shift, d);
          mul_up<VEC>(sum, d, d);
        }
      part[k] = sum.x + sum.y;
    }
    sums(part, 1);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      rstd[k] = 1.f / sqrtf(part[k] / p.n + p.eps);
      if (tid == 0 && p.stats && row + k * step < p.T)
        p.stats[row + k * step] = make_float2(mean[k], rstd[k]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * G + tid) * VEC;
      if (j < N) {
        float g[VEC], b[VEC];
        weights_at<VEC>(p.gamma, j, 1.f, p.gamma16, g);
        weights_at<VEC>(p.beta, j, 0.f, p.beta16, b);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
          if (k > 0 && row + k * step >= p.T) break;
          const int64_t at = (row + k * step) * N + j;
          const float* u = v[k] + c * VEC;
          R o;
          if (p.sum) {
            o.set(u);
            *reinterpret_cast<R*>(static_cast<T*>(p.sum) + at) = o;
          }
          float f[VEC], shift[VEC], by[VEC];
          fill<VEC>(-mean[k], shift);
          fill<VEC>(rstd[k], by);
          add<VEC>(u, shift, f);
          mul<VEC>(f, by, f);
          fma<VEC>(f, g, b, f);
          o.set(f);
          *reinterpret_cast<R*>(static_cast<T*>(p.y) + at) = o;
        }
      }
    }
  }
}

// dgamma[j] or dbeta[j] from its sum
__device__ __forceinline__ void put_sum(float* out, int j, float v, int accumulate) {
  if (out) out[j] = accumulate ? out[j] + v : v;
}

// Groups of W warps side by side in a block of the backward.
__host__ __device__ constexpr int bwd_groups(int W) { return W < kRowWarps ? kRowWarps / W : 1; }

template <typename T, int VEC, int CH, int W>
__global__ void __launch_bounds__(32 * W * bwd_groups(W), W <= 8 ? 2 : 1)
    norm_bwd_kernel(NormBwdArgs p) {
  using R = Raw<T, VEC>;
  constexpr int G = 32 * W, E = CH * VEC, GROUPS = bwd_groups(W);
  __shared__ float2 red[2][32];
  __shared__ float cross[GROUPS > 1 ? 2 * G * E : 1];
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t row = (int64_t)blockIdx.x * GROUPS + group;
  const int N = p.N;
  R rs[CH], rd[CH], ru[CH];
  float2 st = make_float2(0.f, 0.f);
  float dg[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](int64_t r) {
    const T* s = static_cast<const T*>(p.s) + r * N;
    const T* d = static_cast<const T*>(p.dy) + r * N;
    const T* u = static_cast<const T*>(p.dsum) + r * N;
    st = p.stats[r];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * G + tid) * VEC;
      if (j < N) {
        rs[c] = *reinterpret_cast<const R*>(s + j);
        rd[c] = *reinterpret_cast<const R*>(d + j);
        if (p.dsum) ru[c] = *reinterpret_cast<const R*>(u + j);
      }
    }
  };
  int flip = 0;
  if (row < p.T) fetch(row);
  for (; row < p.T; row += step, flip ^= 1) {
    float h[E], g[E];  // normalised values; dy gamma
    R us[CH];
    float2 sg = make_float2(0.f, 0.f), sgh = sg;
    const float2 ms = st;
    float shift[VEC], by[VEC];
    fill<VEC>(-ms.x, shift);
    fill<VEC>(ms.y, by);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * G + tid) * VEC;
      us[c] = ru[c];
      if (j < N) {
        float w[VEC];
        weights_at<VEC>(p.gamma, j, 1.f, p.gamma16, w);
        float *hc = h + c * VEC, *gc = g + c * VEC;
        rs[c].get(hc);
        rd[c].get(gc);
        add<VEC>(hc, shift, hc);
        mul<VEC>(hc, by, hc);
        fma<VEC>(gc, hc, dg + c * VEC, dg + c * VEC);
        add<VEC>(gc, db + c * VEC, db + c * VEC);
        mul<VEC>(gc, w, gc);
        add_up<VEC>(sg, gc);
        mul_up<VEC>(sgh, gc, hc);
      }
    }
    if (row + step < p.T) fetch(row + step);
    const float2 t = group_sum2<W, GROUPS>(sg.x + sg.y, sgh.x + sgh.y, red, flip, group);
    float a[VEC], b[VEC];
    fill<VEC>(-(t.x / p.n), a);
    fill<VEC>(-(t.y / p.n), b);
    T* dx = static_cast<T*>(p.dx) + row * N;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * G + tid) * VEC;
      if (j < N) {
        float f[VEC];
        add<VEC>(g + c * VEC, a, f);
        fma<VEC>(h + c * VEC, b, f, f);
        if (p.dsum) {
          float u[VEC];
          us[c].get(u);
          fma<VEC>(f, by, u, f);
        } else {
          mul<VEC>(f, by, f);
        }
        R o;
        o.set(f);
        *reinterpret_cast<R*>(dx + j) = o;
      }
    }
  }
  // this block's share of the token sums: the groups' in order
  if (GROUPS > 1) {
    for (int k = 0; k < GROUPS; ++k) {
      if (group == k) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (k > 0) dg[i] += cross[i * G + tid], db[i] += cross[(E + i) * G + tid];
          cross[i * G + tid] = dg[i];
          cross[(E + i) * G + tid] = db[i];
        }
      }
      __syncthreads();
    }
    if (group != GROUPS - 1) return;
  }
  const bool last = gridDim.x == 1;
  float* pg = p.parts + (size_t)blockIdx.x * 2 * N;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = (c * G + tid) * VEC;
    if (j < N) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (last) {
          put_sum(p.dgamma, j + i, dg[c * VEC + i], p.accumulate);
          put_sum(p.dbeta, j + i, db[c * VEC + i], p.accumulate);
        } else {
          pg[j + i] = dg[c * VEC + i];
          pg[N + j + i] = db[c * VEC + i];
        }
      }
    }
  }
}

// Sums of the partial rows in row order: 32 columns a block, 32 row slices
// side by side, then the slices in order.
__global__ void __launch_bounds__(1024)
    norm_reduce_kernel(const float* parts, int nparts, int N, float* dgamma, float* dbeta,
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

// ---- rows wider than the registers of a block ----------------------------------
constexpr int kWideThreads = 1024;

template <typename T>
__device__ __forceinline__ float wide_at(const void* p, int64_t i) {
  float f;
  reinterpret_cast<const Raw<T, 1>*>(p)[i].get(&f);
  return f;
}
template <typename T>
__device__ __forceinline__ void wide_put(void* p, int64_t i, float f) {
  reinterpret_cast<Raw<T, 1>*>(p)[i].set(&f);
}

// One block a row, the row read three times (from L2 after the first).
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_fwd_wide_kernel(NormFwdArgs p) {
  __shared__ float2 red[2][32];
  pdl_wait();
  pdl_trigger();
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t o = row * p.N;
    auto value = [&](int j) {
      return wide_at<T>(p.x, o + j) + (p.res ? wide_at<T>(p.res, o + j) : 0.f);
    };
    float part = 0.f;
    for (int j = threadIdx.x; j < p.N; j += kWideThreads) part += value(j);
    const float mean = group_sum<32>(part, red, 0) / p.n;
    part = 0.f;
    for (int j = threadIdx.x; j < p.N; j += kWideThreads) {
      const float d = value(j) - mean;
      part = fmaf(d, d, part);
    }
    const float rstd = 1.f / sqrtf(group_sum<32>(part, red, 1) / p.n + p.eps);
    if (threadIdx.x == 0 && p.stats) p.stats[row] = make_float2(mean, rstd);
    for (int j = threadIdx.x; j < p.N; j += kWideThreads) {
      const float v = value(j);
      if (p.sum) wide_put<T>(p.sum, o + j, v);
      wide_put<T>(p.y, o + j, fmaf((v - mean) * rstd, p.gamma ? __ldg(p.gamma + j) : 1.f,
                                   p.beta ? __ldg(p.beta + j) : 0.f));
    }
  }
}

// dgamma and dbeta of wide rows: a thread a column, rows split over gridDim.y
// (before the dx kernel, which may overwrite dy).
template <typename T>
__global__ void __launch_bounds__(256) norm_cols_wide_kernel(NormBwdArgs p) {
  pdl_wait();
  pdl_trigger();
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= p.N) return;
  float g = 0.f, b = 0.f;
  for (int64_t r = blockIdx.y; r < p.T; r += gridDim.y) {
    const float2 st = p.stats[r];
    const float d = wide_at<T>(p.dy, r * p.N + j);
    g = fmaf(d, (wide_at<T>(p.s, r * p.N + j) - st.x) * st.y, g);
    b += d;
  }
  p.parts[(size_t)blockIdx.y * 2 * p.N + j] = g;
  p.parts[(size_t)blockIdx.y * 2 * p.N + p.N + j] = b;
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_dx_wide_kernel(NormBwdArgs p) {
  __shared__ float2 red[2][32];
  pdl_wait();
  pdl_trigger();
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t o = row * p.N;
    const float2 st = p.stats[row];
    auto h = [&](int j) { return (wide_at<T>(p.s, o + j) - st.x) * st.y; };
    auto g = [&](int j) {
      return wide_at<T>(p.dy, o + j) * (p.gamma ? __ldg(p.gamma + j) : 1.f);
    };
    float sg = 0.f, sgh = 0.f;
    for (int j = threadIdx.x; j < p.N; j += kWideThreads) {
      const float v = g(j);
      sg += v;
      sgh = fmaf(v, h(j), sgh);
    }
    const float a = group_sum<32>(sg, red, 0) / p.n;
    const float b = group_sum<32>(sgh, red, 1) / p.n;
    for (int j = threadIdx.x; j < p.N; j += kWideThreads) {
      const float u = p.dsum ? wide_at<T>(p.dsum, o + j) : 0.f;
      wide_put<T>(p.dx, o + j, st.y * (g(j) - a - h(j) * b) + u);
    }
  }
}

// ---- dispatch --------------------------------------------------------------------
constexpr int kMaxRegRow = 16384;  // widest row held in the registers of a block

// Warps of a row, by its width.  Forward: 1024 values in one warp, else 512 a
// warp.  Backward: 512, since its accumulators take as many registers again
// (16384 x 768 bf16: two warps a row 26 us, one 33 us), and 256 where the values
// come one by one, an address and a predicate each (4095 x 1023 f32: four warps a
// row 18 us, two 31 us).
int fwd_warps(int64_t N) {
  if (N <= 1024) return 1;
  int w = 4;
  while (N > 512 * w) w *= 2;
  return w;
}
int bwd_warps(int64_t N) {
  const int64_t per = N % 4 == 0 || N > 8192 ? 512 : 256;
  int w = 1;
  while (N > per * w) w *= 2;
  return w;
}

// Blocks of the backward: enough to keep an SM's registers in use, no more
// than there are rows, and one block when a second launch for the partial
// sums would cost more than its few rows (one block against two launches: 32 x 768
// 8.4 and 9.6 us, 64 x 768 14.0 and 9.7 us, 64 x 64 6.9 and 9.5 us).
int64_t bwd_blocks(int64_t N, int64_t T) {
  if (N > kMaxRegRow) return T < 64 ? (T < 1 ? 1 : T) : 64;  // row slices of the column sums
  const int rows = bwd_groups(bwd_warps(N));
  const int64_t b = (T + rows - 1) / rows;
  if (T <= 8 * rows) return 1;
  const int64_t most = (int64_t)device_sms() * (bwd_warps(N) <= 8 ? 2 : 1);
  return b < most ? b : most;
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <typename T, int VEC, int CH, int W, bool RES, int ROWS>
cudaError_t fwd_launch(const NormFwdArgs& a, cudaStream_t st) {
  constexpr int rows = W == 1 ? kRowWarps : 1, threads = W == 1 ? 32 * kRowWarps : 32 * W;
  auto kernel = norm_fwd_kernel<T, VEC, CH, W, RES, ROWS>;
  // as many blocks as stay on the SMs, each taking rows in turn
  static PerDevice once;
  static int fit[kMaxDevices] = {};
  int dev = 0;
  const cudaError_t e = once.get([&] {
    int d = 0, n = 0;
    cudaError_t r = cudaGetDevice(&d);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
    fit[d] = n > 0 ? n : 1;
    return r;
  });
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
  const int64_t need = (a.T + rows - 1) / rows, most = (int64_t)device_sms() * fit[dev];
  return launch_ex(kernel, dim3((unsigned)(need < most ? need : most)), dim3(threads), 0, st,
                   false, a);
}
template <typename T, int VEC, int CH, int W>
cudaError_t fwd_go(const NormFwdArgs& a, cudaStream_t st) {
  // Without a residual, and with rows enough for every block, two rows at a time:
  // the weights are read from L1 once for both (their 8 bytes a value, against 2
  // from memory, took 78 % of the L1's rate) and each barrier serves both.  bf16,
  // one -> two rows: 32768 x 4096 119 -> 108 us, 65536 x 2048 115 -> 95, 16384 x
  // 8192 126 -> 116; one warp a row (65536 x 1024) 58 -> 62, 32 warps (8192 x
  // 16384) 134 -> 150, with a residual (16384 x 4096) 89 -> 98: registers.
  if constexpr (VEC < 8) {
    if constexpr (VEC > 1 && W >= 4 && W <= 16) {
      if (!a.res && a.T >= 16 * (int64_t)device_sms())
        return fwd_launch<T, VEC, CH, W, false, 2>(a, st);
    }
    if (!a.res) return fwd_launch<T, VEC, CH, W, false, 1>(a, st);
  }
  return fwd_launch<T, VEC, CH, W, true, 1>(a, st);
}

template <typename T, int V>
cudaError_t fwd_pick(const NormFwdArgs& a, cudaStream_t st) {
  const int N = a.N;
  if (N > kMaxRegRow) {
    const int64_t most = 2 * (int64_t)device_sms();
    return launch_ex(norm_fwd_wide_kernel<T>, dim3((unsigned)(a.T < most ? a.T : most)),
                     dim3(kWideThreads), 0, st, false, a);
  }
  const int w = fwd_warps(N);
  const int e = (N + 32 * w - 1) / (32 * w);  // values a thread
  if (w == 1) {
    if (e <= 8) return fwd_go<T, V, 8 / V, 1>(a, st);
    if (e <= 16) return fwd_go<T, V, 16 / V, 1>(a, st);
    if (e <= 24) return fwd_go<T, V, 24 / V, 1>(a, st);
    return fwd_go<T, V, 32 / V, 1>(a, st);
  }
  if (w == 4) return fwd_go<T, V, 16 / V, 4>(a, st);
  if (w == 8) return fwd_go<T, V, 16 / V, 8>(a, st);
  return w == 16 ? fwd_go<T, V, 16 / V, 16>(a, st) : fwd_go<T, V, 16 / V, 32>(a, st);
}

template <typename T, int VEC, int CH, int W>
cudaError_t bwd_go(const NormBwdArgs& a, int64_t blocks, cudaStream_t st) {
  return launch_ex(norm_bwd_kernel<T, VEC, CH, W>, dim3((unsigned)blocks),
                   dim3(32 * W * bwd_groups(W)), 0, st, false, a);
}

template <typename T, int V>
cudaError_t bwd_pick(const NormBwdArgs& a, int64_t blocks, cudaStream_t st) {
  const int N = a.N;
  constexpr int E = V == 1 ? 8 : 16;  // values a thread
  switch (bwd_warps(N)) {
    case 1:
      if (V > 1 && N <= 256) return bwd_go<T, V, 8 / V, 1>(a, blocks, st);
      return bwd_go<T, V, E / V, 1>(a, blocks, st);
    case 2:
      if (V > 1 && N <= 768) return bwd_go<T, V, 12 / V, 2>(a, blocks, st);
      return bwd_go<T, V, E / V, 2>(a, blocks, st);
    case 4: return bwd_go<T, V, E / V, 4>(a, blocks, st);
    case 8: return bwd_go<T, V, E / V, 8>(a, blocks, st);
    case 16: return bwd_go<T, V, E / V, 16>(a, blocks, st);
    default: return bwd_go<T, V, 16 / V, 32>(a, blocks, st);
  }
}

template <typename T>
cudaError_t bwd_wide(const NormBwdArgs& a, int64_t slices, cudaStream_t st) {
  cudaError_t e = launch_ex(norm_cols_wide_kernel<T>,
                            dim3((unsigned)((a.N + 255) / 256), (unsigned)slices), dim3(256), 0,
                            st, false, a);
  if (e != cudaSuccess) return e;
  const int64_t most = 2 * (int64_t)device_sms();
  return launch_ex(norm_dx_wide_kernel<T>, dim3((unsigned)(a.T < most ? a.T : most)),
                   dim3(kWideThreads), 0, st, false, a);
}

}  // namespace

size_t norm_workspace_bytes(const NormPlan& P, int64_t T) {
  return (size_t)bwd_blocks(P.N, T) * 2 * (size_t)P.N * sizeof(float);
}

}  // namespace ttc

using namespace ttc;

extern "C" {

tt_status tt_norm_plan(const tt_norm_desc* desc, tt_plan_t** out) {
  if (!out) return TT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || desc->N < 1 || !std::isfinite(desc->eps) || !(desc->eps > 0.f) ||
      (desc->flags & ~TT_ACCUMULATE))
    return TT_ERR_INVALID_ARG;
  if (desc->act != TT_DT_F32 && desc->act != TT_DT_BF16 && desc->act != TT_DT_E4M3)
    return TT_ERR_INVALID_ARG;
  if (desc->act == TT_DT_E4M3 || desc->N > (1 << 20)) return TT_ERR_UNSUPPORTED;
  tt_plan_s* p = new (std::nothrow) tt_plan_s();
  if (!p) return TT_ERR_INVALID_ARG;
  p->kind = 4;
  p->norm.N = desc->N;
  p->norm.eps = desc->eps;
  p->norm.act = desc->act;
  p->norm.flags = desc->flags;
  *out = p;
  return TT_OK;
}

tt_status tt_norm_forward(const tt_plan_t* plan, int64_t T, const void* x, const void* res,
                          const float* gamma, const float* beta, void* sum, void* y,
                          float* stats, void* stream) {
  if (!plan || plan->kind != 4 || T < 0) return TT_ERR_INVALID_ARG;
  if (T == 0) return TT_OK;
  if (!x || !y || !aligned_to(x, 16) || !aligned_to(y, 16) || !aligned_to(res, 16) ||
      !aligned_to(sum, 16) || !aligned_to(gamma, 4) || !aligned_to(beta, 4) ||
      !aligned_to(stats, 8))
    return TT_ERR_INVALID_ARG;
  const NormPlan& P = plan->norm;
  NormFwdArgs a;
  a.T = T;
  a.N = (int)P.N;
  a.eps = P.eps;
  a.n = (float)P.N;
  a.x = x;
  a.res = res;
  a.gamma = gamma;
  a.beta = beta;
  a.sum = sum;
  a.y = y;
  a.stats = reinterpret_cast<float2*>(stats);
  a.gamma16 = aligned_to(gamma, 16);
  a.beta16 = aligned_to(beta, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Rows start aligned to four or eight values only when those divide the width.
  // Eight (16 bytes) only with a residual, whose four tensors are most of the loads
  // and stores: 16384 x 768 21.6 -> 19.8 us, 32768 x 2048 88 -> 82; without one the
  // weights are (32 bytes a lane, half of each line of the L1 a load): 32768 x 4096
  // 105 -> 142, 65536 x 1024 57 -> 60.
  prof_begin(kPhElem, st);
  const cudaError_t e =
      P.act == TT_DT_BF16
          ? (res && P.N % 8 == 0 ? fwd_pick<__nv_bfloat16, 8>(a, st)
             : P.N % 4 == 0      ? fwd_pick<__nv_bfloat16, 4>(a, st)
                                 : fwd_pick<__nv_bfloat16, 1>(a, st))
          : (P.N % 4 == 0 ? fwd_pick<float, 4>(a, st) : fwd_pick<float, 1>(a, st));
  prof_end(kPhElem, st);
  count_launches(1);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

tt_status tt_norm_backward(const tt_plan_t* plan, int64_t T, const void* s, const void* dy,
                           const void* dsum, const float* gamma, const float* stats, void* dx,
                           float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                           void* stream) {
  if (!plan || plan->kind != 4 || T < 0) return TT_ERR_INVALID_ARG;
  const NormPlan& P = plan->norm;
  const int acc = (P.flags & TT_ACCUMULATE) != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!aligned_to(dgamma, 4) || !aligned_to(dbeta, 4)) return TT_ERR_INVALID_ARG;
  if (T == 0) {
    if (acc) return TT_OK;
    const size_t n = (size_t)P.N * sizeof(float);
    if (dgamma && cudaMemsetAsync(dgamma, 0, n, st) != cudaSuccess) return TT_ERR_CUDA;
    if (dbeta && cudaMemsetAsync(dbeta, 0, n, st) != cudaSuccess) return TT_ERR_CUDA;
    return TT_OK;
  }
  if (!s || !dy || !stats || !dx || !aligned_to(s, 16) || !aligned_to(dy, 16) ||
      !aligned_to(dsum, 16) || !aligned_to(dx, 16) || !aligned_to(gamma, 4) ||
      !aligned_to(stats, 8))
    return TT_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256) || ws_bytes < norm_workspace_bytes(P, T))
    return TT_ERR_WORKSPACE;
  const int64_t blocks = bwd_blocks(P.N, T);
  const bool wide = P.N > kMaxRegRow;
  NormBwdArgs a;
  a.T = T;
  a.N = (int)P.N;
  a.n = (float)P.N;
  a.s = s;
  a.dy = dy;
  a.dsum = dsum;
  a.gamma = gamma;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.dx = dx;
  a.parts = static_cast<float*>(ws);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.accumulate = acc;
  a.gamma16 = aligned_to(gamma, 16);
  prof_begin(kPhElem, st);
  cudaError_t e;
  if (P.act == TT_DT_BF16)
    e = wide           ? bwd_wide<__nv_bfloat16>(a, blocks, st)
        : P.N % 4 == 0 ? bwd_pick<__nv_bfloat16, 4>(a, blocks, st)
                       : bwd_pick<__nv_bfloat16, 1>(a, blocks, st);
  else
    e = wide           ? bwd_wide<float>(a, blocks, st)
        : P.N % 4 == 0 ? bwd_pick<float, 4>(a, blocks, st)
                       : bwd_pick<float, 1>(a, blocks, st);
  count_launches(wide ? 2 : 1);
  if (e == cudaSuccess && (wide || blocks > 1) && (dgamma || dbeta)) {
    e = launch_ex(norm_reduce_kernel, dim3((unsigned)((2 * P.N + 31) / 32)), dim3(1024), 0, st,
                  false, (const float*)a.parts, (int)blocks, a.N, dgamma, dbeta, acc);
    count_launches(1);
  }
  prof_end(kPhElem, st);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // extern "C"
