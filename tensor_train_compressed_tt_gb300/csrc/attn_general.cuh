// General attention kernels: f32 activations, and bf16 ones whose head width,
// strides or alignment the tensor-core kernels do not take.  Exact fp32
// arithmetic (no tensor-core product holds fp32's error), tiles of 16 MT rows
// in shared memory, 256 threads with MT x MT scores each.
//
// f32, 8 heads, causal: 8 sequences of 2048, heads of 32: forward 662 us, backward
// 1928 us, 26 and 22 TFLOP/s (31 of the seven products done, where a gradient needs
// five) of the fp32 pipes' 80, bound by the reads of shared
// memory that feed them (8 of 16 bytes for 64 multiply-adds); 32 sequences of
// 33 to 97: backward 45 us, the latency of loads and barriers of blocks that have
// two or three tiles each.
#pragma once

#include "attn_seq.cuh"

namespace ttc {
namespace {

constexpr int kGenThreads = 256;

template <typename T>
__device__ __forceinline__ float as_f32(T v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <int DP, int MT>
struct GenShape {
  static constexpr int BT = 16 * MT;   // rows of a tile
  static constexpr int LD = DP + 4;    // pitch: float4 reads of 16 rows hit different banks
  static constexpr int LP = BT + 4;
  static constexpr int TILE = BT * LD;
  static constexpr int DC = (DP + 63) / 64;  // float4 column groups a thread owns
  // heads of 32: the 16 lanes of a row are two sets of 8, with half the sum each
  static constexpr int SETS = DP < 64 ? 64 / DP : 1, LANES = 16 / SETS;
};

// Four elements of a row as floats.
template <typename T>
__device__ __forceinline__ float4 gen_four(const T* x);
template <>
__device__ __forceinline__ float4 gen_four<float>(const float* x) {
  return *reinterpret_cast<const float4*>(x);
}
template <>
__device__ __forceinline__ float4 gen_four<__nv_bfloat16>(const __nv_bfloat16* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(x);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

// Rows r0 .. r0 + BT - 1 of head h (zero past `n` rows and past the head's
// width) into a tile, four elements a load where the tensor's alignment lets it.
template <typename T, int DP, int MT>
__device__ __forceinline__ void gen_load(float* tile, const Heads& x, int64_t base, int h, int r0,
                                         int n, int dim) {
  using S = GenShape<DP, MT>;
  const bool wide = ((reinterpret_cast<uintptr_t>(x.p) / sizeof(T)) | (uintptr_t)x.row |
                     (uintptr_t)x.head | (uintptr_t)dim) % 4 == 0;
  constexpr int Q = DP / 4;
#pragma unroll
  for (int i = 0; i < S::BT * Q; i += kGenThreads) {
    const int e = i + threadIdx.x, r = e / Q, c = e % Q * 4;
    if (S::BT * Q % kGenThreads && e >= S::BT * Q) break;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < n && c < dim) {
      const T* at = x.at<const T>(base + r0 + r, h) + c;
      if (wide) {
        v = gen_four<T>(at);
      } else {
        v.x = as_f32<T>(at[0]);
        if (c + 1 < dim) v.y = as_f32<T>(at[1]);
        if (c + 2 < dim) v.z = as_f32<T>(at[2]);
        if (c + 3 < dim) v.w = as_f32<T>(at[3]);
      }
    }
    *reinterpret_cast<float4*>(tile + r * S::LD + c) = v;
  }
}

// out[a][b] = sum_c A[ty MT + a][c] B[tx + 16 b][c]
template <int DP, int MT>
__device__ __forceinline__ void gen_dot(const float* A, const float* B, int ty, int tx,
                                        float (&out)[MT][MT]) {
  using S = GenShape<DP, MT>;
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b) out[a][b] = 0.f;
#pragma unroll 4
  for (int c = 0; c < DP; c += 4) {
    float4 x[MT], y[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
      x[a] = *reinterpret_cast<const float4*>(A + (ty * MT + a) * S::LD + c);
#pragma unroll
    for (int b = 0; b < MT; ++b)
      y[b] = *reinterpret_cast<const float4*>(B + (tx + 16 * b) * S::LD + c);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < MT; ++b) {
        out[a][b] = fmaf(x[a].x, y[b].x, out[a][b]);
        out[a][b] = fmaf(x[a].y, y[b].y, out[a][b]);
        out[a][b] = fmaf(x[a].z, y[b].z, out[a][b]);
        out[a][b] = fmaf(x[a].w, y[b].w, out[a][b]);
      }
  }
}

// acc[a][4 g + i] += sum_j W[ty MT + a][j] V[j][(16 g + lane) 4 + i], j < n rounded up
// to fours (rows of V past n and their weights are zero); a lane set's share of it.
template <int DP, int MT>
__device__ __forceinline__ void gen_acc(const float* W, const float* V, int n, int ty, int tx,
                                        float (&acc)[MT][4 * GenShape<DP, MT>::DC]) {
  using S = GenShape<DP, MT>;
  const int lane = tx % S::LANES, set = tx / S::LANES;
#pragma unroll 1
  for (int j = 4 * set; j < n; j += 4 * S::SETS) {
    float4 w[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
      w[a] = *reinterpret_cast<const float4*>(W + (ty * MT + a) * S::LP + j);
#pragma unroll
    for (int g = 0; g < S::DC; ++g) {
      const float* col = V + j * S::LD + (16 * g + lane) * 4;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 v = *reinterpret_cast<const float4*>(col + u * S::LD);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const float x = u == 0 ? w[a].x : u == 1 ? w[a].y : u == 2 ? w[a].z : w[a].w;
          acc[a][4 * g + 0] = fmaf(x, v.x, acc[a][4 * g + 0]);
          acc[a][4 * g + 1] = fmaf(x, v.y, acc[a][4 * g + 1]);
          acc[a][4 * g + 2] = fmaf(x, v.z, acc[a][4 * g + 2]);
          acc[a][4 * g + 3] = fmaf(x, v.w, acc[a][4 * g + 3]);
        }
      }
    }
  }
}

// Rows ty MT + a of a tile's accumulators, times mul[a], to the tensor.
template <typename T, int DP, int MT>
__device__ __forceinline__ void gen_store(const Heads& x, int64_t base, int h, int r0, int n,
                                          int dim, int ty, int tx,
                                          const float (&acc)[MT][4 * GenShape<DP, MT>::DC],
                                          const float (&mul)[MT]) {
  using S = GenShape<DP, MT>;
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    const int r = r0 + ty * MT + a;
    T* row = x.at<T>(base + min(r, n - 1), h);
#pragma unroll
    for (int g = 0; g < S::DC; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = acc[a][4 * g + i];
#pragma unroll
        for (int w = S::LANES; w < 16; w *= 2) v += __shfl_xor_sync(0xffffffffu, v, w);
        const int c = (16 * g + tx) * 4 + i;
        if (tx < S::LANES && r < n && c < dim) row[c] = from_f32<T>(v * mul[a]);
      }
  }
}

__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Block -> (sequence, head, tile).  The tiles that see most under a causal mask come
// first for all sequences and heads, so that the last blocks to run are short ones (8
// sequences of 512, heads of 64, backward: 389 us with a sequence's tiles one after
// another, 275 us so; 32 of 33 to 97: 54 and 45 us).
struct GenWork {
  int b, h, tile;
};
__device__ __forceinline__ GenWork gen_work(const AttnArgs& p, int nheads, bool keys, int ntiles) {
  GenWork w;
  const uint32_t per = (uint32_t)p.B * nheads, t = blockIdx.x / per, r = blockIdx.x - t * per;
  w.tile = keys ? (int)t : ntiles - 1 - (int)t;
  w.b = r / nheads;
  w.h = r - w.b * nheads;
  return w;
}

// o and lse of one tile of queries: one pass over the visible keys with the
// running maximum and sum of the softmax.
template <typename T, int DP, int MT>
__global__ void __launch_bounds__(kGenThreads)
    attn_fwd_general(AttnArgs p) {
  using S = GenShape<DP, MT>;
  extern __shared__ float4 gen_smem[];
  float* Q = reinterpret_cast<float*>(gen_smem);
  float* KV = Q + S::TILE;
  float* P = KV + S::TILE;
  pdl_wait();
  pdl_trigger();
  const GenWork w = gen_work(p, p.heads, false, (p.max_q + S::BT - 1) / S::BT);
  Seq s;
  if (!load_seq(p, w.b, &s, threadIdx.x == 0)) return;
  const int t0 = w.tile * S::BT;
  if (t0 >= s.lq) return;
  const int hk = w.h / p.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t0 + s.off();
  const int i1 = min(t0 + S::BT, s.lq) - 1 + s.off();
  gen_load<T, DP, MT>(Q, p.q, s.q0, w.h, t0, s.lq, p.dim);
  float acc[MT][4 * S::DC], m[MT], l[MT];
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * S::DC; ++c) acc[a][c] = 0.f;
  }
  const KeySpan ks = key_span(p, s.lk, i0, i1);
  for (int part = 0; part < 2; ++part) {
    const int hi = part ? ks.b1 : ks.a1;
    for (int j0 = part ? ks.b0 : 0; j0 < hi; j0 += S::BT) {
      __syncthreads();
      gen_load<T, DP, MT>(KV, p.k, s.k0, hk, j0, hi, p.dim);
      __syncthreads();
      float sc[MT][MT];
      gen_dot<DP, MT>(Q, KV, ty, tx, sc);
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        const int i = i0 + ty * MT + a;
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < MT; ++b) {
          const int j = j0 + tx + 16 * b;
          sc[a][b] = j < hi && visible(p, i, j) ? sc[a][b] * p.scale : -INFINITY;
          top = fmaxf(top, sc[a][b]);
        }
        const float mn = fmaxf(m[a], half_warp_max(top));
        const float ref = mn == -INFINITY ? 0.f : mn;  // no key seen yet
        const float fix = expf(m[a] - ref);
        m[a] = mn;
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < MT; ++b) {
          const float e = expf(sc[a][b] - ref);
          sum += e;
          P[(ty * MT + a) * S::LP + tx + 16 * b] = e;
        }
        l[a] = l[a] * fix + half_warp_sum(sum);
#pragma unroll
        for (int c = 0; c < 4 * S::DC; ++c) acc[a][c] *= fix;
      }
      __syncthreads();
      gen_load<T, DP, MT>(KV, p.v, s.k0, hk, j0, hi, p.dim);
      __syncthreads();
      gen_acc<DP, MT>(P, KV, min(S::BT, hi - j0), ty, tx, acc);
    }
  }
  float inv[MT];
#pragma unroll
  for (int a = 0; a < MT; ++a) inv[a] = l[a] > 0.f || l[a] != l[a] ? 1.f / l[a] : 0.f;
  gen_store<T, DP, MT>(p.o, s.q0, w.h, t0, s.lq, p.dim, ty, tx, acc, inv);
  if (p.lse && tx == 0) {
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      const int t = t0 + ty * MT + a;
      if (t < s.lq) p.lse[(int64_t)w.h * p.Tq + s.q0 + t] = m[a] + logf(l[a]);
    }
  }
}

// p and ds of one score; lse is -infinity on a row that sees no key, where
// nothing is visible either.
__device__ __forceinline__ float gen_prob(const AttnArgs& p, float s, float lse, bool vis) {
  return vis ? expf(s * p.scale - lse) : 0.f;
}

// dq of one tile of queries; leaves each row's delta for the other kernel.
template <typename T, int DP, int MT>
__global__ void __launch_bounds__(kGenThreads)
    attn_dq_general(AttnArgs p) {
  using S = GenShape<DP, MT>;
  extern __shared__ float4 gen_smem[];
  float* Q = reinterpret_cast<float*>(gen_smem);
  float* DO = Q + S::TILE;
  float* K = DO + S::TILE;
  float* V = K + S::TILE;
  float* DS = V + S::TILE;
  pdl_wait();
  pdl_trigger();
  const GenWork w = gen_work(p, p.heads, false, (p.max_q + S::BT - 1) / S::BT);
  Seq s;
  if (!load_seq(p, w.b, &s, threadIdx.x == 0)) return;
  const int t0 = w.tile * S::BT;
  if (t0 >= s.lq) return;
  const int hk = w.h / p.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t0 + s.off();
  const int i1 = min(t0 + S::BT, s.lq) - 1 + s.off();
  gen_load<T, DP, MT>(Q, p.q, s.q0, w.h, t0, s.lq, p.dim);
  gen_load<T, DP, MT>(DO, p.dout, s.q0, w.h, t0, s.lq, p.dim);
  __syncthreads();
  float acc[MT][4 * S::DC], lse[MT], delta[MT];
#pragma unroll
  for (int a = 0; a < MT; ++a) {
#pragma unroll
    for (int c = 0; c < 4 * S::DC; ++c) acc[a][c] = 0.f;
    const int r = ty * MT + a;
    const bool in = t0 + r < s.lq;
    const int64_t at = (int64_t)w.h * p.Tq + s.q0 + t0 + r;
    float d = 0.f;
    if (in) {
      const T* o = p.o.at<const T>(s.q0 + t0 + r, w.h);
      for (int c = tx; c < p.dim; c += 16) d = fmaf(as_f32<T>(o[c]), DO[r * S::LD + c], d);
    }
    delta[a] = half_warp_sum(d);
    lse[a] = in ? p.lse_in[at] : 0.f;
  }
  const KeySpan ks = key_span(p, s.lk, i0, i1);
  // A bf16 o has lost the bits that make sum_j ds_j zero on a row of few keys,
  // so its row sums are taken from the weights, in a pass of their own.
  constexpr bool own_delta = sizeof(T) == 2;
  if (own_delta) {
#pragma unroll
    for (int a = 0; a < MT; ++a) delta[a] = 0.f;
  }
  for (int pass = own_delta ? 0 : 1; pass < 2; ++pass) {
    for (int part = 0; part < 2; ++part) {
      const int hi = part ? ks.b1 : ks.a1;
      for (int j0 = part ? ks.b0 : 0; j0 < hi; j0 += S::BT) {
        __syncthreads();
        gen_load<T, DP, MT>(K, p.k, s.k0, hk, j0, hi, p.dim);
        gen_load<T, DP, MT>(V, p.v, s.k0, hk, j0, hi, p.dim);
        __syncthreads();
        float sc[MT][MT], dp[MT][MT];
        gen_dot<DP, MT>(Q, K, ty, tx, sc);
        gen_dot<DP, MT>(DO, V, ty, tx, dp);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const int i = i0 + ty * MT + a;
#pragma unroll
          for (int b = 0; b < MT; ++b) {
            const int j = j0 + tx + 16 * b;
            const bool vis = j < hi && t0 + ty * MT + a < s.lq && visible(p, i, j);
            const float pr = gen_prob(p, sc[a][b], lse[a], vis);
            if (pass == 0)
              delta[a] += vis ? pr * dp[a][b] : 0.f;
            else
              DS[(ty * MT + a) * S::LP + tx + 16 * b] = vis ? pr * (dp[a][b] - delta[a]) : 0.f;
          }
        }
        if (pass == 0) continue;
        __syncthreads();
        gen_acc<DP, MT>(DS, K, min(S::BT, hi - j0), ty, tx, acc);
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int a = 0; a < MT; ++a) delta[a] = half_warp_sum(delta[a]);
    }
  }
  if (tx == 0) {
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      const int t = t0 + ty * MT + a;
      if (t < s.lq) p.delta[(int64_t)w.h * p.Tq + s.q0 + t] = delta[a];
    }
  }
  float mul[MT];
#pragma unroll
  for (int a = 0; a < MT; ++a) mul[a] = p.scale;
  gen_store<T, DP, MT>(p.dq, s.q0, w.h, t0, s.lq, p.dim, ty, tx, acc, mul);
}

// dk and dv of one tile of keys, over every query head that shares it.
template <typename T, int DP, int MT>
__global__ void __launch_bounds__(kGenThreads)
    attn_dkv_general(AttnArgs p) {
  using S = GenShape<DP, MT>;
  extern __shared__ float4 gen_smem[];
  float* K = reinterpret_cast<float*>(gen_smem);
  float* V = K + S::TILE;
  float* Q = V + S::TILE;
  float* DO = Q + S::TILE;
  float* P = DO + S::TILE;
  float* DS = P + S::BT * S::LP;
  pdl_wait();
  pdl_trigger();
  const GenWork w = gen_work(p, p.kv, true, (p.max_k + S::BT - 1) / S::BT);
  Seq s;
  if (!load_seq(p, w.b, &s, threadIdx.x == 0)) return;
  const int j0 = w.tile * S::BT;
  if (j0 >= s.lk) return;
  const int j1 = min(j0 + S::BT, s.lk) - 1;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const RowSpan rs = row_span(p, s, j0, j1);
  gen_load<T, DP, MT>(K, p.k, s.k0, w.h, j0, s.lk, p.dim);
  gen_load<T, DP, MT>(V, p.v, s.k0, w.h, j0, s.lk, p.dim);
  float dk[MT][4 * S::DC], dv[MT][4 * S::DC];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int c = 0; c < 4 * S::DC; ++c) dk[a][c] = dv[a][c] = 0.f;
  for (int g = 0; g < p.group; ++g) {
    const int h = w.h * p.group + g;
    for (int t0 = rs.t0; t0 < rs.t1; t0 += S::BT) {
      __syncthreads();
      gen_load<T, DP, MT>(Q, p.q, s.q0, h, t0, rs.t1, p.dim);
      gen_load<T, DP, MT>(DO, p.dout, s.q0, h, t0, rs.t1, p.dim);
      __syncthreads();
      float sc[MT][MT], dp[MT][MT];
      gen_dot<DP, MT>(K, Q, ty, tx, sc);
      gen_dot<DP, MT>(V, DO, ty, tx, dp);
#pragma unroll
      for (int b = 0; b < MT; ++b) {
        const int t = t0 + tx + 16 * b;
        const bool in = t < rs.t1;
        const int64_t at = (int64_t)h * p.Tq + s.q0 + t;
        const float lse = in ? p.lse_in[at] : 0.f, delta = in ? p.delta[at] : 0.f;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const int j = j0 + ty * MT + a;
          const bool vis = in && j <= j1 && visible(p, t + s.off(), j);
          const float pr = gen_prob(p, sc[a][b], lse, vis);
          P[(ty * MT + a) * S::LP + tx + 16 * b] = pr;
          DS[(ty * MT + a) * S::LP + tx + 16 * b] = vis ? pr * (dp[a][b] - delta) : 0.f;
        }
      }
      __syncthreads();
      gen_acc<DP, MT>(P, DO, min(S::BT, rs.t1 - t0), ty, tx, dv);
      gen_acc<DP, MT>(DS, Q, min(S::BT, rs.t1 - t0), ty, tx, dk);
    }
  }
  float one[MT], sc[MT];
#pragma unroll
  for (int a = 0; a < MT; ++a) one[a] = 1.f, sc[a] = p.scale;
  gen_store<T, DP, MT>(p.dk, s.k0, w.h, j0, s.lk, p.dim, ty, tx, dk, sc);
  gen_store<T, DP, MT>(p.dv, s.k0, w.h, j0, s.lk, p.dim, ty, tx, dv, one);
}

// ---- launches -------------------------------------------------------------------
template <typename T, int DP, int MT>
cudaError_t general_go(const AttnArgs& p, int pass, cudaStream_t st) {
  using S = GenShape<DP, MT>;
  constexpr size_t kFwd = (2 * S::TILE + S::BT * S::LP) * sizeof(float);
  constexpr size_t kDq = (4 * S::TILE + S::BT * S::LP) * sizeof(float);
  constexpr size_t kDkv = (4 * S::TILE + 2 * S::BT * S::LP) * sizeof(float);
  static_assert(kDkv <= 227 * 1024, "shared memory of the general attention kernels");
  static PerDevice once;
  cudaError_t e = once.get([] {
    cudaError_t r = cudaFuncSetAttribute(attn_fwd_general<T, DP, MT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFwd);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(attn_dq_general<T, DP, MT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDq);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(attn_dkv_general<T, DP, MT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDkv);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int64_t rows = pass == 2 ? p.max_k : p.max_q, heads = pass == 2 ? p.kv : p.heads;
  const int64_t blocks = (rows + S::BT - 1) / S::BT * heads * p.B;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(kGenThreads);
  count_launches(1);
  if (pass == 0) return launch_ex(attn_fwd_general<T, DP, MT>, grid, block, kFwd, st, false, p);
  if (pass == 1) return launch_ex(attn_dq_general<T, DP, MT>, grid, block, kDq, st, false, p);
  return launch_ex(attn_dkv_general<T, DP, MT>, grid, block, kDkv, st, false, p);
}

// pass 0: o and lse; 1: dq and delta; 2: dk and dv
template <typename T>
cudaError_t general_pass(const AttnArgs& p, int pass, cudaStream_t st) {
  // Tiles of 32 rows for short sequences, whose last tile of 64 would be mostly
  // padding.  f32, 64 -> 32 rows: sequences of 65, 8 heads of 32: forward 19.6 ->
  // 15.3 us, backward 51 -> 40 us; of 128, 12 heads of 64: 17.4 -> 17.7 and 55 -> 49
  // us; of 512, heads of 32, 49 -> 63 and 150 -> 183 us (tiles of 64 read shared
  // memory half as often).
  const int longest = p.max_q > p.max_k ? p.max_q : p.max_k;
  const bool small = longest <= (pass ? 128 : 96);
  if (p.dim <= 32) return small ? general_go<T, 32, 2>(p, pass, st) : general_go<T, 32, 4>(p, pass, st);
  if (p.dim <= 64) return small ? general_go<T, 64, 2>(p, pass, st) : general_go<T, 64, 4>(p, pass, st);
  if (p.dim <= 128) return general_go<T, 128, 4>(p, pass, st);
  return general_go<T, 256, 2>(p, pass, st);
}

}  // namespace
}  // namespace ttc
