// Attention of a few query rows against long caches: the form for single
// tokens.  There is nothing to tile over the queries, the pass is one read of
// the visible keys and values, so what counts is bytes in flight: the keys of
// a sequence and key head are split over CTAs and warps, and every row of the
// group's query heads uses what a warp read.  The shares of warps and CTAs are
// joined by their maxima, the CTAs' by a second kernel.
//
// bf16: 16 rows x 16 keys a step on warp-level matrix instructions, operands
// straight from global memory in 16-byte pieces (an fp32 dot product by shuffles
// took five times the instructions and 44 us where this takes XX, 32 sequences,
// 16 heads on 4, 1028 keys of 128).  f32: dot products over lanes, exact.
#pragma once

#include "attn_general.cuh"

namespace ttc {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecRows = 16;   // most rows (query heads of a group x queries), bf16
constexpr int kDecRowsF32 = 8;
constexpr int kDecUnroll = 4;  // keys on their way in a lane

struct DecodeCut {
  int splits;
  float* o;    // [split][head][Tq][dim], not yet divided by the sum
  float2* ml;  // [split][head][Tq]: maximum (in powers of two) and sum
};

// 16 bytes as floats
template <typename T>
struct Pack16;
template <>
struct Pack16<float> {
  static constexpr int N = 4;
  static __device__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
};
// The joint softmax state of two shares of a row: the weights of each.
__device__ __forceinline__ float2 join(float ma, float mb, float* m) {
  *m = fmaxf(ma, mb);
  const float ref = *m == -INFINITY ? 0.f : *m;
  return make_float2(exp2f(ma - ref), exp2f(mb - ref));
}

// The warps' shares of a CTA's rows (so: [warp][R][C + 2], o then maximum and
// sum) joined and written: the result, or this split's part of it.
template <typename T, int C>
__device__ __forceinline__ void decode_out(const AttnArgs& p, const DecodeCut& cut, const Seq& s,
                                           int hk, int split, int rows, const float* so, int R) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  for (int r = warp; r < rows; r += kDecWarps) {
    float mm = -INFINITY, ll = 0.f;
    const float* at_w[kDecWarps];
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      at_w[w] = so + (w * R + r) * (C + 2);
      mm = fmaxf(mm, at_w[w][C]);
    }
    const float ref = mm == -INFINITY ? 0.f : mm;
    float f[kDecWarps];
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      f[w] = exp2f(at_w[w][C] - ref);
      ll += at_w[w][C + 1] * f[w];
    }
    const int g = r / s.lq, h = hk * p.group + g;
    const int64_t t = s.q0 + r - g * s.lq;
    const float inv = cut.splits > 1 ? 1.f : ll > 0.f || ll != ll ? 1.f / ll : 0.f;
    const int64_t at = ((int64_t)split * p.heads + h) * p.Tq + t;
    for (int d = lane; d < p.dim; d += 32) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) sum = fmaf(at_w[w][d], f[w], sum);
      if (cut.splits > 1)
        cut.o[at * p.dim + d] = sum;
      else
        p.o.at<T>(t, h)[d] = from_f32<T>(sum * inv);
    }
    if (lane == 0) {
      if (cut.splits > 1)
        cut.ml[at] = make_float2(mm, ll);
      else if (p.lse)
        p.lse[at] = ll > 0.f || ll != ll ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    }
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Lane = (g, t), g = lane / 4, t = lane % 4.  A product's fragments hold, for
// rows or columns g, the pairs 2t, 2t + 1 and 2t + 8, 2t + 9 along the summed
// axis.  That axis may be taken in any order that both operands share, so for
// Q K^T lane t holds 8 channels in a row of every 32 (one 16-byte load), two
// products' worth.  For P V the summed axis is the keys, a column a channel:
// lane g holds 8 channels in a row of the keys 2t, 2t + 1, 2t + 8, 2t + 9, and
// column g of product i stands for its channel i.
// DB: blocks of 32 channels.
template <int DB>
__global__ void __launch_bounds__(32 * kDecWarps, 3)
    attn_decode_mma_kernel(AttnArgs p, DecodeCut cut) {
  constexpr int C = 32 * DB, VB = DB / 2;
  extern __shared__ float dec_smem[];  // [warp][kDecRows][C + 2]
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % cut.splits, rest = blockIdx.x / cut.splits;
  const int hk = rest % p.kv, b = rest / p.kv;
  Seq s;
  if (!load_seq(p, b, &s, threadIdx.x == 0)) return;
  const int rows = p.group * s.lq;
  if (rows == 0) return;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // queries: rows g and g + 8 (row r: query head hk group + r / lq, query r % lq)
  uint4 q[2][DB];
  int pos[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i, gr = r / s.lq, tq = r - gr * s.lq;
    pos[i] = s.off() + tq;
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      const int c = 32 * d + 8 * t;
      q[i][d] = r < rows && c < p.dim
                    ? *reinterpret_cast<const uint4*>(
                          p.q.at<const __nv_bfloat16>(s.q0 + tq, hk * p.group + gr) + c)
                    : zero;
    }
  }
  const float scale = p.scale * 1.4426950408889634f;
  const KeySpan ks = key_span(p, s.lk, s.off(), s.lk - 1);
  const int n = ks.a1 + ks.b1 - ks.b0;  // keys that some row sees, the first tokens first
  const int x0 = (int)((int64_t)n * split / cut.splits);
  const int x1 = (int)((int64_t)n * (split + 1) / cut.splits);
  auto key = [&](int x) { return x < ks.a1 ? x : ks.b0 + x - ks.a1; };
  float o[VB][8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int w = 0; w < VB; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[w][i][e] = 0.f;
  uint4 kk[2][DB], vv[4][VB];
  auto load_k = [&](int x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int y = x + 8 * i + g;
      const __nv_bfloat16* row = p.k.at<const __nv_bfloat16>(s.k0 + key(y), hk);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const int c = 32 * d + 8 * t;
        kk[i][d] = y < x1 && c < p.dim ? *reinterpret_cast<const uint4*>(row + c) : zero;
      }
    }
  };
  auto load_v = [&](int x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int y = x + 2 * t + (i & 1) + 8 * (i >> 1);
      const __nv_bfloat16* row = p.v.at<const __nv_bfloat16>(s.k0 + key(y), hk);
#pragma unroll
      for (int w = 0; w < VB; ++w) {
        const int c = 64 * w + 8 * g;
        vv[i][w] = y < x1 && c < p.dim ? *reinterpret_cast<const uint4*>(row + c) : zero;
      }
    }
  };
  int x = x0 + 16 * warp;
  if (x < x1) {
    load_k(x);
    load_v(x);
  }
#pragma unroll 1
  for (; x < x1; x += 16 * kDecWarps) {
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const uint32_t a0[4] = {q[0][d].x, q[1][d].x, q[0][d].y, q[1][d].y};
        const uint32_t a1[4] = {q[0][d].z, q[1][d].z, q[0][d].w, q[1][d].w};
        mma16816(sc[j], a0, kk[j][d].x, kk[j][d].y);
        mma16816(sc[j], a1, kk[j][d].z, kk[j][d].w);
      }
    }
    const int next = x + 16 * kDecWarps;
    if (next < x1) load_k(next);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int y = x + 8 * j + 2 * t + (e & 1), i = e >> 1;
        const bool see = y < x1 && (s.lq == 1 || visible(p, pos[i], key(y)));
        sc[j][e] = see ? sc[j][e] * scale : -INFINITY;
        top[i] = fmaxf(top[i], sc[j][e]);
      }
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      const float mn = fmaxf(m[i], top[i]);
      f[i] = mn == m[i] ? 1.f : exp2f(m[i] - mn);
      m[i] = mn;
      l[i] *= f[i];
    }
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int w = 0; w < VB; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[w][i][e] *= f[e >> 1];
    }
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = m[i] == -INFINITY ? 0.f : m[i];
        const float u = exp2f(sc[j][2 * i] - ref), v = exp2f(sc[j][2 * i + 1] - ref);
        l[i] += u + v;
        a[2 * j + i] = pack_bf16(u, v);
      }
#pragma unroll
    for (int w = 0; w < VB; ++w) {
      const uint32_t v0[4] = {vv[0][w].x, vv[0][w].y, vv[0][w].z, vv[0][w].w};
      const uint32_t v1[4] = {vv[1][w].x, vv[1][w].y, vv[1][w].z, vv[1][w].w};
      const uint32_t v2[4] = {vv[2][w].x, vv[2][w].y, vv[2][w].z, vv[2][w].w};
      const uint32_t v3[4] = {vv[3][w].x, vv[3][w].y, vv[3][w].z, vv[3][w].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t pick = i & 1 ? 0x7632u : 0x5410u;
        mma16816(o[w][i], a, __byte_perm(v0[i >> 1], v1[i >> 1], pick),
                 __byte_perm(v2[i >> 1], v3[i >> 1], pick));
      }
    }
    if (next < x1) load_v(next);
  }
  float* so = dec_smem + warp * kDecRows * (C + 2);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    float* row = so + (g + 8 * i) * (C + 2);
    if (t == 0) row[C] = m[i], row[C + 1] = l[i];
#pragma unroll
    for (int w = 0; w < VB; ++w)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        row[64 * w + 8 * (2 * t) + k] = o[w][k][2 * i];
        row[64 * w + 8 * (2 * t + 1) + k] = o[w][k][2 * i + 1];
      }
  }
  decode_out<__nv_bfloat16, C>(p, cut, s, hk, split, rows, dec_smem, kDecRows);
}

// R: rows in registers (at least the call's); L lanes a key.
template <typename T, int R, int L>
__global__ void __launch_bounds__(32 * kDecWarps) attn_decode_kernel(AttnArgs p, DecodeCut cut) {
  using P = Pack16<T>;
  constexpr int N = P::N, KEYS = 32 / L, U = kDecUnroll;
  __shared__ float so[kDecWarps][R][L * N + 2];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % L, sub = lane / L;
  const int split = blockIdx.x % cut.splits, rest = blockIdx.x / cut.splits;
  const int hk = rest % p.kv, b = rest / p.kv;
  Seq s;
  if (!load_seq(p, b, &s, threadIdx.x == 0)) return;
  const int rows = p.group * s.lq;
  if (rows == 0) return;
  const bool on = u * N < p.dim;
  // the row r: query head hk group + r / lq, query r % lq
  float q[R][N], o[R][N], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) q[r][e] = o[r][e] = 0.f;
    if (r < rows && on) {
      const int g = r / s.lq;
      P::get(reinterpret_cast<const uint4*>(
                 p.q.at<const T>(s.q0 + r - g * s.lq, hk * p.group + g))[u],
             q[r]);
#pragma unroll
      for (int e = 0; e < N; ++e) q[r][e] *= p.scale * 1.4426950408889634f;
    }
  }
  const KeySpan ks = key_span(p, s.lk, s.off(), s.lk - 1);
  const int n = ks.a1 + ks.b1 - ks.b0;  // keys that some row sees, the first tokens first
  const int x0 = (int)((int64_t)n * split / cut.splits);
  const int x1 = (int)((int64_t)n * (split + 1) / cut.splits);
  constexpr int STEP = kDecWarps * KEYS;
#pragma unroll 1
  for (int x = x0 + warp * KEYS + sub; __any_sync(0xffffffffu, x < x1); x += STEP * U) {
    uint4 kk[U], vv[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int y = x + i * STEP;
      kk[i] = vv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (y < x1 && on) {
        const int j = y < ks.a1 ? y : ks.b0 + y - ks.a1;
        kk[i] = reinterpret_cast<const uint4*>(p.k.at<const T>(s.k0 + j, hk))[u];
        vv[i] = reinterpret_cast<const uint4*>(p.v.at<const T>(s.k0 + j, hk))[u];
      }
    }
    float sc[U][R];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float k[N];
      P::get(kk[i], k);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        sc[i][r] = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) sc[i][r] = fmaf(q[r][e], k[e], sc[i][r]);
      }
    }
#pragma unroll
    for (int w = L / 2; w; w >>= 1)
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) sc[i][r] += __shfl_xor_sync(0xffffffffu, sc[i][r], w);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int y = x + i * STEP;
      const int j = y < ks.a1 ? y : ks.b0 + y - ks.a1;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (y >= x1 || (s.lq > 1 && !visible(p, s.off() + r % s.lq, j))) sc[i][r] = -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = sc[0][r];
#pragma unroll
      for (int i = 1; i < U; ++i) top = fmaxf(top, sc[i][r]);
      if (top > m[r]) {
        const float f = exp2f(m[r] - top);
        m[r] = top;
        l[r] *= f;
#pragma unroll
        for (int e = 0; e < N; ++e) o[r][e] *= f;
      }
      const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        sc[i][r] = exp2f(sc[i][r] - ref);
        l[r] += sc[i][r];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float v[N];
      P::get(vv[i], v);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < N; ++e) o[r][e] = fmaf(sc[i][r], v[e], o[r][e]);
    }
  }
  // the key lanes of a warp, then its warps
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int w = L; w < 32; w <<= 1) {
      float mm;
      const float2 f = join(m[r], __shfl_xor_sync(0xffffffffu, m[r], w), &mm);
      l[r] = l[r] * f.x + __shfl_xor_sync(0xffffffffu, l[r], w) * f.y;
#pragma unroll
      for (int e = 0; e < N; ++e)
        o[r][e] = o[r][e] * f.x + __shfl_xor_sync(0xffffffffu, o[r][e], w) * f.y;
      m[r] = mm;
    }
    if (sub == 0) {
#pragma unroll
      for (int e = 0; e < N; ++e) so[warp][r][u * N + e] = o[r][e];
      if (u == 0) so[warp][r][L * N] = m[r], so[warp][r][L * N + 1] = l[r];
    }
  }
  decode_out<T, L * N>(p, cut, s, hk, split, rows, &so[0][0][0], R);
}

// The splits of a row joined, in their order: a warp a row.
template <typename T>
__global__ void __launch_bounds__(128) attn_join_kernel(AttnArgs p, DecodeCut cut) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint32_t i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int b = (int)(i / (uint32_t)(p.heads * p.max_q));
  if (b >= p.B) return;
  const int rest = (int)(i - (uint32_t)b * (p.heads * p.max_q));
  const int h = rest / p.max_q, t = rest - h * p.max_q;
  Seq s;
  if (!load_seq(p, b, &s, false) || t >= s.lq) return;
  const int64_t row = (int64_t)h * p.Tq + s.q0 + t, step = (int64_t)p.heads * p.Tq;
  float m = -INFINITY;
  for (int k = lane; k < cut.splits; k += 32) m = fmaxf(m, cut.ml[k * step + row].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) o[c] = 0.f;
  for (int k0 = 0; k0 < cut.splits; k0 += 32) {  // lane k: the weight of split k0 + k
    const float2 ml = k0 + lane < cut.splits ? cut.ml[(k0 + lane) * step + row]
                                             : make_float2(-INFINITY, 0.f);
    const float f = exp2f(ml.x - ref);
    const int n = min(32, cut.splits - k0);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k), lk = __shfl_sync(0xffffffffu, ml.y, k);
      l = fmaf(lk, fk, l);
      const float* src = cut.o + ((k0 + k) * step + row) * p.dim;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (32 * c + lane < p.dim) o[c] = fmaf(src[32 * c + lane], fk, o[c]);
    }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (32 * c + lane < p.dim) p.o.at<T>(s.q0 + t, h)[32 * c + lane] = from_f32<T>(o[c] * inv);
  if (lane == 0 && p.lse)
    p.lse[row] = l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ---- launch ---------------------------------------------------------------------
int elems16(int act) { return act == TT_DT_F32 ? 4 : 8; }

// Few enough rows, and heads of whole 16-byte pieces (of up to 128 channels).
bool decode_shape(const AttnPlan& P, const tt_attn_seqs* s) {
  return (int64_t)(P.heads / P.kv) * s->max_q <=
             (P.act == TT_DT_F32 ? kDecRowsF32 : kDecRows) &&
         P.dim % elems16(P.act) == 0 && P.dim <= 128;
}
bool decode_takes(const AttnArgs& p, int act) {
  const int n = elems16(act);
  auto ok = [&](const Heads& x) {
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.row % n == 0 && x.head % n == 0;
  };
  return ok(p.q) && ok(p.k) && ok(p.v);
}

// Splits: as many CTAs as the SMs hold at once (three each), but no fewer than
// 64 keys a CTA (16 a warp).
int decode_splits(const AttnPlan& P, const tt_attn_seqs* s) {
  int64_t keys = s->max_k;
  if (P.left >= 0) {
    const int64_t most = (int64_t)P.left + s->max_q + P.sinks + (P.right > 0 ? P.right : 0);
    if (P.right >= 0 && most < keys) keys = most;
  }
  const int64_t pairs = (int64_t)s->B * P.kv;
  int64_t n = pairs > 0 ? 3 * (int64_t)device_sms() / pairs : 1;
  if (n > keys / 64) n = keys / 64;
  return (int)(n < 1 ? 1 : n > 256 ? 256 : n);
}
size_t decode_bytes(const AttnPlan& P, const tt_attn_seqs* s) {
  if (!decode_shape(P, s)) return 0;
  const int n = decode_splits(P, s);
  if (n == 1) return 0;
  return (size_t)n * P.heads * (size_t)s->Tq * ((size_t)P.dim * sizeof(float) + sizeof(float2));
}

template <int R>
cudaError_t decode_f32(const AttnArgs& p, const DecodeCut& cut, dim3 grid, cudaStream_t st) {
  const dim3 block(32 * kDecWarps);
  if (p.dim <= 32) return launch_ex(attn_decode_kernel<float, R, 8>, grid, block, 0, st, false, p, cut);
  if (p.dim <= 64) return launch_ex(attn_decode_kernel<float, R, 16>, grid, block, 0, st, false, p, cut);
  return launch_ex(attn_decode_kernel<float, R, 32>, grid, block, 0, st, false, p, cut);
}
cudaError_t decode_bf16(const AttnArgs& p, const DecodeCut& cut, dim3 grid, cudaStream_t st) {
  const dim3 block(32 * kDecWarps);
  auto smem = [](int db) { return sizeof(float) * kDecWarps * kDecRows * (32 * db + 2); };
  if (p.dim <= 64)
    return launch_ex(attn_decode_mma_kernel<2>, grid, block, smem(2), st, false, p, cut);
  return launch_ex(attn_decode_mma_kernel<4>, grid, block, smem(4), st, false, p, cut);
}
cudaError_t decode(const AttnPlan& P, const tt_attn_seqs* s, const AttnArgs& p, void* ws,
                   cudaStream_t st) {
  DecodeCut cut;
  cut.splits = decode_splits(P, s);
  cut.ml = static_cast<float2*>(ws);
  cut.o = reinterpret_cast<float*>(cut.ml + (size_t)cut.splits * p.heads * (size_t)p.Tq);
  const int64_t blocks = (int64_t)p.B * p.kv * cut.splits;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  const int rows = p.group * p.max_q;
  const bool f32 = P.act == TT_DT_F32;
  count_launches(1);
  cudaError_t e = !f32        ? decode_bf16(p, cut, grid, st)
                  : rows <= 1 ? decode_f32<1>(p, cut, grid, st)
                  : rows <= 2 ? decode_f32<2>(p, cut, grid, st)
                  : rows <= 4 ? decode_f32<4>(p, cut, grid, st)
                              : decode_f32<8>(p, cut, grid, st);
  if (e == cudaSuccess && cut.splits > 1) {
    const dim3 join((unsigned)(((int64_t)p.B * p.heads * p.max_q + 3) / 4));
    count_launches(1);
    e = f32 ? launch_ex(attn_join_kernel<float>, join, dim3(128), 0, st, false, p, cut)
            : launch_ex(attn_join_kernel<__nv_bfloat16>, join, dim3(128), 0, st, false, p, cut);
  }
  return e;
}

}  // namespace
}  // namespace ttc
