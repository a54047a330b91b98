// Attention of a few query rows against long caches: the form for single
// tokens.  There is nothing to tile over the queries; the pass is one read of the
// visible keys and values, so what counts is bytes in flight and instructions a
// key.  The keys of a sequence and key head are split over the CTAs of a cluster
// and their warps, every row of the group's query heads uses what a warp read,
// and the shares are joined by their maxima through shared memory (across
// clusters, where a sequence has more CTAs than eight, by a second kernel).
//
// bf16: 16 keys a step on warp-level matrix instructions.  The 128-row tiles of
// the tensor-memory kernels would be filled by 4 rows of a group here, and one CTA
// a key head leaves SMs idle.  32 sequences, 1028 visible keys of 128, 16 heads on
// 4 (67 MB): 16.1 us, 4.2 TB/s; by the tiled kernel 39 us; by dot products over
// lanes and a second kernel for every join 50 us; 256 such sequences 87 us, 6.2
// TB/s, tiled 237 us.  One sequence of 8192 keys 24 us, tiled 85 us.
// f32: dot products over lanes, every product in 32 bits: 51 us against 763 us of
// the kernel for any layout (the same shape), bound by its instructions.
#pragma once

#include "attn_general.cuh"

namespace ttc {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecRows = 16;   // most rows (query heads of a group x queries), bf16
constexpr int kDecRowsF32 = 8;
constexpr int kDecStages = 2;
constexpr int kDecUnroll = 4;  // keys on their way in a lane

struct DecodeCut {
  int splits;   // CTAs of a sequence and key head: `cluster` times `parts`
  int cluster;  // CTAs that join through shared memory
  int parts;    // joins left for the second kernel
  float* o;     // [part][query head][query][dim]
  float2* ml;   // [part][query head][query]: maximum, sum
};

// 16 bytes as floats
__device__ __forceinline__ void four(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
// The joint softmax state of two shares of a row: the weights of each.
__device__ __forceinline__ float2 join(float ma, float mb, float* m) {
  *m = fmaxf(ma, mb);
  const float ref = *m == -INFINITY ? 0.f : *m;
  return make_float2(exp2f(ma - ref), exp2f(mb - ref));
}

__device__ __forceinline__ float remote(uint32_t at, int rank) {
  uint32_t there;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
  return x;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The warps' shares of a CTA's rows (so: `stride` floats a warp, rows of C + 4,
// o, then maximum and sum) joined, then those of the cluster's CTAs, a warp a
// row; the result, or this part of it, is written.
template <typename T, int C>
__device__ __forceinline__ void decode_out(const AttnArgs& p, const DecodeCut& cut, const Seq& s,
                                           int hk, int split, int rows, float* so, int stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = split / cut.cluster, rank = split - part * cut.cluster;
  __syncthreads();
  for (int r = warp; r < rows; r += kDecWarps) {
    float* at = so + r * (C + 4);
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, at[w * stride + C]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float f[kDecWarps];
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      f[w] = exp2f(at[w * stride + C] - ref);
      ll += at[w * stride + C + 1] * f[w];
    }
    __syncwarp();
    if (lane == 0) at[C] = mm, at[C + 1] = ll;
#pragma unroll
    for (int d = lane; d < C; d += 32) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) sum = fmaf(at[w * stride + d], f[w], sum);
      at[d] = sum;
    }
  }
  __syncwarp();
  cluster_meet();
  const uint32_t base = su32(so);
  for (int r = rank * kDecWarps + warp; r < rows; r += cut.cluster * kDecWarps) {
    const uint32_t at = base + 4 * r * (C + 4);
    // lane k: maximum and sum of CTA k
    const float m = lane < cut.cluster ? remote(at + 4 * C, lane) : -INFINITY;
    const float l = lane < cut.cluster ? remote(at + 4 * C + 4, lane) : 0.f;
    float mm = m;
#pragma unroll
    for (int w = 4; w; w >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, w));
    const float f = exp2f(m - (mm == -INFINITY ? 0.f : mm));
    float ll = 0.f, o[C / 32];
#pragma unroll
    for (int c = 0; c < C / 32; ++c) o[c] = 0.f;
#pragma unroll 2
    for (int k = 0; k < cut.cluster; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      ll = fmaf(__shfl_sync(0xffffffffu, l, k), fk, ll);
#pragma unroll
      for (int c = 0; c < C / 32; ++c)
        o[c] = fmaf(remote(at + 4 * (32 * c + lane), k), fk, o[c]);
    }
    mm = __shfl_sync(0xffffffffu, mm, 0);
    const int g = r / s.lq, h = hk * p.group + g;
    const int64_t t = s.q0 + r - g * s.lq;
    const float inv = cut.parts > 1 ? 1.f : ll > 0.f || ll != ll ? 1.f / ll : 0.f;
    const int64_t to = ((int64_t)part * p.heads + h) * p.Tq + t;
#pragma unroll
    for (int c = 0; c < C / 32; ++c) {
      const int d = 32 * c + lane;
      if (d >= p.dim) break;
      if (cut.parts > 1)
        cut.o[to * p.dim + d] = o[c];
      else
        p.o.at<T>(t, h)[d] = from_f32<T>(o[c] * inv);
    }
    if (lane == 0) {
      if (cut.parts > 1)
        cut.ml[to] = make_float2(mm, ll);
      else if (p.lse)
        p.lse[to] = ll > 0.f || ll != ll ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncwarp();
  cluster_meet();  // no CTA leaves while another reads its shares
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Products are taken with the keys (or the channels) as the 16 rows of the left
// operand and the call's rows as the 8 columns of the right one, N times 8.
// Lane = (g, t), g = lane / 4, t = lane % 4: a result holds rows g, g + 8 and
// columns 2t, 2t + 1, so a lane keeps the softmax of its columns and the keys'
// maximum is taken over g.  The weights go from a result (keys g) to a right
// operand (keys 2t, 2t + 1) by one 8 x 8 transposition a half.  A warp copies its
// 16 keys and values asynchronously into shared memory of its own, kDecStages - 1
// steps ahead (16-byte pieces of a row turned by row % 8: eight rows' pieces at one
// place lie in eight different bank groups), so only warps meet, not the CTA.
// DB: blocks of 32 channels.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int DB>
constexpr int kDecRing = kDecStages * 32 * (64 * DB);  // bytes a warp: 16 keys, 16 values a stage
template <int DB, int N>
__global__ void __launch_bounds__(32 * kDecWarps, N == 1 ? 3 : 2)
    attn_decode_mma_kernel(AttnArgs p, DecodeCut cut) {
  constexpr int C = 32 * DB, kRow = 2 * C, kRing = kDecRing<DB>, kHalf = 16 * kRow;
  static_assert(kRing >= 32 * N * (C + 4));
  extern __shared__ __align__(128) uint8_t dec_smem[];  // a warp's ring, its share afterwards
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % cut.splits, rest = blockIdx.x / cut.splits;
  const int hk = rest % p.kv, b = rest / p.kv;
  Seq s;
  if (!load_seq(p, b, &s, threadIdx.x == 0)) return;
  const int rows = p.group * s.lq;
  if (rows == 0) return;
  // Steps of 16 keys: those of the first tokens, then those of the window.
  const KeySpan ks = key_span(p, s.lk, s.off(), s.lk - 1);
  const int lead = (ks.a1 + 15) >> 4, steps = lead + ((ks.b1 - ks.b0 + 15) >> 4);
  const int j1 = (int)((int64_t)steps * (split + 1) / cut.splits);
  int j = (int)((int64_t)steps * split / cut.splits) + warp;
  const uint32_t ring = su32(dec_smem) + warp * kRing;
  const __nv_bfloat16* kbase = p.k.at<const __nv_bfloat16>(s.k0, hk);
  const __nv_bfloat16* vbase = p.v.at<const __nv_bfloat16>(s.k0, hk);
  const int krow = (int)p.k.row, vrow = (int)p.v.row;
  constexpr int kPer = 4 * DB, kPass = 32 / kPer;  // lanes a row, rows a pass
  const int r0 = lane / kPer, c0 = lane % kPer;
  const bool in = 8 * c0 < p.dim;
  if (p.dim < C)  // no copy writes the channels above dim: zeros
    for (int i = lane; i < kRing / 16; i += 32)
      *reinterpret_cast<uint4*>(dec_smem + warp * kRing + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  __syncwarp();
  // a step's first key and count; its rows past the count repeat the last one
  auto span = [&](int at, int* key0) {
    const bool first = at < lead;
    *key0 = first ? 16 * at : ks.b0 + 16 * (at - lead);
    return min(16, (first ? ks.a1 : ks.b1) - *key0);
  };
  auto fetch = [&](int at, int stage) {
    int key0;
    const int last = span(at, &key0) - 1;
    const __nv_bfloat16* kp = kbase + key0 * p.k.row + 8 * c0;
    const __nv_bfloat16* vp = vbase + key0 * p.v.row + 8 * c0;
    const uint32_t dst = ring + stage * (2 * kHalf) + r0 * kRow;
    if (in) {
#pragma unroll
      for (int i = 0; i < 16 / kPass; ++i) {
        const int r = r0 + i * kPass, from = min(r, last);
        const uint32_t to = dst + i * kPass * kRow + 16 * (c0 ^ (r & 7));
        copy16(to, kp + (int64_t)from * krow);
        copy16(to + kHalf, vp + (int64_t)from * vrow);
      }
    }
  };
  int stage = 0;
#pragma unroll
  for (int i = 0; i < kDecStages - 1; ++i) {
    if (j + i * kDecWarps < j1) fetch(j + i * kDecWarps, i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // queries: column c is query c % lq of query head hk group + c / lq
  uint32_t q[N][2 * DB][2];
  int pos[N][2];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = 8 * n + g, gr = c / s.lq;
    const __nv_bfloat16* src =
        p.q.at<const __nv_bfloat16>(s.q0 + c - gr * s.lq, hk * p.group + gr) + 2 * t;
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        q[n][i][e] = c < rows && 16 * i + 8 * e < p.dim
                         ? *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * e)
                         : 0u;
#pragma unroll
    for (int e = 0; e < 2; ++e) pos[n][e] = s.off() + (8 * n + 2 * t + e) % s.lq;
  }
  const float scale = p.scale * 1.4426950408889634f;
  float o[N][2 * DB][4], m[N][2], l[N][2];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
  }
  // A 16 x 16 block of keys x channels: matrices (keys 0-7, channels 0-7), (8-15,
  // 0-7), (0-7, 8-15), (8-15, 8-15).  Of values, transposed, with the middle two
  // exchanged (rows are the channels there).
  const int kr = lane & 15, kc = lane >> 4;
  const int vr = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
#pragma unroll 1
  for (; j < j1; j += kDecWarps) {
    const int ahead = j + (kDecStages - 1) * kDecWarps;
    if (ahead < j1) fetch(ahead, stage == 0 ? kDecStages - 1 : stage - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kDecStages - 1) : "memory");
    __syncwarp();
    const uint32_t at = ring + stage * (2 * kHalf);
    stage = stage == kDecStages - 1 ? 0 : stage + 1;
    float sc[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
      uint32_t a[4];
      ldsm4(a, at + kr * kRow + 16 * ((2 * i + kc) ^ (kr & 7)));
#pragma unroll
      for (int n = 0; n < N; ++n) mma16816(sc[n], a, q[n][i][0], q[n][i][1]);
    }
    int key0;
    const int count = span(j, &key0);
    uint32_t w[N][2];
    bool turn = false;
    float f[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = g + 8 * (e >> 1);
        const bool see = k < count && (s.lq == 1 || visible(p, pos[n][e & 1], key0 + k));
        sc[n][e] = see ? sc[n][e] * scale : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(sc[n][e], sc[n][e + 2]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float mn = fmaxf(m[n][e], top);
        const float ref = mn == -INFINITY ? 0.f : mn;
        f[n][e] = ex2(m[n][e] - ref);
        turn |= mn != m[n][e];
        m[n][e] = mn;
        sc[n][e] = ex2(sc[n][e] - ref);
        sc[n][e + 2] = ex2(sc[n][e + 2] - ref);
        l[n][e] = fmaf(l[n][e], f[n][e], sc[n][e] + sc[n][e + 2]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) w[n][h] = transpose8(pack_bf16(sc[n][2 * h], sc[n][2 * h + 1]));
    }
    if (__any_sync(0xffffffffu, turn)) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][i][e] *= f[n][e & 1];
    }
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
      uint32_t a[4];
      ldsm4t(a, at + kHalf + vr * kRow + 16 * ((2 * i + vc) ^ (vr & 7)));
#pragma unroll
      for (int n = 0; n < N; ++n) mma16816(o[n][i], a, w[n][0], w[n][1]);
    }
    __syncwarp();  // every lane has read the stage that the next step fills
  }
  float* so = reinterpret_cast<float*>(dec_smem + warp * kRing);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* row = so + (8 * n + 2 * t + e) * (C + 4);
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
      if (g == 0) row[C] = m[n][e], row[C + 1] = l[n][e];
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) {
        row[16 * i + g] = o[n][i][e];
        row[16 * i + 8 + g] = o[n][i][e + 2];
      }
    }
  decode_out<__nv_bfloat16, C>(p, cut, s, hk, split, rows,
                               reinterpret_cast<float*>(dec_smem), kRing / 4);
}

// R: rows in registers (at least the call's); L lanes a key.
template <int R, int L>
__global__ void __launch_bounds__(32 * kDecWarps) attn_decode_kernel(AttnArgs p, DecodeCut cut) {
  constexpr int N = 4, KEYS = 32 / L, U = kDecUnroll;
  __shared__ float so[kDecWarps][R][L * N + 4];
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
      four(reinterpret_cast<const uint4*>(
                 p.q.at<const float>(s.q0 + r - g * s.lq, hk * p.group + g))[u],
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
        kk[i] = reinterpret_cast<const uint4*>(p.k.at<const float>(s.k0 + j, hk))[u];
        vv[i] = reinterpret_cast<const uint4*>(p.v.at<const float>(s.k0 + j, hk))[u];
      }
    }
    float sc[U][R];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float k[N];
      four(kk[i], k);
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
      four(vv[i], v);
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
  decode_out<float, L * N>(p, cut, s, hk, split, rows, &so[0][0][0], R * (L * N + 4));
}

// The parts of a row (at most 32) joined, in their order: a warp a row.
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
  // lane k: maximum and sum of part k
  const float2 ml =
      lane < cut.parts ? cut.ml[lane * step + row] : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float f = exp2f(ml.x - (m == -INFINITY ? 0.f : m));
  float l = 0.f, o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = 0.f;
#pragma unroll 8
  for (int k = 0; k < cut.parts; ++k) {
    const float fk = __shfl_sync(0xffffffffu, f, k);
    l = fmaf(__shfl_sync(0xffffffffu, ml.y, k), fk, l);
    const float* src = cut.o + (k * step + row) * p.dim;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (32 * c + lane < p.dim) o[c] = fmaf(src[32 * c + lane], fk, o[c]);
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c)
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
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.row % n == 0 && x.head % n == 0 &&
           x.row < (1 << 30) && x.row > -(1 << 30);  // 32 bits in the kernel
  };
  return ok(p.q) && ok(p.k) && ok(p.v);
}

// Splits: as many CTAs as the SMs hold at once, three each, of many rows (whose
// sums take more registers) two, but no fewer than 64 keys a CTA (16 a warp);
// clusters of up to eight, the portable size.  1028 keys, 16 heads on 4: one query
// a sequence 16 us at two and three an SM, 26 us at six (a second wave); 16 rows
// 21 us at two, 28 us at three.  f32 4 rows 51 us at three, 58 us at two; 8 rows
// 74 us at three, 65 us at two.
DecodeCut decode_cut(const AttnPlan& P, const tt_attn_seqs* s) {
  int64_t keys = s->max_k;
  if (P.left >= 0) {
    const int64_t most = (int64_t)P.left + s->max_q + P.sinks + (P.right > 0 ? P.right : 0);
    if (P.right >= 0 && most < keys) keys = most;
  }
  const int64_t pairs = (int64_t)s->B * P.kv;
  const int64_t rows = (int64_t)(P.heads / P.kv) * s->max_q;
  const int an_sm = rows <= (P.act == TT_DT_F32 ? 4 : 8) ? 3 : 2;
  int64_t n = pairs > 0 ? an_sm * (int64_t)device_sms() / pairs : 1;
  if (n > keys / 64) n = keys / 64;
  n = n < 1 ? 1 : n > 256 ? 256 : n;
  DecodeCut cut = {};
  cut.parts = (int)(n + 7) / 8;
  cut.cluster = (int)n / cut.parts;
  cut.splits = cut.parts * cut.cluster;
  return cut;
}
size_t decode_bytes(const AttnPlan& P, const tt_attn_seqs* s) {
  if (!decode_shape(P, s)) return 0;
  const int n = decode_cut(P, s).parts;
  if (n == 1) return 0;
  return (size_t)n * P.heads * (size_t)s->Tq * ((size_t)P.dim * sizeof(float) + sizeof(float2));
}

template <int R>
cudaError_t decode_f32(const AttnArgs& p, const DecodeCut& cut, dim3 grid, cudaStream_t st) {
  const dim3 block(32 * kDecWarps);
  auto go = [&](auto kernel) {
    return launch_cluster(kernel, grid, block, 0, st, cut.cluster, p, cut);
  };
  if (p.dim <= 32) return go(attn_decode_kernel<R, 8>);
  if (p.dim <= 64) return go(attn_decode_kernel<R, 16>);
  return go(attn_decode_kernel<R, 32>);
}
template <int DB, int N>
cudaError_t decode_go(const AttnArgs& p, const DecodeCut& cut, dim3 grid, cudaStream_t st) {
  constexpr int kSmem = kDecRing<DB> * kDecWarps;
  static PerDevice once;
  const cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(attn_decode_mma_kernel<DB, N>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_cluster(attn_decode_mma_kernel<DB, N>, grid, dim3(32 * kDecWarps), kSmem, st,
                        cut.cluster, p, cut);
}
cudaError_t decode_bf16(const AttnArgs& p, const DecodeCut& cut, dim3 grid, cudaStream_t st) {
  const bool one = p.group * p.max_q <= 8;
  if (p.dim <= 64)
    return one ? decode_go<2, 1>(p, cut, grid, st) : decode_go<2, 2>(p, cut, grid, st);
  return one ? decode_go<4, 1>(p, cut, grid, st) : decode_go<4, 2>(p, cut, grid, st);
}
cudaError_t decode(const AttnPlan& P, const tt_attn_seqs* s, const AttnArgs& p, void* ws,
                   cudaStream_t st) {
  DecodeCut cut = decode_cut(P, s);
  cut.ml = static_cast<float2*>(ws);
  cut.o = reinterpret_cast<float*>(cut.ml + (size_t)cut.parts * p.heads * (size_t)p.Tq);
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
  if (e == cudaSuccess && cut.parts > 1) {
    const dim3 join((unsigned)(((int64_t)p.B * p.heads * p.max_q + 3) / 4));
    count_launches(1);
    e = f32 ? launch_ex(attn_join_kernel<float>, join, dim3(128), 0, st, false, p, cut)
            : launch_ex(attn_join_kernel<__nv_bfloat16>, join, dim3(128), 0, st, false, p, cut);
  }
  return e;
}

}  // namespace
}  // namespace ttc
