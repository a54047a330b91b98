// Log probabilities of given tokens with the row's log-sum, entropy and top
// alternatives; their gradient; and both in one pass over the logits.
//
// All are bound by HBM.  In units of log2, with c = scale log2(e) and a reference r near
// the row's maximum:
//   t = c (x - r),  e = 2^t,  s = sum e,  w = sum e t
//   lse = scale r + ln2 log2 s,  log p = ln2 (t - log2 s),  H = ln2 (log2 s - w / s)
//   d L / d x = scale (g ([target] - p) - h p (log p + H))
//             = e (A + B t) + scale g [target]
// One pass finds r, s and w.  A thread's reference is the maximum of the first values
// that it sees and stays until one exceeds it by more than 2^8 in e: raising it at every
// new maximum costs a warp its 20 instructions at nearly every vector, since some lane
// has one (4096 rows of 50001: 17.5 instructions a value).  The threads' sums meet at
// their largest reference.  The difference comes first (one more instruction
// for two values than c x - c r), so a log probability is as exact at logits of a
// thousand as at logits of one, and logits of the type's lowest value do not overflow.
//
// A row is taken by 1 to 32 warps by its width; rows that are few are split over a
// cluster's CTAs, which meet through shared memory.  Rows start anywhere: the elements
// before the first and after the last 16-byte boundary are taken one by one.  The pass
// that also writes the gradient keeps the row in shared memory in between, so it reads it
// from HBM once; of many rows of 24 to 108 KB a block keeps a ring that asynchronous copies
// fill.
//
// Measured in bf16 (of the 6.7 TB/s that a copy reaches): forward 4096 x 50001 67 us, 6.1
// TB/s, with the entropy 69, with four top alternatives as well 87; loss and gradient 8192
// x 32000 163 us, 6.4 TB/s (in one pass a block a row 191); 4096 x 50001 139; 2048 x 131072,
// a row an SM, 210 us, 5.1 TB/s; gradient alone 2048 x 131072 171 us, 6.3 TB/s.
//
// Top alternatives: the maxima of 128 groups of threads give a bound (the k-th
// largest of them, to 16 bits: at least k values are not below it); the few groups that
// reach it are read again, the values not below the bound are ranked by (value, lowest
// index).  Where ties make them too many, k rounds over the row take them in order.
#include <cmath>
#include <new>
#include <type_traits>

#include "rows.cuh"
#include "ttc.h"
#include "ttc_internal.h"

namespace ttc {

cudaError_t read_and_clear_logp_status(DeviceStatus* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(DeviceStatus));
  if (e != cudaSuccess || out->code == 0) return e;
  DeviceStatus z{0, 0};
  return cudaMemcpyToSymbol(g_status, &z, sizeof(z));
}

cudaError_t logp_set_wait_limit(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}

cudaError_t logp_set_debug_skip(int site) {
  return cudaMemcpyToSymbol(g_debug_skip, &site, sizeof(site));
}

namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634074f;
constexpr int kRowsPerBlock = 8;  // of one warp each
constexpr int kMaxCluster = 8;
constexpr int kMaxSlots = 8;  // of the ring of rows
constexpr int kSentAhead = 256 << 10;  // bytes of a long row; those of all SMs stay in L2
constexpr int kMaxTop = 64;
constexpr int kGroups = 128;      // of threads, for the bound of the top values
constexpr int kList = 512;        // candidates; a cluster's kMaxTop each fit too

struct LogpArgs {
  int64_t T;
  int V, top, cluster;
  int staged;  // vectors a thread keeps in shared memory (with a gradient)
  float c, scale;
  const void* x;
  int64_t stride;
  const int32_t* targets;
  float *logp, *lse, *ent;
  int32_t* ids;
  float* tops;
  const float *dlogp, *dent;
  const float *lse_in, *ent_in;  // the gradient alone
  void* dx;
  int64_t dstride;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest value of n vectors of 16 bytes (or of one element each).
template <typename T, int VEC, int N>
__device__ __forceinline__ float raw_max(const Raw<T, VEC>* r) {
  float m = -INFINITY;
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(r);
    __nv_bfloat162 p = h[0];
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) p = __hmax2(p, h[i]);
    m = fmaxf(__low2float(p), __high2float(p));
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float f[VEC];
      r[k].get(f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) m = fmaxf(m, f[i]);
    }
  }
  return m;
}

// Where a row's elements lie: `head` before the first whole vector, `vecs` vectors,
// then the rest.
struct Cut {
  int head = 0, vecs = 0, edges = 0;
  template <typename T, int VEC>
  __device__ void set(const T* x, int V) {
    head = VEC == 1 ? 0 : (int)((0u - (unsigned)(reinterpret_cast<uintptr_t>(x) / sizeof(T))) %
                                (unsigned)VEC);
    if (head > V) head = V;
    vecs = (V - head) / VEC;
    edges = V - vecs * VEC;
  }
  // the i-th element outside the vectors
  template <int VEC>
  __device__ int edge(int i) const {
    return i < head ? i : vecs * VEC + i;
  }
};

// Reference and sums of a thread (and its maximum, where the top values are wanted).
constexpr float kRise = 8.f;
template <bool ENT>
struct Sums {
  float ref = -INFINITY;  // none yet
  float limit = -INFINITY, off = 0.f, most = -INFINITY;
  float2 s = make_float2(0.f, 0.f), w = s;
  __device__ void raise(float to, float c) {
    if (ref > -INFINITY) scale((ref - to) * c);
    ref = to;
    limit = to + kRise / c;
    off = -to;
  }
  // the sums at a reference higher by -by
  __device__ void scale(float by) {
    const float a = ex2(by);
    if (ENT) {
      w.x = a * fmaf(s.x, by, w.x);
      w.y = a * fmaf(s.y, by, w.y);
      if (a == 0.f) w.x = w.y = 0.f;  // by may be -infinity
    }
    s.x *= a;
    s.y *= a;
  }
  __device__ void one(float f, float c) {
    if (f > limit) raise(f, c);
    most = fmaxf(most, f);
    const float t = (f + off) * c, e = ex2(t);
    s.x += e;
    if (ENT) w.x = fmaf(e, fmaxf(t, -256.f), w.x);
  }
  template <typename T, int VEC, int N>
  __device__ __forceinline__ void add(const Raw<T, VEC>* r, float c) {
    const float top = raw_max<T, VEC, N>(r);
    if (top > limit) raise(top, c);
    most = fmaxf(most, top);
    const float2 cc = make_float2(c, c), oo = make_float2(off, off);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float f[VEC];
      r[k].get(f);
      if (VEC == 1) {
        const float t = (f[0] + off) * c, e = ex2(t);
        s.x += e;
        if (ENT) w.x = fmaf(e, fmaxf(t, -256.f), w.x);
      }
#pragma unroll
      for (int i = 0; i + 1 < VEC; i += 2) {
        float2 t = __fmul2_rn(__fadd2_rn(make_float2(f[i], f[i + 1]), oo), cc);
        const float2 e = make_float2(ex2(t.x), ex2(t.y));
        s = __fadd2_rn(s, e);
        if (ENT) {
          t.x = fmaxf(t.x, -256.f);  // 0 times -infinity
          t.y = fmaxf(t.y, -256.f);
          w = __ffma2_rn(e, t, w);
        }
      }
    }
  }
};

// Elements of one vector of the gradient: e (A + B t).
template <int VEC, bool ENT>
__device__ __forceinline__ void grad_of(float* f, float off, float c, float A, float B) {
  if (VEC == 1) {
    const float t = (f[0] + off) * c;
    f[0] = ex2(t) * (ENT ? fmaf(B, fmaxf(t, -256.f), A) : A);
  }
  const float2 cc = make_float2(c, c), oo = make_float2(off, off), aa = make_float2(A, A),
               bb = make_float2(B, B);
#pragma unroll
  for (int i = 0; i + 1 < VEC; i += 2) {
    float2 t = __fmul2_rn(__fadd2_rn(make_float2(f[i], f[i + 1]), oo), cc);
    float2 e = make_float2(ex2(t.x), ex2(t.y));
    if (ENT) {
      t.x = fmaxf(t.x, -256.f);
      t.y = fmaxf(t.y, -256.f);
      e = __fmul2_rn(e, __ffma2_rn(bb, t, aa));
    } else {
      e = __fmul2_rn(e, aa);
    }
    f[i] = e.x, f[i + 1] = e.y;
  }
}

// The target's log probability: 0 without one, -infinity where its logit is (or every one) in
// a row whose sum is a number.
__device__ __forceinline__ float log_p(bool there, float x, float s, float ref, float scale,
                                       float logs) {
  if (!there) return 0.f;
  return s == 0.f || (x == -INFINITY && s == s) ? -INFINITY
                                                : fmaf(x - ref, scale, -kLn2 * logs);
}

template <int W>
__device__ __forceinline__ float team_max(float v, float2 (*red)[32]) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (W == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[0][warp].x = v;
  __syncthreads();
  v = red[0][lane & (W - 1)].x;
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int W>
__device__ __forceinline__ float2 team_sum(float2 v, float2 (*red)[32]) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (W == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[1][warp] = v;
  __syncthreads();
  v = red[1][lane & (W - 1)];
#pragma unroll
  for (int o = W / 2; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// ---- the CTAs of a cluster ----------------------------------------------------------
__device__ __forceinline__ uint32_t peer_at(const void* p, int rank) {
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(su32(p)), "r"(rank));
  return there;
}
__device__ __forceinline__ float peer_float(const float* p, int rank) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(peer_at(p, rank)) : "memory");
  return x;
}
__device__ __forceinline__ uint64_t peer_u64(const uint64_t* p, int rank) {
  uint64_t x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(peer_at(p, rank)) : "memory");
  return x;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// ---- order of the top values ----------------------------------------------------------
// Larger keys come first: by value (-0 as 0, NaN above all numbers).
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// and by index, the lowest first.  0 stands for none.
__device__ __forceinline__ uint64_t entry(uint32_t key, int index) {
  return (uint64_t)key << 32 | (uint32_t)~index;
}

constexpr int kAhead = 4;  // vectors that a thread loads at once
constexpr int kHits = 256;

struct TopShared {
  uint32_t keys[kGroups];
  int groups[kGroups];
  uint64_t list[kList];
  uint64_t best[kMaxTop];
  uint64_t red[8];
  uint4 hits[kHits];   // vectors with a value not below the bound, and where they are
  int hit_at[kHits];
  uint32_t bound;
  int found, chosen, hit;
};

// The slice's k first entries in order into sh.best (0 where there are fewer).
template <typename T, int VEC, int W>
__device__ void top_of_slice(TopShared& sh, const T* x, const Cut& cut, int first, int last,
                             int edges, float most, int k) {
  using R = Raw<T, VEC>;
  constexpr int G = 32 * W, SIDE = G / kGroups;  // threads of a group
  static_assert(G % kGroups == 0 && 32 % SIDE == 0, "groups within a warp");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const R* body = reinterpret_cast<const R*>(x + cut.head);
  uint32_t key = key_of(most);
#pragma unroll
  for (int o = SIDE / 2; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (tid % SIDE == 0) sh.keys[tid / SIDE] = key;
  if (tid == 0) sh.found = sh.hit = 0;
  if (tid < k) sh.best[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    // the largest bound of 16 bits that k groups reach, bit by bit, and those groups
    uint32_t mine[kGroups / 32], bound = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 32; ++j) mine[j] = sh.keys[32 * j + lane];
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t higher = bound | 1u << bit;
      int n = 0;
#pragma unroll
      for (int j = 0; j < kGroups / 32; ++j) n += mine[j] >= higher;
      if (__reduce_add_sync(0xffffffffu, n) >= k) bound = higher;
    }
    int n = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 32; ++j) {
      const unsigned reach = __ballot_sync(0xffffffffu, mine[j] >= bound);
      if (mine[j] >= bound) sh.groups[n + __popc(reach & ((1u << lane) - 1))] = 32 * j + lane;
      n += __popc(reach);
    }
    if (lane == 0) sh.bound = bound, sh.chosen = n;
  }
  __syncthreads();
  const uint32_t bound = sh.bound;
  auto offer = [&](float f, int i) {
    const uint32_t at = key_of(f);
    if (at < bound) return;
    const int n = atomicAdd(&sh.found, 1);
    if (n < kList) sh.list[n] = entry(at, i);
  };
  // half a warp a group, several vectors a lane at once: one or two waits for memory
  constexpr int HALF = 16, ROWS = HALF / SIDE;  // of the group's vectors at a time
  for (int i = tid / HALF; i < sh.chosen; i += G / HALF) {
    const int l = lane % HALF;
    for (int v = first + sh.groups[i] * SIDE + l % SIDE + G * (l / SIDE); v < last;
         v += kAhead * ROWS * G) {
      R r[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (v + k * ROWS * G < last) r[k] = body[v + k * ROWS * G];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (v + k * ROWS * G >= last || key_of(raw_max<T, VEC, 1>(r + k)) < bound) continue;
        const int n = atomicAdd(&sh.hit, 1);
        if (n < kHits) {
          *reinterpret_cast<R*>(sh.hits + n) = r[k];
          sh.hit_at[n] = cut.head + (v + k * ROWS * G) * VEC;
        }
      }
    }
  }
  __syncthreads();
  const int hits = sh.hit;
  for (int i = tid; i < min(hits, kHits) * VEC; i += G) {
    float f;
    (reinterpret_cast<const Raw<T, 1>*>(sh.hits + i / VEC) + i % VEC)->get(&f);
    offer(f, sh.hit_at[i / VEC] + i % VEC);
  }
  if (tid < edges) {
    const int i = cut.edge<VEC>(tid);
    float f;
    reinterpret_cast<const Raw<T, 1>*>(x)[i].get(&f);
    offer(f, i);
  }
  __syncthreads();
  const int n = sh.found;
  if (n <= kList && hits <= kHits) {
    for (int i = tid; i < n; i += G) {
      const uint64_t e = sh.list[i];
      int before = 0;
      for (int j = 0; j < n; ++j) before += sh.list[j] > e;
      if (before < k) sh.best[before] = e;
    }
    __syncthreads();
    return;
  }
  uint64_t prev = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t e = 0;
    auto next = [&](float f, int i) {
      const uint64_t at = entry(key_of(f), i);
      if (at < prev && at > e) e = at;
    };
    for (int v = first + tid; v < last; v += G) {
      float f[VEC];
      body[v].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) next(f[j], cut.head + v * VEC + j);
    }
    if (tid < edges) {
      const int i = cut.edge<VEC>(tid);
      float f;
      reinterpret_cast<const Raw<T, 1>*>(x)[i].get(&f);
      next(f, i);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t b = __shfl_xor_sync(0xffffffffu, e, o);
      if (b > e) e = b;
    }
    if (lane == 0) sh.red[warp] = e;
    __syncthreads();
    e = sh.red[0];
    for (int j = 1; j < W; ++j)
      if (sh.red[j] > e) e = sh.red[j];
    __syncthreads();
    if (tid == 0) sh.best[r] = e;
    prev = e;
  }
  __syncthreads();
}

// Blocks that an SM keeps, by registers: 1536 threads of 40 (1280 of 48 where entropy and
// gradient would spill), or one of a row that fills it.
__host__ __device__ constexpr int kept_blocks(int W, bool ent, bool more) {
  return W == 32 ? 1 : W == 16 ? 3 : (ent && more ? 40 : 48) / (W == 1 ? 8 : W);
}

// One row by a team of W warps (or a cluster of such blocks where p.cluster > 1); `then` is
// the team's next one.
template <typename T, int VEC, int W, bool ENT, bool TOP, bool GRAD>
__device__ __forceinline__ void logp_row(const LogpArgs& p, int64_t row, int64_t then, int rank,
                                         int tid) {
  using R = Raw<T, VEC>;
  constexpr int G = 32 * W;
  extern __shared__ uint4 stage_bytes[];
  __shared__ float2 red[2][32];
  __shared__ float meet[3];
  __shared__ typename std::conditional<TOP, TopShared, int>::type top_shared;
  const T* x = static_cast<const T*>(p.x) + row * p.stride;
  Cut cut;
  cut.set<T, VEC>(x, p.V);
  int first = 0, last = cut.vecs;
  if (W >= 8 && p.cluster > 1) {
    const int per = (cut.vecs + p.cluster - 1) / p.cluster;
    first = min(rank * per, cut.vecs);
    last = min(first + per, cut.vecs);
  }
  const R* body = reinterpret_cast<const R*>(x + cut.head);
  R* stage = reinterpret_cast<R*>(stage_bytes) + threadIdx.x;
  constexpr int stage_step = W == 1 ? 32 * kRowsPerBlock : G;
  const float c = p.c;

  Sums<ENT> sum;
  const int edges = rank == 0 ? cut.edges : 0;
  float lone = 0.f;
  if (tid < edges) {
    reinterpret_cast<const Raw<T, 1>*>(x)[cut.edge<VEC>(tid)].get(&lone);
    sum.one(lone, c);
  }
  const int staged = GRAD ? p.staged : 0;
  int kept = 0, v = first + tid;
  for (; v + (kAhead - 1) * G < last; v += kAhead * G) {
    R r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = body[v + k * G];
    sum.template add<T, VEC, kAhead>(r, c);
    if (GRAD) {
      if (kept + kAhead <= staged) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) stage[(kept + k) * stage_step] = r[k];
      } else {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (kept + k < staged) stage[(kept + k) * stage_step] = r[k];
      }
      kept += kAhead;
    }
  }
  if (v < last) {
    R r[kAhead - 1];
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k)
      if (v + k * G < last) r[k] = body[v + k * G];
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k)
      if (v + k * G < last) {
        sum.template add<T, VEC, 1>(r + k, c);
        if (GRAD && kept + k < staged) stage[(kept + k) * stage_step] = r[k];
      }
  }
  // the target and its logit, which come while the sums meet (asked for at the start
  // they would hold registers through the loop)
  int target = -1;
  float picked = 0.f;
  if (p.targets && (GRAD || (tid == 0 && rank == 0))) {
    target = p.targets[row];
    if (target >= p.V) {
      if (tid == 0 && rank == 0) record_error(TT_ERR_DEVICE, 2);
      target = -1;
    }
    if (target >= 0 && tid == 0 && rank == 0)
      reinterpret_cast<const Raw<T, 1>*>(x)[target].get(&picked);
  }
  // the team's, then the cluster's
  float most = team_max<W>(sum.ref, red);
  if (sum.ref > -INFINITY && sum.ref != most) sum.scale((sum.ref - most) * c);
  float2 sw = team_sum<W>(make_float2(sum.s.x + sum.s.y, sum.w.x + sum.w.y), red);
  if (W >= 8 && p.cluster > 1) {
    if (tid == 0) meet[0] = most, meet[1] = sw.x, meet[2] = sw.y;
    cluster_meet();
    const int lane = tid & 31;
    Sums<ENT> one;
    if (lane < p.cluster) {
      one.ref = peer_float(meet, lane);
      one.s.x = peer_float(meet + 1, lane);
      one.w.x = peer_float(meet + 2, lane);
    }
    most = one.ref;
#pragma unroll
    for (int o = kMaxCluster / 2; o; o >>= 1)
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    most = __shfl_sync(0xffffffffu, most, 0);
    if (one.ref > -INFINITY && one.ref != most) one.scale((one.ref - most) * c);
#pragma unroll
    for (int o = kMaxCluster / 2; o; o >>= 1) {
      one.s.x += __shfl_xor_sync(0xffffffffu, one.s.x, o);
      one.w.x += __shfl_xor_sync(0xffffffffu, one.w.x, o);
    }
    sw.x = __shfl_sync(0xffffffffu, one.s.x, 0);
    sw.y = __shfl_sync(0xffffffffu, one.w.x, 0);
  }
  const float ref = most > -INFINITY ? most : 0.f;
  const float logs = log2f(sw.x);  // -infinity where no logit is above it
  const float ent = sw.x == 0.f ? 0.f : kLn2 * (logs - sw.y / sw.x);
  if (tid == 0 && rank == 0) {
    if (p.lse) p.lse[row] = sw.x == 0.f ? -INFINITY : fmaf(ref, p.scale, kLn2 * logs);
    if (p.logp)
      p.logp[row] = log_p(target >= 0, picked, sw.x, ref, p.scale, logs);
    if (ENT && p.ent) p.ent[row] = ent;
  }

  if constexpr (TOP) {
    top_of_slice<T, VEC, W>(top_shared, x, cut, first, last, edges, sum.most, p.top);
    if (W >= 8 && p.cluster > 1) {
      cluster_meet();
      if (rank == 0) {
        const int n = p.cluster * p.top;
        for (int i = tid; i < n; i += G)
          top_shared.list[i] = peer_u64(top_shared.best + i % p.top, i / p.top);
        __syncthreads();
        for (int i = tid; i < n; i += G) {
          const uint64_t e = top_shared.list[i];
          int before = 0;
          for (int j = 0; j < n; ++j) before += top_shared.list[j] > e;
          if (before < p.top && e) top_shared.best[before] = e;
        }
        __syncthreads();
      }
    }
    if (rank == 0 && tid < p.top) {
      const uint64_t e = top_shared.best[tid];
      const float f = of_key((uint32_t)(e >> 32));
      p.ids[row * p.top + tid] = (int)~(uint32_t)e;
      p.tops[row * p.top + tid] =
          f == -INFINITY && logs == logs ? f : fmaf(f - ref, p.scale, -kLn2 * logs);
    }
  }

  if constexpr (GRAD) {
    if (W == 32 && VEC > 1 && tid == 0 && then < p.T) {
      // the row after this one comes to L2 while this one's gradient is written
      const T* next = static_cast<const T*>(p.x) + then * p.stride;
      Cut there;
      there.set<T, VEC>(next, p.V);
      const int bytes = min(there.vecs, kSentAhead / (int)sizeof(R)) * (int)sizeof(R);
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(next + there.head),
                   "r"(bytes)
                   : "memory");
    }
    if (W == 1) __syncwarp();  // dx may be x: the target's logit is read by now
    T* dx = static_cast<T*>(p.dx) + row * p.dstride;
    R* out = reinterpret_cast<R*>(dx + cut.head);
    const float g = target >= 0 && p.dlogp ? p.dlogp[row] : 0.f;
    const float h = ENT && p.dent ? p.dent[row] : 0.f;
    const bool none = (g == 0.f && h == 0.f) || sw.x == 0.f;
    const float inv = 1.f / sw.x;
    const float A = -p.scale * fmaf(h, ent - kLn2 * logs, g) * inv;
    const float B = -p.scale * kLn2 * h * inv;
    if (tid < edges) {
      const int i = cut.edge<VEC>(tid);
      float d = lone;
      grad_of<1, ENT>(&d, -ref, c, A, B);
      if (i == target) d = fmaf(p.scale, g, d);
      if (none) d = 0.f;
      reinterpret_cast<Raw<T, 1>*>(dx)[i].set(&d);
    }
    const int there = target >= cut.head ? (target - cut.head) / VEC : -1;
    int i = 0;
    if (none) {
      for (int v = first + tid; v < last; v += G) out[v] = R{};
    } else {
      for (int v = first + tid; v < last; v += G, ++i) {
        const R r = i < staged ? stage[i * stage_step] : body[v];
        float f[VEC];
        r.get(f);
        grad_of<VEC, ENT>(f, -ref, c, A, B);
        if (v == there) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (cut.head + v * VEC + j == target) f[j] = fmaf(p.scale, g, f[j]);
        }
        R o;
        o.set(f);
        out[v] = o;
      }
    }
  }
  if (W >= 8 && p.cluster > 1) cluster_meet();  // no CTA leaves while another reads its shares
}

template <typename T, int VEC, int W, bool ENT, bool TOP, bool GRAD>
__global__ void __launch_bounds__(W == 1 ? 32 * kRowsPerBlock : 32 * W, kept_blocks(W, ENT, GRAD))
    logp_kernel(LogpArgs p) {
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if constexpr (W == 32) {  // an SM's rows one after another
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x)
      logp_row<T, VEC, W, ENT, TOP, GRAD>(p, row, row + gridDim.x, 0, tid);
  } else {
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5)
                               : (int64_t)blockIdx.x / p.cluster;
    if (row >= p.T) return;  // whole warps, and only where no barrier is met (W == 1)
    logp_row<T, VEC, W, ENT, TOP, GRAD>(p, row, p.T, W >= 8 ? blockIdx.x % p.cluster : 0, tid);
  }
}

// Both of many rows that fit on an SM at least twice: a block an SM with a ring of rows in
// shared memory.  A row comes by one asynchronous copy of its whole vectors while the rows
// before it are worked on, so the block reads memory all the time (8192 x 32000: blocks that
// each load, sum and write in turn, three an SM, 191 us).  TEAMS teams of W warps take the
// block's rows in turn, so that one sums while another waits for its warps to meet (one team
// of 16 warps 201 us, two 163).
template <typename T, bool ENT, int TEAMS, int W>
__global__ void __launch_bounds__(32 * W * TEAMS, 1)
    logp_ring_kernel(LogpArgs p, int slots, int slot_bytes) {
  constexpr int VEC = 16 / sizeof(T), G = 32 * W;
  using R = Raw<T, VEC>;
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ uint64_t full[kMaxSlots];
  // each warp's reference and sums, and whether its team stops, of every other row
  __shared__ float4 share[TEAMS][2][W];
  __shared__ int abort_flag, sent[kMaxSlots];  // the last of the block's rows sent to a slot
  const int team = threadIdx.x / G, tid = threadIdx.x % G, warp = tid >> 5, lane = tid & 31;
  auto team_sync = [&] {
    if (TEAMS == 1)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(G) : "memory");
  };
  if (threadIdx.x == 0) {
    for (int k = 0; k < slots; ++k) mbar_init(&full[k], 1), sent[k] = -1;
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto row_at = [&](int64_t row, Cut& cut) {
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    cut.set<T, VEC>(x, p.V);
    return x;
  };
  // the block's row n to its slot
  auto send = [&](int n, int slot) {
    const int64_t row = blockIdx.x + (int64_t)n * gridDim.x;
    if (row >= p.T) return;
    __threadfence_block();
    *(volatile int*)&sent[slot] = n;
    if (n == 0 && blockIdx.x == 0 && debug_take(TT_DEBUG_LOGP_LOSS)) return;
    Cut cut;
    const T* x = row_at(row, cut);
    const uint32_t bytes = (uint32_t)(cut.vecs * sizeof(R));
    mbar_expect_tx(&full[slot], bytes);
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(su32(rows + slot * slot_bytes)),
        "l"(x + cut.head), "r"(bytes), "r"(su32(&full[slot]))
        : "memory");
  };
  // Row n is in its slot (false: the wait ran out, or another one did).  The row before it in
  // that slot may be another team's and not even have come: until n is sent the barrier is
  // a phase behind, whose parity is that of the phase after n's.
  auto arrived = [&](int n, int slot, uint32_t parity) {
    int ok = 0;
    if (lane == 0) {
      const uint64_t t0 = gtimer();
      const uint64_t limit = *(volatile unsigned long long*)&g_wait_limit_ns;
      while (!(ok = *(volatile int*)&sent[slot] == n)) {
        if (*(volatile int*)&abort_flag) break;
        if (gtimer() - t0 > limit) {
          *(volatile int*)&abort_flag = 1;
          record_error(TT_ERR_TIMEOUT, 0x701);
          break;
        }
      }
      __threadfence_block();
      ok = ok && wait_bar(&full[slot], parity, &abort_flag, 0x700);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // a shuffle orders no memory: the copy that lane 0 saw, in front of every lane's reads
    __syncwarp();
    return ok != 0;
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < slots; ++k) send(k, k);
  int n = team;
  int64_t row = blockIdx.x + (int64_t)n * gridDim.x;
  const int64_t step = (int64_t)TEAMS * gridDim.x;
  // what of a row does not come by the copy: asked for a row ahead
  Cut cut;
  float lone = 0.f, g = 0.f, h = 0.f;
  int target = -1;
  auto ahead = [&](int64_t r) {
    if (r >= p.T) return;
    const T* x = row_at(r, cut);
    if (tid < cut.edges) reinterpret_cast<const Raw<T, 1>*>(x)[cut.edge<VEC>(tid)].get(&lone);
    target = p.targets ? p.targets[r] : -1;
    g = p.dlogp ? p.dlogp[r] : 0.f;
    h = ENT && p.dent ? p.dent[r] : 0.f;
  };
  ahead(row);
  const float c = p.c;
  int slot = team, flip = 0;
  uint32_t parity = 0;
  for (; row < p.T; row += step, n += TEAMS, flip ^= 1) {
    const Cut at = cut;
    const float mine = lone, h1 = h;
    int goal = target;
    if (goal >= p.V) {
      if (tid == 0) record_error(TT_ERR_DEVICE, 2);
      goal = -1;
    }
    const float g1 = goal >= 0 ? g : 0.f;
    ahead(row + step);
    const R* have = reinterpret_cast<const R*>(rows + slot * slot_bytes);
    Sums<ENT> sum;
    if (tid < at.edges) sum.one(mine, c);
    if (arrived(n, slot, parity)) {
      int v = tid;
      for (; v + (kAhead - 1) * G < at.vecs; v += kAhead * G) {
        R r[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) r[k] = have[v + k * G];
        sum.template add<T, VEC, kAhead>(r, c);
      }
#pragma unroll
      for (int k = 0; k < kAhead - 1; ++k)
        if (v + k * G < at.vecs) {
          const R r = have[v + k * G];
          sum.template add<T, VEC, 1>(&r, c);
        }
    }
    // the warp's sums, then the block's
    auto meet = [&](Sums<ENT>& a, int most) {
      float top = a.ref;
      for (int o = most / 2; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (a.ref > -INFINITY && a.ref != top) a.scale((a.ref - top) * c);
      a.ref = top;
      a.s.x += a.s.y;
      a.w.x += a.w.y;
      for (int o = most / 2; o; o >>= 1) {
        a.s.x += __shfl_xor_sync(0xffffffffu, a.s.x, o);
        if (ENT) a.w.x += __shfl_xor_sync(0xffffffffu, a.w.x, o);
      }
    };
    meet(sum, 32);
    if (lane == 0)
      share[team][flip][warp] =
          make_float4(sum.ref, sum.s.x, sum.w.x, *(volatile int*)&abort_flag ? 1.f : 0.f);
    // the target's logit: from the copy, or from beside it before dx (which may be x) is written
    const int in_copy = goal - at.head;
    const bool copied = goal >= 0 && in_copy >= 0 && in_copy < at.vecs * VEC;
    float picked = 0.f;
    if (tid == 0 && goal >= 0 && !copied)
      (static_cast<const Raw<T, 1>*>(p.x) + row * p.stride + goal)->get(&picked);
    team_sync();
    const float4 all = share[team][flip][lane & (W - 1)];
    // the other team may give up at any time: what this one's warps saw decides for all of it
    if (__any_sync(0xffffffffu, all.w != 0.f)) break;
    Sums<ENT> one;
    one.ref = all.x;
    one.s.x = all.y;
    one.w.x = all.z;
    meet(one, W);
    const float ref = one.ref > -INFINITY ? one.ref : 0.f, s = one.s.x;
    const float logs = log2f(s);
    const float ent = s == 0.f ? 0.f : kLn2 * (logs - one.w.x / s);
    if (tid == 0) {
      if (copied) (reinterpret_cast<const Raw<T, 1>*>(have) + in_copy)->get(&picked);
      if (p.lse) p.lse[row] = s == 0.f ? -INFINITY : fmaf(ref, p.scale, kLn2 * logs);
      if (p.logp)
        p.logp[row] = log_p(goal >= 0, picked, s, ref, p.scale, logs);
      if (ENT && p.ent) p.ent[row] = ent;
    }
    T* dx = static_cast<T*>(p.dx) + row * p.dstride;
    R* out = reinterpret_cast<R*>(dx + at.head);
    const bool none = (g1 == 0.f && h1 == 0.f) || s == 0.f;
    const float inv = 1.f / s;
    const float A = -p.scale * fmaf(h1, ent - kLn2 * logs, g1) * inv;
    const float B = -p.scale * kLn2 * h1 * inv;
    if (tid < at.edges) {
      const int i = at.edge<VEC>(tid);
      float d = mine;
      grad_of<1, ENT>(&d, -ref, c, A, B);
      if (i == goal) d = fmaf(p.scale, g1, d);
      if (none) d = 0.f;
      reinterpret_cast<Raw<T, 1>*>(dx)[i].set(&d);
    }
    const int there = goal >= at.head ? (goal - at.head) / VEC : -1;
    if (none) {
      for (int v = tid; v < at.vecs; v += G) out[v] = R{};
    } else {
#pragma unroll 2
      for (int v = tid; v < at.vecs; v += G) {
        float f[VEC];
        have[v].get(f);
        grad_of<VEC, ENT>(f, -ref, c, A, B);
        if (v == there) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (at.head + v * VEC + j == goal) f[j] = fmaf(p.scale, g1, f[j]);
        }
        R o;
        o.set(f);
        out[v] = o;
      }
    }
    team_sync();  // the slot is read
    if (tid == 0) send(n + slots, slot);
    slot += TEAMS;
    if (slot >= slots) slot -= slots, parity ^= 1;
  }
  __syncthreads();
  if (abort_flag && threadIdx.x == 0)  // the copies on their way end before the block does
    for (int k = 0; k < slots; ++k)
      if (sent[k] >= 0) drain_bar(&full[k], sent[k] / slots & 1);
}

// The largest |lse| that the gradient alone takes its weights from.  Rounded to fp32 an lse is
// off by 2^-24 of itself, and the weight by as much in proportion: 2^-16 here in f32, in bf16
// 2^-12, a sixteenth of the gradient's own half step.  Beyond it (rows whose every logit is a
// mask of -1e9: lse comes in steps of 64 and has lost log V; log-sums beyond the type's range)
// the row's sum is taken again, as the pass that makes both has it.
template <typename T>
constexpr float kFarLse = sizeof(T) == 2 ? 4096.f : 256.f;
constexpr int kGradThreads = 256;

// Such a row by one warp or one block (dx may be x, whose values the sum is of), a vector a
// thread at a time, which leaves the other rows their registers (2048 x 131072 bf16 163 us,
// one row in sixteen far 213, all of them 340).
template <typename T, int VEC, bool SHORT, bool ENT>
__device__ __forceinline__ void logp_far_row(const LogpArgs& p, int64_t row) {
  using R = Raw<T, VEC>;
  constexpr int G = SHORT ? 32 : kGradThreads, W = G / 32;
  __shared__ float2 red[2][32];
  const int tid = threadIdx.x % G;
  const float c = p.c, scale = p.scale;
  const T* x = static_cast<const T*>(p.x) + row * p.stride;
  T* dx = static_cast<T*>(p.dx) + row * p.dstride;
  int target = p.targets ? p.targets[row] : -1;
  if (target >= p.V) {
    if (tid == 0) record_error(TT_ERR_DEVICE, 2);
    target = -1;
  }
  const float g = target >= 0 && p.dlogp ? p.dlogp[row] : 0.f;
  const float h = ENT ? p.dent[row] : 0.f;
  const float A = ENT ? -scale * fmaf(h, p.ent_in[row], g) : -scale * g, B = -scale * h;
  Cut cut;
  cut.set<T, VEC>(x, p.V);
  const R* body = reinterpret_cast<const R*>(x + cut.head);
  R* out = reinterpret_cast<R*>(dx + cut.head);
  Sums<false> sum;
  float lone = 0.f;
  if (tid < cut.edges) {
    reinterpret_cast<const Raw<T, 1>*>(x)[cut.edge<VEC>(tid)].get(&lone);
    sum.one(lone, c);
  }
#pragma unroll 1
  for (int v = tid; v < cut.vecs; v += G) {
    const R r = body[v];
    sum.template add<T, VEC, 1>(&r, c);
  }
  const float most = team_max<W>(sum.ref, red);
  if (sum.ref > -INFINITY && sum.ref != most) sum.scale((sum.ref - most) * c);
  const float s = team_sum<W>(make_float2(sum.s.x + sum.s.y, 0.f), red).x;
  const float ref = most > -INFINITY ? most : 0.f, less = -kLn2 * log2f(s);
  auto grad = [&](float f, int i) {
    const float lp = fmaf(f - ref, scale, less);
    const float d = ex2(lp * kLog2e) * (ENT ? fmaf(B, fmaxf(lp, -256.f), A) : A);
    return s == 0.f ? 0.f : i == target ? fmaf(scale, g, d) : d;  // 0: no logit above -infinity
  };
  // each thread the elements that it read before
  if (tid < cut.edges) {
    const int i = cut.edge<VEC>(tid);
    lone = grad(lone, i);
    reinterpret_cast<Raw<T, 1>*>(dx)[i].set(&lone);
  }
#pragma unroll 1
  for (int v = tid; v < cut.vecs; v += G) {
    float f[VEC];
    body[v].get(f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = grad(f[j], cut.head + v * VEC + j);
    R o;
    o.set(f);
    out[v] = o;
  }
}

// Blocks that an SM keeps, by registers; only far rows spill.  Without a limit their code takes
// the other rows' registers: with the entropy bf16 2048 x 131072 171 -> 179 us, 16384 x 2500 55
// -> 66; f32 2048 x 65536 without it 154 -> 159 (five blocks: 173, 58, 164).
__host__ __device__ constexpr int grad_blocks(int vec, bool brief, bool ent) {
  return vec == 1 ? 8 : brief ? 4 : vec == 4 && !ent ? 7 : 6;
}

// The gradient alone, from the row's log-sum and entropy: a block a piece of a row
// (a warp a row where rows are short).
template <typename T, int VEC, bool SHORT, bool ENT>
__global__ void __launch_bounds__(kGradThreads, grad_blocks(VEC, SHORT, ENT))
    logp_grad_kernel(const __grid_constant__ LogpArgs p, int pieces) {
  using R = Raw<T, VEC>;
  constexpr int G = SHORT ? 32 : kGradThreads;
  const int tid = SHORT ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = SHORT ? (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5)
                            : (int64_t)blockIdx.x / pieces;
  const int piece = SHORT ? 0 : blockIdx.x % pieces;
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;
  const T* x = static_cast<const T*>(p.x) + row * p.stride;
  T* dx = static_cast<T*>(p.dx) + row * p.dstride;
  Cut cut;
  cut.set<T, VEC>(x, p.V);
  const R* body = reinterpret_cast<const R*>(x + cut.head);
  R* out = reinterpret_cast<R*>(dx + cut.head);
  int target = p.targets ? p.targets[row] : -1;
  if (target >= p.V) {
    if (tid == 0 && piece == 0) record_error(TT_ERR_DEVICE, 2);
    target = -1;
  }
  const float lse = p.lse_in[row];
  const float g = target >= 0 && p.dlogp ? p.dlogp[row] : 0.f;
  const float h = ENT ? p.dent[row] : 0.f;
  const bool none = g == 0.f && h == 0.f;
  const float A = ENT ? -p.scale * fmaf(h, p.ent_in[row], g) : -p.scale * g, B = -p.scale * h;
  auto grad = [&](float f) {
    const float lp = fmaf(f, p.scale, -lse);
    return ex2(lp * kLog2e) * (ENT ? fmaf(B, fmaxf(lp, -256.f), A) : A);
  };
  const int there = target >= cut.head ? (target - cut.head) / VEC : -1;
  const int first = SHORT ? 0 : piece * kAhead * G;
  const int last = SHORT ? cut.vecs : min(cut.vecs, first + kAhead * G);
  float lone = 0.f;
  const bool edge = piece == 0 && tid < cut.edges;
  if (edge) reinterpret_cast<const Raw<T, 1>*>(x)[cut.edge<VEC>(tid)].get(&lone);
  const bool far = !none && fabsf(lse) > kFarLse<T>;
  for (int v = first + tid; v < last; v += kAhead * G) {
    R r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (v + k * G < last) r[k] = body[v + k * G];
    if (none || far) break;  // asked behind the loads, which do not wait for lse
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = v + k * G;
      if (at >= last) break;
      float f[VEC];
      r[k].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = grad(f[j]);
      if (at == there) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (cut.head + at * VEC + j == target) f[j] = fmaf(p.scale, g, f[j]);
      }
      R o;
      o.set(f);
      out[at] = o;
    }
  }
  if (far) {
    if (piece == 0) logp_far_row<T, VEC, SHORT, ENT>(p, row);
    return;
  }
  if (none)
    for (int v = first + tid; v < last; v += G) out[v] = R{};
  if (edge) {
    const int i = cut.edge<VEC>(tid);
    float d = grad(lone);
    if (i == target) d = fmaf(p.scale, g, d);
    if (none) d = 0.f;
    reinterpret_cast<Raw<T, 1>*>(dx)[i].set(&d);
  }
}

// ---- dispatch --------------------------------------------------------------------

// Whether row t of x and of dx start at the same distance from a 16-byte boundary.
bool alike(const LogpArgs& a, size_t size) {
  const uintptr_t gap = reinterpret_cast<uintptr_t>(a.x) - reinterpret_cast<uintptr_t>(a.dx);
  return gap % 16 == 0 && (a.T == 1 || ((uint64_t)(a.stride - a.dstride) * size) % 16 == 0);
}

constexpr size_t kStageBytes = 216 << 10;  // most that a CTA keeps of a row

// Clusters for few rows: CTAs for every SM, but no fewer than four vectors a thread of each.
template <int W>
int cluster_of(int64_t rows, int64_t vecs) {
  int n = 1;
  while (n < kMaxCluster && vecs / (2 * n) >= 4 * 32 * W &&
         rows * n < 2 * (int64_t)device_sms())
    n *= 2;
  return n;
}

template <typename T, int VEC, int W, bool ENT, bool TOP, bool GRAD>
cudaError_t go(LogpArgs& a, cudaStream_t st) {
  auto kernel = logp_kernel<T, VEC, W, ENT, TOP, GRAD>;
  constexpr int threads = W == 1 ? 32 * kRowsPerBlock : 32 * W;
  const int64_t rows = W == 1 ? (a.T + kRowsPerBlock - 1) / kRowsPerBlock : a.T;
  const int64_t vecs = a.V / VEC + 1;  // of a row, at most
  a.cluster = W == 8 || W == 16 ? cluster_of<W>(rows, vecs) : 1;
  size_t smem = 0;
  a.staged = 0;
  if (GRAD) {
    const size_t each = sizeof(Raw<T, VEC>) * threads;
    const int64_t need = ((vecs + a.cluster - 1) / a.cluster + 32 * W - 1) / (32 * W);
    a.staged = (int)(need * each <= kStageBytes ? need : kStageBytes / each);
    smem = a.staged * each;
    static PerDevice once;
    const cudaError_t e = once.get([&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)kStageBytes);
    });
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = W == 32 && rows > device_sms() ? device_sms() : rows * a.cluster;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  return a.cluster > 1 ? launch_cluster(kernel, grid, dim3(threads), smem, st, a.cluster, a)
                       : launch_ex(kernel, grid, dim3(threads), smem, st, false, a);
}

template <typename T, bool ENT, int TEAMS, int W>
cudaError_t ring_go(const LogpArgs& a, int slots, size_t bytes, cudaStream_t st) {
  auto kernel = logp_ring_kernel<T, ENT, TEAMS, W>;
  static PerDevice once;
  const cudaError_t e = once.get([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kStageBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_ex(kernel, dim3((unsigned)device_sms()), dim3(32 * W * TEAMS),
                   slots * bytes, st, false, a, slots, (int)bytes);
}

// Warps of a row by its vectors: a warp alone to sixteen a lane (16384 x 1000 bf16 with
// four warps 24.0 us, with one 10.7), then four warps, whose barrier costs little.  With a
// gradient, rows above 24 KB that are many go by the ring: in two slots by one team, three
// or four by two, more by four (16384 x 13000 a block a row 212 us, by the ring 140; 8192 x
// 32000 191 and 163; 16384 x 8000, 16 KB a row, 99 and 112).  Others stay in shared memory
// with 16 warps each, above 108 KB with 32 on an SM of its own, and what exceeds the shared
// memory is read again from L2 (2048 x 131072 in clusters of four 371 us, so 225, and 210 with
// the next row sent for while a gradient is written; f32 4096 x 50001 361, 387 and 312).
template <typename T, int VEC, bool ENT, bool TOP, bool GRAD>
cudaError_t by_width(LogpArgs& a, cudaStream_t st) {
  const int64_t vecs = a.V / VEC;
  if constexpr (!TOP)
    if (vecs <= 512) return go<T, VEC, 1, ENT, TOP, GRAD>(a, st);
  if (vecs <= 1536) return go<T, VEC, 4, ENT, TOP, GRAD>(a, st);
  if constexpr (GRAD) {
    const size_t bytes = ((size_t)vecs * sizeof(Raw<T, VEC>) + 127) / 128 * 128;
    if constexpr (VEC > 1)
      if (2 * bytes <= kStageBytes && a.T >= 4 * (int64_t)device_sms()) {
        const int slots = (int)(kStageBytes / bytes);
        return slots >= 5   ? ring_go<T, ENT, 4, 8>(a, slots < kMaxSlots ? slots : kMaxSlots,
                                                  bytes, st)
               : slots >= 3 ? ring_go<T, ENT, 2, 16>(a, slots, bytes, st)
                            : ring_go<T, ENT, 1, 16>(a, slots, bytes, st);
      }
    if (a.V * (int64_t)sizeof(T) > (108 << 10) && cluster_of<16>(a.T, vecs) == 1)
      return go<T, VEC, 32, ENT, TOP, GRAD>(a, st);
    return go<T, VEC, 16, ENT, TOP, GRAD>(a, st);
  } else {
    return go<T, VEC, 8, ENT, TOP, GRAD>(a, st);
  }
}

template <typename T>
cudaError_t forward(LogpArgs& a, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  if (a.top)
    return a.ent ? by_width<T, VEC, true, true, false>(a, st)
                 : by_width<T, VEC, false, true, false>(a, st);
  return a.ent ? by_width<T, VEC, true, false, false>(a, st)
               : by_width<T, VEC, false, false, false>(a, st);
}
template <typename T>
cudaError_t loss(LogpArgs& a, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  const bool ent = a.ent || a.dent;
  if (!alike(a, sizeof(T)))
    return ent ? by_width<T, 1, true, false, true>(a, st)
               : by_width<T, 1, false, false, true>(a, st);
  return ent ? by_width<T, VEC, true, false, true>(a, st)
             : by_width<T, VEC, false, false, true>(a, st);
}
template <typename T, int VEC, bool ENT>
cudaError_t grad_go(LogpArgs& a, cudaStream_t st) {
  const int64_t vecs = a.V / VEC;
  const int64_t pieces = (vecs + kAhead * kGradThreads - 1) / (kAhead * kGradThreads);
  const bool brief = vecs <= 128;
  const int64_t blocks = brief ? (a.T + kRowsPerBlock - 1) / kRowsPerBlock : a.T * pieces;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_ex(brief ? logp_grad_kernel<T, VEC, true, ENT>
                         : logp_grad_kernel<T, VEC, false, ENT>,
                   dim3((unsigned)blocks), dim3(kGradThreads), 0, st, false, a, (int)pieces);
}
template <typename T>
cudaError_t backward(LogpArgs& a, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  if (!alike(a, sizeof(T)))
    return a.dent ? grad_go<T, 1, true>(a, st) : grad_go<T, 1, false>(a, st);
  return a.dent ? grad_go<T, VEC, true>(a, st) : grad_go<T, VEC, false>(a, st);
}

// The arguments that every call has.
bool common_ok(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
               const int32_t* targets, LogpArgs* a) {
  if (!plan || plan->kind != 8 || T < 0 || T > 0x7FFFFFFF) return false;
  const LogpPlan& P = plan->logits;
  if (stride < P.V || stride > (int64_t)1 << 31 || !aligned_to(targets, 4) ||
      !aligned_to(logits, P.act == TT_DT_F32 ? 4 : 2) || (T > 0 && !logits))
    return false;
  *a = LogpArgs{};
  a->T = T;
  a->V = (int)P.V;
  a->c = P.scale * kLog2e;
  a->scale = P.scale;
  a->x = logits;
  a->stride = stride;
  a->targets = targets;
  return true;
}

tt_status done(cudaError_t e, cudaStream_t st) {
  prof_end(kPhElem, st);
  count_launches(1);
  return e == cudaErrorInvalidConfiguration ? TT_ERR_UNSUPPORTED
         : e == cudaSuccess                 ? TT_OK
                                            : TT_ERR_CUDA;
}

}  // namespace
}  // namespace ttc

using namespace ttc;

extern "C" {

tt_status tt_logp_plan(const tt_logp_desc* desc, tt_plan_t** out) {
  if (!out) return TT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || desc->V < 1 || !(desc->scale >= 1e-6f) || !(desc->scale <= 1e6f) ||
      desc->top < 0 || desc->top > desc->V)
    return TT_ERR_INVALID_ARG;
  if (desc->act != TT_DT_F32 && desc->act != TT_DT_BF16 && desc->act != TT_DT_E4M3)
    return TT_ERR_INVALID_ARG;
  if (desc->act == TT_DT_E4M3 || desc->V > (1 << 24) || desc->top > kMaxTop)
    return TT_ERR_UNSUPPORTED;
  tt_plan_s* p = new (std::nothrow) tt_plan_s();
  if (!p) return TT_ERR_INVALID_ARG;
  p->kind = 8;
  p->logits.V = desc->V;
  p->logits.scale = desc->scale;
  p->logits.top = desc->top;
  p->logits.act = desc->act;
  *out = p;
  return TT_OK;
}

tt_status tt_logp_forward(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                          const int32_t* targets, float* logp, float* lse, float* entropy,
                          int32_t* top, float* top_logp, void* stream) {
  LogpArgs a;
  if (!common_ok(plan, T, logits, stride, targets, &a) || (logp && !targets) ||
      (!top) != (!top_logp) || (top && !plan->logits.top) || !aligned_to(logp, 4) ||
      !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(top, 4) ||
      !aligned_to(top_logp, 4))
    return TT_ERR_INVALID_ARG;
  if (T == 0) return TT_OK;
  a.logp = logp;
  a.lse = lse;
  a.ent = entropy;
  a.top = top ? plan->logits.top : 0;
  a.ids = top;
  a.tops = top_logp;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  return done(plan->logits.act == TT_DT_BF16 ? forward<__nv_bfloat16>(a, st)
                                             : forward<float>(a, st), st);
}

tt_status tt_logp_backward(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                           const int32_t* targets, const float* lse, const float* dlogp,
                           const float* entropy, const float* dentropy, void* dlogits,
                           int64_t dstride, void* stream) {
  LogpArgs a;
  if (!common_ok(plan, T, logits, stride, targets, &a) || dstride < a.V ||
      dstride > (int64_t)1 << 31 || (dlogp && !targets) || (dentropy && !entropy) ||
      (T > 0 && ((!dlogp && !dentropy) || !lse || !dlogits)) || !aligned_to(lse, 4) ||
      !aligned_to(dlogp, 4) || !aligned_to(entropy, 4) || !aligned_to(dentropy, 4) ||
      !aligned_to(dlogits, plan->logits.act == TT_DT_F32 ? 4 : 2))
    return TT_ERR_INVALID_ARG;
  if (T == 0) return TT_OK;
  a.lse_in = lse;
  a.dlogp = dlogp;
  a.ent_in = entropy;
  a.dent = dentropy;
  a.dx = dlogits;
  a.dstride = dstride;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  return done(plan->logits.act == TT_DT_BF16 ? backward<__nv_bfloat16>(a, st)
                                             : backward<float>(a, st), st);
}

tt_status tt_logp_loss(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                       const int32_t* targets, const float* dlogp, const float* dentropy,
                       float* logp, float* lse, float* entropy, void* dlogits, int64_t dstride,
                       void* stream) {
  LogpArgs a;
  if (!common_ok(plan, T, logits, stride, targets, &a) || dstride < a.V ||
      dstride > (int64_t)1 << 31 || ((dlogp || logp) && !targets) ||
      (T > 0 && ((!dlogp && !dentropy) || !dlogits)) || !aligned_to(logp, 4) ||
      !aligned_to(lse, 4) ||
      !aligned_to(entropy, 4) || !aligned_to(dlogp, 4) || !aligned_to(dentropy, 4) ||
      !aligned_to(dlogits, plan->logits.act == TT_DT_F32 ? 4 : 2))
    return TT_ERR_INVALID_ARG;
  if (T == 0) return TT_OK;
  a.logp = logp;
  a.lse = lse;
  a.ent = entropy;
  a.dlogp = dlogp;
  a.dent = dentropy;
  a.dx = dlogits;
  a.dstride = dstride;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  return done(plan->logits.act == TT_DT_BF16 ? loss<__nv_bfloat16>(a, st) : loss<float>(a, st),
              st);
}

}  // extern "C"
