// Norm of queries and keys for each head with the rotation by position in the
// same pass: forward (into dense tensors or into the rows of a cache), backward
// with the reduction of the weight gradients.
//
// Both are bound by HBM: a head's values are read once into registers and written
// once.  A warp holds 32 / group heads side by side, the same ones for every token it
// takes: its pointers step from row to row, its weights stay in registers, and so do
// the backward's sums.  A lane holds both channels of each of its pairs (two chunks of
// P consecutive channels half a rotation apart, or one run of 2 P where neighbours are
// pairs), so the rotation needs no exchange and the norm's sums only those over a
// head's lanes.  The warp's lanes compute the angles of its token, a pair each, and
// share them through shared memory: each warp of a token does so again, which takes
// fewer instructions than a warp that goes through all of a token's heads spends on
// finding them (16384 tokens of 24 heads of 64 in bf16: 36 us, backward 98).
//
// An angle is pos f modulo a turn.  The frequency is held as a 64-bit fraction of a
// turn, so the product modulo 2^64 is that reduction itself, without rounding: the
// error is the frequency's own (2^-52 of it, times the position), at any position
// of 31 bits.  The nearest quarter turn is taken off; sine and cosine of the rest, an
// eighth of a turn at most, come from the hardware's approximation in bf16 (off by
// 2^-20, where the output's half step is 2^-8), in f32 from their Taylor series to the
// ninth and tenth power, whose next terms are below 2^-28 at an eighth of a turn.
#include <cmath>
#include <new>

#include "rows.cuh"
#include "ttc.h"
#include "ttc_internal.h"

namespace ttc {

cudaError_t read_and_clear_rope_status(DeviceStatus* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(DeviceStatus));
  if (e != cudaSuccess || out->code == 0) return e;
  DeviceStatus z{0, 0};
  return cudaMemcpyToSymbol(g_status, &z, sizeof(z));
}

namespace {

constexpr int kMaxPairs = 128;  // of a head of 256
constexpr int kWarps = 8;       // warps a block

struct RopeArgs {
  int64_t T;
  int heads, kv, dim, rot;
  int group;       // lanes of a head
  int side;        // heads side by side in a warp: 32 / group
  int chunks;      // chunks of a head: the rotated ones, then the rest
  int turned;      // rotated chunks
  int passes;      // warps of a token
  int norm;        // 0: rotation alone
  float inv_n, eps;
  const int32_t* pos;
  const int32_t* rows;  // k and v go to these rows of ko and vo
  int64_t cache_rows;
  Heads q, k, v, qo, ko, vo;  // backward: qo, ko are the gradients of q and k
  Heads dq, dk;
  int values;                 // v is copied too
  const float *gq, *gk;
  float* sums;                // backward: [gridDim.x][2 dim] shares of dgq, dgk
  float *dgq, *dgk;           // written directly by a grid of one block
  int accumulate;
  uint64_t turn[kMaxPairs];   // frequencies, as fractions of a turn
};

// cos and sin of pos frequency
template <typename T>
__device__ __forceinline__ void angle(int64_t pos, uint64_t turn, float* cosine, float* sine) {
  const uint64_t a = (uint64_t)pos * turn;
  const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
  // in [-2^61, 2^61), where 2^63 is half a turn; 2^-31 of it fits 31 bits
  const int32_t rest = (int32_t)((int64_t)(a - ((uint64_t)quarter << 62)) >> 31);
  const float x = (float)rest * (float)(3.14159265358979323846 * 0x1p-32);
  float s, c;
  if (sizeof(T) == 2) {
    s = __sinf(x);
    c = __cosf(x);
  } else {
    const float y = x * x;
    s = fmaf(y, 1.f / 362880, -1.f / 5040);
    s = fmaf(y, s, 1.f / 120);
    s = fmaf(y, s, -1.f / 6);
    s = fmaf(x * y, s, x);
    c = fmaf(y, -1.f / 3628800, 1.f / 40320);
    c = fmaf(y, c, -1.f / 720);
    c = fmaf(y, c, 1.f / 24);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.f);
  }
  const float u = quarter & 1 ? -s : c, v = quarter & 1 ? c : s;
  *cosine = quarter & 2 ? -u : u;
  *sine = quarter & 2 ? -v : v;
}

// A lane's share of a head: the first channels of its pairs and the second ones.
template <int P>
struct Pairs {
  float a[P], b[P];
};

// Where that lies: two runs of P channels as they are in memory.  PAIRS: neighbouring
// channels are a pair.  The channels that are not rotated are dealt in the same runs.
template <typename T, int P, bool PAIRS>
struct Place {
  using R = Raw<T, P>;
  int at, at2;      // channels
  bool has, has2;
  __device__ void set(const RopeArgs& p, int i) {
    has = i < p.chunks;
    if (i < p.turned) {
      at = PAIRS ? 2 * P * i : P * i;
      at2 = PAIRS ? at + P : p.rot / 2 + P * i;
    } else {
      at = p.rot + 2 * P * (i - p.turned);
      at2 = at + P;
    }
    has2 = has && at2 < p.dim;
  }
  __device__ void load(const T* x, R& u, R& v) const {
    if (has) u = *reinterpret_cast<const R*>(x + at);
    if (has2) v = *reinterpret_cast<const R*>(x + at2);
  }
  // runs to pairs and back
  __device__ static void split(const float* u, const float* v, Pairs<P>& x) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int k = 2 * j;
      x.a[j] = !PAIRS || P == 1 ? u[j] : k < P ? u[k] : v[k - P];
      x.b[j] = !PAIRS || P == 1 ? v[j] : k < P ? u[k + 1] : v[k + 1 - P];
    }
  }
  __device__ static void join(const Pairs<P>& x, float* u, float* v) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      u[j] = !PAIRS || P == 1 ? x.a[j] : j % 2 ? x.b[j / 2] : x.a[j / 2];
      v[j] = !PAIRS || P == 1 ? x.b[j] : j % 2 ? x.b[(P + j) / 2] : x.a[(P + j) / 2];
    }
  }
  __device__ void get(const R& ru, const R& rv, Pairs<P>& x) const {
    float u[P], v[P];
    ru.get(u);
    rv.get(v);
    split(u, v, x);
  }
  __device__ void put(T* y, const Pairs<P>& x) const {
    float u[P], v[P];
    join(x, u, v);
    R o;
    o.set(u);
    if (has) *reinterpret_cast<R*>(y + at) = o;
    o.set(v);
    if (has2) *reinterpret_cast<R*>(y + at2) = o;
  }
  // the channels of pair n of a head
  __device__ static void pair(const RopeArgs& p, int n, int& a, int& b) {
    Place q;
    q.set(p, n / P);
    a = q.at + (PAIRS ? 2 * (n % P) : n % P);
    b = PAIRS ? a + 1 : q.at2 + n % P;
  }
};

template <int P>
__device__ __forceinline__ void from_shared(const float* p, float* f) {
  if constexpr (P < 4) {
#pragma unroll
    for (int j = 0; j < P; ++j) f[j] = p[j];
  } else {
#pragma unroll
    for (int j = 0; j < P; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + j);
      f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
    }
  }
}

// x turned by the angle, or back.
template <int P>
__device__ __forceinline__ void turn_by(const float* cosine, const float* sine, bool back,
                                        Pairs<P>& x) {
  float c[P], s[P], m[P], u[P], v[P];
  from_shared<P>(cosine, c);
  from_shared<P>(sine, s);
#pragma unroll
  for (int j = 0; j < P; ++j) {
    m[j] = -s[j];
  }
  mul<P>(x.a, c, u);
  mul<P>(x.b, c, v);
  fma<P>(x.b, back ? s : m, u, u);
  fma<P>(x.a, back ? m : s, v, x.b);
#pragma unroll
  for (int j = 0; j < P; ++j) x.a[j] = u[j];
}

// 1 / sqrt(x): the hardware's approximation and one step of Newton's iteration, which has no
// meaning for an infinity (a sum of squares beyond fp32): 0, as the quotient is.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return x < INFINITY ? fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r) : r;
}

// The sum over the lanes of each head, lane i of which this one is.  Known powers of two by
// exchanges; else from the upper lanes to the lower, in the same steps for every number
// (a loop's branches cost heads of ten lanes a sixth of their instructions), then from the
// first lane to all.  `takes`: bit k where step k adds a lane's value to this one.
__device__ __forceinline__ uint32_t sum_steps(int group, int i) {
  uint32_t takes = 0;
#pragma unroll
  for (int k = 0; k < 5; ++k) takes |= (uint32_t)(i < 1 << k && i + (1 << k) < group) << k;
  return takes;
}
template <int GROUP>
__device__ __forceinline__ float head_sum(float v, uint32_t takes, int first) {
  if constexpr (GROUP > 0) {
#pragma unroll
    for (int o = GROUP / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
#pragma unroll
  for (int k = 4; k >= 0; --k) {
    const float u = __shfl_down_sync(0xffffffffu, v, 1 << k);
    v += takes >> k & 1 ? u : 0.f;
  }
  return __shfl_sync(0xffffffffu, v, first);
}

// A lane's loads on their way: copied asynchronously to slots of its own in shared
// memory, two tokens ahead.  (In registers one token ahead, a warp waited for memory
// in four of ten cycles: backward of 16384 tokens of 24 heads of 64 38.4 us.)  Single bf16
// values, which the asynchronous copy does not take, go one token ahead in registers.
constexpr int kDepth = 3;
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if constexpr (BYTES == 16)
    copy_async16(to, from);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(su32(to)), "l"(from),
                 "n"(BYTES)
                 : "memory");
}

// Blocks of 256 threads that an SM holds.
constexpr int kGradPerSm = 2, kPerSm = 3;

// Shared memory of a block's copies: two runs a lane of x, and of dy.
template <typename T, int P, int CH, bool GRAD>
constexpr size_t ring_bytes() {
  return P * sizeof(T) >= 4 ? (size_t)kDepth * kWarps * 32 * CH * P * sizeof(T) * (GRAD ? 4 : 2)
                            : 0;
}

// GROUP: the lanes of a head where they are known (16 and 32 bytes a lane of heads of 64
// and 128), else 0.
template <typename T, int P, int CH, bool PAIRS, bool GRAD, int GROUP>
__global__ void __launch_bounds__(32 * kWarps, GRAD ? kGradPerSm : kPerSm)
    rope_kernel(const __grid_constant__ RopeArgs p) {
  using R = Raw<T, P>;
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ __align__(16) float cosines[kWarps][kMaxPairs], sines[kWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][2][kMaxPairs];  // of q and k, by pairs
  __shared__ float cross[GRAD ? kWarps : 1][GRAD ? 2 * 2 * kMaxPairs : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.rot / 2; i += 32 * kWarps) turn[i] = p.turn[i];
  for (int i = p.rot / 2 + lane; i < kMaxPairs; i += 32) {  // what is not rotated
    cosines[warp][i] = 1.f;
    sines[warp][i] = 0.f;
  }
  pdl_wait();
  pdl_trigger();
  if (p.norm)
    for (int i = threadIdx.x; i < 2 * kMaxPairs; i += 32 * kWarps) {
      const float* g = i < kMaxPairs ? p.gq : p.gk;
      int a, b;
      Place<T, P, PAIRS>::pair(p, i % kMaxPairs, a, b);
      weights[i / kMaxPairs][0][i % kMaxPairs] = a < p.dim ? g ? __ldg(g + a) : 1.f : 0.f;
      weights[i / kMaxPairs][1][i % kMaxPairs] = b < p.dim ? g ? __ldg(g + b) : 1.f : 0.f;
    }
  __syncthreads();
  // this lane's head and channels
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t step = (int64_t)gridDim.x * kWarps / p.passes;
  const int group = GROUP ? GROUP : p.group, side = GROUP ? 32 / GROUP : p.side;
  const int beside = lane / group, li = lane - beside * group;
  const uint32_t takes = GROUP ? 0 : sum_steps(group, li);
  int h = (int)(w % p.passes) * side + beside;
  int64_t t = w / p.passes;
  if (t >= step) t = p.T;
  const int which = h < p.heads ? 0 : h < p.heads + p.kv ? 1 : 2;
  h -= which == 0 ? 0 : which == 1 ? p.heads : p.heads + p.kv;
  const bool here = beside < side && (which == 0 || (h < p.kv && (which == 1 || p.values)));
  Place<T, P, PAIRS> at[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    at[c].set(p, c * group + li);
    if (!here) at[c].has = at[c].has2 = false;
  }
  const int share = li * P;  // its pairs in the table of angles
  const float* mine = &weights[which == 0 ? 0 : 1][0][share];
  auto weight = [&](int c, Pairs<P>& g) {
    from_shared<P>(mine + group * P * c, g.a);
    from_shared<P>(mine + kMaxPairs + group * P * c, g.b);
  };
  // where the head starts in the tensors' first row
  const bool reads = !GRAD || p.norm;
  if (!here) h = 0;
  const T* x = which == 0 ? p.q.at<T>(t, h) : which == 1 ? p.k.at<T>(t, h) : p.v.at<T>(t, h);
  const int64_t step_in = step * (which == 0 ? p.q.row : which == 1 ? p.k.row : p.v.row);
  const T* d = which == 0 ? p.dq.at<T>(t, h) : p.dk.at<T>(t, h);
  const int64_t step_grad = step * (which == 0 ? p.dq.row : p.dk.row);
  T* y = which == 0 ? p.qo.at<T>(0, h) : which == 1 ? p.ko.at<T>(0, h) : p.vo.at<T>(0, h);
  const int64_t row_out = which == 0 ? p.qo.row : which == 1 ? p.ko.row : p.vo.row;

  R xu[CH] = {}, xv[CH] = {}, du[GRAD ? CH : 1] = {}, dv[GRAD ? CH : 1] = {};
  int pos = 0, row = 0;
  // One token's loads; with copies into slot k of the lane, and of the warp for the position.
  extern __shared__ uint4 ring[];
  __shared__ int at_pos[kWarps][kDepth], at_row[kWarps][kDepth];
  constexpr bool copies = sizeof(R) >= 4;
  constexpr int runs = (GRAD ? 4 : 2) * CH;
  R* slots = reinterpret_cast<R*>(ring) + warp * kDepth * runs * 32 + lane;
  auto fetch = [&](int64_t t, int k) {
    if constexpr (copies) {
      constexpr int bytes = sizeof(R);
      R* to = slots + k * runs * 32;
      if (t < p.T) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          R* mine = to + c * (GRAD ? 128 : 64);
          if (reads && at[c].has) copy_async<bytes>(mine, x + at[c].at);
          if (reads && at[c].has2) copy_async<bytes>(mine + 32, x + at[c].at2);
          if constexpr (GRAD) {
            if (at[c].has) copy_async<bytes>(mine + 64, d + at[c].at);
            if (at[c].has2) copy_async<bytes>(mine + 96, d + at[c].at2);
          }
        }
        if (lane == 0 && p.pos) copy_async<4>(&at_pos[warp][k], p.pos + t);
        if (lane == 0 && !GRAD && p.rows) copy_async<4>(&at_row[warp][k], p.rows + t);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else if (t < p.T) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (reads) at[c].load(x, xu[c], xv[c]);
        if constexpr (GRAD) at[c].load(d, du[c], dv[c]);
      }
      pos = p.pos ? p.pos[t] : (int)t;
      row = !GRAD && p.rows && which > 0 ? p.rows[t] : (int)t;
    }
    x += step_in;
    if constexpr (GRAD) d += step_grad;
  };
  Pairs<P> sum[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) fill<P>(0.f, sum[c].a), fill<P>(0.f, sum[c].b);

  if constexpr (copies) {
    // channels and heads that are not there stay zeros
    for (int i = 0; i < kDepth * runs; ++i) slots[i * 32] = R{};
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) fetch(t + k * step, k);
  } else {
    fetch(t, 0);
  }
  int slot = 0;
  for (; t < p.T; t += step) {
    if constexpr (copies) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      __syncwarp();
      pos = p.pos ? at_pos[warp][slot] : (int)t;
      row = !GRAD && p.rows && which > 0 ? at_row[warp][slot] : (int)t;
      const R* have = slots + slot * runs * 32;
#pragma unroll
      for (int c = 0; c < CH; ++c, have += GRAD ? 128 : 64) {
        xu[c] = have[0], xv[c] = have[32];
        if constexpr (GRAD) du[c] = have[64], dv[c] = have[96];
      }
    } else {
      __syncwarp();
    }
    for (int i = lane; i < p.rot / 2; i += 32)
      angle<T>(pos, turn[i], &cosines[warp][i], &sines[warp][i]);
    __syncwarp();
    bool kept = here;
    if (!GRAD && p.rows && which > 0) {
      if (row < 0 || row >= p.cache_rows) {
        if (row >= 0) record_error(TT_ERR_DEVICE, 1);
        kept = false;
      }
    }
    T* out = y + (int64_t)(kept ? row : 0) * row_out;
    Pairs<P> u[CH], e[GRAD ? CH : 1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      at[c].get(xu[c], xv[c], u[c]);
      if constexpr (GRAD) {
        at[c].get(du[c], dv[c], e[c]);
      } else if (which == 2 && kept) {  // v goes as it is
        if (at[c].has) *reinterpret_cast<R*>(out + at[c].at) = xu[c];
        if (at[c].has2) *reinterpret_cast<R*>(out + at[c].at2) = xv[c];
      }
    }
    // the slot that the token before this one was in
    fetch(t + (copies ? kDepth - 1 : 1) * step, slot == 0 ? kDepth - 1 : slot - 1);
    slot = slot == kDepth - 1 ? 0 : slot + 1;

    if constexpr (!GRAD) {
      if (p.norm) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) mul_up<P>(s2, u[c].a, u[c].a), mul_up<P>(s2, u[c].b, u[c].b);
        float s = s2.x + s2.y;
        s = head_sum<GROUP>(s, takes, lane - li);
        float r[P];
        fill<P>(inverse_root(fmaf(s, p.inv_n, p.eps)), r);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Pairs<P> g;
          weight(c, g);
          mul<P>(u[c].a, r, u[c].a), mul<P>(u[c].a, g.a, u[c].a);
          mul<P>(u[c].b, r, u[c].b), mul<P>(u[c].b, g.b, u[c].b);
        }
      }
      if (kept && which < 2) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = group * P * c + share;
          turn_by<P>(&cosines[warp][i], &sines[warp][i], false, u[c]);
          at[c].put(out, u[c]);
        }
      }
    } else {
      // du = R^T dy; h = x r; g' = du g; dx = r (g' - h mean(g' h)); dg = sum du h
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = group * P * c + share;
        turn_by<P>(&cosines[warp][i], &sines[warp][i], true, e[c]);
      }
      if (p.norm) {
        float2 s2 = make_float2(0.f, 0.f), m2 = s2;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float gu[P];
          Pairs<P> g;
          weight(c, g);
          mul_up<P>(s2, u[c].a, u[c].a), mul_up<P>(s2, u[c].b, u[c].b);
          mul<P>(e[c].a, u[c].a, gu), mul_up<P>(m2, gu, g.a);
          mul<P>(e[c].b, u[c].b, gu), mul_up<P>(m2, gu, g.b);
        }
        float s = s2.x + s2.y, m = m2.x + m2.y;
        s = head_sum<GROUP>(s, takes, lane - li);
        m = head_sum<GROUP>(m, takes, lane - li);
        const float one = inverse_root(fmaf(s, p.inv_n, p.eps));
        float r[P], less[P];
        fill<P>(one, r);
        // less mean(g' h): 0 where h is, although the sum of g' x may be an infinity there
        fill<P>(one == 0.f ? 0.f : -one * m * p.inv_n, less);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Pairs<P> g;
          weight(c, g);
          mul<P>(u[c].a, r, u[c].a), mul<P>(u[c].b, r, u[c].b);
          fma<P>(e[c].a, u[c].a, sum[c].a, sum[c].a);
          fma<P>(e[c].b, u[c].b, sum[c].b, sum[c].b);
          mul<P>(e[c].a, g.a, e[c].a), mul<P>(e[c].b, g.b, e[c].b);
          fma<P>(u[c].a, less, e[c].a, e[c].a), fma<P>(u[c].b, less, e[c].b, e[c].b);
          mul<P>(e[c].a, r, e[c].a), mul<P>(e[c].b, r, e[c].b);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) at[c].put(out, e[c]);
    }
  }

  if constexpr (GRAD) {
    if (!p.norm || !p.sums) return;
    // the warp's heads of q and of k, then the block's warps in order
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float u[2 * P];
      Place<T, P, PAIRS>::join(sum[c], u, u + P);
      Place<T, P, PAIRS> own;  // the channels, whether or not this lane's head exists
      own.set(p, c * group + li);
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) {
        float a = here && which == 0 ? u[j] : 0.f, b = here && which == 1 ? u[j] : 0.f;
        for (int o = group; o < 32; o <<= 1) {  // the first of each two, four, .. heads
          const float x = __shfl_down_sync(0xffffffffu, a, o);
          const float y = __shfl_down_sync(0xffffffffu, b, o);
          if (lane + o < 32) a += x, b += y;
        }
        if (lane < group && (j < P ? own.has : own.has2)) {
          const int i = j < P ? own.at + j : own.at2 + j - P;
          cross[warp][i] = a;
          cross[warp][p.dim + i] = b;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += 32 * kWarps) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += cross[k][i];
      if (gridDim.x > 1)
        p.sums[(size_t)blockIdx.x * 2 * p.dim + i] = v;
      else if (i < p.dim)
        put_sum(p.dgq, i, v, p.accumulate);
      else
        put_sum(p.dgk, i - p.dim, v, p.accumulate);
    }
  }
}

// ---- dispatch --------------------------------------------------------------------

int pow2_above(int n) {
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

// Blocks for T tokens of `passes` warps each, `fit` of which stay on the SMs: as few as
// give every warp no more tokens than that many would.
int64_t blocks_of(int64_t T, int64_t passes, int64_t fit) {
  const int64_t most = fit * kWarps;                             // warps
  int64_t side = most / passes;                                  // tokens side by side
  if (side < 1) side = 1;
  const int64_t rounds = (T + side - 1) / side;
  side = (T + rounds - 1) / rounds;
  return (side * passes + kWarps - 1) / kWarps;
}

// A backward of few heads in all runs as one block: a second launch for the partial
// sums would cost more.
int64_t grad_blocks(int64_t T, int64_t passes, int64_t fit) {
  return T * passes <= 4 * kWarps && passes <= kWarps ? 1 : blocks_of(T, passes, fit);
}
// No launch of T tokens or fewer has more blocks, with any number of heads side by side in a
// warp.  blocks_of evens out the tokens of its warps, so that one token more can halve its
// blocks (24 heads of 64: 303 for 101 tokens, 153 for 102): this bound leaves the evening out
// and never falls, and a workspace serves every batch up to the one that it was made for.
int64_t most_grad_blocks(const RopePlan& R, int64_t T) {
  const int64_t warps = (int64_t)device_sms() * kGradPerSm * kWarps;
  int64_t most = 1;
  for (int side = 1; side <= 32; ++side) {
    const int64_t passes = (R.heads + R.kv + side - 1) / side;
    const int64_t beside = warps / passes < 1 ? 1 : warps / passes;  // tokens side by side
    const int64_t b = ((T < beside ? T : beside) * passes + kWarps - 1) / kWarps;
    if (b > most) most = b;
  }
  return most;
}

// Whether chunks of P channels fit the layout: whole chunks in each half of the
// rotated channels and in the rest, and every head at a multiple of P elements.
bool fits(const RopePlan& R, const RopeArgs& a, int P, bool grad) {
  const int size = R.act == TT_DT_F32 ? 4 : 2;
  if ((R.inter ? R.rot % (2 * P) : (R.rot / 2) % P) || (R.dim - R.rot) % (2 * P)) return false;
  const Heads* all[8] = {&a.q, &a.k, &a.qo, &a.ko, &a.v, &a.vo, &a.dq, &a.dk};
  for (int i = 0; i < 8; ++i) {
    if ((i == 4 || i == 5) && !a.values) continue;
    if (i >= 6 && !grad) continue;
    if (grad && i < 2 && !a.norm) continue;
    if (!aligned_to(all[i]->p, (size_t)P * size) || all[i]->row % P || all[i]->head % P)
      return false;
  }
  return true;
}

template <typename T, int P, int CH, bool PAIRS, bool GRAD, int GROUP>
cudaError_t go(RopeArgs& a, int64_t* blocks, cudaStream_t st) {
  a.passes = (a.heads + a.kv + (a.values ? a.kv : 0) + a.side - 1) / a.side;
  const int64_t sms = device_sms();
  *blocks = GRAD ? grad_blocks(a.T, a.passes, sms * kGradPerSm)
                 : blocks_of(a.T, a.passes, sms * kPerSm);
  auto kernel = rope_kernel<T, P, CH, PAIRS, GRAD, GROUP>;
  constexpr size_t smem = ring_bytes<T, P, CH, GRAD>();
  static PerDevice once;
  const cudaError_t e = once.get([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  return launch_ex(kernel, dim3((unsigned)*blocks), dim3(32 * kWarps), smem, st, false, a);
}

template <typename T, int P, bool PAIRS, bool GRAD>
cudaError_t by_group(RopeArgs& a, int64_t* blocks, cudaStream_t st) {
  constexpr int of64 = 32 / P, of128 = 64 / P;  // lanes of heads of 64 and of 128
  if (a.group == of64) return go<T, P, 1, PAIRS, GRAD, of64>(a, blocks, st);
  if (a.group == of128) return go<T, P, 1, PAIRS, GRAD, of128>(a, blocks, st);
  return go<T, P, 1, PAIRS, GRAD, 0>(a, blocks, st);
}

template <typename T, bool GRAD>
cudaError_t pick(const RopePlan& R, RopeArgs& a, int64_t* blocks, cudaStream_t st) {
  auto shape = [&](int P, int CH) {
    a.turned = R.rot / 2 / P;
    a.chunks = a.turned + (R.dim - R.rot + 2 * P - 1) / (2 * P);
    // a power of two, whose sums take fewer exchanges, unless more heads fit without
    // it (4099 x 20 heads of 80 in f32, ten lanes a head: 29.3 us by sixteens)
    const int lanes = (a.chunks + CH - 1) / CH;
    a.group = pow2_above(lanes);
    if (32 / lanes > 32 / a.group) a.group = lanes;
    a.side = 32 / a.group;
  };
  // 16 bytes a run (f32 with eight pairs a lane, 32 bytes: 4099 x 20 heads of 80 26.3 ->
  // 28.6 us)
  if constexpr (sizeof(T) == 2) {
    if (fits(R, a, 8, GRAD)) {
      shape(8, 1);
      return R.inter ? by_group<T, 8, true, GRAD>(a, blocks, st)
                     : by_group<T, 8, false, GRAD>(a, blocks, st);
    }
  }
  if (fits(R, a, 4, GRAD)) {
    shape(4, 1);
    return R.inter ? by_group<T, 4, true, GRAD>(a, blocks, st)
                   : by_group<T, 4, false, GRAD>(a, blocks, st);
  }
  // Halves of a rotation, or rests, that four do not divide: runs of two or one, with eight
  // values a lane all the same, so that a warp holds as many heads (backward of 20000 x 24
  // heads of 40 in bf16: 20 channels rotated 71 us with one run a lane, 41 with two; ten
  // channels 212 with one, 55 with four)
  if (fits(R, a, 2, GRAD)) {
    shape(2, 2);
    return R.inter ? go<T, 2, 2, true, GRAD, 0>(a, blocks, st)
                   : go<T, 2, 2, false, GRAD, 0>(a, blocks, st);
  }
  shape(1, 4);
  return R.inter ? go<T, 1, 4, true, GRAD, 0>(a, blocks, st)
                 : go<T, 1, 4, false, GRAD, 0>(a, blocks, st);
}

void fill(const RopePlan& R, int64_t T, const int32_t* pos, RopeArgs* a) {
  a->T = T;
  a->heads = R.heads;
  a->kv = R.kv;
  a->dim = R.dim;
  a->rot = R.rot;
  a->norm = R.eps > 0.f;
  a->inv_n = 1.f / (float)R.dim;
  a->eps = R.eps;
  a->pos = pos;
  for (int i = 0; i < R.rot / 2; ++i) a->turn[i] = R.turn[i];
}

}  // namespace

size_t rope_workspace_bytes(const RopePlan& R, int64_t T) {
  return R.eps > 0.f ? (size_t)most_grad_blocks(R, T) * 2 * (size_t)R.dim * sizeof(float) : 0;
}

}  // namespace ttc

using namespace ttc;

extern "C" {

tt_status tt_rope_plan(const tt_rope_desc* desc, tt_plan_t** out) {
  if (!out) return TT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || desc->heads < 1 || desc->heads > 1024 || desc->kv_heads < 1 ||
      desc->heads % desc->kv_heads || desc->dim < 1 || desc->rot < 0 || desc->rot > desc->dim ||
      desc->rot % 2 || !std::isfinite(desc->eps) || desc->eps < 0.f ||
      (desc->flags & ~TT_ACCUMULATE) || (desc->rot == 0 && desc->eps == 0.f))
    return TT_ERR_INVALID_ARG;
  if (desc->act != TT_DT_F32 && desc->act != TT_DT_BF16 && desc->act != TT_DT_E4M3)
    return TT_ERR_INVALID_ARG;
  if (desc->rot > 0 && !desc->freqs && (!std::isfinite(desc->base) || !(desc->base > 0.)))
    return TT_ERR_INVALID_ARG;
  if (desc->act == TT_DT_E4M3 || desc->dim > 2 * kMaxPairs) return TT_ERR_UNSUPPORTED;
  tt_plan_s* p = new (std::nothrow) tt_plan_s();
  if (!p) return TT_ERR_INVALID_ARG;
  p->kind = 6;
  RopePlan& R = p->rope;
  R.heads = desc->heads;
  R.kv = desc->kv_heads;
  R.dim = desc->dim;
  R.rot = desc->rot;
  R.inter = desc->interleaved != 0;
  R.eps = desc->eps;
  R.act = desc->act;
  R.flags = desc->flags;
  for (int i = 0; i < R.rot / 2; ++i) {
    const double f = desc->freqs ? desc->freqs[i] : std::pow(desc->base, -2.0 * i / R.rot);
    if (!std::isfinite(f)) {
      delete p;
      return TT_ERR_INVALID_ARG;
    }
    double turns = f * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= std::floor(turns);
    // a fraction below 1 has 53 bits at most: the product is below 2^64
    R.turn[i] = turns < 1. ? (uint64_t)(turns * 18446744073709551616.0) : 0;
  }
  *out = p;
  return TT_OK;
}

tt_status tt_rope_forward(const tt_plan_t* plan, int64_t T, const int32_t* pos,
                          const tt_heads* q, const tt_heads* k, const float* gq,
                          const float* gk, const tt_heads* q_out, const tt_heads* k_out,
                          const tt_heads* v, const tt_heads* v_out, const int32_t* rows,
                          int64_t cache_rows, void* stream) {
  if (!plan || plan->kind != 6 || T < 0 || T > 0x7FFFFFFF || cache_rows < 0)
    return TT_ERR_INVALID_ARG;
  const RopePlan& R = plan->rope;
  RopeArgs a = {};
  fill(R, T, pos, &a);
  const int64_t kept = rows ? cache_rows : T;
  if (!heads_ok(q, T, R.act, &a.q) || !heads_ok(k, T, R.act, &a.k) ||
      !heads_ok(q_out, T, R.act, &a.qo) || !heads_ok(k_out, kept, R.act, &a.ko) ||
      !aligned_to(pos, 4) || !aligned_to(rows, 4) || !aligned_to(gq, 4) || !aligned_to(gk, 4) ||
      (!v) != (!v_out) || (!a.norm && (gq || gk)))
    return TT_ERR_INVALID_ARG;
  a.values = v != nullptr;
  if (v && (!heads_ok(v, T, R.act, &a.v) || !heads_ok(v_out, kept, R.act, &a.vo)))
    return TT_ERR_INVALID_ARG;
  if (T == 0) return TT_OK;
  a.rows = rows;
  a.cache_rows = cache_rows;
  a.gq = gq;
  a.gk = gk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  int64_t blocks = 0;
  const cudaError_t e = R.act == TT_DT_BF16 ? pick<__nv_bfloat16, false>(R, a, &blocks, st)
                                            : pick<float, false>(R, a, &blocks, st);
  prof_end(kPhElem, st);
  count_launches(1);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

tt_status tt_rope_backward(const tt_plan_t* plan, int64_t T, const int32_t* pos,
                           const tt_heads* q, const tt_heads* k, const float* gq,
                           const float* gk, const tt_heads* dq_out, const tt_heads* dk_out,
                           const tt_heads* dq, const tt_heads* dk, float* dgq, float* dgk,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!plan || plan->kind != 6 || T < 0 || T > 0x7FFFFFFF) return TT_ERR_INVALID_ARG;
  const RopePlan& R = plan->rope;
  RopeArgs a = {};
  fill(R, T, pos, &a);
  if (!heads_ok(dq_out, T, R.act, &a.dq) || !heads_ok(dk_out, T, R.act, &a.dk) ||
      !heads_ok(dq, T, R.act, &a.qo) || !heads_ok(dk, T, R.act, &a.ko) || !aligned_to(pos, 4) ||
      !aligned_to(gq, 4) || !aligned_to(gk, 4) || !aligned_to(dgq, 4) || !aligned_to(dgk, 4) ||
      (!a.norm && (gq || gk || dgq || dgk)))
    return TT_ERR_INVALID_ARG;
  if (a.norm && (!heads_ok(q, T, R.act, &a.q) || !heads_ok(k, T, R.act, &a.k)))
    return TT_ERR_INVALID_ARG;
  a.accumulate = (R.flags & TT_ACCUMULATE) != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (a.accumulate) return TT_OK;
    const size_t n = (size_t)R.dim * sizeof(float);
    if (dgq && cudaMemsetAsync(dgq, 0, n, st) != cudaSuccess) return TT_ERR_CUDA;
    if (dgk && cudaMemsetAsync(dgk, 0, n, st) != cudaSuccess) return TT_ERR_CUDA;
    return TT_OK;
  }
  const size_t need = rope_workspace_bytes(R, T);
  if (need && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return TT_ERR_WORKSPACE;
  a.gq = gq;
  a.gk = gk;
  const bool sums = a.norm && (dgq || dgk);
  a.sums = sums ? static_cast<float*>(ws) : nullptr;
  a.dgq = dgq;
  a.dgk = dgk;
  prof_begin(kPhElem, st);
  int64_t blocks = 0;
  cudaError_t e = R.act == TT_DT_BF16 ? pick<__nv_bfloat16, true>(R, a, &blocks, st)
                                      : pick<float, true>(R, a, &blocks, st);
  count_launches(1);
  if (e == cudaSuccess && sums && blocks > 1) {
    e = launch_ex(sum_parts_kernel, dim3((unsigned)((2 * R.dim + 31) / 32)), dim3(1024), 0, st,
                  false, (const float*)a.sums, (int)blocks, R.dim, dgq, dgk, a.accumulate);
    count_launches(1);
  }
  prof_end(kPhElem, st);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // extern "C"
