// Norm of queries and keys for each head with the rotation by position in the
// same pass: forward (into dense tensors or into the rows of a cache), backward
// with the reduction of the weight gradients.
//
// Both are bound by HBM: a head's values are read once into registers and written
// once.  A warp takes a token; its lanes are dealt so that a lane holds both
// channels of each of its pairs (two chunks of P consecutive channels half a
// rotation apart, or one run of 2 P where neighbours are pairs), so the rotation
// needs no exchange and the norm's sums only those over a head's lanes.  The
// angles of a token are common to its heads: the warp's lanes compute them once, a
// pair each, and share them through shared memory.
//
// An angle is pos f modulo a turn.  The frequency is held as a 64-bit fraction of a
// turn, so the product modulo 2^64 is that reduction itself, without rounding: the
// error is the frequency's own (2^-52 of it, times the position), at any position
// of 31 bits.  The nearest quarter turn is taken off, and what is left, at most an
// eighth of a turn either way, is rounded to fp32 for sincospi.
#include <cmath>
#include <new>

#include "rows.cuh"
#include "ttc.h"
#include "ttc_internal.h"

namespace ttc {

cudaError_t read_and_clear_rope_status(DeviceStatus* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status, sizeof(DeviceStatus));
  if (e != cudaSuccess) return e;
  DeviceStatus z{0, 0};
  return cudaMemcpyToSymbol(g_status, &z, sizeof(z));
}

namespace {

constexpr int kMaxPairs = 128;  // of a head of 256
constexpr int kWarps = 8;       // warps a block

struct RopeArgs {
  int64_t T;
  int heads, kv, dim, rot;
  int group;       // lanes of a head: a power of two
  int chunks;      // chunks of a head; the first rotated ones, then the rest
  int turned;      // rotated chunks
  int parts;       // warps of a token
  int norm;        // 0: rotation alone
  float n, eps;
  const int32_t* pos;
  const int32_t* rows;  // k and v go to these rows of ko and vo
  int64_t cache_rows;
  Heads q, k, v, qo, ko, vo;  // backward: qo, ko are the gradients of q and k
  Heads dq, dk;
  int values;                 // v is copied too
  const float *gq, *gk;
  int gq16, gk16;             // 16-byte aligned
  float* sums;                // backward: [gridDim.x][2 dim] shares of dgq, dgk
  float *dgq, *dgk;           // written directly by a grid of one block
  int accumulate;
  uint64_t turn[kMaxPairs];   // frequencies, as fractions of a turn
};

// cos and sin of pos frequency
__device__ __forceinline__ float2 angle(int64_t pos, uint64_t turn) {
  const uint64_t a = (uint64_t)pos * turn;
  const uint64_t quarter = (a + (1ull << 61)) >> 62;
  // in [-2^61, 2^61): 2^63 is half a turn
  const int64_t rest = (int64_t)(a - (quarter << 62));
  float s, c;
  sincospif((float)(int32_t)(rest >> 31) * 0x1p-32f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// What a lane holds of a head: CH chunks of P pairs.  PAIRS: neighbouring channels
// are a pair.
template <typename T, int P, int CH, bool PAIRS>
struct Lane {
  using R = Raw<T, P>;
  int at[CH], at2[CH];       // channels of a chunk's two halves
  bool has[CH], has2[CH];
  float2 cs[CH][P];

  __device__ void place(const RopeArgs& p, int lane) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * 32 + (lane & (p.group - 1));
      has[c] = i < p.chunks;
      if (i < p.turned) {
        at[c] = PAIRS ? 2 * P * i : P * i;
        at2[c] = PAIRS ? at[c] + P : p.rot / 2 + P * i;
      } else {
        at[c] = p.rot + 2 * P * (i - p.turned);
        at2[c] = at[c] + P;
      }
      has2[c] = has[c] && at2[c] < p.dim;
    }
  }
  // the table of the token's angles: a lane keeps those of its pairs
  __device__ void angles(const RopeArgs& p, int64_t pos, const uint64_t* turn, float2* table,
                         int lane) {
    __syncwarp();
    for (int i = lane; i < p.rot / 2; i += 32) table[i] = angle(pos, turn[i]);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * 32 + (lane & (p.group - 1));
#pragma unroll
      for (int j = 0; j < P; ++j)
        cs[c][j] = i < p.turned ? table[i * P + j] : make_float2(1.f, 0.f);
    }
  }
  __device__ void turn_by(int c, float (&u)[2 * P], bool back) const {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      float& a = u[PAIRS ? 2 * j : j];
      float& b = u[PAIRS ? 2 * j + 1 : P + j];
      const float co = cs[c][j].x, si = back ? -cs[c][j].y : cs[c][j].y;
      const float t = fmaf(a, co, -b * si);
      b = fmaf(a, si, b * co);
      a = t;
    }
  }
  __device__ void load(const T* x, R (&a)[CH], R (&b)[CH]) const {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (has[c]) a[c] = *reinterpret_cast<const R*>(x + at[c]);
      if (has2[c]) b[c] = *reinterpret_cast<const R*>(x + at2[c]);
    }
  }
  __device__ void get(int c, const R (&a)[CH], const R (&b)[CH], float (&u)[2 * P]) const {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) u[j] = 0.f;
    if (has[c]) a[c].get(u);
    if (has2[c]) b[c].get(u + P);
  }
  __device__ void put(T* y, int c, const float (&u)[2 * P]) const {
    R o;
    if (has[c]) {
      o.set(u);
      *reinterpret_cast<R*>(y + at[c]) = o;
    }
    if (has2[c]) {
      o.set(u + P);
      *reinterpret_cast<R*>(y + at2[c]) = o;
    }
  }
  __device__ void weights(const float* g, bool aligned, int c, float (&w)[2 * P]) const {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) w[j] = 0.f;
    if (has[c]) weights_at<P>(g, at[c], 1.f, aligned, w);
    if (has2[c]) weights_at<P>(g, at2[c], 1.f, aligned, w + P);
  }
};

__device__ __forceinline__ float head_sum(float v, int group) {
  for (int o = group >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp's passes over a token: its lanes hold 32 / group heads at a time, first
// those of q, then of k, then of v.  With `parts` warps a token each takes every
// parts-th pass.  The next pass is loaded while one is worked on.
template <typename T, int P, int CH, bool PAIRS, bool GRAD>
__global__ void __launch_bounds__(32 * kWarps, GRAD ? 2 : 3) rope_kernel(RopeArgs p) {
  using L = Lane<T, P, CH, PAIRS>;
  using R = typename L::R;
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ float2 tables[kWarps][kMaxPairs];
  __shared__ float cross[GRAD ? kWarps : 1][GRAD ? 2 * 2 * kMaxPairs : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.rot / 2; i += 32 * kWarps) turn[i] = p.turn[i];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  L at;
  at.place(p, lane);
  const int side = 32 / p.group, mine = lane / p.group;  // heads of a pass; this lane's
  const int nq = (p.heads + side - 1) / side, nk = (p.kv + side - 1) / side;
  const int passes = nq + nk + (p.values ? nk : 0);
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t step = (int64_t)gridDim.x * kWarps / p.parts;
  const int part = (int)(w % p.parts);
  int64_t t = w / p.parts;
  if (t >= step) t = p.T;
  int s = part;

  R xa[CH], xb[CH], da[GRAD ? CH : 1], db[GRAD ? CH : 1];
  int64_t pos = 0, row = 0;
  auto fetch = [&](int64_t t, int s) {
    const int which = s < nq ? 0 : s < nq + nk ? 1 : 2;
    const int h = (s - (which == 0 ? 0 : which == 1 ? nq : nq + nk)) * side + mine;
    if (h >= (which == 0 ? p.heads : p.kv)) return;
    if (!GRAD || p.norm) {
      const Heads& from = which == 0 ? p.q : which == 1 ? p.k : p.v;
      at.load(from.at<T>(t, h), xa, xb);
    }
    if constexpr (GRAD) at.load((which == 0 ? p.dq : p.dk).at<T>(t, h), da, db);
  };
  auto fetch_token = [&](int64_t t) {
    pos = p.pos ? p.pos[t] : t;
    row = p.rows ? p.rows[t] : t;
  };
  float accq[CH][2 * P], acck[CH][2 * P];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) accq[c][j] = acck[c][j] = 0.f;

  int64_t to = 0;  // the row that the token's keys go to
  bool fresh = true;
  if (t < p.T) {
    fetch_token(t);
    fetch(t, s);
  }
  while (t < p.T) {
    if (fresh) {
      at.angles(p, pos, turn, tables[warp], lane);
      to = row;
      if (!GRAD && p.rows && to >= p.cache_rows) {
        if (lane == 0) record_error(TT_ERR_DEVICE, 1);
        to = -1;
      }
    }
    const int which = s < nq ? 0 : s < nq + nk ? 1 : 2;
    const int h = (s - (which == 0 ? 0 : which == 1 ? nq : nq + nk)) * side + mine;
    const bool here = h < (which == 0 ? p.heads : p.kv);
    float u[CH][2 * P], d[GRAD ? CH : 1][2 * P];
    R va[CH], vb[CH];  // v goes as it is
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      at.get(c, xa, xb, u[c]);
      if constexpr (GRAD)
        at.get(c, da, db, d[c]);
      else
        va[c] = xa[c], vb[c] = xb[c];
    }
    const int64_t now = t;
    s += p.parts;
    fresh = s >= passes;
    if (fresh) {
      s = part;
      t += step;
      if (t < p.T) fetch_token(t);
    }
    if (t < p.T) fetch(t, s);

    const float* g = which == 0 ? p.gq : p.gk;
    const bool g16 = which == 0 ? p.gq16 : p.gk16;
    if constexpr (!GRAD) {
      const bool kept = here && (which == 0 || to >= 0);
      const int64_t out = which == 0 ? now : to;
      if (which == 2) {
        if (kept) {
          T* y = p.vo.at<T>(out, h);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (at.has[c]) *reinterpret_cast<R*>(y + at.at[c]) = va[c];
            if (at.has2[c]) *reinterpret_cast<R*>(y + at.at2[c]) = vb[c];
          }
        }
        continue;
      }
      if (p.norm) {
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) sum = fmaf(u[c][j], u[c][j], sum);
        sum = head_sum(sum, p.group);
        const float r = 1.f / sqrtf(sum / p.n + p.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float f[2 * P];
          at.weights(g, g16, c, f);
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) u[c][j] = u[c][j] * r * f[j];
        }
      }
      if (kept) {
        T* y = (which == 0 ? p.qo : p.ko).at<T>(out, h);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          at.turn_by(c, u[c], false);
          at.put(y, c, u[c]);
        }
      }
    } else {
      // du = R^T dy; h = x r; g' = du g; dx = r (g' - h mean(g' h)); dg = sum du h.
      // Lanes of a head that the token lacks hold zeros or what the pass before
      // left: they join the exchanges of other lanes' groups, not their sums.
#pragma unroll
      for (int c = 0; c < CH; ++c) at.turn_by(c, d[c], true);
      if (p.norm) {
        float sx = 0.f, sg = 0.f, f[CH][2 * P];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          at.weights(g, g16, c, f[c]);
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) {
            sx = fmaf(u[c][j], u[c][j], sx);
            f[c][j] *= d[c][j];
            sg = fmaf(f[c][j], u[c][j], sg);
          }
        }
        for (int o = p.group >> 1; o; o >>= 1) {
          sx += __shfl_xor_sync(0xffffffffu, sx, o);
          sg += __shfl_xor_sync(0xffffffffu, sg, o);
        }
        const float r = 1.f / sqrtf(sx / p.n + p.eps);
        const float m = r * sg / p.n;  // mean(g' h)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) {
            const float x = u[c][j] * r;
            if (here) {
              if (which == 0)
                accq[c][j] = fmaf(d[c][j], x, accq[c][j]);
              else
                acck[c][j] = fmaf(d[c][j], x, acck[c][j]);
            }
            d[c][j] = r * fmaf(-x, m, f[c][j]);
          }
      }
      if (here) {
        T* y = (which == 0 ? p.qo : p.ko).at<T>(now, h);
#pragma unroll
        for (int c = 0; c < CH; ++c) at.put(y, c, d[c]);
      }
    }
  }

  if constexpr (GRAD) {
    if (!p.norm || !p.sums) return;
    // the warp's heads, then the block's warps in order
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) {
        float a = accq[c][j], b = acck[c][j];
        for (int o = p.group; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        const bool real = j < P ? at.has[c] : at.has2[c];
        const int i = j < P ? at.at[c] + j : at.at2[c] + j - P;
        if (mine == 0 && real) {
          cross[warp][i] = a;
          cross[warp][p.dim + i] = b;
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

// Warps that the card keeps busy; a token is split over several where there are
// fewer tokens.
int64_t most_warps() { return (int64_t)device_sms() * 2 * kWarps; }

int64_t grad_blocks(int64_t T) {
  const int64_t b = (T + kWarps - 1) / kWarps;
  if (T <= 4 * kWarps) return 1;  // a second launch would cost more than the rows
  const int64_t most = (int64_t)device_sms() * 2;
  return b < most ? b : most;
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

template <typename T, int P, int CH, bool PAIRS, bool GRAD>
cudaError_t go(RopeArgs& a, cudaStream_t st) {
  auto kernel = rope_kernel<T, P, CH, PAIRS, GRAD>;
  const int side = 32 / a.group;
  const int nk = (a.kv + side - 1) / side;
  const int passes = (a.heads + side - 1) / side + nk + (a.values ? nk : 0);
  int64_t blocks;
  if (GRAD) {
    blocks = grad_blocks(a.T);
    a.parts = 1;
  } else {
    int64_t parts = most_warps() / a.T;
    a.parts = parts < 1 ? 1 : parts > passes ? passes : (int)parts;
    const int64_t need = (a.T * a.parts + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)device_sms() * 3;
    blocks = need < most ? need : most;
  }
  return launch_ex(kernel, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, false, a);
}

template <typename T, bool GRAD>
cudaError_t pick(const RopePlan& R, RopeArgs& a, cudaStream_t st) {
  auto shape = [&](int P) {
    a.turned = R.rot / 2 / P;
    a.chunks = a.turned + (R.dim - R.rot + 2 * P - 1) / (2 * P);
    a.group = a.chunks > 32 ? 32 : pow2_above(a.chunks);
  };
  if constexpr (sizeof(T) == 2) {
    if (fits(R, a, 8, GRAD)) {
      shape(8);
      return R.inter ? go<T, 8, 1, true, GRAD>(a, st) : go<T, 8, 1, false, GRAD>(a, st);
    }
  }
  if (fits(R, a, 4, GRAD)) {
    shape(4);
    return R.inter ? go<T, 4, 1, true, GRAD>(a, st) : go<T, 4, 1, false, GRAD>(a, st);
  }
  shape(1);
  if (R.inter)
    return a.chunks <= 32 ? go<T, 1, 1, true, GRAD>(a, st)
                          : go<T, 1, 4, true, GRAD>(a, st);
  return a.chunks <= 32 ? go<T, 1, 1, false, GRAD>(a, st)
                        : go<T, 1, 4, false, GRAD>(a, st);
}

void fill(const RopePlan& R, int64_t T, const int32_t* pos, RopeArgs* a) {
  a->T = T;
  a->heads = R.heads;
  a->kv = R.kv;
  a->dim = R.dim;
  a->rot = R.rot;
  a->norm = R.eps > 0.f;
  a->n = (float)R.dim;
  a->eps = R.eps;
  a->pos = pos;
  for (int i = 0; i < R.rot / 2; ++i) a->turn[i] = R.turn[i];
}

}  // namespace

size_t rope_workspace_bytes(const RopePlan& R, int64_t T) {
  return R.eps > 0.f ? (size_t)grad_blocks(T) * 2 * (size_t)R.dim * sizeof(float) : 0;
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
  a.gq16 = aligned_to(gq, 16);
  a.gk16 = aligned_to(gk, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(kPhElem, st);
  const cudaError_t e = R.act == TT_DT_BF16 ? pick<__nv_bfloat16, false>(R, a, st)
                                            : pick<float, false>(R, a, st);
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
  a.gq16 = aligned_to(gq, 16);
  a.gk16 = aligned_to(gk, 16);
  const bool sums = a.norm && (dgq || dgk);
  a.sums = sums ? static_cast<float*>(ws) : nullptr;
  a.dgq = dgq;
  a.dgk = dgk;
  prof_begin(kPhElem, st);
  cudaError_t e = R.act == TT_DT_BF16 ? pick<__nv_bfloat16, true>(R, a, st)
                                      : pick<float, true>(R, a, st);
  count_launches(1);
  const int64_t blocks = grad_blocks(T);
  if (e == cudaSuccess && sums && blocks > 1) {
    e = launch_ex(sum_parts_kernel, dim3((unsigned)((2 * R.dim + 31) / 32)), dim3(1024), 0, st,
                  false, (const float*)a.sums, (int)blocks, R.dim, dgq, dgk, a.accumulate);
    count_launches(1);
  }
  prof_end(kPhElem, st);
  return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // extern "C"
