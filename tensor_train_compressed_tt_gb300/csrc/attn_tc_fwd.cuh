// Tensor-core forward of windowed attention (bf16, heads of up to 128
// channels in multiples of 8).
//
// A CTA takes tiles of 128 queries of one head, one after another, and passes
// once over the keys that a tile sees (the first tokens and the window, in
// tiles of KT keys; a short tile's products and exponentials shrink to its
// width): S = Q K^T into tensor memory, the weights exp2(c s - m) over it as
// bf16, O += P V beside it, l += sum p in registers (thread = row).
//
// The reference m of a row need not be its maximum, only near enough that
// nothing overflows: bf16 and fp32 share their exponents, and the division by
// l takes m out again.  So m is the maximum of the first 32 keys that the row
// sees, and stays while the scores keep within 60 powers of two of it: no pass for
// the maximum, no rescaling of O.  Scores that rise further show in a tile's sum of
// weights, before the tile's product is taken, and the row's m, l, weights of the
// tile and O are brought to a higher reference there (far_tile; by the writing warps,
// which wait at that time).  Nothing of it is in the softmax loop but a comparison a tile:
// the check before each 32 keys' weights are written 69 us where this takes 59 (its
// latency is in the chain), the raise called from the loop itself 200 us (registers).
// 128 queries and 12000 causal keys, two heads of 64: 0.17 ms with level scores, 0.39 ms
// with scores that rise by 0.7 powers of two a key (a raise a tile), 5.3 ms with two (192
// powers a tile: its scores computed again, 42 us a tile).
//
// Roles: warps 0-3 softmax, warp 4 finds the work and loads it, warp 5 issues S,
// warp 6 O += P V, warps 7-10 write the output.  S has two buffers, so that the
// next S is computed during a softmax, and two CTAs on an SM fill each other's
// waits.
//
// 128 sequences of 128, window +-64, 12 heads of 64: 24.2 us (101 MB: 4.2 TB/s);
// 64 sequences of 257 to 512, window +-128, 16 heads of 64: 59.1 us (203 MB), the
// tensor pipe 25 % and the issue slots 51 % busy: bound by the chain of a tile,
// whose 96 columns take a softmax warp 1700 cycles, half of them waiting for
// tensor memory, exponentials and the other warps of its scheduler.  Measured and
// not kept (the second case, 59.5): columns in 16s 63 us; in 16s with the next
// ones loaded ahead 82 us (twice the code); one buffer of S and four CTAs an SM 76
// us, three 73 us; the softmax warps writing the output themselves 62 us.
//
// What held the kernel back was not a pipe.  The loops are not unrolled more
// than the softmax needs: with the code at twice its size the kernel waited
// for instructions (the cache that several SMs share answered at 90 % of its
// rate) and took 1.6 times as long.  And each role's own code between two
// hand-overs is kept short (tile lists that step, one barrier for a key and a
// value tile, two warps for the two products): one thread that does the
// bookkeeping of a whole tile takes as long as the tile.
#pragma once

#include "attn_tc.cuh"

namespace ttc {
namespace {

// One tile of queries of one head and the keys it passes over.
struct FwdItem {
  int64_t q0, k0;      // the sequence's first rows
  int h, t0, nq, i0;   // head, first row, rows, position of the first row
  TileList keys;
  int nt;              // key tiles; < 0: no more work
};

template <int NB>
struct TcFwd {
  // Two buffers of S and one O share 256 columns of tensor memory (two CTAs
  // an SM): 96 + 96 + 64, or 64 + 64 + 128.
  static constexpr int KT = NB == 1 ? 96 : 64;  // keys of a tile
  static constexpr int QS = NB == 1 ? 2 : 1;    // query tiles in flight
  static constexpr int KP = NB == 1 ? 3 : 2;    // pairs of a key and a value tile in flight
  static constexpr int ITEMS = 4;               // pieces of work told to the roles
  static constexpr int CTAS = 2;                // CTAs an SM
  static constexpr int KBOX = KT * 128, UNIT = NB * KBOX;
  static constexpr uint32_t O_COL = 2 * KT, COLS = 256;
  struct Shared {
    uint64_t q_full[QS], q_empty[QS], k_full[KP], k_empty[KP], v_full[KP], v_empty[KP];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free, fin, fin2;  // [tile & 1]
    uint64_t stat_full[4], stat_free[4];  // a message of a softmax warp to its writing warp
    uint64_t item_full[ITEMS], item_empty[ITEMS], clc;
    FwdItem item[ITEMS];
    uint4 answer;
    // the messages: an item's m and l (far = -1), or m and the tile's sum of a tile with
    // far rows (its number), answered by m, sum and the scale of l
    float m[AT], l[AT], f[AT];
    int far[4];
    int rows[2 * KP];  // keys of a tile, by its number (a key tile's place is free before
                       // the product of its values has read this)
    uint32_t tmem;
    WaitFlags flags, never;
  };
  static constexpr size_t kSmem = QS * NB * ABOX + 2 * KP * UNIT + sizeof(Shared) + 1024;
};

constexpr int kTcThreads = 352;

// CTA number -> tile.  The tiles of one sequence and head come one after
// another, so that they share its keys in L2; the last ones, which see the
// most keys under a causal mask, first.  Under a causal mask without a window,
// where a long sequence's tiles differ most, they come in that order over all
// sequences and heads, so that the last to run are short: 8 sequences of 2048, 16
// heads of 64, 105 -> 91 us, 16 of 1000, 8 heads of 128, 56 -> 50 us; but 64 of 512,
// 12 heads of 64, 56 -> 63 us, and the windowed 64 of 257 to 512 59 -> 70 us.
// False: nothing to do.
__device__ __forceinline__ bool long_first(const AttnArgs& p, uint32_t ntiles) {
  return p.left < 0 && p.right >= 0 && ntiles >= 8;
}
template <int KT>
__device__ __forceinline__ bool fwd_item(const AttnArgs& p, uint32_t item, uint32_t ntiles,
                                         FwdItem* w) {
  const bool across = long_first(p, ntiles);
  const uint32_t per = across ? (uint32_t)p.B * p.heads : ntiles;
  const uint32_t a = item / per, c = item - a * per, r = across ? c : a;
  const int tile = (int)(ntiles - 1 - (across ? a : c));
  const uint32_t b = r / (uint32_t)p.heads;
  w->h = (int)(r - b * p.heads);
  Seq s;
  if (!load_seq(p, (int)b, &s, true)) return false;
  w->q0 = s.q0;
  w->k0 = s.k0;
  w->t0 = tile * AT;
  if (w->t0 >= s.lq) return false;
  w->nq = min(AT, s.lq - w->t0);
  w->i0 = w->t0 + s.off();
  const KeySpan ks = key_span(p, s.lk, w->i0, w->i0 + w->nq - 1);
  w->keys = key_list(ks, w->h / p.group);
  w->nt = (ks.a1 + KT - 1) / KT + (ks.b1 - ks.b0 + KT - 1) / KT;
  return true;
}

// The sum of weights over a tile from which a row's reference is raised: weights of up to
// 2^60 times bf16 values of up to 2^68 stay finite in O.
constexpr float kFar = 1152921504606846976.f;  // 2^60
// The sum from which a weight may have overflowed (bf16 rounds up to infinity a little below
// fp32's largest number): 2^127.
constexpr float kOver = 1.7014118346046923e38f;

// In keys from a tile's first, j0, on: the last one that the first of a warp's rows sees,
// the first one that its last row sees, the end of the first tokens.  A later row sees
// one key more on the right and one less on the left.  iw: position of the first row.
struct TileView {
  int nk, wh, wl, sk;
  __device__ __forceinline__ TileView(const AttnArgs& p, int iw, int j0, int n) {
    nk = n;
    wh = p.right < 0 ? kAttnMaxLen : iw + p.right - j0;
    wl = p.left < 0 ? -kAttnMaxLen : iw + 31 - p.left - j0;
    sk = p.sinks - j0;
  }
  // bit e: this lane's row sees key q + e of the tile
  __device__ __forceinline__ uint32_t sees(int q, int lane) const {
    return bit_span(0, min(nk - 1, wh + lane) - q) &
           (bit_span(wl - 31 + lane - q, 31) | bit_span(0, sk - 1 - q));
  }
};

// A tile in which some rows of a warp are far above their reference m (their sums ts of
// weights are kFar or more): those rows get a reference higher by a whole number of powers
// of two, so that the tile's weights and O, scaled to it, keep their bits.  Where a weight
// may have overflowed (kOver), the row's scores are computed again from q and the tile's
// keys (the weights lie over them), rounded before the reference is taken from them (a
// score beyond 2^24 is rounded by whole powers of two), and the reference becomes their
// maximum.  Returns the reference, the tile's sum, and the scale of l.
__device__ __forceinline__ float3 far_tile(const AttnArgs& p, const FwdItem& w, int t, int KT,
                                           uint32_t sp, uint32_t o_at, float m, float ts) {
  const int lane = threadIdx.x & 31, row = 32 * ((threadIdx.x >> 5) & 3) + lane;
  const int first = (w.keys.lim - w.keys.r + KT - 1) / KT;  // tiles before the list's second part
  const int j0 = t < first ? w.keys.r + t * KT : w.keys.r2 + (t - first) * KT;
  const int nk = min(KT, (t < first ? w.keys.lim : w.keys.lim2) - j0);
  const int o_cols = t == 0 ? 0 : (p.dim + 15) & ~15;
  const TileView view(p, w.i0 + row - lane, j0, nk);
  const float c = p.scale * kLog2e;
  const bool far = ts >= kFar && row < w.nq, over = far && ts >= kOver;
  const bool any_over = __any_sync(0xffffffffu, over);
  const __nv_bfloat16* q = p.q.at<const __nv_bfloat16>(w.q0 + w.t0 + row, w.h);
  const __nv_bfloat16* k = p.k.at<const __nv_bfloat16>(w.k0 + j0, w.h / p.group);
  float top = -INFINITY;
#pragma unroll 1
  for (int x = 0; any_over && x < nk; x += 4) {  // the scores of 4 keys, over S
    float s[4], old[4];
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = 0.f;
#pragma unroll 1
    for (int d = 0; over && d < p.dim; d += 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(q + d);
      const uint32_t qa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 b = *reinterpret_cast<const uint4*>(k + min(x + e, nk - 1) * p.k.row + d);
        const uint32_t kb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[e] = fmaf(__uint_as_float(qa[i] << 16), __uint_as_float(kb[i] << 16), s[e]);
          s[e] = fmaf(__uint_as_float(qa[i] & 0xFFFF0000u), __uint_as_float(kb[i] & 0xFFFF0000u),
                      s[e]);
        }
      }
    }
    __syncwarp();
    const uint32_t see = view.sees(x, lane);
    tmem_ld4_async(sp + x, old);
    tmem_wait_ld();
    tmem_landed(old);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = see & (1u << e) ? __fmul_rn(s[e], c) : -INFINITY;
      top = fmaxf(top, s[e]);
      u[e] = __float_as_uint(over ? s[e] : old[e]);  // the other rows' weights stay
    }
    tmem_st4(sp + x, u);
  }
  tmem_wait_st();
  const float up = over ? ceilf(top - m) : ceilf(log2f(ts));
  const float to = !far ? m : over && !(up < 8388608.f) ? top : m + up;
  const float f = far ? exp2f(m - to) : 1.f;
  float sum = 0.f;
  // 8 weights lie in 4 columns; the scores they come from are read before, and weights
  // are never written over scores that are still to come.  The product takes 16 keys a
  // step: the weights of those past the tile's end, where scores may lie, become zero.
#pragma unroll 1
  for (int x = 0; x < nk || x % 16; x += 8) {
    float old[4], z[2][4];
    uint32_t u[4];
    tmem_ld4_async(sp + (x >> 1), old);
    tmem_ld4_async(sp + x, z[0]);
    tmem_ld4_async(sp + x + 4, z[1]);
    tmem_wait_ld();
    tmem_landed(old);
    tmem_landed(z[0]);
    tmem_landed(z[1]);
    const uint32_t see = view.sees(x, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = __float_as_uint(old[e]);
      float y0 = __uint_as_float(b << 16) * f, y1 = __uint_as_float(b & 0xFFFF0000u) * f;
      if (over) {
        y0 = see & (1u << (2 * e)) ? ex2(z[e >> 1][2 * (e & 1)] - to) : 0.f;
        y1 = see & (2u << (2 * e)) ? ex2(z[e >> 1][2 * (e & 1) + 1] - to) : 0.f;
        sum += y0 + y1;
      }
      u[e] = pack_bf16(y0, y1);
    }
    __syncwarp();
    tmem_st4(sp + (x >> 1), u);
    tmem_wait_st();
  }
#pragma unroll 1
  for (int x = 0; x < o_cols; x += 4) {
    float o[4];
    uint32_t u[4];
    tmem_ld4_async(o_at + x, o);
    tmem_wait_ld();
    tmem_landed(o);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(o[e] * f);
    tmem_st4(o_at + x, u);
  }
  tmem_wait_st();
  return make_float3(to, over ? sum : ts * f, f);
}

// A writing warp's messages from the first one of a far tile on to the item's end.
// Returns the number of messages taken, 0 after an abort.
template <int NB>
__device__ __forceinline__ uint32_t serve_far(const AttnArgs& p, typename TcFwd<NB>::Shared& S,
                                              const FwdItem& w, int g0, uint32_t lanes,
                                              uint32_t msgs) {
  using C = TcFwd<NB>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = 32 * quad + lane;
  while (true) {
    const int g = S.far[quad];
    // O holds the products up to the last tile's (of this item)
    if (g > g0 && !wait_all(&S.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &S.flags, 114))
      return 0;
    tc_fence_after();
    const float3 r = far_tile(p, w, g - g0, C::KT, lanes + (g & 1) * C::KT, lanes + C::O_COL,
                              S.m[row], S.l[row]);
    S.m[row] = r.x;
    S.l[row] = r.y;
    S.f[row] = r.z;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.stat_free[quad]);
    if (!wait_all(&S.stat_full[quad], msgs & 1, &S.flags, 113)) return 0;
    ++msgs;
    if (S.far[quad] < 0) return msgs;
  }
}

// A softmax warp's side of it: m, the tile's sum, the scale of l, and 0 after an abort.
template <int NB>
__device__ __noinline__ float4 ask_far(typename TcFwd<NB>::Shared& S, int g, uint32_t msgs,
                                       float m, float ts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = threadIdx.x;
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!wait_all(&S.stat_free[warp], (msgs & 1) ^ 1, &S.flags, 110)) return none;
  S.m[row] = m;
  S.l[row] = ts;
  if (lane == 0) S.far[warp] = g;
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.stat_full[warp]);
  if (!wait_all(&S.stat_free[warp], msgs & 1, &S.flags, 115)) return none;
  tc_fence_after();
  return make_float4(S.m[row], S.l[row], S.f[row], 1.f);
}

template <int NB>
__global__ void __launch_bounds__(kTcThreads, TcFwd<NB>::CTAS)
    attn_fwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs p) {
  using C = TcFwd<NB>;
  constexpr int KT = C::KT, KP = C::KP, QS = C::QS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qbuf = align1k(smem_raw);
  uint8_t* kvbuf = qbuf + QS * NB * ABOX;  // K and V of pair s: units 2 s and 2 s + 1
  auto& S = *reinterpret_cast<typename C::Shared*>(kvbuf + 2 * KP * C::UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < QS; ++i) mbar_init(&S.q_full[i], 1), mbar_init(&S.q_empty[i], 1);
#pragma unroll 1
    for (int i = 0; i < KP; ++i) {
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.v_empty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.pv_done[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < C::ITEMS; ++i)
      mbar_init(&S.item_full[i], 1), mbar_init(&S.item_empty[i], 10);
    mbar_init(&S.o_free, 4);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) mbar_init(&S.stat_full[i], 1), mbar_init(&S.stat_free[i], 1);
    mbar_init(&S.clc, 1);
    mbar_init(&S.fin, 1);
    mbar_init(&S.fin2, 1);
    S.flags = S.never = WaitFlags{0, 0};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) tmem_take(&S.tmem, C::COLS);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  volatile WaitFlags* flags = &S.flags;

  if (warp == 4) {
    // ---------------- work and loads
    if (lane == 0) {
      const uint32_t ntiles = (p.max_q + AT - 1) / AT;
      int n = 0, nload = 0, s = 0, loads = 0;
      uint32_t ph = 1, clc = 0;  // parity of the ring's empty barriers; of the next answer
      bool ok = true, first = true;
      // test hook: the first CTA leaves its first tile of keys unloaded
      const int from = blockIdx.x == 0 && debug_take(TT_DEBUG_ATTN_FWD);
      int cta = (int)blockIdx.x;
      FwdItem cur, w;
      cur.nt = -1;
#pragma unroll 1
      while (true) {
        // The next piece of work: told to the roles, its rows sent for from memory, before
        // the loads of the current one, so that its own loads find them in L2.
        w.nt = -1;
#pragma unroll 1
        while (cta >= 0) {
          if (!first) {
            // After an abort the CTAs that have not started are still taken over, and do
            // nothing.
            cta = wait_one(&S.clc, clc, &S.never, 95) ? clc_take(&S.answer) : -1;
            clc ^= 1;
            if (cta < 0) break;
          }
          first = false;
          clc_ask(&S.answer, &S.clc);
          if (!ok || !fwd_item<KT>(p, (uint32_t)cta, ntiles, &w)) {
            w.nt = -1;
            continue;
          }
          const int slot = n % C::ITEMS;
          ok = wait_one(&S.item_empty[slot], ((n / C::ITEMS) & 1) ^ 1, flags, 96);
          if (!ok) {
            w.nt = -1;
            continue;
          }
          S.item[slot] = w;
          mbar_arrive(&S.item_full[slot]);
          ++n;
          if (w.nt > 0) {
            const int span = min(w.keys.lim2 - w.keys.r2, 4 * KT);
            prefetch_rows<NB>(&tm_q, AT, w.h, (int)w.q0 + w.t0, w.nq);
            prefetch_rows<NB>(&tm_k, KT, w.keys.h, (int)w.k0 + w.keys.r2, span);
            prefetch_rows<NB>(&tm_v, KT, w.keys.h, (int)w.k0 + w.keys.r2, span);
          }
          break;
        }
        if (ok && cur.nt > 0) {
          const int qs = nload % QS;
          ok = wait_one(&S.q_empty[qs], ((nload / QS) & 1) ^ 1, flags, 97);
          if (ok) {
            mbar_expect_tx(&S.q_full[qs], NB * ABOX);
            load_tile<NB>(qbuf + qs * NB * ABOX, ABOX, &tm_q, &S.q_full[qs], cur.h,
                          (int)cur.q0 + cur.t0);
            ++nload;
          }
          TileList l = cur.keys;
#pragma unroll 1
          for (int t = 0; ok && t < cur.nt; ++t) {
            ok = wait_one(&S.k_empty[s], ph, flags, 98);
            if (!ok) break;
            S.rows[loads % (2 * KP)] = l.rows(KT);
            uint8_t* dst = kvbuf + 2 * s * C::UNIT;
            if (loads >= from) {
              mbar_expect_tx(&S.k_full[s], C::UNIT);
              load_tile<NB>(dst, C::KBOX, &tm_k, &S.k_full[s], l.h, (int)cur.k0 + l.r);
            }
            ok = wait_one(&S.v_empty[s], ph, flags, 94);
            if (!ok) {
              drain_one(&S.k_full[s], ph ^ 1);
              break;
            }
            mbar_expect_tx(&S.v_full[s], C::UNIT);
            load_tile<NB>(dst + C::UNIT, C::KBOX, &tm_v, &S.v_full[s], l.h, (int)cur.k0 + l.r);
            l.next(KT);
            ++loads;
            if (++s == KP) s = 0, ph ^= 1;
          }
        }
        if (w.nt < 0) break;
        cur = w;
      }
      if (ok && wait_one(&S.item_empty[n % C::ITEMS], ((n / C::ITEMS) & 1) ^ 1, flags, 99)) {
        S.item[n % C::ITEMS].nt = -1;
        mbar_arrive(&S.item_full[n % C::ITEMS]);
      }
      // nothing is in flight into shared memory when the CTA leaves
#pragma unroll 1
      for (int i = 1; i <= QS && i <= nload; ++i)
        drain_one(&S.q_full[(nload - i) % QS], (uint32_t)(((nload - i) / QS) & 1));
#pragma unroll 1
      for (int i = 0; i < KP && i < loads; ++i) {
        if (--s < 0) s = KP - 1, ph ^= 1;
        drain_one(&S.k_full[s], ph ^ 1);  // the last loads into pair s
        drain_one(&S.v_full[s], ph ^ 1);
      }
    }
  } else if (warp == 5) {
    // ---------------- S of every tile
    const int ksteps = (p.dim + 15) >> 4;
    int g = 0, nload = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 100)) break;
      const int nt = S.item[n % C::ITEMS].nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (nt < 0) break;
      if (nt == 0) continue;
      const int qs = nload % QS;
      ok = wait_all(&S.q_full[qs], (nload / QS) & 1, flags, 101);
      const uint64_t q = kdesc(su32(qbuf + qs * NB * ABOX));
#pragma unroll 1
      for (int t = 0; ok && t < nt; ++t, ++g) {
        // S of tile g goes where P of tile g - 2 was
        ok = wait_all(&S.k_full[s], ph, flags, 102) &&
             (g < 2 || wait_all(&S.pv_done[g & 1], ((g >> 1) - 1) & 1, flags, 103));
        if (!ok) break;
        tc_fence_after();
        const int nk = S.rows[g % (2 * KP)];
        if (elect_lane()) {
          dot_tile(tmem + (g & 1) * KT, q, ABOX, kdesc(su32(kvbuf + 2 * s * C::UNIT)), C::KBOX,
                   idesc(128, (nk + 15) & ~15, 0, 0), ksteps);
          mma_commit(&S.s_full[g & 1]);
          mma_commit(&S.k_empty[s]);
          if (t == nt - 1) mma_commit(&S.q_empty[qs]);
        }
        __syncwarp();
        if (++s == KP) s = 0, ph ^= 1;
      }
      ++nload;
    }
    if (elect_lane()) {
      mma_commit(&S.fin);
      drain_one(&S.fin, 0);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ---------------- O (+)= P V of every tile
    const uint32_t id = idesc(128, ((p.dim + 15) >> 4) * 16, 0, 1);
    int g = 0, nload = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 104)) break;
      const int nt = S.item[n % C::ITEMS].nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (nt < 0) break;
      if (nt == 0) continue;
#pragma unroll 1
      for (int t = 0; ok && t < nt; ++t, ++g) {
        ok = wait_all(&S.v_full[s], ph, flags, 105);
        if (!ok) break;
        const int nk = S.rows[g % (2 * KP)];
        uint8_t* vt = kvbuf + (2 * s + 1) * C::UNIT;
        zero_tail<NB>(vt, C::KBOX, nk, lane);
        // (the first: the item before has read its O)
        ok = (t > 0 || wait_all(&S.o_free, (nload & 1) ^ 1, flags, 106)) &&
             wait_all(&S.p_full[g & 1], (g >> 1) & 1, flags, 107);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane()) {
          sum_ts(tmem + C::O_COL, tmem + (g & 1) * KT, mndesc(su32(vt), C::KBOX), id,
                 (nk + 15) >> 4, t > 0);
          mma_commit(&S.pv_done[g & 1]);
          mma_commit(&S.v_empty[s]);
          flags->tile = g;
        }
        __syncwarp();
        if (++s == KP) s = 0, ph ^= 1;
      }
      ++nload;
    }
    if (elect_lane()) {
      mma_commit(&S.fin2);
      drain_one(&S.fin2, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------- softmax: thread = row
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    const int row = 32 * warp + lane;
    const float c = p.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    int g = 0;
    uint32_t msgs = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 108)) break;
      const FwdItem w = S.item[n % C::ITEMS];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (w.nt < 0) break;
      const int iw = w.i0 + 32 * warp;  // position of the warp's first row
      float m = -INFINITY, l = 0.f;
      bool fresh = true;  // some row of the warp has seen no key
      TileList keys = w.keys;
#pragma unroll 1
      for (int t = 0; t < w.nt; ++t, ++g, keys.next(KT)) {
        const int j0 = keys.r, nk = keys.rows(KT);
        const uint32_t sp = tmem + lane_off + (g & 1) * KT;  // S, and P over it
        const TileView view(p, iw, j0, nk);
        const int wh = view.wh, wl = view.wl, sk = view.sk;
        const int end = 32 * warp < w.nq ? min(nk, wh + 32) : 0;  // past the keys of any row
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if (!wait_all(&S.s_full[g & 1], (g >> 1) & 1, flags, 109)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < nk; q += 32) {
          uint32_t w16[16];
          if (q >= end || (q + 62 < wl && q >= sk)) {  // keys that no row of the warp sees
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = 0u;
          } else {
            float v[32];
            tmem_ld32_async(sp + q, v);
            tmem_wait_ld();
            tmem_landed(v);
            if (q + 32 > min(nk, wh + 1) || (q < wl && q + 32 > sk)) {  // not all see all of them
              const uint32_t see = view.sees(q, lane);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = see & (1u << e) ? v[e] : -INFINITY;
            }
            if (fresh) {  // a row's first keys give its reference
              float mx[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(v[e], v[e + 4]);
#pragma unroll
              for (int e = 8; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], v[e]);
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
              if (m == -INFINITY) m = top;
              fresh = __any_sync(0xffffffffu, m == -INFINITY && row < w.nq);
            }
            const float ref = m == -INFINITY ? 0.f : -m;
            const float2 r2 = make_float2(ref, ref);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 z = fma2(make_float2(v[e], v[e + 1]), c2, r2);
              const float2 y = make_float2(ex2(z.x), ex2(z.y));
              s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], y);
              w16[e >> 1] = pack_bf16(y.x, y.y);
            }
          }
          tmem_st16(sp + (q >> 1), w16);  // the piece of S under it has been read
        }
        const float ts = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        if (__any_sync(0xffffffffu, ts >= kFar && row < w.nq)) {
          tmem_wait_st();
          const float4 r = ask_far<NB>(S, g, msgs, m, ts);
          ok = r.w != 0.f;
          if (!ok) break;
          ++msgs;
          m = r.x;
          l = fmaf(l, r.z, r.y);
        } else {
          l += ts;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[g & 1]);
      }
      ok = ok && wait_all(&S.stat_free[warp], (msgs & 1) ^ 1, flags, 110);
      if (!ok) break;
      ++msgs;
      S.m[row] = m;
      S.l[row] = l;
      if (lane == 0) S.far[warp] = -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.stat_full[warp]);
    }
  } else {
    // ---------------- output: thread = row of the warp's quarter of tensor memory
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int row = 32 * (warp & 3) + lane;
    const bool wide = wide_rows(p.o);
    const int quad = warp & 3;
    int g = 0;
    uint32_t msgs = 0;
#pragma unroll 1
    for (int n = 0;; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 112)) break;
      if (S.item[n % C::ITEMS].nt < 0) break;
      if (!wait_all(&S.stat_full[quad], msgs & 1, flags, 113)) break;
      ++msgs;
      if (S.far[quad] >= 0) {
        msgs = serve_far<NB>(p, S, S.item[n % C::ITEMS], g, tmem + lane_off, msgs);
        if (msgs == 0) break;
      }
      const FwdItem w = S.item[n % C::ITEMS];
      const float m = S.m[row], l = S.l[row];
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.item_empty[n % C::ITEMS]);
        mbar_arrive(&S.stat_free[quad]);
      }
      g += w.nt;
      const bool in = row < w.nq;
      if (p.lse && in)
        p.lse[(int64_t)w.h * p.Tq + w.q0 + w.t0 + row] =
            l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
      __nv_bfloat16* out = p.o.at<__nv_bfloat16>(w.q0 + w.t0 + row, w.h);
      if (w.nt == 0) {  // no query of the tile sees a key
        if (in)
          for (int e = 0; e < p.dim; e += 8)
            *reinterpret_cast<uint4*>(out + e) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      // One barrier for even and one for odd tiles: the product of tile g - 3 was
      // done before S of tile g - 1 came, and that before the statistics, so the
      // parity is not taken for another's.
      if (!wait_all(&S.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, flags, 111)) break;
      tc_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
      for (int d = 0; d < p.dim; d += 32) {
        float o[32];
        tmem_ld32_async(tmem + lane_off + C::O_COL + d, o);
        tmem_wait_ld();
        tmem_landed(o);
        if (d + 32 >= p.dim) {  // the last of O: the next item's product may begin
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.o_free);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (in) st_row32(out + d, o, p.dim - d, wide);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_give(tmem, C::COLS);
}

// ---- launch ---------------------------------------------------------------------
bool tc_fwd_takes(const AttnArgs& p) {
  return p.dim % 8 == 0 && p.dim <= 128 && p.scale > 0.f && tc_heads(p.q, p.Tq, p.heads) &&
         tc_heads(p.k, p.Tk, p.kv) && tc_heads(p.v, p.Tk, p.kv) && tc_heads(p.o, p.Tq, p.heads);
}

template <int NB>
cudaError_t tc_fwd_go(const AttnArgs& p, cudaStream_t st) {
  using C = TcFwd<NB>;
  static_assert(C::CTAS * (C::kSmem + 1024) <= 228 * 1024, "CTAs an SM");
  static PerDevice once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(attn_fwd_tc<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!make_heads_map(&mq, p.q, p.Tq, p.heads, p.dim, AT) ||
      !make_heads_map(&mk, p.k, p.Tk, p.kv, p.dim, C::KT) ||
      !make_heads_map(&mv, p.v, p.Tk, p.kv, p.dim, C::KT))
    return cudaErrorInvalidValue;
  const int64_t items = (int64_t)((p.max_q + AT - 1) / AT) * p.heads * p.B;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  count_launches(1);
  return launch_ex(attn_fwd_tc<NB>, dim3((unsigned)items), dim3(kTcThreads), C::kSmem, st, false,
                   mq, mk, mv, p);
}

cudaError_t tc_fwd(const AttnArgs& p, cudaStream_t st) {
  return p.dim <= 64 ? tc_fwd_go<1>(p, st) : tc_fwd_go<2>(p, st);
}

}  // namespace
}  // namespace ttc
