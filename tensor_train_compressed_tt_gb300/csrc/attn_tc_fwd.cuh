// Tensor-core forward of windowed attention (bf16, heads of up to 128
// channels in multiples of 8).
//
// A CTA takes tiles of 128 queries of one head, one after another, and passes
// once over the keys that a tile sees (the first tokens and the window, in
// tiles of up to 128 keys; a short tile's products and exponentials shrink to
// its width): S = Q K^T into tensor memory, the softmax with its running
// maximum and sum in registers (thread = row), the weights back into tensor
// memory as bf16, O += P V there.  A larger maximum rescales O only when it
// grew by more than 2^8: the weights of a row share one reference, which the
// final division takes out again, and fp32 sums hold the range.
//
// Roles: warps 0-3 softmax and output, warp 4 TMA, warp 5 MMA.  Two CTAs on an
// SM keep the tensor and exponential units busy in turn.  Heads of up to 64
// channels keep P beside S (the next S is computed during the softmax);
// wider ones put P over S, since O takes the columns.
#pragma once

#include "attn_tc.cuh"

namespace ttc {
namespace {

template <int NB>
struct TcFwd {
  static constexpr int QS = NB == 1 ? 2 : 1;   // query tiles in flight
  static constexpr int KS = NB == 1 ? 4 : 2;   // key / value tiles in flight
  static constexpr int UNIT = NB * ABOX;
  static constexpr uint32_t S_COL = 0, P_COL = NB == 1 ? 128 : 0, O_COL = NB == 1 ? 192 : 128;
  static constexpr uint32_t COLS = 256;
  static constexpr bool kOver = NB == 2;       // P lies over S
  struct Shared {
    uint64_t q_full[QS], q_empty[QS], kv_full[KS], kv_empty[KS];
    uint64_t s_full, s_free, p_full, pv_done, o_free, fin;
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr size_t kSmem = (QS + KS) * UNIT + sizeof(Shared) + 1024;
};

constexpr int kTcThreads = 192;

// One tile of queries of one head and the keys it passes over.
struct FwdItem {
  Seq s;
  int h, t0, nq, i0;  // head, first row, rows, position of the first row
  KeySpan ks;
  int n1, nt;         // key tiles of the first span, of both
  __device__ void tile(int t, int* j0, int* n) const {
    if (t < n1) {
      *j0 = AT * t;
      *n = min(AT, ks.a1 - *j0);
    } else {
      *j0 = ks.b0 + AT * (t - n1);
      *n = min(AT, ks.b1 - *j0);
    }
  }
};

// Work item -> tile.  Tiles of one index of every sequence and head come one
// after another, the last index first: dealt round-robin, each CTA gets a
// like share of every index, and the tiles that see the most keys under a
// causal mask are not left for the end.  False: nothing to do.
__device__ __forceinline__ bool fwd_item(const AttnArgs& p, uint32_t item, uint32_t ntiles,
                                         FwdItem* w) {
  const uint32_t per = (uint32_t)p.heads * (uint32_t)p.B;
  const uint32_t back = item / per, r = item - back * per;
  const int tile = (int)(ntiles - 1 - back);
  const uint32_t b = r / (uint32_t)p.heads;
  w->h = (int)(r - b * p.heads);
  if (!load_seq(p, (int)b, &w->s)) return false;
  w->t0 = tile * AT;
  if (w->t0 >= w->s.lq) return false;
  w->nq = min(AT, w->s.lq - w->t0);
  w->i0 = w->t0 + w->s.off();
  w->ks = key_span(p, w->s.lk, w->i0, w->i0 + w->nq - 1);
  w->n1 = (w->ks.a1 + AT - 1) / AT;
  w->nt = w->n1 + (w->ks.b1 - w->ks.b0 + AT - 1) / AT;
  return true;
}

template <int NB>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_fwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, AttnArgs p, uint32_t nitems) {
  using C = TcFwd<NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qbuf = align1k(smem_raw);
  uint8_t* kvbuf = qbuf + C::QS * C::UNIT;
  auto& S = *reinterpret_cast<typename C::Shared*>(kvbuf + C::KS * C::UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::QS; ++i) mbar_init(&S.q_full[i], 1), mbar_init(&S.q_empty[i], 4);
    for (int i = 0; i < C::KS; ++i) mbar_init(&S.kv_full[i], 1), mbar_init(&S.kv_empty[i], 1);
    mbar_init(&S.s_full, 1);
    mbar_init(&S.s_free, 4);
    mbar_init(&S.p_full, 4);
    mbar_init(&S.pv_done, 1);
    mbar_init(&S.o_free, 4);
    mbar_init(&S.fin, 1);
    S.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) tmem_take(&S.tmem, C::COLS);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  volatile int* abort_flag = &S.abort_flag;
  const int ntiles = (p.max_q + AT - 1) / AT;
  const int ksteps = (p.dim + 15) >> 4;

  if (warp == 4) {
    // ---------------- TMA
    if (lane == 0) {
      int it = 0, n = 0;
      bool ok = true;
      int q_par[C::QS], kv_par[C::KS];
      for (int i = 0; i < C::QS; ++i) q_par[i] = -1;
      for (int i = 0; i < C::KS; ++i) kv_par[i] = -1;
      for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
        FwdItem w;
        if (!fwd_item(p, item, ntiles, &w) || w.nt == 0) continue;
        const int hk = w.h / p.group;
        const int qs = n % C::QS;
        if (!wait_bar(&S.q_empty[qs], ((n / C::QS) & 1) ^ 1, abort_flag, 100)) break;
        load_tile<NB>(qbuf + qs * C::UNIT, &tm_q, &S.q_full[qs], w.h, (int)w.s.q0 + w.t0, w.nq);
        q_par[qs] = (n / C::QS) & 1;
        ++n;
        for (int t = 0; ok && t < w.nt; ++t) {
          int j0, nk;
          w.tile(t, &j0, &nk);
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int s = it % C::KS;
            if (!wait_bar(&S.kv_empty[s], ((it / C::KS) & 1) ^ 1, abort_flag, 101)) {
              ok = false;
              break;
            }
            load_tile<NB>(kvbuf + s * C::UNIT, kv ? &tm_v : &tm_k, &S.kv_full[s], hk,
                          (int)w.s.k0 + j0, nk);
            kv_par[s] = (it / C::KS) & 1;
          }
        }
      }
      // nothing is in flight into shared memory when the CTA leaves
      for (int i = 0; i < C::QS; ++i)
        if (q_par[i] >= 0) drain_bar(&S.q_full[i], (uint32_t)q_par[i]);
      for (int i = 0; i < C::KS; ++i)
        if (kv_par[i] >= 0) drain_bar(&S.kv_full[i], (uint32_t)kv_par[i]);
    }
  } else if (warp == 5) {
    // ---------------- MMA: S of tile g beside O += P V of tile g - 1
    int g = 0, n = 0;
    bool ok = true;
    struct {
      int nk, first;
    } prev = {0, 0};
    int o_items = 0;
    auto pv = [&](int gp) {  // O (+)= P V of tile gp
      const int s = (2 * gp + 1) % C::KS;
      if (!warp_wait(&S.kv_full[s], ((2 * gp + 1) / C::KS) & 1, abort_flag, 102)) return false;
      zero_tail<NB>(kvbuf + s * C::UNIT, prev.nk, lane);
      if (prev.first) {  // the last tile's O has been read
        if (!warp_wait(&S.o_free, (o_items & 1) ^ 1, abort_flag, 103)) return false;
        ++o_items;
      }
      if (!warp_wait(&S.p_full, gp & 1, abort_flag, 104)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t v = su32(kvbuf + s * C::UNIT);
        const uint32_t id = idesc(128, ksteps * 16, 0, 1);
        const int steps = (prev.nk + 15) >> 4;
        for (int k = 0; k < steps; ++k)
          mma_ts(tmem + C::O_COL, tmem + C::P_COL + 8 * k, mndesc(v, ABOX) + 128 * k, id,
                 !prev.first || k != 0);
        mma_commit(&S.kv_empty[s]);
        mma_commit(&S.pv_done);
      }
      __syncwarp();
      return true;
    };
    for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
      FwdItem w;
      if (!fwd_item(p, item, ntiles, &w) || w.nt == 0) continue;
      const int qs = n % C::QS;
      for (int t = 0; ok && t < w.nt; ++t, ++g) {
        int j0, nk;
        w.tile(t, &j0, &nk);
        if (C::kOver && g > 0) {
          // P of tile g - 1 is read before S of tile g is written over it
          if (!pv(g - 1) || !warp_wait(&S.pv_done, (g - 1) & 1, abort_flag, 106)) {
            ok = false;
            break;
          }
        }
        // (after the last item's product: a single query buffer is not refilled before it)
        if (t == 0 && !warp_wait(&S.q_full[qs], (n / C::QS) & 1, abort_flag, 105)) {
          ok = false;
          break;
        }
        const int s = (2 * g) % C::KS;
        if (!warp_wait(&S.kv_full[s], ((2 * g) / C::KS) & 1, abort_flag, 107) ||
            !warp_wait(&S.s_free, (g & 1) ^ 1, abort_flag, 108)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t q = su32(qbuf + qs * C::UNIT), k = su32(kvbuf + s * C::UNIT);
          const uint32_t id = idesc(128, (nk + 15) & ~15, 0, 0);
          for (int c = 0; c < ksteps; ++c) {
            const uint32_t box = (c >> 2) * ABOX;
            mma(tmem + C::S_COL, kdesc(q + box) + 2 * (c & 3), kdesc(k + box) + 2 * (c & 3), id,
                c != 0);
          }
          mma_commit(&S.kv_empty[s]);
          mma_commit(&S.s_full);
        }
        __syncwarp();
        if (!C::kOver && g > 0 && !pv(g - 1)) { ok = false; break; }
        prev.nk = nk;
        prev.first = t == 0;
      }
      ++n;
    }
    if (ok && g > 0) ok = pv(g - 1);
    if (lane == 0) {
      mma_commit(&S.fin);
      drain_bar(&S.fin, 0);
    }
    __syncwarp();
  } else {
    // ---------------- softmax and output: thread = row
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    const int row = 32 * warp + lane;
    const float c = p.scale * kLog2e;
    int g = 0, n = 0;
    bool ok = true;
    for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
      FwdItem w;
      if (!fwd_item(p, item, ntiles, &w)) continue;
      const int i = w.i0 + row;
      float m = -INFINITY, l = 0.f;
      const int iw = w.i0 + 32 * warp;  // the warp's first row
      for (int t = 0; t < w.nt; ++t, ++g) {
        int j0, nk;
        w.tile(t, &j0, &nk);
        const int nq = (nk + 31) >> 5;
        const int hi = min(nk - 1, p.right < 0 ? nk - 1 : i + p.right - j0);
        const int lo = p.left < 0 ? 0 : i - p.left - j0;
        const int sunk = p.sinks - 1 - j0;
        if (!warp_wait(&S.s_full, g & 1, abort_flag, 109)) { ok = false; break; }
        tc_fence_after();
        // first pass over S: each row's maximum.  32-key pieces that none of
        // the warp's rows sees are skipped, those that all see need no mask.
        uint32_t none = 0, all = 0;
        float top = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < nq; ++q) {
          const int jc = j0 + 32 * q;
          if ((p.right >= 0 && jc > iw + 31 + p.right) ||
              (p.left >= 0 && jc + 31 < iw - p.left && jc >= p.sinks)) {
            none |= 1u << q;
            continue;
          }
          float v[32];
          tmem_ld32_async(tmem + lane_off + C::S_COL + 32 * q, v);
          tmem_wait_ld();
          tmem_landed(v);
          if (32 * q + 32 <= nk && (p.right < 0 || jc + 31 <= iw + p.right) &&
              (p.left < 0 || jc >= iw + 31 - p.left || jc + 32 <= p.sinks)) {
            all |= 1u << q;
          } else {
            const uint32_t see = (bit_span(lo - 32 * q, 31) | bit_span(0, sunk - 32 * q)) &
                                 bit_span(0, hi - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = see & (1u << e) ? v[e] : -INFINITY;
          }
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(v[e], v[e + 4]);
#pragma unroll
          for (int e = 8; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], v[e]);
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        }
        top *= c;
        // P and O of the tile before are done with
        if (g > 0 && !warp_wait(&S.pv_done, (g - 1) & 1, abort_flag, 110)) { ok = false; break; }
        tc_fence_after();
        const bool up = top > m + 8.f;
        if (__any_sync(0xffffffffu, up)) {
          const float f = up ? ex2(m - top) : 1.f;
          if (up) m = top;
          l *= f;
          if (t > 0) {
#pragma unroll 1
            for (int q = 0; 32 * q < p.dim; ++q) {
              float o[32];
              const uint32_t at = tmem + lane_off + C::O_COL + 32 * q;
              tmem_ld32_async(at, o);
              tmem_wait_ld();
              tmem_landed(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(at, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;  // a row that has seen no key yet
        // second pass: weights and their sum
#pragma unroll 1
        for (int q = 0; q < nq; ++q) {
          uint32_t w16[16];
          if (none & (1u << q)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = 0u;
          } else {
            float v[32];
            tmem_ld32_async(tmem + lane_off + C::S_COL + 32 * q, v);
            tmem_wait_ld();
            tmem_landed(v);
            if (!(all & (1u << q))) {
              const uint32_t see = (bit_span(lo - 32 * q, 31) | bit_span(0, sunk - 32 * q)) &
                                   bit_span(0, hi - 32 * q);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = see & (1u << e) ? v[e] : -INFINITY;
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float a = ex2(fmaf(v[e], c, -ref));
              const float b = ex2(fmaf(v[e + 1], c, -ref));
              sum[e & 2] += a;
              sum[(e & 2) + 1] += b;
              w16[e >> 1] = pack_bf16(a, b);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          // (over S, the piece's own columns have been read)
          tmem_st16(tmem + lane_off + C::P_COL + 16 * q, w16);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.s_free);
          mbar_arrive(&S.p_full);
        }
      }
      if (!ok) break;
      // output: through the query tile's shared memory, so that rows leave in whole lines
      const bool in = row < w.nq;
      if (p.lse && in) {
        float ls = -INFINITY;
        if (w.nt > 0 && (l > 0.f || l != l)) ls = (m + log2f(l)) * kLn2;
        p.lse[(int64_t)w.h * p.Tq + w.s.q0 + w.t0 + row] = ls;
      }
      if (w.nt == 0) {  // no query of the tile sees a key
        if (in) {
          uint4* o = reinterpret_cast<uint4*>(
              p.o.at<__nv_bfloat16>(w.s.q0 + w.t0 + row, w.h));
          for (int e = 0; e < p.dim / 8; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      if (!warp_wait(&S.pv_done, (g - 1) & 1, abort_flag, 111)) { ok = false; break; }
      tc_fence_after();
      const int qs = n % C::QS;
      uint8_t* stage = qbuf + qs * C::UNIT;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
      for (int q = 0; 32 * q < p.dim; ++q) {
        float o[32];
        tmem_ld32_async(tmem + lane_off + C::O_COL + 32 * q, o);
        tmem_wait_ld();
        tmem_landed(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        st_tile_half(stage + (q >> 1) * ABOX, row, q & 1, o);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.o_free);
      const int units = p.dim / 8;  // 16-byte units of a row
      for (int e = lane; e < 32 * units; e += 32) {
        const int r = e / units, u = e - r * units;
        const int rr = 32 * warp + r;
        if (rr >= w.nq) break;
        const uint4 x = *reinterpret_cast<const uint4*>(stage + (u >> 3) * ABOX + rr * 128 +
                                                        (((u & 7) ^ (rr & 7)) << 4));
        *reinterpret_cast<uint4*>(p.o.at<__nv_bfloat16>(w.s.q0 + w.t0 + rr, w.h) + 8 * u) = x;
      }
      fence_async_smem();  // the next query tile comes in through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_empty[qs]);
      ++n;
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
  static_assert(2 * (C::kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  static PerDevice once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(attn_fwd_tc<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!make_heads_map(&mq, p.q, p.Tq, p.heads, p.dim) ||
      !make_heads_map(&mk, p.k, p.Tk, p.kv, p.dim) || !make_heads_map(&mv, p.v, p.Tk, p.kv, p.dim))
    return cudaErrorInvalidValue;
  const int64_t items = (int64_t)((p.max_q + AT - 1) / AT) * p.heads * p.B;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const int64_t most = 2 * (int64_t)device_sms();
  count_launches(1);
  return launch_ex(attn_fwd_tc<NB>, dim3((unsigned)(items < most ? items : most)),
                   dim3(kTcThreads), C::kSmem, st, false, mq, mk, mv, p, (uint32_t)items);
}

cudaError_t tc_fwd(const AttnArgs& p, cudaStream_t st) {
  return p.dim <= 64 ? tc_fwd_go<1>(p, st) : tc_fwd_go<2>(p, st);
}

}  // namespace
}  // namespace ttc
