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
// sees, and stays; a later piece of 32 whose weights sum to more than 2^16
// (m too low by that much) takes a new reference and rescales l, O and the
// weights already written.  That leaves no pass for the maximum and, in
// practice, no rescaling.
//
// Roles: warps 0-3 softmax and output, warp 4 TMA, warp 5 MMA.  S has two
// buffers, so that the next S is computed during a softmax, and two CTAs on
// an SM fill each other's waits.
#pragma once

#include "attn_tc.cuh"

namespace ttc {
namespace {

template <int NB>
struct TcFwd {
  // Two buffers of S and one O share 256 columns of tensor memory (two CTAs
  // an SM): 96 + 96 + 64, or 64 + 64 + 128.
  static constexpr int KT = NB == 1 ? 96 : 64;  // keys of a tile
  static constexpr int QS = NB == 1 ? 2 : 1;    // query tiles in flight
  static constexpr int KS = NB == 1 ? 6 : 4;    // key / value tiles in flight
  static constexpr int KBOX = KT * 128;
  static constexpr uint32_t O_COL = 2 * KT, COLS = 256;
  struct Shared {
    uint64_t q_full[QS], q_empty[QS], kv_full[KS], kv_empty[KS];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free, fin;  // [tile & 1]
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr size_t kSmem = QS * NB * ABOX + KS * NB * KBOX + sizeof(Shared) + 1024;
};

constexpr int kTcThreads = 192;

// One tile of queries of one head and the keys it passes over.
template <int KT>
struct FwdItem {
  Seq s;
  int h, t0, nq, i0;  // head, first row, rows, position of the first row
  KeySpan ks;
  int n1, nt;         // key tiles of the first span, of both
  __device__ void tile(int t, int* j0, int* n) const {
    if (t < n1) {
      *j0 = KT * t;
      *n = min(KT, ks.a1 - *j0);
    } else {
      *j0 = ks.b0 + KT * (t - n1);
      *n = min(KT, ks.b1 - *j0);
    }
  }
};

// Work item -> tile.  Tiles of one index of every sequence and head come one
// after another, the last index first: dealt round-robin, each CTA gets a
// like share of every index, and the tiles that see the most keys under a
// causal mask are not left for the end.  False: nothing to do.
template <int KT>
__device__ __forceinline__ bool fwd_item(const AttnArgs& p, uint32_t item, uint32_t ntiles,
                                         FwdItem<KT>* w) {
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
  w->n1 = (w->ks.a1 + KT - 1) / KT;
  w->nt = w->n1 + (w->ks.b1 - w->ks.b0 + KT - 1) / KT;
  return true;
}

template <int NB>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_fwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, AttnArgs p, uint32_t nitems) {
  using C = TcFwd<NB>;
  constexpr int KT = C::KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qbuf = align1k(smem_raw);
  uint8_t* kvbuf = qbuf + C::QS * NB * ABOX;
  auto& S = *reinterpret_cast<typename C::Shared*>(kvbuf + C::KS * NB * C::KBOX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::QS; ++i) mbar_init(&S.q_full[i], 1), mbar_init(&S.q_empty[i], 1);
    for (int i = 0; i < C::KS; ++i) mbar_init(&S.kv_full[i], 1), mbar_init(&S.kv_empty[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&S.s_full[i], 1), mbar_init(&S.p_full[i], 4), mbar_init(&S.pv_done[i], 1);
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
  const uint32_t ntiles = (p.max_q + AT - 1) / AT;

  if (warp == 4) {
    // ---------------- TMA
    if (lane == 0) {
      int it = 0, n = 0;
      bool ok = true;
      for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
        FwdItem<KT> w;
        if (!fwd_item(p, item, ntiles, &w) || w.nt == 0) continue;
        const int hk = w.h / p.group;
        const int qs = n % C::QS;
        if (!wait_bar(&S.q_empty[qs], ((n / C::QS) & 1) ^ 1, abort_flag, 100)) break;
        load_tile<NB>(qbuf + qs * NB * ABOX, ABOX, &tm_q, &S.q_full[qs], w.h,
                      (int)w.s.q0 + w.t0, w.nq);
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
            load_tile<NB>(kvbuf + s * NB * C::KBOX, C::KBOX, kv ? &tm_v : &tm_k, &S.kv_full[s],
                          hk, (int)w.s.k0 + j0, nk);
          }
        }
      }
      // nothing is in flight into shared memory when the CTA leaves
      for (int i = 0; i < C::QS; ++i)
        if (n > i) drain_bar(&S.q_full[i], (uint32_t)(((n - 1 - i) / C::QS) & 1));
      for (int i = 0; i < C::KS; ++i)
        if (it > i) drain_bar(&S.kv_full[i], (uint32_t)(((it - 1 - i) / C::KS) & 1));
    }
  } else if (warp == 5) {
    // ---------------- MMA: S of tile g, then O += P V of tile g - 1
    const int ksteps = (p.dim + 15) >> 4;
    const uint32_t id_o = idesc(128, ksteps * 16, 0, 1);
    int g = 0, n = 0, o_items = 0, prev_nk = 0;
    bool ok = true, prev_first = false;
    auto pv = [&](int gp) {
      const int s = (2 * gp + 1) % C::KS;
      uint8_t* vt = kvbuf + s * NB * C::KBOX;
      if (!warp_wait(&S.kv_full[s], ((2 * gp + 1) / C::KS) & 1, abort_flag, 102)) return false;
      zero_tail<NB>(vt, C::KBOX, prev_nk, lane);
      if (prev_first) {  // the last item's O has been read
        if (!warp_wait(&S.o_free, (o_items & 1) ^ 1, abort_flag, 103)) return false;
        ++o_items;
      }
      if (!warp_wait(&S.p_full[gp & 1], (gp >> 1) & 1, abort_flag, 104)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t v = mndesc(su32(vt), C::KBOX);
        const uint32_t pc = tmem + (gp & 1) * KT;
        const int steps = (prev_nk + 15) >> 4;
        if (steps == KT / 16) {  // descriptors known before the loop: the products follow closer
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_ts(tmem + C::O_COL, pc + 8 * k, v + 128 * k, id_o, k != 0 || !prev_first);
        } else {
#pragma unroll 1
          for (int k = 0; k < steps; ++k)
            mma_ts(tmem + C::O_COL, pc + 8 * k, v + 128 * k, id_o, k != 0 || !prev_first);
        }
        mma_commit(&S.kv_empty[s]);
        mma_commit(&S.pv_done[gp & 1]);
      }
      __syncwarp();
      return true;
    };
    for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
      FwdItem<KT> w;
      if (!fwd_item(p, item, ntiles, &w) || w.nt == 0) continue;
      const int qs = n % C::QS;
      for (int t = 0; t < w.nt; ++t, ++g) {
        int j0, nk;
        w.tile(t, &j0, &nk);
        // An item's first S waits for its queries, whose buffer is free once the
        // S of the item before is done: no product stands behind it here.
        const int s = (2 * g) % C::KS;
        if ((t == 0 && !warp_wait(&S.q_full[qs], (n / C::QS) & 1, abort_flag, 105)) ||
            !warp_wait(&S.kv_full[s], ((2 * g) / C::KS) & 1, abort_flag, 107) ||
            (g > 1 && !warp_wait(&S.pv_done[g & 1], ((g >> 1) - 1) & 1, abort_flag, 106))) {
          ok = false;  // (the last: P of tile g - 2 lay where S of g goes)
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t q = kdesc(su32(qbuf + qs * NB * ABOX));
          const uint64_t k = kdesc(su32(kvbuf + s * NB * C::KBOX));
          const uint32_t id = idesc(128, (nk + 15) & ~15, 0, 0);
          const uint32_t sc = tmem + (g & 1) * KT;
          if (ksteps == 4 * NB) {
#pragma unroll
            for (int c = 0; c < 4 * NB; ++c)
              mma(sc, q + (c >> 2) * (ABOX >> 4) + 2 * (c & 3),
                  k + (c >> 2) * (C::KBOX >> 4) + 2 * (c & 3), id, c != 0);
          } else {
#pragma unroll 1
            for (int c = 0; c < ksteps; ++c)
              mma(sc, q + (c >> 2) * (ABOX >> 4) + 2 * (c & 3),
                  k + (c >> 2) * (C::KBOX >> 4) + 2 * (c & 3), id, c != 0);
          }
          mma_commit(&S.kv_empty[s]);
          if (t == w.nt - 1) mma_commit(&S.q_empty[qs]);
          mma_commit(&S.s_full[g & 1]);
        }
        __syncwarp();
        if (g > 0 && !pv(g - 1)) { ok = false; break; }
        prev_nk = nk;
        prev_first = t == 0;
      }
      ++n;
    }
    if (ok && g > 0) pv(g - 1);
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
    const float2 c2 = make_float2(c, c);
    const bool wide = wide_rows(p.o);
    int g = 0;
    bool ok = true;
    for (uint32_t item = blockIdx.x; ok && item < nitems; item += gridDim.x) {
      FwdItem<KT> w;
      if (!fwd_item(p, item, ntiles, &w)) continue;
      const int i = w.i0 + row;
      const int iw = w.i0 + 32 * warp;  // the warp's first row
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < w.nt; ++t, ++g) {
        int j0, nk;
        w.tile(t, &j0, &nk);
        const int nq = (nk + 31) >> 5;
        const uint32_t sp = tmem + lane_off + (g & 1) * KT;  // S, and P over it
        if (!warp_wait(&S.s_full[g & 1], (g >> 1) & 1, abort_flag, 109)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < nq; ++q) {
          const int jc = j0 + 32 * q;
          uint32_t w16[16];
          // a piece that none of the warp's rows sees
          if (32 * warp >= w.nq || (p.right >= 0 && jc > iw + 31 + p.right) ||
              (p.left >= 0 && jc + 31 < iw - p.left && jc >= p.sinks)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = 0u;
            tmem_st16(sp + 16 * q, w16);
            continue;
          }
          float v[32];
          tmem_ld32_async(sp + 32 * q, v);
          tmem_wait_ld();
          tmem_landed(v);
          if (!(32 * q + 32 <= nk && (p.right < 0 || jc + 31 <= iw + p.right) &&
                (p.left < 0 || jc >= iw + 31 - p.left || jc + 32 <= p.sinks))) {
            const int hi = min(nk - 1 - 32 * q, p.right < 0 ? 31 : i + p.right - jc);
            uint32_t see = bit_span(0, hi);
            if (p.left >= 0) see &= bit_span(i - p.left - jc, 31) | bit_span(0, p.sinks - 1 - jc);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = see & (1u << e) ? v[e] : -INFINITY;
          }
          float sum;
          auto weights = [&] {
            const float ref = m == -INFINITY ? 0.f : -m;
            const float2 r2 = make_float2(ref, ref);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = fma2(make_float2(v[e], v[e + 1]), c2, r2);
              const float2 y = make_float2(ex2(x.x), ex2(x.y));
              s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], y);
              w16[e >> 1] = pack_bf16(y.x, y.y);
            }
            const float2 s1 = add2(s2[0], s2[1]);
            sum = s1.x + s1.y;
          };
          auto maximum = [&] {
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(v[e], v[e + 4]);
#pragma unroll
            for (int e = 8; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], v[e]);
            return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          };
          if (__any_sync(0xffffffffu, m == -INFINITY)) {  // a row's first keys
            const float top = maximum();
            if (m == -INFINITY) m = top;
          }
          weights();
          if (__any_sync(0xffffffffu, !(sum < 65536.f))) {
            const float top = maximum();
            const bool up = top > m + 8.f;  // (not a NaN in the sum)
            const float f = up ? ex2(m - top) : 1.f;
            if (up) m = top;
            l *= f;
            // O holds the tiles before, which are done; this tile's pieces before
            // lie in P
            if (g > 0 &&
                !warp_wait(&S.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, 110)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (t > 0) {
#pragma unroll 1
              for (int d = 0; 32 * d < p.dim; ++d) {
                float o[32];
                const uint32_t at = tmem + lane_off + C::O_COL + 32 * d;
                tmem_ld32_async(at, o);
                tmem_wait_ld();
                tmem_landed(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(at, o);
              }
            }
#pragma unroll 1
            for (int d = 0; d < q; ++d) {
              uint32_t o[16];
              tmem_wait_st();
              tmem_ld16_async(sp + 16 * d, o);
              tmem_wait_ld();
              tmem_landed(o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = pack_bf16(__uint_as_float(o[e] << 16) * f,
                                 __uint_as_float(o[e] & 0xFFFF0000u) * f);
              tmem_st16(sp + 16 * d, o);
            }
            weights();
          }
          l += sum;
          tmem_st16(sp + 16 * q, w16);  // the columns under it have been read
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[g & 1]);
      }
      if (!ok) break;
      const bool in = row < w.nq;
      if (p.lse && in)
        p.lse[(int64_t)w.h * p.Tq + w.s.q0 + w.t0 + row] =
            l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
      __nv_bfloat16* out = p.o.at<__nv_bfloat16>(w.s.q0 + w.t0 + row, w.h);
      if (w.nt == 0) {  // no query of the tile sees a key
        if (in)
          for (int e = 0; e < p.dim; e += 8)
            *reinterpret_cast<uint4*>(out + e) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      // One barrier for even and one for odd tiles: the product of tile g - 3 was
      // done before S of tile g - 1 came, so the parity is not taken for another's.
      if (!warp_wait(&S.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, 111)) break;
      tc_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d) {
        if (32 * d < p.dim) {
          float o[32];
          tmem_ld32_async(tmem + lane_off + C::O_COL + 32 * d, o);
          tmem_wait_ld();
          tmem_landed(o);
          if (32 * d + 32 >= p.dim) {  // the last of O: the next item's product may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.o_free);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (in) st_row32(out + 32 * d, o, p.dim - 32 * d, wide);
        }
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
