// Tensor-core backward of windowed attention (bf16, heads of up to 128
// channels in multiples of 8), as two passes of one kernel.
//
// With s = c q.k - lse (in powers of two), p = exp2(s), dp = do.v and
// ds = p (dp - delta), delta = sum_j p dp = o.do:
//   dq = scale ds k   needs a tile of queries and every key it sees,
//   dk = scale ds^T q, dv = p^T do   a tile of keys and every query that sees it.
// One kernel for both would add one of the two into memory from many CTAs: an
// fp32 buffer of dq's size read and written again and again, in an order that
// changes.  Two passes compute s and dp twice (7 products instead of 5, twice
// the exponentials), keep every sum in tensor memory in a fixed order, and
// write each gradient once.
//
// Both passes have the same shape.  X1, X2 are the 128 rows that a CTA works
// on (Q and dO, or K and V), Y1, Y2 tiles of YT of the others' rows (K and V,
// or Q and dO):  S = X1 Y1^T and dP = X2 Y2^T into tensor memory, the softmax
// warps (thread = row) put p and ds over them as bf16, and the accumulators
// take  acc0 += dS Y1  and  acc1 += P Y  (over keys dk and dv; over queries dq
// and P K, see below).
//
// delta comes from the stored o, whose rounding shows in rows of few keys:
// with e = sum_j ds_j, which should vanish, delta + e is right (the p_j add up
// to 1).  Over queries e is known at the end, and dq = scale (acc0 - e P K);
// the pass over keys gets the corrected delta.
//
// Roles as in the forward (one warp issues S and dP, another the sums).  What
// bounds the passes is the chain of hand-overs of a tile, S and dP (0.35 us),
// softmax (1 us), sums (0.3 us), 2.2 us with the waits between, so the one CTA of
// an SM keeps as many tiles in turn as the tensor memory holds: three buffers
// of S and dP for heads of up to 64 channels, two for wider ones, each with its
// own four softmax warps.  Four more warps write the gradients, so that the
// softmax goes on with the next item meanwhile.
//
// 128 sequences of 128, window +-64, 12 heads of 64: 75 us (dq 40, dk and dv 40);
// 64 sequences of 257 to 512, window +-128, 16 heads of 64: 228 us (110 and 124),
// 1.3 TB/s and 27 % of the tensor pipe: the chain above.  One sequence of 16384,
// the last 1024 keys, 8 heads of 128 on 2: 335 us (150, 177, and 11 for the
// pieces), 47 % of the tensor pipe.  The product P K costs the last 20 us, and
// with it dq's error is that of the bf16 weights alone.  Causal without a window,
// long tiles first over all sequences: 4 sequences of 4096, 8 heads of 128, 619 ->
// 492 us (698 TFLOP/s of the five products that a gradient needs; 977 of the seven done).
//
// The pass over keys: the first tokens are seen by every later query, so their
// tile is cut into pieces of its list of query tiles, each the work of one
// item; so is every tile when there are fewer tiles than SMs.  The pieces'
// sums go to the workspace in fp32 and are added in order by one more kernel.
#pragma once

#include "attn_tc.cuh"
#include "attn_tc_fwd.cuh"

namespace ttc {
namespace {

struct BwdCut {
  int tiles;           // key tiles of the longest sequence
  int lead;            // of them, those that hold first tokens outside the window's bound
  int lead_pieces, pieces;
  int64_t lead_slots;  // partial slots of all lead tiles (the others' follow)
  float* parts;        // [slot][2][128][dim]
};

struct BwdItem {
  int64_t x0, y0;      // first rows of the sequence in X and in Y
  int hx, r0, nx;      // head of X, first row and rows of the tile
  int off, sinks;      // position of query row 0; first tokens
  TileList list;       // tiles of Y
  int nt;              // their number; < 0: no more work
  int slot;            // partial sums go here (-1: the gradients themselves)
};

template <bool KV, int NB>
struct TcBwd {
  static constexpr int BUF = NB == 1 ? 3 : 2;     // buffers of S and dP
  static constexpr int YT = 64;                   // rows of a Y tile
  static constexpr int NX = KV ? 2 : 3;           // X tiles: over queries o, too
  static constexpr int XS = NB == 1 ? 2 : 1;      // sets of X tiles in flight
  static constexpr int KP = NB == 1 ? 6 : KV ? 4 : 3;  // pairs of Y tiles in flight
  static constexpr int ITEMS = 4;                 // items told to the roles
  static constexpr int YBOX = YT * 128, UNIT = NB * YBOX, XSET = NX * NB * ABOX;
  static constexpr uint32_t ACC = BUF * 2 * YT, COLS = 512;
  static constexpr int WARPS = 4 * BUF;           // softmax warps
  static constexpr int THREADS = 32 * (WARPS + 7);        // and four that write, three that issue
  struct Shared {
    uint64_t x_full[XS], x_empty[XS], y_full[KP], y_empty[KP];
    uint64_t s_full[BUF], p_full[BUF], done[BUF], acc_full, acc_free, fin, fin2;
    uint64_t item_full[ITEMS], item_empty[ITEMS], clc;
    uint64_t col_full[BUF], half_full[2], half_free[2];  // [item & 1]
    BwdItem item[ITEMS];
    uint4 answer;
    int rows[KP];  // rows of the pair's tile
    alignas(16) float col[KV ? BUF : 1][2][2][KV ? YT : 4];  // lse and delta of a tile's queries
    float half[2][KV ? 1 : BUF + 1][KV ? 1 : AT];  // each buffer's sums of ds, then delta
    uint32_t tmem;
    WaitFlags flags, never;
  };
  static constexpr size_t kSmem = XS * XSET + 2 * KP * UNIT + sizeof(Shared) + 1024;
  static_assert(ACC + 2 * 64 * NB <= COLS, "tensor memory");
};

// CTA number -> item.  False: nothing to do.
template <bool KV, int YT>
__device__ __forceinline__ bool bwd_item(const AttnArgs& p, const BwdCut& cut, uint32_t cta,
                                         BwdItem* w) {
  Seq s;
  w->sinks = p.sinks;
  w->slot = -1;
  if (KV) {
    const uint32_t lead = cut.lead * cut.lead_pieces;
    const uint32_t per = lead + (cut.tiles - cut.lead) * cut.pieces;
    const bool across = long_first(p, cut.tiles);
    const uint32_t row = across ? (uint32_t)p.B * p.kv : per;
    const uint32_t i = cta / row, j = cta - i * row, r = across ? j : i, e = across ? i : j;
    const uint32_t b = r / (uint32_t)p.kv;
    w->hx = (int)(r - b * p.kv);
    int tile, piece, pieces;
    if (e < lead) {
      pieces = cut.lead_pieces;
      tile = e / pieces;
      piece = e - tile * pieces;
      if (pieces > 1) w->slot = (int)(r * lead + e);
    } else {
      pieces = cut.pieces;
      tile = (e - lead) / pieces;
      piece = e - lead - tile * pieces;
      if (pieces > 1)
        w->slot = (int)(cut.lead_slots + r * (per - lead) + (e - lead));
      tile += cut.lead;
    }
    if (!load_seq(p, (int)b, &s, true)) return false;
    w->r0 = tile * AT;
    if (w->r0 >= s.lk) return false;
    w->x0 = s.k0;
    w->y0 = s.q0;
    w->nx = min(AT, s.lk - w->r0);
    const RowSpan rs = row_span(p, s, w->r0, w->r0 + w->nx - 1);
    // the tiles of every head that shares the keys, one head after another
    const int ntq = (rs.t1 - rs.t0 + YT - 1) / YT, all = ntq * p.group;
    const int u0 = (int)((int64_t)all * piece / pieces);
    w->nt = (int)((int64_t)all * (piece + 1) / pieces) - u0;
    const int g0 = ntq ? u0 / ntq : 0;
    w->list.h = w->hx * p.group + g0;
    w->list.r = rs.t0 + YT * (u0 - g0 * ntq);
    w->list.lim = w->list.lim2 = rs.t1;
    w->list.r2 = rs.t0;
    w->list.dh = 1;
  } else {
    const uint32_t ntiles = (p.max_q + AT - 1) / AT;
    const bool across = long_first(p, ntiles);
    const uint32_t row = across ? (uint32_t)p.B * p.heads : ntiles;
    const uint32_t i = cta / row, j = cta - i * row, r = across ? j : i;
    const int tile = (int)(ntiles - 1 - (across ? i : j));
    const uint32_t b = r / (uint32_t)p.heads;
    w->hx = (int)(r - b * p.heads);
    if (!load_seq(p, (int)b, &s, true)) return false;
    w->r0 = tile * AT;
    if (w->r0 >= s.lq) return false;
    w->x0 = s.q0;
    w->y0 = s.k0;
    w->nx = min(AT, s.lq - w->r0);
    const int i0 = w->r0 + s.off();
    const KeySpan ks = key_span(p, s.lk, i0, i0 + w->nx - 1);
    w->list = key_list(ks, w->hx / p.group);
    w->nt = (ks.a1 + YT - 1) / YT + (ks.b1 - ks.b0 + YT - 1) / YT;
  }
  w->off = s.off();
  return true;
}

// sum over the channels of o do, of a row of two swizzled tiles
template <int NB>
__device__ __forceinline__ float row_delta(const uint8_t* o, const uint8_t* d, int row, int dim) {
  float s[2] = {0.f, 0.f};
#pragma unroll 1
  for (int e = 0; 8 * e < dim; ++e) {
    const int at = (e >> 3) * ABOX + row * 128 + (((e & 7) ^ (row & 7)) << 4);
    const uint4 a = *reinterpret_cast<const uint4*>(o + at);
    const uint4 b = *reinterpret_cast<const uint4*>(d + at);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[0] = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s[0]);
      s[1] = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s[1]);
    }
  }
  return s[0] + s[1];
}

template <bool KV, int NB>
__global__ void __launch_bounds__(TcBwd<KV, NB>::THREADS, 1)
    attn_bwd_tc(const __grid_constant__ CUtensorMap tm_x1, const __grid_constant__ CUtensorMap tm_x2,
                const __grid_constant__ CUtensorMap tm_y1, const __grid_constant__ CUtensorMap tm_y2,
                const __grid_constant__ CUtensorMap tm_o,
                const __grid_constant__ AttnArgs p, const __grid_constant__ BwdCut cut) {
  using C = TcBwd<KV, NB>;
  constexpr int YT = C::YT, KP = C::KP, BUF = C::BUF, WARPS = C::WARPS, XS = C::XS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* xbuf = align1k(smem_raw);      // sets of X1, X2 and, over queries, o
  uint8_t* ybuf = xbuf + XS * C::XSET;    // Y1 and Y2 of pair s: units 2 s and 2 s + 1
  auto& S = *reinterpret_cast<typename C::Shared*>(ybuf + 2 * KP * C::UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < XS; ++i)
      mbar_init(&S.x_full[i], 1), mbar_init(&S.x_empty[i], KV ? 1 : 1 + WARPS);
#pragma unroll 1
    for (int i = 0; i < KP; ++i) mbar_init(&S.y_full[i], 1), mbar_init(&S.y_empty[i], 1);
#pragma unroll 1
    for (int i = 0; i < BUF; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.done[i], 1);
      mbar_init(&S.col_full[i], 4);
    }
#pragma unroll 1
    for (int i = 0; i < C::ITEMS; ++i)
      mbar_init(&S.item_full[i], 1), mbar_init(&S.item_empty[i], WARPS + 6);
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      mbar_init(&S.half_full[i], WARPS), mbar_init(&S.half_free[i], 4);
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_free, 4);
    mbar_init(&S.clc, 1);
    mbar_init(&S.fin, 1);
    mbar_init(&S.fin2, 1);
    S.flags = S.never = WaitFlags{0, 0};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARPS + 5) tmem_take(&S.tmem, C::COLS);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  volatile WaitFlags* flags = &S.flags;

  if (warp == WARPS + 4) {
    // ---------------- work and loads
    if (lane == 0) {
      int n = 0, nload = 0, s = 0, loads = 0;
      uint32_t ph = 1, clc = 0;  // parity of the ring's empty barriers; of the next answer
      bool ok = true, first = true;
      // test hook: the first CTA leaves its first pair of tiles unloaded
      const int from =
          blockIdx.x == 0 && debug_take(KV ? TT_DEBUG_ATTN_BWD_KEYS : TT_DEBUG_ATTN_BWD_QUERIES);
      int cta = (int)blockIdx.x;
      BwdItem cur, w;
      cur.nt = -1;
#pragma unroll 1
      while (true) {
        // The next item: told to the roles, its first rows sent for from memory, before
        // the loads of the current one, so that its own loads find them in L2.
        w.nt = -1;
#pragma unroll 1
        while (cta >= 0) {
          if (!first) {
            // After an abort the CTAs that have not started are still taken over, and do
            // nothing.
            cta = wait_one(&S.clc, clc, &S.never, 123) ? clc_take(&S.answer) : -1;
            clc ^= 1;
            if (cta < 0) break;
          }
          first = false;
          clc_ask(&S.answer, &S.clc);
          if (!ok || !bwd_item<KV, YT>(p, cut, (uint32_t)cta, &w)) {
            w.nt = -1;
            continue;
          }
          const int slot = n % C::ITEMS;
          ok = wait_one(&S.item_empty[slot], ((n / C::ITEMS) & 1) ^ 1, flags, 120);
          if (!ok) {
            w.nt = -1;
            continue;
          }
          S.item[slot] = w;
          mbar_arrive(&S.item_full[slot]);
          ++n;
          if (w.nt > 0) {
            prefetch_rows<NB>(&tm_x1, AT, w.hx, (int)w.x0 + w.r0, w.nx);
            prefetch_rows<NB>(&tm_x2, AT, w.hx, (int)w.x0 + w.r0, w.nx);
            if (!KV) prefetch_rows<NB>(&tm_o, AT, w.hx, (int)w.x0 + w.r0, w.nx);
            // (over queries the window: the first tokens are in L2)
            const int r = KV ? w.list.r : w.list.r2, rows = min(w.list.lim2 - r, 4 * YT);
            prefetch_rows<NB>(&tm_y1, YT, w.list.h, (int)w.y0 + r, rows);
            prefetch_rows<NB>(&tm_y2, YT, w.list.h, (int)w.y0 + r, rows);
          }
          break;
        }
        if (ok && cur.nt > 0) {
          const int xs = nload % XS;
          ok = wait_one(&S.x_empty[xs], ((nload / XS) & 1) ^ 1, flags, 121);
          if (ok) {
            const int row = (int)cur.x0 + cur.r0;
            uint8_t* dst = xbuf + xs * C::XSET;
            mbar_expect_tx(&S.x_full[xs], C::XSET);
            load_tile<NB>(dst, ABOX, &tm_x1, &S.x_full[xs], cur.hx, row);
            load_tile<NB>(dst + NB * ABOX, ABOX, &tm_x2, &S.x_full[xs], cur.hx, row);
            if (!KV) load_tile<NB>(dst + 2 * NB * ABOX, ABOX, &tm_o, &S.x_full[xs], cur.hx, row);
            ++nload;
          }
          TileList l = cur.list;
#pragma unroll 1
          for (int t = 0; ok && t < cur.nt; ++t) {
            ok = wait_one(&S.y_empty[s], ph, flags, 122);
            if (!ok) break;
            S.rows[s] = l.rows(YT);
            uint8_t* dst = ybuf + 2 * s * C::UNIT;
            if (loads >= from) {
              mbar_expect_tx(&S.y_full[s], 2 * C::UNIT);
              load_tile<NB>(dst, C::YBOX, &tm_y1, &S.y_full[s], l.h, (int)cur.y0 + l.r);
              load_tile<NB>(dst + C::UNIT, C::YBOX, &tm_y2, &S.y_full[s], l.h,
                            (int)cur.y0 + l.r);
            }
            l.next(YT);
            ++loads;
            if (++s == KP) s = 0, ph ^= 1;
          }
        }
        if (w.nt < 0) break;
        cur = w;
      }
      if (ok && wait_one(&S.item_empty[n % C::ITEMS], ((n / C::ITEMS) & 1) ^ 1, flags, 124)) {
        S.item[n % C::ITEMS].nt = -1;
        mbar_arrive(&S.item_full[n % C::ITEMS]);
      }
      // nothing is in flight into shared memory when the CTA leaves
#pragma unroll 1
      for (int i = 1; i <= XS && i <= nload; ++i)
        drain_one(&S.x_full[(nload - i) % XS], (uint32_t)(((nload - i) / XS) & 1));
#pragma unroll 1
      for (int i = 0; i < KP && i < loads; ++i) {
        if (--s < 0) s = KP - 1, ph ^= 1;
        drain_one(&S.y_full[s], ph ^ 1);  // the last load into pair s
      }
    }
  } else if (warp == WARPS + 5) {
    // ---------------- S and dP of every tile
    const int ksteps = (p.dim + 15) >> 4;
    int nload = 0, s = 0, b = 0;
    uint32_t ph = 0, pb = 1;  // parity of the pair; of the buffer's last sums
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 125)) break;
      const int nt = S.item[n % C::ITEMS].nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (nt < 0) break;
      if (nt == 0) continue;
      const int xs = nload % XS;
      ok = wait_all(&S.x_full[xs], (nload / XS) & 1, flags, 126);
      const uint64_t x = kdesc(su32(xbuf + xs * C::XSET));
#pragma unroll 1
      for (int t = 0; ok && t < nt; ++t) {
        // the p and ds that lie over the buffer have been summed
        ok = wait_all(&S.y_full[s], ph, flags, 128) &&
             wait_all(&S.done[b], pb, flags, 127);
        if (!ok) break;
        tc_fence_after();
        const int ny = S.rows[s];
        if (elect_lane()) {
          const uint64_t y = kdesc(su32(ybuf + 2 * s * C::UNIT));
          const uint32_t id = idesc(128, (ny + 15) & ~15, 0, 0), to = tmem + b * 2 * YT;
          dot_tile(to, x, ABOX, y, C::YBOX, id, ksteps);
          dot_tile(to + YT, x + NB * (ABOX >> 4), ABOX, y + (C::UNIT >> 4), C::YBOX, id, ksteps);
          mma_commit(&S.s_full[b]);
          if (t == nt - 1) mma_commit(&S.x_empty[xs]);
        }
        __syncwarp();
        if (++s == KP) s = 0, ph ^= 1;
        if (++b == BUF) b = 0, pb ^= 1;
      }
      ++nload;
    }
    if (elect_lane()) {
      mma_commit(&S.fin);
      drain_one(&S.fin, 0);
    }
    __syncwarp();
  } else if (warp == WARPS + 6) {
    // ---------------- the sums
    const uint32_t id = idesc(128, ((p.dim + 15) >> 4) * 16, 0, 1);
    int nload = 0, s = 0, b = 0;
    uint32_t ph = 0, pb = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 139)) break;
      const int nt = S.item[n % C::ITEMS].nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (nt < 0) break;
      if (nt == 0) continue;
#pragma unroll 1
      for (int t = 0; ok && t < nt; ++t) {
        ok = wait_all(&S.y_full[s], ph, flags, 140);
        if (!ok) break;
        const int ny = S.rows[s];
        uint8_t* y = ybuf + 2 * s * C::UNIT;
        zero_tail<NB>(y, C::YBOX, ny, lane);
        if (KV) zero_tail<NB>(y + C::UNIT, C::YBOX, ny, lane);
        // (the first: the item before has read its accumulators)
        ok = (t > 0 || wait_all(&S.acc_free, (nload & 1) ^ 1, flags, 129)) &&
             wait_all(&S.p_full[b], pb, flags, 130);
        if (!ok) break;
        tc_fence_after();
        if (elect_lane()) {
          const int steps = (ny + 15) >> 4;
          const uint64_t y1 = mndesc(su32(y), C::YBOX);
          const uint32_t w = tmem + b * 2 * YT;
          sum_ts(tmem + C::ACC + 64 * NB, w, y1 + (KV ? C::UNIT >> 4 : 0), id, steps, t > 0);
          sum_ts(tmem + C::ACC, w + YT, y1, id, steps, t > 0);
          mma_commit(&S.done[b]);
          mma_commit(&S.y_empty[s]);
          if (t == nt - 1) mma_commit(&S.acc_full);
          flags->tile = t;
        }
        __syncwarp();
        if (++s == KP) s = 0, ph ^= 1;
        if (++b == BUF) b = 0, pb ^= 1;
      }
      ++nload;
    }
    if (elect_lane()) {
      mma_commit(&S.fin2);
      drain_one(&S.fin2, 0);
    }
    __syncwarp();
  } else if (warp < WARPS) {
    // ---------------- p and ds: thread = row of X
    const int buf = warp >> 2;                // every BUF-th tile, from the buf-th on
    const int quad = warp & 3, tid = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const int row = 32 * quad + lane;
    const float c = p.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    int turn = 0, nload = 0;  // buffer of the next tile
    uint32_t ps = 0, flip = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 131)) break;
      const BwdItem w = S.item[n % C::ITEMS];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (w.nt < 0) break;
      const bool in = row < w.nx;
      const int xw = w.r0 + 32 * quad + (KV ? 0 : w.off);  // position of the warp's first row
      float2 rl = make_float2(0.f, 0.f);      // - lse (in powers of two) and - delta of the row
      float2 ds2 = make_float2(0.f, 0.f);     // sum of the row's ds
      if (!KV && in) {
        const float ls = p.lse_in[(int64_t)w.hx * p.Tq + w.x0 + w.r0 + row];
        rl.x = ls == -INFINITY ? 0.f : -ls * kLog2e;  // (sees no key)
      }
      if (!KV && w.nt > 0) {
        const int xs = nload % XS;
        if (!wait_all(&S.x_full[xs], (nload / XS) & 1, flags, 138)) break;
        const uint8_t* x = xbuf + xs * C::XSET;
        if (in) rl.y = -row_delta<NB>(x + 2 * NB * ABOX, x + NB * ABOX, row, p.dim);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.x_empty[xs]);
      }
      TileList list = w.list;
#pragma unroll 1
      for (int t = 0; t < w.nt; ++t, list.next(YT)) {
        const bool mine = turn == buf;
        if (++turn == BUF) turn = 0;
        if (!mine) continue;
        const int h = list.h, r = list.r, ny = list.rows(YT);
        const uint32_t sp = tmem + lane_off + buf * 2 * YT;  // S, then dP
        // In columns of the tile: the last that the warp's first row sees, the first
        // that its last row sees, and (over keys) the end of the first tokens.
        int wh, wl, sk = 0, up, low;  // up: no row sees a column past it; low: none before it
        float cv = 0.f;
        if (KV) {
          const int ip = r + w.off;  // position of the tile's first query
          const bool sunk = xw < w.sinks;
          wl = p.right < 0 ? -kAttnMaxLen : xw + 31 - p.right - ip;
          wh = p.left < 0 ? kAttnMaxLen : xw + p.left - ip;
          low = wl - 31;
          up = p.left < 0 || sunk ? kAttnMaxLen : wh + 31;
          // this thread's share of the tile's lse and delta
          const int e = tid < YT ? tid : tid - YT;
          if (e < ny) {
            const int64_t at = (int64_t)h * p.Tq + w.y0 + r + e;
            if (tid < YT) {
              cv = p.lse_in[at];
              cv = cv == -INFINITY ? 0.f : -cv * kLog2e;
            } else {
              cv = -p.delta[at];
            }
          }
        } else {
          wh = p.right < 0 ? kAttnMaxLen : xw + p.right - r;
          wl = p.left < 0 ? -kAttnMaxLen : xw + 31 - p.left - r;
          sk = w.sinks - r;
          up = wh + 31;
          low = wl - 31;
        }
        const int end = 32 * quad < w.nx ? min(ny, up + 1) : 0;
        if (!wait_all(&S.s_full[buf], ps, flags, 132)) { ok = false; break; }
        ps ^= 1;
        tc_fence_after();
        const float* col = nullptr;
        if (KV) {
          // (two buffers in turn: a warp that is still at the last tile reads the other)
          float* dst = &S.col[KV ? buf : 0][flip][0][0];
          dst[tid] = cv;
          col = dst;
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.col_full[buf]);
          if (!wait_all(&S.col_full[buf], flip, flags, 134)) { ok = false; break; }
          flip ^= 1;
        }
        // 16 columns at a time: more would not fit the registers of as many warps
#pragma unroll 1
        for (int q = 0; q < ny; q += 16) {
          uint32_t p8[8], d8[8];
          if (q >= end || (q + 15 < low && (KV || q >= sk))) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p8[e] = d8[e] = 0u;
          } else {
            float v[16], d[16];
            tmem_ld16_async(sp + q, v);
            tmem_ld16_async(sp + YT + q, d);
            tmem_wait_ld();
            tmem_landed(v);
            tmem_landed(d);
            if (q + 16 > min(ny, wh + 1) || (q < wl && (KV || q + 16 > sk))) {
              uint32_t see;
              if (KV) {
                const bool sink = w.r0 + row < w.sinks;
                see = bit_span(wl - 31 + lane - q, sink ? ny - 1 - q : min(ny - 1, wh + lane) - q);
              } else {
                see = bit_span(0, min(ny - 1, wh + lane) - q) &
                      (bit_span(wl - 31 + lane - q, 31) | bit_span(0, sk - 1 - q));
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const bool vis = see & (1u << e);
                v[e] = vis ? v[e] : -INFINITY;
                d[e] = vis ? d[e] : 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float4 ml = make_float4(rl.x, rl.x, rl.x, rl.x);
              float4 md = make_float4(rl.y, rl.y, rl.y, rl.y);
              if (KV) {
                ml = *reinterpret_cast<const float4*>(col + q + e);
                md = *reinterpret_cast<const float4*>(col + YT + q + e);
              }
#pragma unroll
              for (int f = 0; f < 4; f += 2) {
                const float2 z = fma2(make_float2(v[e + f], v[e + f + 1]), c2,
                                      f ? make_float2(ml.z, ml.w) : make_float2(ml.x, ml.y));
                const float2 y = make_float2(ex2(z.x), ex2(z.y));
                const float2 dd = add2(make_float2(d[e + f], d[e + f + 1]),
                                       f ? make_float2(md.z, md.w) : make_float2(md.x, md.y));
                const float2 x = mul2(y, dd);
                if (!KV) ds2 = add2(ds2, x);
                p8[(e + f) >> 1] = pack_bf16(y.x, y.y);
                d8[(e + f) >> 1] = pack_bf16(x.x, x.y);
              }
            }
          }
          // over the pieces of S and dP that have been read
          tmem_st8(sp + (q >> 1), p8);
          tmem_st8(sp + YT + (q >> 1), d8);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[buf]);
      }
      if (!ok) break;
      if (w.nt > 0) {
        if (!KV) {  // for the warps that write
          const int half = nload & 1;
          if (!wait_all(&S.half_free[half], ((nload >> 1) & 1) ^ 1, flags, 134)) break;
          S.half[half][buf][row] = ds2.x + ds2.y;
          if (buf == 0) S.half[half][KV ? 0 : BUF][row] = -rl.y;
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.half_full[half]);
        }
        ++nload;
      }
    }
  } else {
    // ---------------- the gradients
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + C::ACC;
    int nload = 0, turn = 0;  // turn: buffer of the item's first tile
#pragma unroll 1
    for (int n = 0;; ++n) {
      if (!wait_all(&S.item_full[n % C::ITEMS], (n / C::ITEMS) & 1, flags, 141)) break;
      const BwdItem w = S.item[n % C::ITEMS];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n % C::ITEMS]);
      if (w.nt < 0) break;
      const bool in = row < w.nx, some = w.nt > 0;
      const int64_t xr = w.x0 + w.r0 + row;
      float err = 0.f, delta = 0.f;  // sum of the row's ds
      if (!KV && some) {
        const int half = nload & 1;
        if (!wait_all(&S.half_full[half], (nload >> 1) & 1, flags, 135)) break;
        // In the order of the tiles: which buffer an item begins with depends on the
        // items that the CTA has taken before.
#pragma unroll
        for (int i = 0; i < BUF; ++i) {
          err += S.half[half][KV ? 0 : turn][row];
          if (++turn == BUF) turn = 0;
        }
        turn = (turn + w.nt) % BUF;
        delta = S.half[half][KV ? 0 : BUF][row] + err;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.half_free[half]);
      }
      if (!KV && in) p.delta[(int64_t)w.hx * p.Tq + xr] = delta;
      if (some) {
        if (!wait_all(&S.acc_full, nload & 1, flags, 133)) break;
        tc_fence_after();
        ++nload;
      }
      // dk = scale acc0 and dv = acc1, or dq = scale (acc0 - err acc1)
#pragma unroll 1
      for (int a = 0; a < (KV ? 2 : 1); ++a) {
        const Heads& out = KV ? (a ? p.dv : p.dk) : p.dq;
        const float mul = a ? 1.f : p.scale, back = -mul * err;
        const bool wide = wide_rows(out);
        __nv_bfloat16* dst = out.at<__nv_bfloat16>(xr, w.hx);
        float* part = cut.parts + (((int64_t)w.slot * 2 + a) * AT + row) * p.dim;
#pragma unroll 1
        for (int d = 0; d < p.dim; d += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
          if (some) {
            tmem_ld32_async(acc + a * 64 * NB + d, o);
            tmem_wait_ld();
            tmem_landed(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= mul;
            if (!KV) {
              float m[32];
              tmem_ld32_async(acc + 64 * NB + d, m);
              tmem_wait_ld();
              tmem_landed(m);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(m[e], back, o[e]);
            }
            if (d + 32 >= p.dim && (!KV || a)) {  // the accumulators have been read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&S.acc_free);
            }
          }
          if (!in) continue;
          if (KV && w.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (d + e < p.dim)
                *reinterpret_cast<float4*>(part + d + e) =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
            st_row32(dst + d, o, p.dim - d, wide);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == WARPS + 5) tmem_give(tmem, C::COLS);
}

// dk and dv of the key tiles that were worked on in pieces: the pieces' sums
// in order.  A block takes 8 rows of a tile.
__global__ void __launch_bounds__(256) attn_pieces_kernel(AttnArgs p, BwdCut cut) {
  pdl_wait();
  pdl_trigger();
  const bool lead_only = cut.pieces <= 1;
  const uint32_t first = cut.lead_pieces > 1 ? 0 : cut.lead;  // the first tile in pieces
  const uint32_t tiles = (lead_only ? cut.lead : cut.tiles) - first;
  const uint32_t block = blockIdx.x >> 4, rows8 = blockIdx.x & 15;
  const uint32_t r = block / tiles;
  const int tile = (int)(first + block - r * tiles);
  const int b = (int)(r / p.kv), h = (int)(r - (uint32_t)b * p.kv);
  Seq s;
  if (!load_seq(p, b, &s, false)) return;
  const int n = min(AT, s.lk - tile * AT);
  const bool lead = tile < cut.lead;
  const int pieces = lead ? cut.lead_pieces : cut.pieces;
  const int64_t slot = lead ? ((int64_t)r * cut.lead + tile) * pieces
                            : cut.lead_slots +
                                  ((int64_t)r * (cut.tiles - cut.lead) + tile - cut.lead) * pieces;
  const int quads = p.dim / 4;
  for (int e = threadIdx.x; e < 2 * 8 * quads; e += 256) {
    const int a = e / (8 * quads), f = e - a * 8 * quads;
    const int row = rows8 * 8 + f / quads, d = 4 * (f % quads);
    if (row >= n) continue;
    const float* src = cut.parts + ((slot * 2 + a) * AT + row) * p.dim + d;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)i * 2 * AT * p.dim);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    __nv_bfloat16* dst = (a ? p.dv : p.dk).at<__nv_bfloat16>(s.k0 + tile * AT + row, h) + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
  }
}

// ---- launch ---------------------------------------------------------------------
// (without the tensors' layouts: the workspace holds the partial sums in either case)
bool tc_bwd_shape(const AttnPlan& P) {
  return P.act == TT_DT_BF16 && P.dim % 8 == 0 && P.dim <= 128 && P.scale > 0.f;
}
bool tc_bwd_takes(const AttnArgs& p) {
  return p.dim % 8 == 0 && p.dim <= 128 && p.scale > 0.f && tc_heads(p.q, p.Tq, p.heads) &&
         tc_heads(p.k, p.Tk, p.kv) && tc_heads(p.v, p.Tk, p.kv) && tc_heads(p.o, p.Tq, p.heads) &&
         tc_heads(p.dout, p.Tq, p.heads) && tc_heads(p.dq, p.Tq, p.heads) &&
         tc_heads(p.dk, p.Tk, p.kv) && tc_heads(p.dv, p.Tk, p.kv);
}

// How the pass over keys is cut (see the top of the file); *slots: partial slots.
BwdCut bwd_cut(const AttnPlan& P, const tt_attn_seqs* s, int64_t* slots) {
  constexpr int YT = 64;
  BwdCut c = {};
  const int group = P.heads / P.kv;
  c.tiles = (s->max_k + AT - 1) / AT;
  if (P.left >= 0 && P.sinks > 0) {
    c.lead = (P.sinks + AT - 1) / AT;
    if (c.lead > c.tiles) c.lead = c.tiles;
  }
  const int64_t all = (int64_t)group * ((s->max_q + YT - 1) / YT);  // a lead tile's list at most
  int64_t list = all;                                               // another tile's
  if (P.left >= 0 && P.right >= 0) {
    const int64_t span = (int64_t)AT + P.left + P.right;
    const int64_t l = group * ((span + YT - 1) / YT + 1);
    if (l < list) list = l;
  }
  // a lead tile: pieces of about another tile's length; every tile: enough
  // pieces to reach the SMs once
  const int64_t ctas = device_sms();
  const int64_t items = (int64_t)c.tiles * P.kv * s->B;
  int64_t cut = items > 0 && items < ctas ? ctas / items : 1;
  if (cut > list / 4) cut = list / 4;  // no piece under four tiles
  if (cut < 1) cut = 1;
  c.pieces = (int)cut;
  const int64_t len = (list + cut - 1) / cut;
  int64_t lead = len > 0 ? (all + len - 1) / len : 1;
  if (2 * all < 3 * len) lead = 1;
  c.lead_pieces = (int)(lead < 1 ? 1 : lead);
  c.lead_slots = c.lead_pieces > 1 ? (int64_t)s->B * P.kv * c.lead * c.lead_pieces : 0;
  *slots = c.lead_slots +
           (c.pieces > 1 ? (int64_t)s->B * P.kv * (c.tiles - c.lead) * c.pieces : 0);
  return c;
}
size_t bwd_parts_bytes(const AttnPlan& P, const tt_attn_seqs* s) {
  if (!tc_bwd_shape(P)) return 0;
  int64_t slots = 0;
  bwd_cut(P, s, &slots);
  return (size_t)slots * 2 * AT * P.dim * sizeof(float);
}

template <bool KV, int NB>
cudaError_t tc_bwd_go(const AttnArgs& p, const BwdCut& cut, cudaStream_t st) {
  using C = TcBwd<KV, NB>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory of the attention backward");
  static PerDevice once;
  cudaError_t e = once.get([] {
    return cudaFuncSetAttribute(attn_bwd_tc<KV, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, md, mo;
  constexpr int xq = KV ? C::YT : AT, xk = KV ? AT : C::YT;  // rows of a box
  if (!make_heads_map(&mq, p.q, p.Tq, p.heads, p.dim, xq) ||
      !make_heads_map(&mk, p.k, p.Tk, p.kv, p.dim, xk) ||
      !make_heads_map(&mv, p.v, p.Tk, p.kv, p.dim, xk) ||
      !make_heads_map(&md, p.dout, p.Tq, p.heads, p.dim, xq) ||
      !make_heads_map(&mo, p.o, p.Tq, p.heads, p.dim, AT))
    return cudaErrorInvalidValue;
  const int64_t items =
      KV ? (int64_t)p.B * p.kv *
               ((int64_t)cut.lead * cut.lead_pieces + (int64_t)(cut.tiles - cut.lead) * cut.pieces)
         : (int64_t)((p.max_q + AT - 1) / AT) * p.heads * p.B;
  if (items == 0) return cudaSuccess;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  count_launches(1);
  return launch_ex(attn_bwd_tc<KV, NB>, dim3((unsigned)items), dim3(C::THREADS), C::kSmem, st,
                   false, KV ? mk : mq, KV ? mv : md, KV ? mq : mk, KV ? md : mv, mo, p, cut);
}

cudaError_t tc_bwd(const AttnPlan& P, const tt_attn_seqs* s, const AttnArgs& p, float* parts,
                   cudaStream_t st) {
  int64_t slots = 0;
  BwdCut cut = bwd_cut(P, s, &slots);
  cut.parts = parts;
  cudaError_t e = p.dim <= 64 ? tc_bwd_go<false, 1>(p, cut, st) : tc_bwd_go<false, 2>(p, cut, st);
  if (e == cudaSuccess)
    e = p.dim <= 64 ? tc_bwd_go<true, 1>(p, cut, st) : tc_bwd_go<true, 2>(p, cut, st);
  if (e == cudaSuccess && slots > 0) {
    const int first = cut.lead_pieces > 1 ? 0 : cut.lead;
    const int tiles = (cut.pieces > 1 ? cut.tiles : cut.lead) - first;
    const int64_t blocks = (int64_t)p.B * p.kv * tiles * 16;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (blocks > 0) {
      count_launches(1);
      e = launch_ex(attn_pieces_kernel, dim3((unsigned)blocks), dim3(256), 0, st, false, p, cut);
    }
  }
  return e;
}

}  // namespace
}  // namespace ttc
