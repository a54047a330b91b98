// What the tensor-core attention kernels share: tiles of 128 rows in
// 128-byte-swizzled shared memory boxes of 64 channels, products with one
// operand in tensor memory, masks as bit words.
#pragma once

#include "attn_seq.cuh"

namespace ttc {
namespace {

constexpr int AT = 128;                  // rows of an accumulator tile
constexpr int ABOX = AT * 128;           // bytes of [128 rows][64 bf16]
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                          int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The rows of one box of the map from `row` on, head h, into NB boxes of 64
// channels, `box` bytes apart.  Rows past the sequence, and channels past the
// head's width (zeros), come along.
template <int NB>
__device__ __forceinline__ void load_tile(uint8_t* dst, int box, const CUtensorMap* map,
                                          uint64_t* bar, int h, int row) {
#pragma unroll
  for (int b = 0; b < NB; ++b) tma_load3(dst + b * box, map, bar, 64 * b, h, row);
}
// n rows on their way from memory to L2 (`box` rows at a time): what the next
// piece of work reads first.
template <int NB>
__device__ __noinline__ void prefetch_rows(const CUtensorMap* map, int box, int h, int row,
                                           int n) {
#pragma unroll 1
  for (int r = 0; r < n; r += box)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(64 * b), "r"(h), "r"(row + r)
                   : "memory");
}

// The list of tiles that a piece of work passes over: rows [r, lim) of head h
// in steps of a tile, then [r2, lim2) of head h + dh, and so on.
struct TileList {
  int h, r, lim, r2, lim2, dh;
  __device__ __forceinline__ int rows(int step) const { return min(step, lim - r); }
  __device__ __forceinline__ void next(int step) {
    r += step;
    if (r >= lim) {
      r = r2;
      lim = lim2;
      h += dh;
    }
  }
};
// The keys that a tile of queries sees: the first tokens, then the window.
__device__ __forceinline__ TileList key_list(const KeySpan& ks, int h) {
  TileList l;
  l.h = h;
  l.r = ks.a1 > 0 ? 0 : ks.b0;
  l.lim = ks.a1 > 0 ? ks.a1 : ks.b1;
  l.r2 = ks.b0;
  l.lim2 = ks.b1;
  l.dh = 0;
  return l;
}

// The wait for a load of one's own on the way out.
__device__ __noinline__ void drain_one(uint64_t* b, uint32_t parity) { drain_bar(b, parity); }

// What a CTA's waits look at: set when one has run out, and the number of the tile whose
// product was issued last.
struct WaitFlags {
  int abort, tile;
};

// Waits of these kernels: one try in line, everything else out of line.  The
// roles of all CTAs of an SM share its instruction cache, and a hand-over
// between two roles is short, so the out-of-line part polls for a while
// before it looks at the timer, whose limit is a load from global memory.  The
// limit counts from the last tile that was worked on: the warps that write wait for all
// of an item, and its list of tiles may be as long as the sequences are.
__device__ __noinline__ bool wait_long(uint64_t* b, uint32_t parity, volatile WaitFlags* flags,
                                       unsigned where) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait(b, parity)) return true;
  const uint64_t limit = *(volatile unsigned long long*)&g_wait_limit_ns;
  uint64_t since = gtimer();
  int tile = flags->tile;
  while (!mbar_try_wait(b, parity)) {
    if (flags->abort) return false;
    const int now = flags->tile;
    if (now != tile) {
      tile = now;
      since = gtimer();
    } else if (gtimer() - since > limit) {
      flags->abort = 1;
      record_error(TT_ERR_TIMEOUT, where);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_one(uint64_t* b, uint32_t parity, volatile WaitFlags* flags,
                                         unsigned where) {
  return mbar_try_wait(b, parity) || wait_long(b, parity, flags, where);
}
// Every lane of a converged warp waits; the warp is converged after it.
__device__ __forceinline__ bool wait_all(uint64_t* b, uint32_t parity, volatile WaitFlags* flags,
                                         unsigned where) {
  return __all_sync(0xffffffffu, wait_one(b, parity, flags, where));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(p));
  return p != 0;
}

// D (tensor memory) += A (tensor memory, two bf16 of consecutive K a column) . B (shared)
__device__ __forceinline__ void mma_ts(uint32_t dtmem, uint32_t atmem, uint64_t b, uint32_t id,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(dtmem),
      "r"(atmem), "l"(b), "r"(id), "r"(acc));
}

// The products of one tile, by one thread.  dot: over the channels, both
// operands K-major tiles of 64-channel boxes (abox, bbox bytes apart).  sum_ts:
// over rows of b (MN-major), the weights in tensor memory.  In fours where they
// come in fours: with known offsets the products follow one another closer.
__device__ __forceinline__ void dot_tile(uint32_t to, uint64_t a, int abox, uint64_t b, int bbox,
                                         uint32_t id, int ksteps) {
#pragma unroll 1
  for (int c = 0; c < ksteps; c += 4) {
    const uint64_t x = a + (c >> 2) * (abox >> 4), y = b + (c >> 2) * (bbox >> 4);
    if (c + 4 <= ksteps) {
#pragma unroll
      for (int e = 0; e < 4; ++e) mma(to, x + 2 * e, y + 2 * e, id, c + e != 0);
    } else {
#pragma unroll 1
      for (int e = 0; c + e < ksteps; ++e) mma(to, x + 2 * e, y + 2 * e, id, c + e != 0);
    }
  }
}
__device__ __forceinline__ void sum_ts(uint32_t to, uint32_t w, uint64_t b, uint32_t id, int steps,
                                       bool add) {
#pragma unroll 1
  for (int k = 0; k < steps; k += 2) {
    mma_ts(to, w + 8 * k, b + 128 * k, id, k != 0 || add);
    if (k + 1 < steps) mma_ts(to, w + 8 * k + 8, b + 128 * k + 128, id, 1);
  }
}
// 32 columns of this thread's lane, not yet readable: tmem_landed orders the
// uses after the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float (&v)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " TT_LD32_REGS ", [%32];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
                 "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
                 "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
                 "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
                 "=f"(v[30]), "=f"(v[31])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_landed(float (&v)[32]) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]));
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}

// 16 packed columns (32 bf16) of this thread's lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]));
}
// 8 packed columns (16 bf16), and 16 f32 columns, of this thread's lane
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_landed(float (&v)[16]) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
// 4 columns: for what is rare and has to do with few registers
__device__ __forceinline__ void tmem_ld4_async(uint32_t taddr, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_landed(float (&v)[4]) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_take(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   su32(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_give(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
               : "memory");
}

// Two f32 in one 64-bit register: x * m + a, and a + b.
__device__ __forceinline__ float2 fma2(float2 x, float2 m, float2 a) {
  return __ffma2_rn(x, m, a);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// 32 values as bf16 to global memory, `n` (a multiple of 8) of them.  wide: the
// address is 32-byte aligned and whole sectors can be written at once.
__device__ __forceinline__ void st_row32(__nv_bfloat16* dst, const float (&v)[32], int n,
                                         bool wide) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (wide && 16 * q + 16 <= n) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * q),
                   "r"(w[8 * q]), "r"(w[8 * q + 1]), "r"(w[8 * q + 2]), "r"(w[8 * q + 3]),
                   "r"(w[8 * q + 4]), "r"(w[8 * q + 5]), "r"(w[8 * q + 6]), "r"(w[8 * q + 7])
                   : "memory");
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (16 * q + 8 * u < n)
          *reinterpret_cast<uint4*>(dst + 16 * q + 8 * u) =
              make_uint4(w[8 * q + 4 * u], w[8 * q + 4 * u + 1], w[8 * q + 4 * u + 2],
                         w[8 * q + 4 * u + 3]);
    }
  }
}
__device__ __forceinline__ bool wide_rows(const Heads& x) {
  return ((reinterpret_cast<uintptr_t>(x.p) | (uintptr_t)(x.row * 2) | (uintptr_t)(x.head * 2)) &
          31) == 0;
}

// Rows n .. (n rounded up to 16) - 1 of a tile's boxes set to zero by one
// warp: the products read keys in steps of 16, and what lies past a
// sequence's end may hold anything (0 * NaN is NaN).
template <int NB>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int box, int n, int lane) {
  const int units = ((16 - (n & 15)) & 15) * 8;  // 16-byte units of a box
  if (!units) return;
#pragma unroll 1
  for (int i = lane; i < units; i += 32)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      *reinterpret_cast<uint4*>(tile + b * box + n * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_async_smem();
  __syncwarp();
}

// The next piece of work of a grid that has one CTA a piece: a running CTA
// takes over a CTA that has not started (cluster launch control), so pieces of
// unlike cost even out and each CTA sets itself up once.  clc_ask requests
// one; the answer (16 bytes) lands on `bar`, and clc_take reads it: the CTA's
// number, or -1 when none is left.
__device__ __forceinline__ void clc_ask(uint4* answer, uint64_t* bar) {
  mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(su32(answer)),
      "r"(su32(bar))
      : "memory");
}
__device__ __forceinline__ int clc_take(const uint4* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n"
      " ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n"
      " mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
      : "=r"(got), "=r"(x)
      : "r"(su32(answer))
      : "memory");
  fence_async_smem();  // the next answer is written through the async proxy
  return got ? (int)x : -1;
}

// Bits [lo, hi] of a word (none when lo > hi), lo and hi any integers.
__device__ __forceinline__ uint32_t bit_span(int lo, int hi) {
  const uint32_t a = lo <= 0 ? 0xFFFFFFFFu : lo > 31 ? 0u : 0xFFFFFFFFu << lo;
  const uint32_t b = hi >= 31 ? 0xFFFFFFFFu : hi < 0 ? 0u : 0xFFFFFFFFu >> (31 - hi);
  return a & b;
}

// (T, heads, dim) tensor as TMA sees it: boxes of 64 channels x 1 head x `rows`
// rows, 128-byte swizzle, zeros outside.
bool make_heads_map(CUtensorMap* m, const Heads& x, int64_t T, int heads, int dim, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
  // the stride of an axis of one is not used; any legal value does
  const int64_t row = T > 1 ? x.row : 64, head = heads > 1 ? x.head : 64;
  cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x.p, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The layouts that the tensor-core kernels take: 16-byte aligned rows of
// whole 16-byte units, strides within the tensor map's 40 bits.
bool tc_heads(const Heads& x, int64_t T, int heads) {
  auto stride_ok = [](int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t(1) << 38); };
  return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && T > 0 && (T == 1 || stride_ok(x.row)) &&
         (heads == 1 || stride_ok(x.head));
}

}  // namespace
}  // namespace ttc
