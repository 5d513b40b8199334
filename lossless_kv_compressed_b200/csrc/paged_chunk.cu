// Paged attention of many rows (prefill chunks, verify blocks) on the 5th-generation tensor
// cores: tcgen05 with TMEM accumulators, pages by TMA.
//
// Mathematics as in paged_rows.cu: tiles of keys, log2-domain scores against a running
// reference that is raised only when a tile's maximum exceeds it by more than 2^8, weights
// in bf16 (what they are rounded from is summed for l).  A row's 8-bit keys and values enter
// the products as their codes, exact in bf16; the key's scale multiplies the score, the
// value's scale the weight before its rounding.
//
// One persistent CTA per SM takes an equal share of the line of key tiles (Deal): units of
// 256 rows (row r = token * g + head, two UMMA M-tiles of 128) by 64 keys.
//   warp 0      producer: K and V tiles [64 keys x D] (128-byte swizzle) of the unit's pages
//               into a ring of tile slots, a lane per box of a page
//   warp 1, 2   UMMA issuer of M-tile 0, 1: S = Q K^T (both from shared memory), then
//               O += P V with P from TMEM; the ring is released by commits of both
//   warp 3      bf16 pages: zeroes the value rows behind a sequence's last token (those
//               slots may hold NaN, and 0 * NaN is no 0) before the tile is handed on
//   warps 4-11  softmax, a thread per row; M-tile 1's row r sits in lane r ^ kFlip
//   warps 12-19 8-bit pages: codes (a ring of their own) to bf16 tiles, four warps for K and
//               four for V
// Each M-tile has two S buffers of 64 columns in TMEM, and P overwrites the S that it came
// from: the products of tile j + 1 run while the softmax is at tile j, and S of tile j + 2
// follows the P V of tile j.  (One S buffer of 128 keys instead, D 128, 2048 new tokens over
// 32K: the chain S - softmax - P V - S took 5100 cycles per 128 keys, of which the softmax
// 2600; 1231 us.)
//
// Measured (32 heads over 8, D 128, a call in a loop): 2048 new tokens over 32K in bf16
// 955-985 us = 1.08-1.12 PFLOP/s, e4m3 1375 us; 8 sequences of 32 tokens over 32K (one M-tile)
// 200 us = 5.4 TB/s, of 33 tokens (a second M-tile of four rows) 247 us, e4m3 363 us; D 64, 2048
// tokens 824 us.  Bound: the softmax, a chain of 1750 cycles a tile of which 1110 are the
// exponentials of two warps on a sub-partition (640 for one), against 1024 of tensor work; with
// the power cap on long bf16 chunks; 8-bit pages the same chain, whose sub-partitions the
// conversion shares.  Tried: the columns of a row split over two warps, which halves a warp's
// chain but adds a barrier a tile, 1172 us for 1075 then; the last 16 rows of an M-tile by
// mma.sync, e4m3 622 us for 393; tiles prefetched into L2 three ahead, 1026 us for 1000.
//
// Every wait is bounded as in verify_attn.cu: on expiry the CTA raises the device error
// word, lets its copies and products land, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "paged.cuh"
#include "paged_internal.h"
#include "paged_io.cuh"
#include "tc05.cuh"
#include "vc_internal.h"

namespace vc {
namespace paged {

constexpr int kCG = 256;                 // rows of a unit
constexpr int kCK = 64;                  // keys of a tile
constexpr float kCRaise = 8.f;

__device__ int g_chunks_error;           // bit 1: a bounded wait expired

template <int D, int PT>
struct ChunkCfg {
  static constexpr bool k8 = PT != VC_PAGE_BF16;
  static constexpr int kThreads = k8 ? 640 : 384;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kTile = kCK * D * 2;              // K or V tile in bf16
  // stages of a K and a V tile: bf16 for the UMMAs, and for 8-bit pages the codes before
  // their conversion
  static constexpr int kStages = D == 128 ? (k8 ? 3 : 5) : (k8 ? 4 : 8);
  static constexpr int kRaw = k8 ? kCK * D : kTile;      // bytes of K, or V, that TMA brings
  static constexpr int kRawStages = k8 ? (D == 128 ? 3 : 4) : 0;
  // A tile's scales are read until its softmax is done.  The load of tile t + 8 waits for
  // the conversion of tile t + 8 - kRawStages, which waits for the P V of tile
  // t + 8 - kRawStages - kStages.
  static constexpr int kScaleSlots = 8;
  static_assert(8 - kRawStages - kStages >= 0, "scale slots");
  // Of eight pairs of exponentials, those on the FMA pipe (2048 tokens over 32K, bf16, none to
  // three: 978, 971, 962, 964 us, D 64 889, 860, 834, 849; 8-bit, whose FMA pipe has the scales:
  // none 1564, two 1680); registers of weights stored at a time.
  static constexpr int kPoly = k8 ? 0 : 2;
  static constexpr int kPw = k8 ? 16 : 32;
  // Places the first rows of a part-filled second M-tile on sub-partition 3 (96) or 2 (64).
  // 33 rows e4m3 359 us with 96, 371 with 64; bf16 244 and 247, but whole tiles 962 and 953.
  static constexpr int kFlip = k8 ? 96 : 64;
  static constexpr int kQ0 = 0;
  static constexpr int kRing = 2 * kQTile;
  static constexpr int kRawRing = kRing + kStages * 2 * kTile;
  static constexpr int kScale = kRawRing + kRawStages * 2 * kRaw;
  // scales of a tile: boxes of 16 rows on 128-byte boundaries (TMA), larger ones packed
  static constexpr int kScaleTile = kCK / 16 * 128;
  static constexpr int kBar = kScale + (k8 ? kScaleSlots * 2 * kScaleTile : 0);
  static constexpr int kNBar = 2 * kStages + 2 * (k8 ? kRawStages : kStages) + 2 + 4 + 4 + 2 + 1;
  static constexpr int kTmemSlot = kBar + kNBar * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;
  static constexpr uint32_t kColO = 0;
  static constexpr uint32_t kColS = 2 * D;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColS + 4 * kCK <= kTmemCols, "TMEM columns");
  static_assert(kAlloc <= 232448, "shared memory");
};

struct ChunkParams {
  const __nv_bfloat16* q;
  int64_t q_tok, q_head;
  const int32_t* table;
  int32_t max_pages, n_pages, page, page_shift, rows_per_box;
  int32_t Hq;
  float qk2;
  void* out;
  float* lse;
  int32_t out_f32;
  float* ws_o;                  // [workers, 2, 256, D]
  float* ws_ml;                 // [workers, 2, 256, 2]
  Cut* cut;                     // [workers]
  int32_t* err_flag;
  uint64_t wait_ns;
};

// Registers of a thread from here on (whole warpgroups; the shares add up to at most what
// the block was launched with).
template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}
// The scales of 32 keys from number k on, every load issued before any is used (volatile: the
// compiler otherwise loads four at a time and waits for each).
__device__ __forceinline__ void scales32(uint32_t at, int k, int gap, float (&f)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(f[4 * c]), "=f"(f[4 * c + 1]), "=f"(f[4 * c + 2]), "=f"(f[4 * c + 3])
                 : "r"(at + (k + 4 * c) * 4 + (k + 4 * c) / 16 * gap));
}
// The largest of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[16]) { tc::tmem_st16(t, r); }
__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[32]) { tc::tmem_st32(t, r); }

// ------------------------------------------------------------------ packed fp32 pairs
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of two numbers in [-inf, 2^7) on the FMA pipe: x = n + r with n the nearest integer,
// 2^r by the polynomial of degree 4 with the least relative error on [-1/2, 1/2] (2.7e-6,
// coefficients from a Remez iteration), n added to the exponent.  Under 2^-125 it stays there.
__device__ __forceinline__ void ex2_poly(uint64_t x, float& a, float& b) {
  f2_get(x, a, b);
  x = f2(fmaxf(a, -125.f), fmaxf(b, -125.f));
  const uint64_t big = f2(12582912.f, 12582912.f);           // 1.5 * 2^23: n in the low bits
  const uint64_t t = f2_add(x, big);
  const uint64_t r = f2_fma(f2_add(t, f2(-12582912.f, -12582912.f)), f2(-1.f, -1.f), x);
  uint64_t y = f2_fma(r, f2(0.009570102207362652f, 0.009570102207362652f),
                      f2(0.05591785907745361f, 0.05591785907745361f));
  y = f2_fma(r, y, f2(0.240247443318367f, 0.240247443318367f));
  y = f2_fma(r, y, f2(0.6931217908859253f, 0.6931217908859253f));
  y = f2_fma(r, y, f2(0.9999992847442627f, 0.9999992847442627f));
  float ta, tb;
  f2_get(t, ta, tb);
  f2_get(y, a, b);
  a = __uint_as_float(__float_as_uint(a) + (__float_as_uint(ta) << 23));
  b = __uint_as_float(__float_as_uint(b) + (__float_as_uint(tb) << 23));
}

// ------------------------------------------------------------------ codes to bf16
// codes_to_bf16 takes an e4m3 NaN (0x7f, 0xff) for the 480 that its bits would be; this makes it
// one again.
__device__ __forceinline__ void put_nan(uint2& r) {
  r.x |= __vcmpeq2(r.x & 0x7fff7fffu, 0x43f043f0u) & 0x7fff7fffu;
  r.y |= __vcmpeq2(r.y & 0x7fff7fffu, 0x43f043f0u) & 0x7fff7fffu;
}
// Four codes of a word as bf16 pairs, exactly.  most: the largest e4m3 magnitude bits so far in
// each half, which are 0x07f0 if one of the codes is a NaN (and the pairs then need put_nan).
template <int PT>
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t& most) {
  uint32_t r[2], mag[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (PT == VC_PAGE_E4M3) {
      // code s eeee fff as bf16 s 0000eeee fff0000 is 2^-120 of its value (subnormal codes
      // too, as subnormal bf16)
      const uint32_t x = __byte_perm(w, 0, i ? 0x3424 : 0x1404);       // codes in the high bytes
      mag[i] = (x >> 4) & 0x07f007f0u;
      const uint32_t y = mag[i] | (x & 0x80008000u);
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(y), "r"(0x7b807b80u));   // 2^120
    } else {
      // 128 + low 7 bits, less 128, or 256 where the sign bit is set
      const uint32_t x = __byte_perm(w, 0, i ? 0x4342 : 0x4140);       // codes in the low bytes
      const uint32_t a = (x & 0x007f007fu) | 0x43004300u;
      const uint32_t b = (x & 0x00800080u) | 0x43004300u;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(a), "r"(b));
    }
  }
  if constexpr (PT == VC_PAGE_E4M3) most = __vimax3_u16x2(most, mag[0], mag[1]);
  return make_uint2(r[0], r[1]);
}

template <int D, int PT>
__global__ void __launch_bounds__(ChunkCfg<D, PT>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmKS,
                       const __grid_constant__ CUtensorMap tmVS, const Deal<kCG, kCK> deal,
                       const ChunkParams p) {
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
    if constexpr (PT != VC_PAGE_BF16) {
      tc::prefetch_tmap(&tmKS);
      tc::prefetch_tmap(&tmVS);
    }
  }
  pdl_wait();
  pdl_trigger();
  using L = ChunkCfg<D, PT>;
  constexpr bool k8 = L::k8;
  constexpr int NS = L::kStages, NR = k8 ? L::kRawStages : L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // every role walks the same units by a cursor of its own
  typename Deal<kCG, kCK>::Lane l0;
  const int64_t total = deal.total(lane, l0);
  const Shares sh(total, deal.workers(total));
  const int64_t w = blockIdx.x;
  const int64_t t0 = w < sh.W ? sh.first(w) : total;
  const int n = w < sh.W ? (int)(sh.first(w + 1) - t0) : 0;    // tiles of this worker
  Cursor<kCG, kCK> cur;
  if (n > 0) cur.seek(deal, l0, t0, lane);
  if (warp == 0) note_cut(p.cut + w, deal, sh, cur, t0, n, lane);
  if (n == 0) return;

  auto bar = [&](int i) -> uint32_t { return sb + L::kBar + 8 * i; };
  auto b_full = [&](int s) { return bar(s); };             // tile ready for the UMMAs
  auto b_empty = [&](int s) { return bar(NS + s); };       // released by both issuers
  // arrived, still to be converted, or (bf16) cut at the end
  auto b_raw = [&](int s) { return bar(2 * NS + s); };
  auto b_raw_empty = [&](int s) { return bar(2 * NS + NR + s); };
  constexpr int kB = 2 * NS + 2 * NR;
  auto b_q = [&](int mt) { return bar(kB + mt); };
  auto b_s = [&](int mt, int buf) { return bar(kB + 2 + 2 * mt + buf); };
  auto b_p = [&](int mt, int buf) { return bar(kB + 6 + 2 * mt + buf); };
  auto b_o = [&](int mt) { return bar(kB + 10 + mt); };
  const uint32_t b_teardown = bar(kB + 12);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(b_full(s), k8 ? 8 : 1);
      tc::mbar_init(b_empty(s), 2);
    }
    for (int s = 0; s < NR; ++s) {
      tc::mbar_init(b_raw(s), 1);
      tc::mbar_init(b_raw_empty(s), 8);
    }
    for (int mt = 0; mt < 2; ++mt) {
      tc::mbar_init(b_q(mt), 4);
      for (int buf = 0; buf < 2; ++buf) {
        tc::mbar_init(b_s(mt, buf), 1);
        tc::mbar_init(b_p(mt, buf), 4);
      }
      tc::mbar_init(b_o(mt), 1);
    }
    tc::mbar_init(b_teardown, 2);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async();
  }
  if (warp == 1) tc::tmem_alloc(sb + L::kTmemSlot, L::kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlot);

  auto raise = [&]() {
    *abort_flag = 1;
    atomicOr(&g_chunks_error, 2);
  };
  auto rows_of = [&](const Cursor<kCG, kCK>& c) -> int {
    return (int)min((int64_t)kCG, (int64_t)c.q.nq * deal.g - (int64_t)c.rg * kCG);
  };

  // 8-bit pages launch with 640 x 96 registers: 56 + 2 x 152 + 2 x 56 <= 5 x 96.  (The roles of 56
  // spill 484 bytes, 1.2% of the instructions executed.)
  if (warp < 4) {
    if constexpr (k8) set_regs_down<56>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      constexpr int kHalves = k8 ? 1 : D / 64;
      const int nb = kCK / p.rows_per_box;                   // boxes of a tile (per half)
      // lanes 0-15 load K, 16-31 V: a lane a box
      const int kv = lane >> 4, box_of = (lane & 15) % nb, half = (lane & 15) / nb;
      const bool mine = (lane & 15) < nb * kHalves;
      const CUtensorMap* map = kv ? &tmV : &tmK;
      const CUtensorMap* smap = kv ? &tmVS : &tmKS;
      int chunk = -1, ids = 0, ahead = 0;
      auto load_ids = [&](int ch) -> int {
        const int64_t pos = ((int64_t)ch * 32 + lane) * p.rows_per_box;
        int id = p.n_pages;                                  // out of range: TMA fills zeros
        if (pos < cur.q.len) {
          id = __ldg(p.table + (int64_t)cur.b * p.max_pages + (pos >> p.page_shift));
          if ((unsigned)id >= (unsigned)p.n_pages) {
            id = p.n_pages;
            if (p.err_flag) atomicOr(p.err_flag, VC_PAGED_BAD_PAGE);
          }
        }
        return id;
      };
      int st = 0, use = 0;
      uint32_t tails = 0, tail_use = 0;    // bf16: stages whose last use went by b_raw, its parity
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int box = cur.tile * nb;
        if ((box >> 5) != chunk) {
          ids = (chunk >= 0 && (box >> 5) == chunk + 1) ? ahead : load_ids(box >> 5);
          chunk = box >> 5;
          ahead = load_ids(chunk + 1);
        }
        const int id = __shfl_sync(0xffffffffu, ids, (box + box_of) & 31);
        const int y = (int)(((int64_t)box + box_of) * p.rows_per_box & (p.page - 1));
        if (use > 0)
          ok = warp_wait(k8 ? b_raw_empty(st) : b_empty(st), (use - 1) & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        // tiles with slots behind the last token pass through warp 3, 8-bit ones through the
        // conversion
        const bool by_raw = k8 || (cur.tile + 1) * (int64_t)kCK > cur.q.len;
        const uint32_t fb = by_raw ? b_raw(st) : b_full(st);
        if (!k8) {
          if (by_raw) {
            tails |= 1u << st;
            tail_use ^= 1u << st;
          } else {
            tails &= ~(1u << st);
          }
        }
        if (lane == 0) tc::mbar_expect_tx(fb, 2 * (L::kRaw + (k8 ? kCK * 4 : 0)));
        __syncwarp();
        if (mine) {
          const uint32_t dst = sb + (k8 ? L::kRawRing : L::kRing) + (2 * st + kv) * L::kRaw;
          tma_load_5d(dst + (k8 ? box_of * p.rows_per_box * D
                                : half * (kCK * 128) + box_of * p.rows_per_box * 128),
                      map, fb, 0, y, half, cur.kvh, id);
          if constexpr (k8)
            tc::tma_load_3d(sb + L::kScale + (2 * (i % L::kScaleSlots) + kv) * L::kScaleTile +
                                box_of * max(p.rows_per_box * 4, 128),
                            smap, fb, y, cur.kvh, id);
        }
        if (++st == NR) { st = 0; ++use; }
        if (++cur.tile == cur.n_tiles && i + 1 < n) {
          const int b = cur.b;
          cur.next_unit(deal);
          if (cur.b != b) chunk = -1;
        }
      }
      if (!ok && lane == 0) raise();
      // loads in flight land before the shared memory is given back: every stage's last use
      for (int s = 0; s < NR; ++s) {
        const int uses = use + (s < st ? 1 : 0);
        if (uses == 0) continue;
        if (k8) {
          tc::mbar_wait(b_raw(s), (uses - 1) & 1, nullptr, 1000000000ull);
        } else if (tails >> s & 1) {
          tc::mbar_wait(b_raw(s), (tail_use >> s & 1) ^ 1, nullptr, 1000000000ull);
        } else {
          tc::mbar_wait(b_full(s), (uses - 1) & 1, nullptr, 1000000000ull);
        }
      }
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------------------ UMMA issuers
      // The whole warp walks and waits, so that descriptors are warp-uniform values (they sit
      // in uniform registers); one elected lane issues.
      const int mt = warp - 1;
      const uint32_t id_qk = tc::idesc_bf16_f32(128, kCK, false, false);
      const uint32_t id_pv = tc::idesc_bf16_f32(128, D, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t s_t = tm + L::kColS + 2 * mt * kCK, o_t = tm + L::kColO + mt * D;
      const uint64_t q_desc = tc::sdesc_sw128(sb + L::kQ0 + mt * L::kQTile, 16, 1024);
      const uint64_t k_desc = tc::sdesc_sw128(sb + L::kRing, 16, 1024);
      const uint64_t v_desc = tc::sdesc_sw128(sb + L::kRing, kCK * 128, 1024);
      constexpr uint32_t kTileStep = L::kTile >> 4;          // descriptor steps (16 bytes)
      auto qk = [&](int s, int buf) {
        const uint64_t kd = k_desc + 2 * s * kTileStep;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t in = (ks & 3) * 2;
          tc::umma_ss(s_t + buf * kCK, q_desc + (ks >> 2) * (128 * 128 / 16) + in,
                      kd + (ks >> 2) * (kCK * 128 / 16) + in, id_qk, ks > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](int s, int buf, bool fresh) {
        const uint64_t vd = v_desc + (2 * s + 1) * kTileStep;
        const uint32_t pt = s_t + buf * kCK;
        tc::umma_ts(o_t, pt, vd, id_pv, fresh ? 0u : 1u);
#pragma unroll
        for (int ks = 1; ks < kCK / 16; ++ks)
          tc::umma_ts(o_t, pt + ks * 8, vd + ks * (16 * 128 / 16), id_pv, 1u);
      };
      auto wait = [&](uint32_t b, int phase) -> bool {
        return warp_wait(b, phase & 1, abort_flag, p.wait_ns);
      };
      int k_st = 0, k_use = 0, v_st = 0;   // stages of the tiles whose K, and V, come next
      auto next = [&](int& s) -> int { return ++s == NS ? (s = 0, 1) : 0; };
      int tiles = 0, units = 0;            // done by this M-tile
      bool ok = true;
      for (int i = 0; i < n && ok;) {
        const int m = __shfl_sync(0xffffffffu, min(cur.n_tiles - cur.tile, n - i), 0);
        const bool active = __shfl_sync(0xffffffffu, rows_of(cur), 0) > mt * 128;
        if (active) {
          if (!(ok = wait(b_q(mt), units))) break;
          for (int j = 0; j < min(m, 2); ++j) {
            if (!(ok = wait(b_full(k_st), k_use))) break;
            tc::tc_fence_after();
            const int buf = (tiles + j) & 1;
            if (tc::elect_one()) {
              qk(k_st, buf);
              tc::umma_commit(b_s(mt, buf));
            }
            __syncwarp();
            k_use += next(k_st);
          }
          if (!ok) break;
          for (int j = 0; j < m; ++j, ++tiles) {
            // tile j's V came with its K
            const int buf = tiles & 1;
            const bool more = j + 2 < m;
            if (!(ok = (!more || wait(b_full(k_st), k_use)) && wait(b_p(mt, buf), tiles >> 1))) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
              pv(v_st, buf, j == 0);
              tc::umma_commit(b_o(mt));
              tc::umma_commit(b_empty(v_st));
            }
            __syncwarp();
            if (more) {
              // S of tile j + 2 takes the place of P of tile j, and only products of one
              // accumulator and shape keep the order of their issue: wait for P V. (Without:
              // 2048 tokens over 32K bf16 1007 us instead of 1020, 128 rows 207 instead of 234
              // then; waiting for tile j + 2 here too, and not above: 1052.)
              if (!(ok = wait(b_o(mt), tiles))) break;
              tc::tc_fence_after();
              if (tc::elect_one()) {
                qk(k_st, buf);
                tc::umma_commit(b_s(mt, buf));
              }
              __syncwarp();
            }
            next(v_st);
            if (more) k_use += next(k_st);
          }
          if (!ok) break;
          ++units;
        } else {
          // no rows here: release the unit's stages in step
          for (int j = 0; j < m; ++j) {
            if (!(ok = wait(b_full(k_st), k_use))) break;
            if (tc::elect_one()) tc::mbar_arrive(b_empty(k_st));
            __syncwarp();
            next(v_st);
            k_use += next(k_st);
          }
          if (!ok) break;
        }
        i += m;
        if (i < n) cur.next_unit(deal);
      }
      if (!ok && lane == 0) raise();
      // every product issued retires before TMEM is released
      if (tc::elect_one()) tc::umma_commit(b_teardown);
      __syncwarp();
      tc::mbar_wait(b_teardown, 0, nullptr, 1000000000ull);
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------ value rows behind the end
      if constexpr (!k8) {
        uint32_t parity = 0;
        int done = 0;
        while (done < n) {
          const int m = min(cur.n_tiles - cur.tile, n - done);
          const int last = cur.tile + m - 1;
          const int64_t left = cur.q.len - (int64_t)last * kCK;
          if (left < kCK) {                  // only a unit's last tile can be cut
            const int st = (done + m - 1) % NS;
            if (!warp_wait(b_raw(st), parity >> st & 1, abort_flag, p.wait_ns)) {
              if (lane == 0) raise();
              break;
            }
            parity ^= 1u << st;
            const uint32_t v0 = sb + L::kRing + (2 * st + 1) * L::kTile;
            for (int i = (int)left * 8 + lane; i < kCK * 8; i += 32)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};"
                             :: "r"(v0 + h * (kCK * 128) + i * 16), "r"(0u) : "memory");
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(b_full(st));
          }
          done += m;
          if (done < n) cur.next_unit(deal);
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    if constexpr (k8) set_regs_up<152>();
    const int mt = (warp - 4) >> 2, q4 = warp & 3;
    const int flip = mt ? L::kFlip : 0;
    const int rl = 32 * q4 + lane;                   // TMEM lane, row of the Q tile
    const int r = mt * 128 + (rl ^ flip);            // row of the unit
    const uint32_t lane_t = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t o_t = lane_t + L::kColO + mt * D;
    const int gap = p.rows_per_box == 16 ? 64 : 0;   // behind each 16 rows' scales
    int tiles = 0, sc = 0;
    bool ok = true, first_unit = true;
    for (int done = 0; done < n && ok;) {
      const int m_tiles = min(cur.n_tiles - cur.tile, n - done);
      const int rows = rows_of(cur);
      const int seg0 = cur.tile;
      if (rows > mt * 128) {
        const int grow = cur.rg * kCG + r;
        const int tok = grow / deal.g, h = grow - tok * deal.g;
        const bool row_ok = r < rows;
        const bool warp_ok = mt * 128 + ((32 * q4) ^ flip) < rows;
        {
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (int64_t)(cur.q.q0 + tok) * p.q_tok + (int64_t)(cur.kvh * deal.g + h) * p.q_head);
          uint8_t* dst = smem + L::kQ0 + mt * L::kQTile + rl * 128;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint4 x = row_ok ? __ldg(src + ch) : make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(dst + (ch >> 3) * (128 * 128) + (((ch & 7) ^ (rl & 7)) << 4)) = x;
          }
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(b_q(mt));
        }
        // keys this row sees; rows that are not there see any
        const int vis = row_ok ? cur.q.len - cur.q.nq + tok + 1 : INT_MAX;
        float m_ref = -INFINITY;
        uint64_t l2[4];                                // partial sums, two each
#pragma unroll
        for (int u = 0; u < 4; ++u) l2[u] = f2(0.f, 0.f);
        for (int j = 0; j < m_tiles; ++j) {
          const int buf = tiles & 1;
          const uint32_t s_t = lane_t + L::kColS + (2 * mt + buf) * kCK;
          ok = warp_wait(b_s(mt, buf), (tiles >> 1) & 1, abort_flag, p.wait_ns);
          if (!ok) break;
          const int scj = (sc + j) % L::kScaleSlots;
          tc::tc_fence_after();
          if (warp_ok) {
            const int key0 = (seg0 + j) * kCK;
            uint32_t s[kCK];
#pragma unroll
            for (int c = 0; c < kCK / 32; ++c)
              tc::tmem_ld32(s_t + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
            // 8-bit pages: log2-domain scores against the reference so far, by the keys' scales
            // (times qk2 already)
            float ref = m_ref == -INFINITY ? 0.f : m_ref;
            if constexpr (k8) {
              const uint32_t ks = sb + L::kScale + scj * 2 * L::kScaleTile;
              const uint64_t nref = f2(-ref, -ref);
              float f[32];
              scales32(ks, 0, gap, f);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < kCK; c += 2) {
                if (c == 32) scales32(ks, 32, gap, f);
                float a, b;
                f2_get(f2_fma(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                              f2(f[c & 31], f[(c & 31) + 1]), nref), a, b);
                s[c] = __float_as_uint(a);
                s[c + 1] = __float_as_uint(b);
              }
            } else {
              tc::tmem_wait_ld();
            }
            const int hi = min(vis, cur.q.len) - key0;       // columns seen
            const bool cut = __any_sync(0xffffffffu, hi < kCK);
            if (cut) {
#pragma unroll
              for (int c = 0; c < kCK; ++c)
                if (c >= hi) s[c] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = __uint_as_float(s[u]);
#pragma unroll
            for (int c = 4; c < kCK; c += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mx[u] = max3(mx[u], __uint_as_float(s[c + u]),
                             c + 4 < kCK ? __uint_as_float(s[(c + 4 + u) & (kCK - 1)]) : mx[u]);
            float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
            top = k8 ? top + ref : top * p.qk2;
            // a NaN goes up too, and makes the reference, l and O NaN
            const bool up = !(top <= m_ref + kCRaise);
            if (__any_sync(0xffffffffu, up)) {
              // O may be touched once the P V of the tile before is done
              if (j > 0) {
                ok = warp_wait(b_o(mt), (tiles - 1) & 1, abort_flag, p.wait_ns);
                if (!ok) break;
                tc::tc_fence_after();
              }
              const float alpha = up ? ex2(m_ref - top) : 1.f;
              // inf - inf is NaN in a softmax.  A NaN stays: a masked tile behind it has a maximum
              // of -inf, and that as the reference would say that the row has seen nothing.
              if (up) m_ref = top == INFINITY || m_ref != m_ref ? NAN : top;
              if constexpr (k8) {                      // to the new reference
                const float by = ref - (m_ref == -INFINITY ? 0.f : m_ref);
#pragma unroll
                for (int c = 0; c < kCK; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) + by);
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) l2[u] = f2_mul(l2[u], f2(alpha, alpha));
              if (j > 0) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t o[16];
                  tc::tmem_ld16(o_t + 16 * c, o);
                  tc::tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                  tc::tmem_st16(o_t + 16 * c, o);
                }
              }
            }
            ref = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t nref = f2(-ref, -ref), q2 = f2(p.qk2, p.qk2);
            const uint32_t vs = sb + L::kScale + (scj * 2 + 1) * L::kScaleTile;
            // kCut: columns behind the row's last key (weight exactly 0, the scales there may be
            // anything); else kPoly of eight pairs go to the FMA pipe
            auto weights = [&](auto cut_tag) {
              constexpr bool kCut = decltype(cut_tag)::value;
              constexpr int kPw = L::kPw, kPoly = L::kPoly;
#pragma unroll
              for (int c = 0; c < kCK / kPw / 2; ++c) {
                uint32_t pw[kPw];
                [[maybe_unused]] float f[32];
                if constexpr (k8) scales32(vs, 32 * c, gap, f);
#pragma unroll
                for (int e = 0; e < kPw; e += 2) {
                  float a[4];
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const int k = 2 * (kPw * c + e + x);
                    uint64_t y = f2(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                    if constexpr (!k8) y = f2_fma(y, q2, nref);
                    if (!kCut && ((e + x) * kPoly) % 8 < kPoly) {
                      ex2_poly(y, a[2 * x], a[2 * x + 1]);
                    } else {
                      float u, v;
                      f2_get(y, u, v);
                      a[2 * x] = ex2(u);
                      a[2 * x + 1] = ex2(v);
                    }
                    l2[(e + x) & 3] = f2_add(l2[(e + x) & 3], f2(a[2 * x], a[2 * x + 1]));
                  }
                  if constexpr (k8) {
                    f2_get(f2_mul(f2(a[0], a[1]), f2(f[2 * e], f[2 * e + 1])), a[0], a[1]);
                    f2_get(f2_mul(f2(a[2], a[3]), f2(f[2 * e + 2], f[2 * e + 3])), a[2], a[3]);
                    if constexpr (kCut) {
                      const int k = 2 * (kPw * c + e);
#pragma unroll
                      for (int x = 0; x < 4; ++x)
                        if (k + x >= hi) a[x] = 0.f;
                    }
                  }
                  pw[e] = pack_bf16x2(a[0], a[1]);
                  pw[e + 1] = pack_bf16x2(a[2], a[3]);
                }
                st_cols(s_t + kPw * c, pw);
              }
            };
            if (cut) weights(std::true_type{});
            else weights(std::false_type{});
            tc::tmem_wait_st();
          }
          // A barrier's parity tells a phase from the one before it only: the wait for the unit's
          // last P V starts when all but that one are known to be done (from S just read: all
          // but the last two), and before this P lets it begin.
          if (j > 0 && j + 1 == m_tiles) {
            ok = warp_wait(b_o(mt), (tiles - 1) & 1, abort_flag, p.wait_ns);
            if (!ok) break;
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(b_p(mt, buf));
          ++tiles;
        }
        if (ok)
          ok = warp_wait(b_o(mt), (tiles - 1) & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        tc::tc_fence_after();
        if (warp_ok) {
          float la, lb;
          f2_get(f2_add(f2_add(l2[0], l2[1]), f2_add(l2[2], l2[3])), la, lb);
          // (all scores -inf: what ex2_poly makes of them does not count)
          const float l = m_ref == -INFINITY ? 0.f : la + lb;
          const bool whole = seg0 == 0 && seg0 + m_tiles == cur.n_tiles;
          const int64_t part = ((w * 2 + (first_unit ? 0 : 1)) * kCG + r);
          const int64_t o_row = (int64_t)(cur.q.q0 + tok) * p.Hq + cur.kvh * deal.g + h;
          const float f = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(o_t + 32 * c, o);
            tc::tmem_wait_ld();
            if (row_ok) {
              if (whole && !p.out_f32) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o_row * D + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t y[4];
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    y[x] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * x]) * f,
                                       __uint_as_float(o[8 * e + 2 * x + 1]) * f);
                  dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
                }
              } else {
                float4* dst = reinterpret_cast<float4*>((whole ? static_cast<float*>(p.out) + o_row * D
                                                               : p.ws_o + part * D) + 32 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  dst[e] = make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                       __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
              }
            }
          }
          if (row_ok) {
            if (!whole) {
              *reinterpret_cast<float2*>(p.ws_ml + part * 2) = make_float2(m_ref, l);
            } else if (p.lse) {
              p.lse[o_row] = l == 0.f ? -INFINITY : (m_ref + lg2(l)) * kLn2;
            }
          }
        }
        // the next unit's first P V overwrites O: these reads are done before its P is given
        tc::tc_fence_before();
      }
      first_unit = false;
      sc = (sc + m_tiles) % L::kScaleSlots;
      done += m_tiles;
      if (done < n) cur.next_unit(deal);
    }
    if (!ok && lane == 0) raise();
  } else {
    // ------------------------------------------------------------ codes to bf16
    if constexpr (k8) {
      // warps 12-15 the keys, 16-19 the values
      set_regs_down<56>();
      const int kv = (warp - 12) >> 2, tid = (threadIdx.x - 384) & 127;
      constexpr int kRowPieces = D / 16;           // 16-byte pieces of a row
      constexpr int kRowsPer = 128 / kRowPieces;   // rows that the 128 threads take at a time
      constexpr int kPer = kCK / kRowsPer;         // pieces of a thread
      const int row0 = tid / kRowPieces;
      // which 16 codes of the row lie there (the pool's boxes are swizzled)
      const int piece = (tid % kRowPieces) ^ (D == 128 ? row0 & 7 : (row0 >> 1) & 3);
      int st = 0, use = 0, rs = 0, r_use = 0, left_tiles = min(cur.n_tiles - cur.tile, n);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int live = (int)min((int64_t)kCK, (int64_t)cur.q.len - (int64_t)cur.tile * kCK);
        ok = warp_wait(b_raw(rs), r_use & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        // the keys' scales times qk2, for the softmax
        if (kv == 0 && tid < kCK)
          *reinterpret_cast<float*>(smem + L::kScale + 2 * (i % L::kScaleSlots) * L::kScaleTile + tid * 4 +
                                    (p.rows_per_box == 16 ? tid / 16 * 64 : 0)) *= p.qk2;
        uint4 x[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y)
          x[y] = *reinterpret_cast<const uint4*>(smem + L::kRawRing + (2 * rs + kv) * L::kRaw +
                                                 (y * 128 + tid) * 16);
        if (use > 0) {
          ok = warp_wait(b_empty(st), (use - 1) & 1, abort_flag, p.wait_ns);
          if (!ok) break;
        }
        uint8_t* at = smem + L::kRing + (2 * st + kv) * L::kTile;
        uint32_t most = 0;
        auto put = [&](int y, uint4 codes, auto nan_tag) {
          const int row = y * kRowsPer + row0;
          uint2 c0 = codes_to_bf16<PT>(codes.x, most), c1 = codes_to_bf16<PT>(codes.y, most);
          uint2 c2 = codes_to_bf16<PT>(codes.z, most), c3 = codes_to_bf16<PT>(codes.w, most);
          if constexpr (decltype(nan_tag)::value) {
            put_nan(c0);
            put_nan(c1);
            put_nan(c2);
            put_nan(c3);
          }
          if (kv == 1 && row >= live) c0 = c1 = c2 = c3 = make_uint2(0u, 0u);
          const uint4 a = make_uint4(c0.x, c0.y, c1.x, c1.y), b = make_uint4(c2.x, c2.y, c3.x, c3.y);
          // pieces 2 piece, 2 piece + 1 of the bf16 row; at D 128 the two halves' lanes write
          // them in opposite order, so that eight lanes cover all banks
          uint8_t* dst = at + (piece >> 2) * (kCK * 128) + row * 128;
          const int p0 = (2 * piece) & 7, flip = D == 128 ? piece >> 2 : 0;
          const uint4 fst = flip ? b : a, snd = flip ? a : b;
          *reinterpret_cast<uint4*>(dst + (((p0 + flip) ^ (row & 7)) << 4)) = fst;
          *reinterpret_cast<uint4*>(dst + (((p0 + 1 - flip) ^ (row & 7)) << 4)) = snd;
        };
#pragma unroll
        for (int y = 0; y < kPer; ++y) put(y, x[y], std::false_type{});
        // A NaN is put in behind the plain conversion.  Looking for it costs 32 rows over 32K 321 ->
        // 343 us, 33 rows 359 -> 363, a 2048-token chunk nothing (in the loop itself: 360, 378 and
        // 1371 -> 1438; from the codes, before the wait: 336, 364 and 1389).
        if (PT == VC_PAGE_E4M3 && ((most + 0x00100010u) & 0x08000800u)) {
#pragma unroll 1
          for (int y = 0; y < kPer; ++y)
            put(y, *reinterpret_cast<const uint4*>(smem + L::kRawRing + (2 * rs + kv) * L::kRaw +
                                                   (y * 128 + tid) * 16), std::true_type{});
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(b_full(st));
          tc::mbar_arrive(b_raw_empty(rs));
        }
        if (++st == NS) { st = 0; ++use; }
        if (++rs == NR) { rs = 0; ++r_use; }
        ++cur.tile;
        if (--left_tiles == 0 && i + 1 < n) {
          cur.next_unit(deal);
          left_tiles = min(cur.n_tiles, n - i - 1);
        }
      }
      if (!ok && lane == 0) raise();
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ------------------------------------------------------------------ host side
PartSet chunk_parts(int D, char* ws) {
  PartSet p;
  p.n = num_sms();
  p.rows = kCG;
  p.o = reinterpret_cast<float*>(ws);
  p.ml = p.o + (size_t)p.n * 2 * p.rows * D;
  p.cut = reinterpret_cast<Cut*>(p.ml + (size_t)p.n * 2 * p.rows * 2);
  return p;
}

size_t chunks_workspace_bytes(int D) {
  const PartSet p = chunk_parts(D, nullptr);
  return ((size_t)p.n * (2 * p.rows * (D + 2) * sizeof(float) + sizeof(Cut)) + 255) & ~(size_t)255;
}

vc_status read_chunks_error(int32_t* value, int clear) {
  VC_CUDA(cudaMemcpyFromSymbol(value, g_chunks_error, sizeof(int)));
  if (clear) {
    const int z = 0;
    VC_CUDA(cudaMemcpyToSymbol(g_chunks_error, &z, sizeof(int)));
  }
  return VC_OK;
}

template <int D, int PT>
static vc_status run_chunks(const AttnCall& a, const PartSet& parts, cudaStream_t stream) {
  using L = ChunkCfg<D, PT>;
  const vc_paged_cache* c = a.cache;
  const int rows = std::min(c->page, kCK);
  CUtensorMap mk, mv, mks, mvs;
  bool ok = make_pool_map(&mk, c, true, rows, L::k8) && make_pool_map(&mv, c, false, rows, L::k8);
  if (L::k8) {
    ok = ok && make_scale_map(&mks, c, true, rows) && make_scale_map(&mvs, c, false, rows);
  } else {
    mks = mk;
    mvs = mv;
  }
  if (!ok) return fail(VC_ERR_CUDA, "paged_attn: cuTensorMapEncodeTiled failed");
  Deal<kCG, kCK> deal;
  deal.s = seqs_of(a);
  deal.g = a.Hq / c->Hkv;
  deal.Hkv = c->Hkv;
  deal.rows_over = few_rows(c->type, c->D);
  deal.rows_upto = INT32_MAX;
  deal.n_workers = parts.n;
  deal.min_tiles = 1;
  ChunkParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_tok = a.q_tok;
  p.q_head = a.q_head;
  p.table = c->page_table;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.page = c->page;
  p.page_shift = __builtin_ctz((unsigned)c->page);
  p.rows_per_box = rows;
  p.Hq = a.Hq;
  p.qk2 = a.scale * kLog2e;
  p.out = a.out;
  p.lse = a.lse;
  p.out_f32 = a.flags & VC_OUT_F32 ? 1 : 0;
  p.ws_o = parts.o;
  p.ws_ml = parts.ml;
  p.cut = parts.cut;
  p.err_flag = c->err_flag;
  p.wait_ns = wait_limit_ns();
  VC_CUDA(grant_smem((const void*)paged_chunk_kernel<D, PT>, L::kAlloc));
  VC_CUDA(launch_pdl(paged_chunk_kernel<D, PT>, dim3(parts.n), dim3(L::kThreads), L::kAlloc,
                     stream, 1, mk, mv, mks, mvs, deal, p));
  return VC_OK;
}

vc_status launch_chunks(const AttnCall& a, const PartSet& parts, cudaStream_t stream) {
  const int D = a.cache->D;
  switch (a.cache->type) {
    case VC_PAGE_BF16:
      return D == 128 ? run_chunks<128, VC_PAGE_BF16>(a, parts, stream) : run_chunks<64, VC_PAGE_BF16>(a, parts, stream);
    case VC_PAGE_E4M3:
      return D == 128 ? run_chunks<128, VC_PAGE_E4M3>(a, parts, stream) : run_chunks<64, VC_PAGE_E4M3>(a, parts, stream);
    default:
      return D == 128 ? run_chunks<128, VC_PAGE_INT8>(a, parts, stream) : run_chunks<64, VC_PAGE_INT8>(a, parts, stream);
  }
}

}  // namespace paged
}  // namespace vc
