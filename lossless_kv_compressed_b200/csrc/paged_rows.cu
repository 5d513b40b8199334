// Paged attention of few rows (few_rows): every group of up to 16 query rows (new token, head of
// the GQA group) of a (sequence, kv head) against the sequence's pages, on mma.sync.
//
// Mathematics.  For each row the keys come tile by tile; with the running reference m of
// the log2-domain scores x_t = (q . k_t) scale log2(e), l = sum 2^(x_t - m) and
// O = sum 2^(x_t - m) v_t; m is raised (and l, O rescaled) only when a tile's maximum
// exceeds it by more than 2^8, so weights stay below 2^8 and no rescaling runs in most
// tiles.  o = O / l, lse = (m + log2 l) ln 2.
//
// 8-bit rows are not turned into real values: the codes are exact in fp16, so q (as fp16
// scaled by a power of two per row) times the codes is exact up to fp32 accumulation, and
// the key's scale multiplies the score.  A value's scale joins its weight:
// w_t = 2^(x_t + log2 vs_t - m) enters the product in fp16 with m the running reference of
// x_t + log2 vs_t, while l sums 2^(x_t - m).  fp16 weights are off by 2^-12 at most and
// 2^-25 in absolute terms, against a largest weight of 2^-8 .. 2^8.
// bf16 rows take bf16 weights; blocks of at most 8 rows put each weight's bf16 remainder
// into the idle rows 8-15 of the same products, so the weights carry 16 bits at no cost.
//
// Bound: bf16 HBM (each K/V byte is used for at most 16 rows); 8-bit the chain of a warp's tile,
// codes to fp16, products, exponentials (1.9 of 4 instructions a cycle from eight warps an SM, 64%
// of DRAM; with 4 live rows of 16, three quarters of the products are for nobody).  Every warp is a worker of its
// own: an equal share of the line of key tiles (see Deal), a private ring of 8 KB stages
// (K and V of one tile) filled by TMA from the pages, one lane per box, and no barrier
// with other warps.  Eight warps with three stages keep 192 KB in flight per SM.
// Measured (32 heads over 8, D 128, a call in a loop): 8 sequences of 4 tokens over 32K in bf16
// 184 us = 5.8 TB/s, e4m3 122 us = 4.5 TB/s; a token each of 64 sequences over 16K in e4m3
// 409 us = 5.4 TB/s; one token over 1009 keys 10.6 us of the GPU (deal, one tile, merge).  Tiles
// prefetched into L2 three ahead: 196 us, e4m3 64 x 16K of 32 heads 410 -> 466.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>

#include "paged.cuh"
#include "paged_internal.h"
#include "paged_io.cuh"
#include "tc05.cuh"
#include "vc_internal.h"

namespace vc {
namespace paged {

constexpr int kRowGroup = 16;        // rows of a unit
constexpr int kRowWarps = 8;
constexpr int kRowStages = 3;
constexpr float kRaise = 8.f;        // a maximum this far above the reference raises it

template <int D, int PT>
struct RowCfg {
  static constexpr int kEs = PT == VC_PAGE_BF16 ? 2 : 1;
  static constexpr int kRowBytes = D * kEs;
  static constexpr int kTileBytes = 4096;                       // K (or V) of one tile
  static constexpr int kKT = kTileBytes / kRowBytes;            // keys of a tile: 16, 32, 64
  static constexpr int kW = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in smem
  static constexpr int kScaleBytes = PT == VC_PAGE_BF16 ? 0 : kKT / 16 * 128;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kRing = kRowWarps * kRowStages;
  static constexpr int kScale0 = kRing * kStage;
  static constexpr int kBar0 = kScale0 + kRing * 2 * kScaleBytes;
  static constexpr int kAlloc = kBar0 + kRing * 8 + 1024;
};

struct RowParams {
  const __nv_bfloat16* q;
  int64_t q_tok, q_head;
  const int32_t* table;
  int32_t max_pages, n_pages, page, page_shift, rows_per_box;
  int32_t Hq;
  float qk2;                    // scale * log2(e)
  void* out;
  float* lse;
  int32_t out_f32;
  float* ws_o;                  // [workers, 2, 16, D]
  float* ws_ml;                 // [workers, 2, 16, 2]
  Cut* cut;                     // [workers]
  int32_t* err_flag;
  uint64_t wait_ns;
};

__device__ int g_rows_error;    // bit 1: a bounded wait expired

// Two e4m3 codes (low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(x));
  return r;
}
// Two int8 codes with the sign bit flipped (bytes u = code + 128 under 0x64: fp16 1024 + u)
// as fp16: 1024 + u - 1152, exactly.
__device__ __forceinline__ uint32_t biased_f16x2(uint32_t x) {
  const uint32_t c = 0x64806480u;
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(c));
  return r;
}
// Four codes of a word as two fp16 pairs (bytes 0,1 and 2,3).
template <int PT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (PT == VC_PAGE_E4M3) {
    lo = e4m3x2_f16x2(w);
    hi = e4m3x2_f16x2(w >> 16);
  } else {
    w ^= 0x80808080u;
    lo = biased_f16x2(__byte_perm(w, 0x64646464u, 0x4140));
    hi = biased_f16x2(__byte_perm(w, 0x64646464u, 0x4342));
  }
}

template <int D, int PT>
__global__ void __launch_bounds__(kRowWarps * 32, 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmKS,
                      const __grid_constant__ CUtensorMap tmVS,
                      const Deal<kRowGroup, RowCfg<D, PT>::kKT> deal, const RowParams p) {
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
  using C = RowCfg<D, PT>;
  constexpr int KT = C::kKT, NT = KT / 8, KS = D / 16, NO = D / 8;
  constexpr bool k8 = PT != VC_PAGE_BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rl = lane >> 2, c = lane & 3;        // fragment row, column pair

  typename Deal<kRowGroup, KT>::Lane l0;
  const int64_t total = deal.total(lane, l0);
  const Shares sh(total, deal.workers(total));
  const int64_t w = (int64_t)warp * gridDim.x + blockIdx.x;   // neighbours on other SMs
  const int64_t t0 = w < sh.W ? sh.first(w) : total;
  const int n = w < sh.W ? (int)(sh.first(w + 1) - t0) : 0;
  Cursor<kRowGroup, KT> cur;
  if (n > 0) cur.seek(deal, l0, t0, lane);
  note_cut(p.cut + w, deal, sh, cur, t0, n, lane);
  if (n == 0) return;

  const int ring0 = warp * kRowStages;
  auto bar = [&](int st) -> uint32_t { return sb + C::kBar0 + (ring0 + st) * 8; };
  auto k_at = [&](int st) -> uint32_t { return sb + (ring0 + st) * C::kStage; };
  auto v_at = [&](int st) -> uint32_t { return k_at(st) + C::kTileBytes; };
  auto scale_off = [&](int st) -> int { return C::kScale0 + (ring0 + st) * 2 * C::kScaleBytes; };
  if (lane == 0) {
    for (int st = 0; st < kRowStages; ++st) tc::mbar_init(bar(st), 1);
    tc::fence_barrier_init();
    tc::fence_proxy_async();
  }
  __syncwarp();

  // ------------------------------------------------------------ page loads
  // Lane j holds the page of box chunk * 32 + j of the sequence the loads are at (the
  // next 32 in ahead); a box is rows_per_box rows of one page.
  Cursor<kRowGroup, KT> pc = cur;
  const int nb = KT / p.rows_per_box;            // boxes of a tile
  const bool half_line = p.rows_per_box == 16;   // scales of a box fill half of their 128 bytes
  int chunk = -1, ids = 0, ahead = 0;
  auto load_ids = [&](int ch) -> int {
    const int64_t pos = ((int64_t)ch * 32 + lane) * p.rows_per_box;
    int id = p.n_pages;                          // out of range: TMA fills zeros
    if (pos < pc.q.len) {
      id = __ldg(p.table + (int64_t)pc.b * p.max_pages + (pos >> p.page_shift));
      if ((unsigned)id >= (unsigned)p.n_pages) {
        id = p.n_pages;
        if (p.err_flag) atomicOr(p.err_flag, VC_PAGED_BAD_PAGE);
      }
    }
    return id;
  };
  int produced = 0;
  auto produce = [&]() {
    const int st = produced % kRowStages;
    const int box = pc.tile * nb;
    if ((box >> 5) != chunk) {
      ids = (chunk >= 0 && (box >> 5) == chunk + 1) ? ahead : load_ids(box >> 5);
      chunk = box >> 5;
      ahead = load_ids(chunk + 1);
    }
    const int id = __shfl_sync(0xffffffffu, ids, (box + lane) & 31);
    if (lane == 0) tc::mbar_expect_tx(bar(st), C::kStage + (k8 ? 2 * KT * 4 : 0));
    __syncwarp();
    if (lane < nb) {
      const int y = (int)((int64_t)(box + lane) * p.rows_per_box & (p.page - 1));
      const uint32_t off = lane * p.rows_per_box * C::kW;
      tma_load_5d(k_at(st) + off, &tmK, bar(st), 0, y, 0, pc.kvh, id);
      tma_load_5d(v_at(st) + off, &tmV, bar(st), 0, y, 0, pc.kvh, id);
      if constexpr (k8) {
        const uint32_t s0 = sb + scale_off(st) + lane * max(p.rows_per_box * 4, 128);
        tc::tma_load_3d(s0, &tmKS, bar(st), y, pc.kvh, id);
        tc::tma_load_3d(s0 + C::kScaleBytes, &tmVS, bar(st), y, pc.kvh, id);
      }
    }
    ++produced;
    if (++pc.tile == pc.n_tiles && produced < n) {
      const int b = pc.b;
      pc.next_unit(deal);
      if (pc.b != b) chunk = -1;
    }
  };
  for (int i = 0; i < min(n, kRowStages); ++i) produce();

  // ------------------------------------------------------------ per unit
  uint32_t qf[KS][4];
  float qs[2];                                   // scale of the scores of rows rl, rl + 8
  float acc[NO][4], m[2], l[2];
  int vis[2], vis0, R, seg0;
  bool pairs;                                    // rows 8-15 carry the weights' remainders
  bool first_unit = true;
  auto begin_unit = [&]() {
    const int g = deal.g;
    const int row0 = cur.rg * kRowGroup;
    R = (int)min((int64_t)kRowGroup, (int64_t)cur.q.nq * g - row0);
    pairs = !k8 && R <= 8;
    seg0 = cur.tile;
    vis0 = cur.q.len - cur.q.nq + row0 / g + 1;
    const __nv_bfloat16* src[2];
    bool ok[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = rl + (u && !pairs ? 8 : 0);
      ok[u] = r < R;
      const int i = (row0 + r) / g, h = (row0 + r) - i * g;
      src[u] = p.q + (int64_t)(cur.q.q0 + i) * p.q_tok + (int64_t)(cur.kvh * g + h) * p.q_head;
      vis[u] = ok[u] ? cur.q.len - cur.q.nq + i + 1 : INT_MAX;   // rows that are not there: any
      m[u] = -INFINITY;
      l[u] = 0.f;
    }
    if constexpr (!k8) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int u = x & 1, d = ks * 16 + 2 * c + (x >> 1) * 8;
          qf[ks][x] = ok[u] ? __ldg(reinterpret_cast<const uint32_t*>(src[u] + d)) : 0u;
        }
      }
      qs[0] = qs[1] = p.qk2;
    } else {
      // q as fp16: each row times the power of two that brings its largest value to
      // [2^13, 2^14), so that the products with the codes are exact
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint2 raw[KS];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d = (ks >> 2) * 64 + 16 * c + 4 * (ks & 3);
          raw[ks] = ok[u] ? __ldg(reinterpret_cast<const uint2*>(src[u] + d)) : make_uint2(0u, 0u);
          top = fmaxf(fmaxf(fmaxf(fabsf(bf16_lo(raw[ks].x)), fabsf(bf16_hi(raw[ks].x))),
                            fmaxf(fabsf(bf16_lo(raw[ks].y)), fabsf(bf16_hi(raw[ks].y)))), top);
        }
        top = warp_max_xor(top, 2);
        const int e = top > 0.f ? max(-100, (int)((__float_as_uint(top) >> 23) & 255) - 127) : 0;
        const float f = __uint_as_float((uint32_t)(127 + 13 - min(e, 126)) << 23);
        qs[u] = p.qk2 * __uint_as_float((uint32_t)(127 - 13 + min(e, 126)) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][u] = pack_f16x2(bf16_lo(raw[ks].x) * f, bf16_hi(raw[ks].x) * f);
          qf[ks][2 + u] = pack_f16x2(bf16_lo(raw[ks].y) * f, bf16_hi(raw[ks].y) * f);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NO; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[t][x] = 0.f;
  };

  // 8-bit rows of 128 bytes: within 8 keys (or 16-byte pieces of a row) number i sits at
  // (i >> 1) | (i & 1) << 2, which spreads a quarter-warp's 16-byte reads over all banks.
  auto spread = [](int i) -> int { return D == 128 ? (i >> 1) | ((i & 1) << 2) : i; };
  // key (within the tile) of a thread's score column e (0, 1) in the 8 keys of group j
  auto key_of = [&](int j, int e) -> int {
    return k8 && D == 128 ? 8 * j + c + 4 * e : 8 * j + 2 * c + e;
  };

  auto store_unit = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    }
    const bool whole = seg0 == 0 && cur.tile == cur.n_tiles;
    const int64_t part = (w * 2 + (first_unit ? 0 : 1)) * kRowGroup;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = rl + 8 * u;
      if ((u == 1 && pairs) || r >= R) continue;
      const int row = cur.rg * kRowGroup + r;
      const int i = row / deal.g, h = row - i * deal.g;
      const int64_t o = (int64_t)(cur.q.q0 + i) * p.Hq + cur.kvh * deal.g + h;
      const float f = !whole ? 1.f : l[u] == 0.f ? 0.f : 1.f / l[u];
      void* dst = whole ? p.out : p.ws_o;
      const int f32 = whole ? p.out_f32 : 1;
      const int64_t at = (whole ? o : part + r) * D;
      if constexpr (!k8) {
#pragma unroll
        for (int t = 0; t < NO; ++t) {
          float a = acc[t][2 * u], b = acc[t][2 * u + 1];
          if (u == 0 && pairs) {
            a += acc[t][2];
            b += acc[t][3];
          }
          st_pair(dst, f32, at + 8 * t + 2 * c, a * f, b * f);
        }
      } else {
        // column n of product t is dim spread(n) * 16 + t (D 128) or 8 n + t (D 64)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t d0 = at + (D == 128 ? 16 * spread(2 * c + e) : 8 * (2 * c + e));
#pragma unroll
          for (int t = 0; t < NO; t += 2)
            st_pair(dst, f32, d0 + t, acc[t][2 * u + e] * f, acc[t + 1][2 * u + e] * f);
        }
      }
      if (c == 0) {
        if (!whole) {
          *reinterpret_cast<float2*>(p.ws_ml + (part + r) * 2) = make_float2(m[u], l[u]);
        } else if (p.lse) {
          p.lse[o] = l[u] == 0.f ? -INFINITY : (m[u] + lg2(l[u])) * kLn2;
        }
      }
    }
    first_unit = false;
  };

  begin_unit();
  bool ok = true;
  int it = 0;
  for (; it < n; ++it) {
    const int st = it % kRowStages;
    ok = warp_wait(bar(st), (it / kRowStages) & 1, nullptr, p.wait_ns);
    if (!ok) break;
    const int key0 = cur.tile * KT;
    const int left = cur.q.len - key0;           // live keys of this tile (at least one)
    if (left < KT) {
      // slots past the sequence's end may hold anything: their values must not meet the
      // zero weights
      for (int i = left * C::kRowBytes / 16 + lane; i < C::kTileBytes / 16; i += 32) {
        // 16-byte piece i of the tile counted by rows, in its half of the dims
        const int row = i / (C::kRowBytes / 16), ch = i % (C::kRowBytes / 16);
        const int half = ch * 16 / C::kW;
        const int sw = C::kW == 128 ? (ch & 7) ^ (row & 7) : ch ^ ((row >> 1) & 3);
        const uint32_t a = v_at(st) + half * KT * C::kW + row * C::kW + sw * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" :: "r"(a), "r"(0u) : "memory");
      }
      tc::fence_proxy_async();                   // before a later load overwrites them
      __syncwarp();
    }

    // ---- scores
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[j][x] = 0.f;
    if constexpr (!k8) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int ch = (ks & 3) * 2 + ((lane >> 3) & 1);
#pragma unroll
        for (int j2 = 0; j2 < NT / 2; ++j2) {
          const int key = j2 * 16 + (lane >> 4) * 8 + (lane & 7);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(k_at(st) + (ks >> 2) * KT * 128 + key * 128 + ((ch ^ (key & 7)) << 4), b0, b1,
                  b2, b3);
          mma_bf16(s[2 * j2], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
          mma_bf16(s[2 * j2 + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2, b3);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int key = 8 * j + spread(rl);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const int ch = 4 * h + c;
          const int sw = D == 128 ? ch ^ (key & 7) : ch ^ ((key >> 1) & 3);
          uint4 x;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(k_at(st) + key * C::kW + sw * 16) : "memory");
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            codes_f16<PT>(xs[i], b0, b1);
            const int ks = 4 * h + i;
            mma_f16(s[j], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
          }
        }
      }
    }

    // ---- log2-domain scores, running reference, weights
    float lv[NT][2];                             // log2 of the value scales
    float mx[2] = {-INFINITY, -INFINITY};
    const bool whole_seen = key0 + KT <= vis0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key_of(j, e);
        float f0 = qs[0], f1 = qs[1];
        if constexpr (k8) {
          const int at = scale_off(st) + 4 * (half_line ? (key >> 4) * 32 + (key & 15) : key);
          const float ksc = *reinterpret_cast<const float*>(smem + at);
          const float vsc = *reinterpret_cast<const float*>(smem + at + C::kScaleBytes);
          f0 *= ksc;
          f1 *= ksc;
          lv[j][e] = fmaxf(lg2(vsc), -90.f);
        } else {
          lv[j][e] = 0.f;
        }
        s[j][e] *= f0;
        s[j][2 + e] *= f1;
        if (!whole_seen) {
          if (key0 + key >= vis[0] || key >= left) s[j][e] = -INFINITY;
          if (key0 + key >= vis[1] || key >= left) s[j][2 + e] = -INFINITY;
          if (k8 && key >= left) lv[j][e] = 0.f;
        }
        mx[0] = fmaxf(mx[0], s[j][e] + lv[j][e]);
        mx[1] = fmaxf(mx[1], s[j][2 + e] + lv[j][e]);
      }
    }
    float ref[2], alpha[2];
    bool raise = false;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = warp_max_xor(mx[u], 2);
      alpha[u] = 1.f;
      if (mx[u] > m[u] + kRaise) {
        alpha[u] = ex2(m[u] - mx[u]);            // 0 at the first keys
        m[u] = mx[u];
        raise = true;
      }
      ref[u] = m[u] == -INFINITY ? 0.f : m[u];
    }
    if (__any_sync(0xffffffffu, raise)) {
      l[0] *= alpha[0];
      l[1] *= alpha[1];
#pragma unroll
      for (int t = 0; t < NO; ++t) {
        acc[t][0] *= alpha[0];
        acc[t][1] *= alpha[0];
        acc[t][2] *= alpha[1];
        acc[t][3] *= alpha[1];
      }
    }
    uint32_t wf[NT][2];                          // weights of rows rl, rl + 8, two keys each
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = ex2(s[j][i] - ref[i >> 1]);
        l[i >> 1] += x[i];
        if constexpr (k8) x[i] = ex2(s[j][i] + lv[j][i & 1] - ref[i >> 1]);
      }
      if constexpr (k8) {
        wf[j][0] = pack_f16x2(x[0], x[1]);
        wf[j][1] = pack_f16x2(x[2], x[3]);
      } else {
        wf[j][0] = pack_bf16x2(x[0], x[1]);
        if (pairs) {
          x[2] -= bf16_lo(wf[j][0]);
          x[3] -= bf16_hi(wf[j][0]);
        }
        wf[j][1] = pack_bf16x2(x[2], x[3]);
      }
    }

    // ---- O += w V
#pragma unroll
    for (int j2 = 0; j2 < NT / 2; ++j2) {
      const uint32_t a0 = wf[2 * j2][0], a1 = wf[2 * j2][1], a2 = wf[2 * j2 + 1][0],
                     a3 = wf[2 * j2 + 1][1];
      if constexpr (!k8) {
#pragma unroll
        for (int t2 = 0; t2 < NO / 2; ++t2) {
          const int key = j2 * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
          const int d = t2 * 16 + (lane >> 4) * 8;
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(v_at(st) + (d >> 6) * KT * 128 + key * 128 +
                        ((((d & 63) >> 3) ^ (key & 7)) << 4),
                    b0, b1, b2, b3);
          mma_bf16(acc[2 * t2], a0, a1, a2, a3, b0, b1);
          mma_bf16(acc[2 * t2 + 1], a0, a1, a2, a3, b2, b3);
        }
      } else {
        // a thread's four keys of the product (columns 2c, 2c+1, 2c+8, 2c+9), its piece of
        // D / 8 dims of each
        constexpr int NW = D / 32;               // words of the piece
        uint32_t x[4][NW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key_of(2 * j2 + (i >> 1), i & 1);
          if constexpr (D == 128) {
            const uint32_t a = v_at(st) + key * 128 + ((spread(rl) ^ (key & 7)) << 4);
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                         : "r"(a) : "memory");
          } else {
            const uint32_t a = v_at(st) + key * 64 + (((rl >> 1) ^ ((key >> 1) & 3)) << 4) +
                               (rl & 1) * 8;
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                         : "=r"(x[i][0]), "=r"(x[i][1]) : "r"(a) : "memory");
          }
        }
#pragma unroll
        for (int wd = 0; wd < NW; ++wd) {
          uint32_t f[2][4];                      // [keys 0,1 | keys 2,3][dim of the word]
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            codes_f16<PT>(__byte_perm(x[2 * y][wd], x[2 * y + 1][wd], 0x5140), f[y][0], f[y][1]);
            codes_f16<PT>(__byte_perm(x[2 * y][wd], x[2 * y + 1][wd], 0x7362), f[y][2], f[y][3]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f16(acc[4 * wd + i], a0, a1, a2, a3, f[0][i], f[1][i]);
        }
      }
    }

    __syncwarp();                                // every lane has read the stage
    if (produced < n) produce();
    ++cur.tile;
    if (cur.tile == cur.n_tiles || it + 1 == n) {
      store_unit();
      if (it + 1 < n) {
        cur.next_unit(deal);
        begin_unit();
      }
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(&g_rows_error, 2);
    // copies in flight land before the block's shared memory is given back
    for (; it < produced; ++it)
      tc::mbar_wait(bar(it % kRowStages), (it / kRowStages) & 1, nullptr, 1000000000ull);
  }
}

// ------------------------------------------------------------------ host side
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess || q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

bool make_pool_map(CUtensorMap* m, const vc_paged_cache* c, bool key, int rows, bool whole_rows) {
  auto fn = encoder();
  if (!fn) return false;
  const bool b16 = c->type == VC_PAGE_BF16;
  const int es = b16 ? 2 : 1;
  const int width = b16 ? 64 : c->D;                 // elements of the innermost box
  const cuuint64_t row = (cuuint64_t)(key ? c->k_row_stride : c->v_row_stride) * es;
  const cuuint64_t head = (cuuint64_t)(key ? c->k_head_stride : c->v_head_stride) * es;
  const cuuint64_t pg = (cuuint64_t)(key ? c->k_page_stride : c->v_page_stride) * es;
  cuuint64_t dims[5] = {(cuuint64_t)width, (cuuint64_t)c->page, (cuuint64_t)(c->D / width),
                        (cuuint64_t)c->Hkv, (cuuint64_t)c->n_pages};
  // strides of one-entry dimensions are never used: any valid number will do
  cuuint64_t strides[4] = {row, 128, c->Hkv > 1 ? head : 128, c->n_pages > 1 ? pg : 128};
  cuuint32_t box[5] = {(cuuint32_t)width, (cuuint32_t)rows,
                       whole_rows ? (cuuint32_t)(c->D / width) : 1u, 1, 1};
  cuuint32_t es1[5] = {1, 1, 1, 1, 1};
  return fn(m, b16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 5,
            key ? c->k : c->v, dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE,
            width * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_scale_map(CUtensorMap* m, const vc_paged_cache* c, bool key, int rows) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)c->page, (cuuint64_t)c->Hkv, (cuuint64_t)c->n_pages};
  cuuint64_t strides[2] = {(cuuint64_t)c->page * 4, (cuuint64_t)c->page * c->Hkv * 4};
  cuuint32_t box[3] = {(cuuint32_t)rows, 1, 1};
  cuuint32_t es1[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, key ? c->k_scale : c->v_scale, dims, strides,
            box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

vc_status read_rows_error(int32_t* value, int clear) {
  VC_CUDA(cudaMemcpyFromSymbol(value, g_rows_error, sizeof(int)));
  if (clear) {
    const int z = 0;
    VC_CUDA(cudaMemcpyToSymbol(g_rows_error, &z, sizeof(int)));
  }
  return VC_OK;
}

PartSet rows_parts(int D, char* ws) {
  PartSet p;
  p.n = num_sms() * kRowWarps;
  p.rows = kRowGroup;
  p.o = reinterpret_cast<float*>(ws);
  p.ml = p.o + (size_t)p.n * 2 * p.rows * D;
  p.cut = reinterpret_cast<Cut*>(p.ml + (size_t)p.n * 2 * p.rows * 2);
  return p;
}

size_t rows_workspace_bytes(int D) {
  const PartSet p = rows_parts(D, nullptr);
  return ((size_t)p.n * (2 * p.rows * (D + 2) * sizeof(float) + sizeof(Cut)) + 255) & ~(size_t)255;
}

template <int D, int PT>
static vc_status run_rows(const AttnCall& a, const PartSet& parts, cudaStream_t stream) {
  using C = RowCfg<D, PT>;
  const vc_paged_cache* c = a.cache;
  const int rows = std::min(c->page, (int32_t)C::kKT);
  CUtensorMap mk, mv, mks, mvs;
  bool ok = make_pool_map(&mk, c, true, rows, true) && make_pool_map(&mv, c, false, rows, true);
  if (PT != VC_PAGE_BF16) {
    ok = ok && make_scale_map(&mks, c, true, rows) && make_scale_map(&mvs, c, false, rows);
  } else {
    mks = mk;
    mvs = mv;
  }
  if (!ok) return fail(VC_ERR_CUDA, "paged_attn: cuTensorMapEncodeTiled failed");
  Deal<kRowGroup, C::kKT> deal;
  deal.s = seqs_of(a);
  deal.g = a.Hq / c->Hkv;
  deal.Hkv = c->Hkv;
  deal.rows_over = 0;
  deal.rows_upto = few_rows(c->type, c->D);
  deal.n_workers = parts.n;
  deal.min_tiles = 2;       // one tile each: 11.7 us for one token over 1009 keys against 10.6; four: 11.8
  RowParams p;
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
  VC_CUDA(grant_smem((const void*)paged_rows_kernel<D, PT>, C::kAlloc));
  VC_CUDA(launch_pdl(paged_rows_kernel<D, PT>, dim3(num_sms()), dim3(kRowWarps * 32), C::kAlloc,
                     stream, 1, mk, mv, mks, mvs, deal, p));
  return VC_OK;
}

vc_status launch_rows(const AttnCall& a, const PartSet& parts, cudaStream_t stream) {
  const int D = a.cache->D;
  switch (a.cache->type) {
    case VC_PAGE_BF16:
      return D == 128 ? run_rows<128, VC_PAGE_BF16>(a, parts, stream)
                      : run_rows<64, VC_PAGE_BF16>(a, parts, stream);
    case VC_PAGE_E4M3:
      return D == 128 ? run_rows<128, VC_PAGE_E4M3>(a, parts, stream)
                      : run_rows<64, VC_PAGE_E4M3>(a, parts, stream);
    default:
      return D == 128 ? run_rows<128, VC_PAGE_INT8>(a, parts, stream)
                      : run_rows<64, VC_PAGE_INT8>(a, parts, stream);
  }
}

}  // namespace paged
}  // namespace vc
