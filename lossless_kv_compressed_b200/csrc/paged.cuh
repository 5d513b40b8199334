// Device helpers of the paged cache: lengths of a sequence, page lookup, and the deal of
// attention work to workers from the lengths on the device.
#pragma once

#include <stdint.h>

#include "vc_common.cuh"

namespace vc {
namespace paged {

// A call's sequences: new rows by cu_q (or uni rows each) and cached tokens by kv_len.
struct Seqs {
  const int32_t* cu_q;      // [B + 1] or NULL
  const int32_t* kv_len;    // [B]
  int32_t B, N, uni;
  int32_t cap;              // max_pages * page
};

struct SeqLen {
  int q0, nq, len;          // first new row, new rows, cached tokens (all clamped)
};

__host__ __device__ __forceinline__ SeqLen seq_len(const Seqs& s, int b) {
  SeqLen r;
  if (s.cu_q) {
    r.q0 = min(max(s.cu_q[b], 0), s.N);
    r.nq = min(max(s.cu_q[b + 1], r.q0), s.N) - r.q0;
  } else {
    r.q0 = b * s.uni;
    r.nq = s.uni;
  }
  r.len = min(max(s.kv_len[b], 0), s.cap);
  return r;
}

// Whether sequence b's lengths are what the interface asks for.
__device__ __forceinline__ bool lengths_ok(const Seqs& s, int b) {
  bool ok = s.kv_len[b] >= 0 && s.kv_len[b] <= s.cap;
  if (s.cu_q) ok = ok && s.cu_q[b] >= 0 && s.cu_q[b] <= s.cu_q[b + 1] && s.cu_q[b + 1] <= s.N;
  return ok;
}

// a / b for a >= 0, b > 0 (the short division where it serves).
__host__ __device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// S(n, m, a, b) = sum_{i < n} floor((a i + b) / m) for n, a, b >= 0, m > 0.  Whole multiples of m
// in a and b give closed sums.  What is left, a, b < m, counts the lattice points (i, j) with
// 1 <= j <= (a i + b) / m under a line that rises to h = floor((a (n - 1) + b) / m).  Counted by
// rows instead, row j has n - ceil((j m - b) / a) of them, so that
//   S(n, m, a, b) = n h - sum_{j = 1..h} ceil((j m - b) / a) = n h - S(h, a, m, m - b + a - 1),
// where (a, m) goes the way of Euclid's algorithm: a logarithmic number of steps.
__host__ __device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  bool minus = false;
  while (n > 0) {
    const int64_t qa = div64(a, m), qb = div64(b, m);
    a -= qa * m;
    b -= qb * m;
    const int64_t h = div64(a * (n - 1) + b, m);
    const int64_t part = n * (n - 1) / 2 * qa + n * (qb + h);
    sum += minus ? -part : part;
    minus = !minus;
    b = m - b + a - 1;
    n = h;
    const int64_t step = a;
    a = m;
    m = step;
  }
  return sum;
}

// Equal shares of a line of `total` pieces for W workers, W <= total: worker w has
// [first(w), first(w + 1)); owner(t) is the worker of piece t.
struct Shares {
  int64_t total, size, more;     // the first `more` workers get size + 1, the others size
  int64_t W;
  __host__ __device__ __forceinline__ Shares(int64_t t, int64_t workers)
      : total(t), size(div64(t, workers)), more(0), W(workers) {
    more = total - size * W;
  }
  __host__ __device__ __forceinline__ int64_t first(int64_t w) const {
    return w * size + (w < more ? w : more);
  }
  __host__ __device__ __forceinline__ int64_t owner(int64_t t) const {
    const int64_t big = more * (size + 1);
    return t < big ? div64(t, size + 1) : more + div64(t - big, size);
  }
};

// The deal of attention work.  The rows (token, head of the group) of a (sequence, kv
// head) form groups of RG; a group is a unit, its work the key tiles of KT keys up to
// the last key that its last row sees.  All units' tiles, in the order sequence, kv head,
// group, tile, form one line [0, total) that the workers cut into equal parts; a unit cut by
// a border is merged afterwards.  The numbers follow from cu_q and kv_len alone and are
// computed by every warp for itself: lanes sum 32 sequences at a time, a sequence's groups
// in closed form.  Only sequences whose row count lies in (rows_over, rows_upto] count.
template <int RG, int KT>
struct Deal {
  Seqs s;
  int32_t g, Hkv;
  int32_t rows_over, rows_upto;
  int32_t n_workers;        // workers launched
  int32_t min_tiles;        // tiles a worker gets at least (fewer workers then take part)

  __host__ __device__ __forceinline__ bool mine(const SeqLen& q) const {
    const int64_t r = (int64_t)q.nq * g;
    return r > rows_over && r <= rows_upto;
  }
  __host__ __device__ __forceinline__ int groups(const SeqLen& q) const {
    return (int)(((int64_t)q.nq * g + RG - 1) / RG);
  }
  // keys that the last row of group rg sees
  __host__ __device__ __forceinline__ int visible(const SeqLen& q, int rg) const {
    const int64_t last = min((int64_t)q.nq * g, (int64_t)RG * (rg + 1)) - 1;
    return max(0, q.len - q.nq + (int)(last / g) + 1);
  }
  __host__ __device__ __forceinline__ int tiles(const SeqLen& q, int rg) const {
    return (visible(q, rg) + KT - 1) / KT;
  }
  // tiles of groups 0 .. n-1.  A group but the last has
  //   ceil((len - nq + floor((RG (rg + 1) - 1) / g) + 1) / KT)
  //     = floor((RG rg + RG - 1 + g (len - nq + KT)) / (g KT))
  // tiles, none while its last row sits at a negative position.
  __host__ __device__ __forceinline__ int64_t tiles_before(const SeqLen& q, int n) const {
    const int ng = groups(q);
    int64_t sum = 0;
    if (n == ng && n > 0) {
      sum = tiles(q, ng - 1);
      --n;
    }
    if (n <= 0) return sum;
    const int64_t base = (int64_t)q.len - q.nq;
    int64_t rg0 = 0;
    if (base < 0) rg0 = max((int64_t)0, (-base * g - RG + 1 + RG - 1) / RG);
    if (rg0 >= n) return sum;
    return sum + floor_sum(n - rg0, (int64_t)g * KT, RG,
                           RG * rg0 + RG - 1 + (int64_t)g * (base + KT));
  }
  __host__ __device__ __forceinline__ int64_t seq_tiles(const SeqLen& q) const {   // of one kv head
    return mine(q) ? tiles_before(q, groups(q)) : 0;
  }

  // What a lane keeps of the first 32 sequences between total() and Cursor::seek().
  struct Lane {
    SeqLen q;
    int64_t tiles;
  };
  // Whole warp: tiles of all sequences and heads.
  __device__ __forceinline__ int64_t total(int lane, Lane& l) const {
    l.tiles = 0;
    l.q = {0, 0, 0};
    if (lane < s.B) {
      l.q = seq_len(s, lane);
      l.tiles = seq_tiles(l.q);
    }
    int64_t t = l.tiles;
    for (int b = lane + 32; b < s.B; b += 32) t += seq_tiles(seq_len(s, b));
    t *= Hkv;
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
  }
  __host__ __device__ __forceinline__ int64_t workers(int64_t total_tiles) const {
    const int64_t w = (total_tiles + min_tiles - 1) / min_tiles;
    return w < n_workers ? (w > 1 ? w : 1) : n_workers;
  }
};

// A place on the line of tiles.
template <int RG, int KT>
struct Cursor {
  int b, kvh, rg, tile, n_tiles, n_groups;
  SeqLen q;

  // Whole warp: move to tile t of the line (0 <= t < total).
  __device__ __forceinline__ void seek(const Deal<RG, KT>& d, const typename Deal<RG, KT>::Lane& l0,
                                       int64_t t, int lane) {
    int64_t base = 0, per_head = 0;
    for (int b0 = 0; b0 < d.s.B; b0 += 32) {
      SeqLen sl = l0.q;
      int64_t w = l0.tiles;
      if (b0 > 0) {
        w = 0;
        if (b0 + lane < d.s.B) {
          sl = seq_len(d.s, b0 + lane);
          w = d.seq_tiles(sl);
        }
      }
      int64_t incl = w * d.Hkv;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
      if (t < base + sum) {
        const unsigned m = __ballot_sync(0xffffffffu, base + incl > t);
        const int l = __ffs(m) - 1;
        b = b0 + l;
        q.q0 = __shfl_sync(0xffffffffu, sl.q0, l);
        q.nq = __shfl_sync(0xffffffffu, sl.nq, l);
        q.len = __shfl_sync(0xffffffffu, sl.len, l);
        per_head = __shfl_sync(0xffffffffu, w, l);
        t -= base + __shfl_sync(0xffffffffu, incl, l) - per_head * d.Hkv;
        break;
      }
      base += sum;
    }
    n_groups = d.groups(q);
    kvh = (int)div64(t, per_head);
    t -= kvh * per_head;
    // the last group with tiles_before(group) <= t, by lanes in parallel
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int c = lo + lane * step;
      const bool le = c < hi && d.tiles_before(q, c) <= t;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      const int last = 31 - __clz(m);            // lane 0 always holds
      lo += last * step;
      hi = min(hi, lo + step);
    }
    rg = lo;
    n_tiles = d.tiles(q, rg);
    tile = (int)(t - d.tiles_before(q, rg));
  }
  // To the first tile of the next unit that has any; the caller stops at its last tile.
  __device__ __forceinline__ void next_unit(const Deal<RG, KT>& d) {
    tile = 0;
    do {
      if (++rg >= n_groups) {
        rg = 0;
        if (++kvh >= d.Hkv) {
          kvh = 0;
          do {
            if (++b >= d.s.B) {                  // past the end of the line
              n_tiles = 0;
              return;
            }
            q = seq_len(d.s, b);
          } while (!d.mine(q) || q.len == 0);
          n_groups = d.groups(q);
        }
      }
      n_tiles = d.tiles(q, rg);
    } while (n_tiles == 0);
  }
};

// A unit that was cut, to be merged: filled in by the worker that has its last tile (rows 0
// in the entries of workers without one).
struct Cut {
  int32_t rows;            // of the unit
  int32_t q0, row0, kvh;   // first new row of its sequence, its first row (token x group + head)
  int32_t w0;              // its first worker; this entry's worker is the last
  int32_t late;            // whether w0 began before the unit (its part is in slot 1)
};

// Whole warp: worker w's entry.  cur is at its first tile t0, n its tiles (0: no tiles).
template <int RG, int KT>
__device__ __forceinline__ void note_cut(Cut* out, const Deal<RG, KT>& d, const Shares& sh,
                                         const Cursor<RG, KT>& cur, int64_t t0, int64_t n, int lane) {
  Cut c = {0, 0, 0, 0, 0, 0};
  if (n > 0 && cur.tile > 0 && cur.n_tiles - cur.tile <= n) {
    const int64_t rows = (int64_t)cur.q.nq * d.g - (int64_t)cur.rg * RG;
    c.rows = (int)(rows < RG ? rows : RG);
    c.q0 = cur.q.q0;
    c.row0 = cur.rg * RG;
    c.kvh = cur.kvh;
    const int64_t u0 = t0 - cur.tile;
    c.w0 = (int)sh.owner(u0);
    c.late = sh.first(c.w0) < u0;
  }
  if (lane == 0) *out = c;
}

}  // namespace paged
}  // namespace vc
