// Acceptance by sampling (the counterpart of greedy acceptance, accept.cu): drafted tokens
// against the target's probabilities, with given random numbers.
//
// With p, q the softmax of the target's and the drafting side's logits over T, draft d_i
// stays while u_i q(d_i) < p(d_i); at the first refusal the token is drawn from
// max(p - q, 0), after the last draft from p, as the first index whose running sum passes
// u times the total.  Committed tokens are then distributed as samples of p.
//
// Kernel 1 (HBM-bound: every logit once): rows over a grid of (slice, row), per slice the
//   largest logit with its first index and sum 2^((x - max) c), c = log2(e) / T in two fp32
//   parts, so the exponent's error is its rounding alone.  fp32 terms, fp64 across threads.
// Kernel 2: every block of a sequence decides the drafts for itself from kernel 1's parts
//   (a warp a position), then adds up segments of 512 values of the one row that is drawn
//   from, a warp a segment, in fp64: e^x_p, and e^x_q where both rows matter.  fp32 would not
//   do here: a running sum off by 1e-7 crosses another border once in some hundred draws from
//   a flat row of 128K.
// Kernel 3 (draft_logits given): segment sums of max(p - q, 0).
// Kernel 4: picks the segment, then the index in it, and writes the outputs.
// Where one block serves a sequence, kernels 2 to 4 are one launch.
// Measured, a call: 8 x 65 rows (33 and 32 of each side) of 128256 fp32 64 us, of which kernel 1
// 44 (267 MB at 6.1 TB/s) and the rest the decisions and two fp64 passes over 16 rows; 64 x 4
// bf16 rows 42 us; 9 rows of 8192 13 us of the GPU, three launches' latency.
// The fp64 exponential is a table of 2^(j/64) and a polynomial of degree 4 (the table method
// published by P. T. P. Tang, "Table-driven implementation of the exponential function",
// 1989): 10 fp64 operations, relative error under 1e-13.
#include <algorithm>
#include <climits>

#include "vc_common.cuh"
#include "vc_internal.h"

namespace vc {
namespace {

constexpr int kStatThreads = 256;
constexpr int kPassThreads = 512;
constexpr int kPassWarps = kPassThreads / 32;
constexpr int kSeg = 512;            // values of a segment
constexpr int kMostSplits = 16;      // of a row in kernel 1 (half a warp reads them)
constexpr int kStatBlocks = 6;       // of kernel 1 on an SM
constexpr float kColdest = 8.673617379884035e-19f;   // 2^-60: colder is greedy

struct Stat {            // one slice of one row
  double s;              // sum 2^((x - m) c)
  float m;               // largest logit (-inf: none above)
  int idx;               // its first index
  int bad;               // a NaN
  int pad;
};

enum Mode : int { kGreedy = 0, kBadRow = 1, kFromP = 2, kWithoutDraft = 3, kResidual = 4 };

struct State {           // kernel 2's decision for a sequence
  double inv_t;
  double wp, wq;         // kernel 3's: one over the sums of the two rows
  float mp, mq;          // largest logits of the two rows
  int a, mode, token, err;
};

struct SampleArgs {
  const void* logits;
  const void* draft_logits;
  const int32_t* drafts;
  const double* u;
  const float* temperature;
  const int32_t* n_drafts;
  int32_t B, n_q, V;
  int32_t splits;        // slices of a row in kernel 1
  int32_t n_seg;         // segments of a row in kernels 2 to 4
  Stat* stat;            // [B * n_q + B * k, splits]
  double* sums;          // [3, B, n_seg]: e^x_p, e^x_q, residual
  State* state;          // [B]
  int32_t* accept_len;
  int32_t* commit;
  int32_t* n_commit;
  int32_t* err_flag;
};

__device__ __forceinline__ int live_drafts(const SampleArgs& a, int b) {
  const int k = a.n_q - 1;
  return a.n_drafts ? min(max(a.n_drafts[b], 0), k) : k;
}
// 0 for greedy sequences.
__device__ __forceinline__ float temp_of(const SampleArgs& a, int b, bool& bad) {
  const float t = a.temperature ? a.temperature[b] : 1.f;
  bad = !(t >= 0.f && t < INFINITY);
  return bad || t < kColdest ? 0.f : t;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[i]);
    else return i & 1 ? bf16_hi(r[i >> 1]) : bf16_lo(r[i >> 1]);
  }
};

// ------------------------------------------------------------------ kernel 1
struct Acc {
  float m = -INFINITY, s = 0.f;
  int best = INT_MAX;      // where m came from first (the caller's number of the batch)
};

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

// The exponent's factor log2(e) / T in two parts, both > 0: a part of a -inf logit is then -inf
// whatever the other is, and so is one that overflows.  (At least the smallest fp32 number: next
// to a factor of 1e-38, for T near the largest, more would count.)
struct Factor {
  float hi, lo;
};
__device__ __forceinline__ Factor factor_of(float t) {
  const double c = 1.4426950408889634 / (double)t;
  Factor f;
  f.hi = __double2float_rz(c);
  f.lo = fmaxf((float)(c - (double)f.hi), 1.4e-45f);
  return f;
}
// 2^(d (hi + lo)) for d <= 0.
__device__ __forceinline__ float weight_of(float d, Factor f) { return ex2(fmaf(d, f.hi, d * f.lo)); }

// A batch of N logits, number `id` of the thread, ascending in index.  A NaN or a +inf makes the
// sum NaN.
template <int N>
__device__ __forceinline__ void take(Acc& a, const float (&x)[N], Factor f, int id) {
  float t[4] = {x[0], x[0], x[0], x[0]};
#pragma unroll
  for (int i = 1; i < N; ++i) t[i & 3] = fmaxf(t[i & 3], x[i]);
  const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
  if (top > a.m) {
    a.s *= weight_of(a.m - top, f);
    a.m = top;
    a.best = id;
  }
  if (a.m > -INFINITY) {
    if constexpr (N % 2 == 0) {
      const uint64_t nm = pair(-a.m, -a.m), hi = pair(f.hi, f.hi), lo = pair(f.lo, f.lo);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        uint64_t y;
        asm("{\n .reg .b64 d, e;\n add.rn.f32x2 d, %1, %2;\n mul.rn.f32x2 e, d, %4;\n"
            " fma.rn.f32x2 %0, d, %3, e;\n}\n"
            : "=l"(y) : "l"(pair(x[i], x[i + 1])), "l"(nm), "l"(hi), "l"(lo));
        float u, v;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(u), "=f"(v) : "l"(y));
        s[0] += ex2(u);
        s[1] += ex2(v);
      }
      a.s += s[0] + s[1];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) a.s += weight_of(x[i] - a.m, f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (x[i] != x[i]) a.s = NAN;       // nothing above -inf yet
  }
}

template <typename T>
__global__ void __launch_bounds__(kStatThreads, kStatBlocks) sample_stat_kernel(const SampleArgs a) {
  pdl_wait();
  pdl_trigger();
  const int k = a.n_q - 1;
  const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  const int64_t n_target = (int64_t)a.B * a.n_q;
  // (rows that fill up the grid's last plane are nobody's, whether or not there are draft rows)
  if (row >= n_target + (a.draft_logits ? (int64_t)a.B * k : 0)) return;
  const bool draft = row >= n_target;
  const int b = (int)(draft ? (row - n_target) / k : row / a.n_q);
  const int i = (int)(draft ? (row - n_target) % k : row % a.n_q);
  const int n = live_drafts(a, b);
  bool bad_t;
  const float t = temp_of(a, b, bad_t);
  if (draft ? (i >= n || t == 0.f) : i > n) return;       // never looked at
  const Factor f = factor_of(t == 0.f ? 1.f : t);          // (greedy: for the NaN alone)
  const T* x = static_cast<const T*>(draft ? a.draft_logits : a.logits) +
               (draft ? row - n_target : row) * (int64_t)a.V;

  // 16-byte vectors between the first aligned value and the last whole one; slice 0 takes
  // the values before them, the last slice those behind
  constexpr int N = Vec<T>::kN, U = 4;
  const int head = min(a.V, (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
  const int nv = (a.V - head) / N;
  const int lo = (int)((int64_t)nv * blockIdx.x / a.splits);
  const int hi = (int)((int64_t)nv * (blockIdx.x + 1) / a.splits);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  Acc acc;
  // batches are numbered by their first vector, single values by -1 - index
  auto single = [&](int j) {
    const float v[1] = {to_f32(x[j])};
    take(acc, v, f, -1 - j);
  };
  if (blockIdx.x == 0)
    for (int j = threadIdx.x; j < head; j += kStatThreads) single(j);
  for (int v0 = lo + (int)threadIdx.x; v0 < hi; v0 += kStatThreads * U) {
    Vec<T> r[U];
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (v0 + q * kStatThreads < hi) r[q].raw = __ldcs(xv + v0 + q * kStatThreads);
    if (v0 + (U - 1) * kStatThreads < hi) {
      // 16 values a batch
      constexpr int G = 16 / N;
#pragma unroll
      for (int q = 0; q < U; q += G) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = r[q + e / N].get(e % N);
        take(acc, v, f, v0 + q * kStatThreads);
      }
    } else {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        if (v0 + q * kStatThreads < hi) {
          float v[N];
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = r[q].get(e);
          take(acc, v, f, v0 + q * kStatThreads);
        }
      }
    }
  }
  if ((int)blockIdx.x == a.splits - 1)
    for (int j = head + nv * N + threadIdx.x; j < a.V; j += kStatThreads) single(j);

  // block: the largest, its first index (read again by the threads that have it), and the
  // sums brought to it
  __shared__ float sh_m[kStatThreads / 32];
  __shared__ int sh_n[kStatThreads / 32], sh_i;
  __shared__ double sh_s[kStatThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) sh_i = INT_MAX;
  const float wm = warp_max_xor(acc.m, 5);
  if (lane == 0) sh_m[warp] = wm;
  __syncthreads();
  float m = sh_m[0];
#pragma unroll
  for (int w = 1; w < kStatThreads / 32; ++w) m = fmaxf(m, sh_m[w]);
  const float d = acc.m == -INFINITY ? 0.f : acc.m - m;
  double s = (double)acc.s * (double)weight_of(d, f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const bool nan = __any_sync(0xffffffffu, acc.s != acc.s);
  if (lane == 0) { sh_s[warp] = s; sh_n[warp] = nan; }
  if (acc.m == m && m > -INFINITY) {
    int idx = INT_MAX;
    if (acc.best < 0) {
      idx = -1 - acc.best;
    } else {
      for (int q = 16 / N - 1; q >= 0; --q) {
        const int v = acc.best + q * kStatThreads;
        if (v < hi)
          for (int e = N - 1; e >= 0; --e) {
            const int j = head + v * N + e;
            if (to_f32(x[j]) == m) idx = j;
          }
      }
    }
    atomicMin(&sh_i, idx);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Stat r;
    r.m = m;
    r.idx = sh_i;
    r.s = 0.0;
    r.bad = 0;
    for (int w = 0; w < kStatThreads / 32; ++w) {
      r.s += sh_s[w];
      r.bad |= sh_n[w];
    }
    r.pad = 0;
    a.stat[row * a.splits + blockIdx.x] = r;
  }
}

// ------------------------------------------------------------------ fp64 exponential
// table[j] = 2^(j / 64), filled by the block.
constexpr int kTable = 64;
__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < kTable) table[threadIdx.x] = exp2(threadIdx.x * (1.0 / kTable));
}
// Weights e^((x - m) / T) of a row: with k = 64 / (T ln 2), d = x - m, d k = n + r, |r| <= 1/2,
//   e^((x - m) / T) = 2^(n / 64) e^(r ln 2 / 64);
// 0 where d k < -64512 (2^-1008), and for x = -inf.  The difference is taken first: it is 0 at
// the largest logit whatever m / T is (m k alone may be large enough for its rounding to pass
// the ends of the exponent).
struct Expo {
  double k, m;
  double least;              // of d
};
__device__ __forceinline__ Expo expo_of(float m, double inv_t) {
  Expo e;
  e.k = 92.33248261689366 * inv_t;                      // 64 / ln 2
  e.m = (double)m;
  e.least = -64512.0 / e.k;
  return e;
}
__device__ __forceinline__ double weight64(double x, Expo e, const double* table) {
  const double d = x - e.m;
  if (!(d > e.least)) return 0.0;
  const double shift = 6755399441055744.0;              // 1.5 * 2^52: rounds to an integer
  const double z = fma(d, e.k, shift);
  const int n = __double2loint(z);
  const double r = fma(d, e.k, shift - z);
  // (ln 2 / 64)^i / i!
  double p = fma(r, 5.732851688640402e-10, 2.1173137155464774e-07);
  p = fma(r, p, 5.864904955056169e-05);
  p = fma(r, p, 0.010830424696249146);
  p *= r;
  const double t = table[n & 63];
  const double w = fma(t, p, t);
  return __hiloint2double(__double2hiint(w) + ((n >> 6) << 20), __double2loint(w));
}

// max(p - q, 0) from the weights of both rows and one over their sums.  Both products are rounded
// (fused, one of them would be exact and p - p its rounding), so that it is 0 where p == q, and
// the pick meets the very numbers that were summed.
__device__ __forceinline__ double residual_of(double e_p, double w_p, double e_q, double w_q) {
  return fmax(__dsub_rn(__dmul_rn(e_p, w_p), __dmul_rn(e_q, w_q)), 0.0);
}

// Sum over the block, in the same order every time; sh: kPassWarps values.
__device__ __forceinline__ double block_sum(double s, double* sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();                                      // sh of an earlier sum is read
  if (lane == 0) sh[warp] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kPassWarps; ++w) t += sh[w];
  return t;
}
__device__ __forceinline__ double sum_of(const double* x, int n, double* sh) {
  double s = 0.0;
  for (int j = threadIdx.x; j < n; j += kPassThreads) s += x[j];
  return block_sum(s, sh);
}
// Running sum over the block's threads (their own value included); all: the total.
__device__ __forceinline__ double block_scan(double s, double* sh, double& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += up;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  double before = 0.0;
  all = 0.0;
#pragma unroll
  for (int w = 0; w < kPassWarps; ++w) {
    if (w < warp) before += sh[w];
    all += sh[w];
  }
  return before + s;
}

struct RowStat {
  float m;
  int idx;
  double z;              // sum e^((x - m) / T)
  bool bad;
};

// A row's parts, merged by the 16 lanes of a half-warp (the same in each of them).
__device__ __forceinline__ RowStat row_stat(const SampleArgs& a, int64_t row, bool wanted,
                                            double inv_t, const double* table, int lane) {
  Stat st;
  st.m = -INFINITY;
  st.idx = INT_MAX;
  st.s = 0.0;
  st.bad = 0;
  const int j = lane & 15;
  if (wanted && j < a.splits) st = a.stat[row * a.splits + j];
  RowStat r = {st.m, st.idx, 0.0, st.bad != 0};
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, r.m, o);
    const int oi = __shfl_xor_sync(0xffffffffu, r.idx, o);
    r.bad |= __shfl_xor_sync(0xffffffffu, (int)r.bad, o) != 0;
    if (om > r.m || (om == r.m && oi < r.idx)) { r.m = om; r.idx = oi; }
  }
  r.bad |= !(r.m > -INFINITY && r.m < INFINITY);
  if (!r.bad && st.m > -INFINITY) r.z = st.s * weight64(st.m, expo_of(r.m, inv_t), table);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) r.z += __shfl_xor_sync(0xffffffffu, r.z, o);
  return r;
}

// The rows that sequence b draws from.
template <typename T>
__device__ __forceinline__ const T* target_row(const SampleArgs& a, int b, int i) {
  return static_cast<const T*>(a.logits) + ((int64_t)b * a.n_q + i) * a.V;
}
template <typename T>
__device__ __forceinline__ const T* draft_row(const SampleArgs& a, int b, int i) {
  return static_cast<const T*>(a.draft_logits) + ((int64_t)b * (a.n_q - 1) + i) * a.V;
}
// The first segment of a block out of `blocks`.
__device__ __forceinline__ int seg_at(const SampleArgs& a, int block, int blocks) {
  return (int)((int64_t)a.n_seg * block / blocks);
}
// A warp's values of a segment of row x: 16 a lane, in vectors where the row is aligned
// (-inf behind the row's end); value i of a lane has the index seg_index(...).
template <typename T>
struct SegValues {
  float v[kSeg / 32];
  bool vec;
  // `aligned`: whether x lies on 16 bytes (for two rows read side by side: whether both do)
  __device__ __forceinline__ void load(const T* x, int V, int seg, int lane, bool aligned) {
    const int lo = seg * kSeg;
    constexpr int N = Vec<T>::kN;
    vec = lo + kSeg <= V && aligned;
    if (vec) {
      const uint4* p = reinterpret_cast<const uint4*>(x + lo) + lane;
      Vec<T> r[kSeg / 32 / N];
#pragma unroll
      for (int q = 0; q < kSeg / 32 / N; ++q) r[q].raw = __ldg(p + 32 * q);
#pragma unroll
      for (int i = 0; i < kSeg / 32; ++i) v[i] = r[i / N].get(i % N);
    } else {
#pragma unroll
      for (int i = 0; i < kSeg / 32; ++i) {
        const int j = lo + 32 * i + lane;
        v[i] = j < V ? to_f32(x[j]) : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ int index(int seg, int lane, int i) const {
    constexpr int N = Vec<T>::kN;
    return seg * kSeg + (vec ? (i / N * 32 + lane) * N + i % N : 32 * i + lane);
  }
};
template <typename T>
__device__ __forceinline__ bool aligned16(const T* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

__device__ __forceinline__ double warp_sum(double s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// ------------------------------------------------------------------ kernel 2
template <typename T>
__device__ __forceinline__ void sum_part(const SampleArgs& a, int b, int block, int blocks,
                                         const double* table) {
  __shared__ int first;
  __shared__ State st;
  // what a position gives, by its warp
  struct Seen {
    float mp, mq;
    int idx, d;
    unsigned char bad_p, bad_q, odd;
  };
  __shared__ Seen seen[257];
  const int k = a.n_q - 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) first = INT_MAX;
  __syncthreads();
  const int n = live_drafts(a, b);
  bool bad_t;
  const float t = temp_of(a, b, bad_t);
  const double inv_t = t == 0.f ? 0.0 : 1.0 / (double)t;
  const bool with_q = a.draft_logits != nullptr && t != 0.f;
  // positions 0 .. n: lanes 0-15 look at the target's row, 16-31 at the draft's
#pragma unroll 2
  for (int i = warp; i <= n; i += kPassWarps) {
    const bool is_q = lane >= 16;
    const int64_t row = is_q ? (int64_t)a.B * a.n_q + (int64_t)b * k + i : (int64_t)b * a.n_q + i;
    const bool wanted = !is_q || (with_q && i < n);
    int d = 0;
    double u = 0.0;
    if (i < n) {
      d = a.drafts[(int64_t)b * k + i];
      u = a.u[(int64_t)b * a.n_q + i];
    }
    const bool out = i < n && (d < 0 || d >= a.V);
    float x = 0.f;                                 // the draft's logit in this half's row
    if (i < n && !out && wanted)
      x = to_f32(is_q ? draft_row<T>(a, b, i)[d] : target_row<T>(a, b, i)[d]);
    const RowStat r = row_stat(a, row, wanted, inv_t, table, lane);
    const double e = weight64(x, expo_of(r.m, inv_t), table);
    const double eq = __shfl_sync(0xffffffffu, e, 16), zq = __shfl_sync(0xffffffffu, r.z, 16);
    const float mq = __shfl_sync(0xffffffffu, r.m, 16);
    const bool bad_q = __shfl_sync(0xffffffffu, (int)r.bad, 16) != 0;
    if (lane == 0) {
      const bool odd = r.bad || out || (with_q && i < n && bad_q);
      bool refuse = out || r.bad;
      if (!refuse && i < n) {
        if (t == 0.f) refuse = d != r.idx;
        else refuse = !(u * r.z * (with_q && !bad_q ? eq / zq : 1.0) < e);
      }
      seen[i] = {r.m, mq, r.idx, d, r.bad, bad_q, odd};
      if (refuse && i < n) atomicMin(&first, i);
    }
  }
  __syncthreads();
  const int pos = min(first, n);
  bool odd = false;
  for (int i = threadIdx.x; i <= pos; i += kPassThreads) odd |= seen[i].odd != 0;
  odd = __syncthreads_or(odd);
  if (threadIdx.x == 0) {
    const Seen s = seen[pos];
    State r;
    r.inv_t = inv_t;
    r.a = pos;
    r.mp = s.mp;
    r.mq = s.mq;
    r.token = s.idx;
    r.mode = s.bad_p ? kBadRow : t == 0.f ? kGreedy : kFromP;
    if (pos < n && r.mode == kFromP) {
      const bool in = s.d >= 0 && s.d < a.V;
      if (with_q && !s.bad_q) r.mode = kResidual;
      else if (in) r.mode = kWithoutDraft;
      if (r.mode == kWithoutDraft) r.token = s.d;
    }
    const int nd = a.n_drafts ? a.n_drafts[b] : k;
    r.err = odd || bad_t || nd < 0 || nd > k ? 1 : 0;
    st = r;
    if (block == 0) a.state[b] = r;
  }
  __syncthreads();
  const int mode = st.mode;
  if (mode == kGreedy || mode == kBadRow) return;
  const T* xp = target_row<T>(a, b, st.a);
  const Expo ep = expo_of(st.mp, st.inv_t), eq = expo_of(st.mq, st.inv_t);
  const int skip = mode == kWithoutDraft ? st.token : -1;
  const T* xq = mode == kResidual ? draft_row<T>(a, b, st.a) : xp;
  const int end = seg_at(a, block + 1, blocks);
  for (int seg = seg_at(a, block, blocks) + warp; seg < end; seg += kPassWarps) {
    SegValues<T> vp, vq;
    vp.load(xp, a.V, seg, lane, aligned16(xp));
    if (mode == kResidual) vq.load(xq, a.V, seg, lane, aligned16(xq));
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kSeg / 32; ++i)
      s[i & 3] += vp.index(seg, lane, i) == skip ? 0.0 : weight64(vp.v[i], ep, table);
    const double sp = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (lane == 0) a.sums[(int64_t)b * a.n_seg + seg] = sp;
    if (mode == kResidual) {
      s[0] = s[1] = s[2] = s[3] = 0.0;
#pragma unroll
      for (int i = 0; i < kSeg / 32; ++i) s[i & 3] += weight64(vq.v[i], eq, table);
      const double sq = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
      if (lane == 0) a.sums[((int64_t)a.B + b) * a.n_seg + seg] = sq;
    }
  }
}

// ------------------------------------------------------------------ kernel 3
template <typename T>
__device__ __forceinline__ void residual_part(const SampleArgs& a, int b, int block, int blocks,
                                              const double* table) {
  __shared__ double sh[kPassWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const State st = a.state[b];
  if (st.mode != kResidual) return;
  const double wp = 1.0 / sum_of(a.sums + (int64_t)b * a.n_seg, a.n_seg, sh);
  const double wq = 1.0 / sum_of(a.sums + ((int64_t)a.B + b) * a.n_seg, a.n_seg, sh);
  if (block == 0 && threadIdx.x == 0) {
    a.state[b].wp = wp;
    a.state[b].wq = wq;
  }
  const Expo ep = expo_of(st.mp, st.inv_t), eq = expo_of(st.mq, st.inv_t);
  const T* xp = target_row<T>(a, b, st.a);
  const T* xq = draft_row<T>(a, b, st.a);
  const int end = seg_at(a, block + 1, blocks);
  for (int seg = seg_at(a, block, blocks) + warp; seg < end; seg += kPassWarps) {
    SegValues<T> vp, vq;
    const bool both = aligned16(xp) && aligned16(xq);
    vp.load(xp, a.V, seg, lane, both);
    vq.load(xq, a.V, seg, lane, both);
    double r[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kSeg / 32; ++i)
      r[i & 3] += residual_of(weight64(vp.v[i], ep, table), wp, weight64(vq.v[i], eq, table), wq);
    const double s = warp_sum((r[0] + r[1]) + (r[2] + r[3]));
    if (lane == 0) a.sums[(2 * (int64_t)a.B + b) * a.n_seg + seg] = s;
  }
}

// ------------------------------------------------------------------ kernel 4
template <typename T>
__device__ __forceinline__ void pick_part(const SampleArgs& a, int b, const double* table) {
  __shared__ double sh[kPassWarps];
  __shared__ int found, last, seg_sh;
  __shared__ double left_sh;
  const int k = a.n_q - 1, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    found = seg_sh = INT_MAX;
    last = -1;
  }
  __syncthreads();
  const State st = a.state[b];
  int mode = st.mode, token = st.token;
  if (mode == kBadRow) {
    // vc_accept's argmax: the first NaN, else the first largest value (index 0 if all -inf)
    const T* x = target_row<T>(a, b, st.a);
    int nan = INT_MAX, idx = INT_MAX;
    float m = -INFINITY;
    for (int j = tid; j < a.V; j += kPassThreads) {
      const float v = to_f32(x[j]);
      if (v != v) nan = min(nan, j);
      else if (v > m || idx == INT_MAX) { m = v; idx = j; }
    }
    __shared__ float sm[kPassWarps];
    __shared__ int si[kPassWarps];
    atomicMin(&found, nan);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o);
      const int oi = __shfl_xor_sync(0xffffffffu, idx, o);
      if (om > m || (om == m && oi < idx)) { m = om; idx = oi; }
    }
    if (lane == 0) { sm[warp] = m; si[warp] = idx; }
    __syncthreads();
    for (int w = 0; w < kPassWarps; ++w)
      if (sm[w] > m || (sm[w] == m && si[w] < idx)) { m = sm[w]; idx = si[w]; }
    token = found != INT_MAX ? found : idx;
  } else if (mode != kGreedy) {
    const double* sp = a.sums + (int64_t)b * a.n_seg;
    const double* sr = a.sums + (2 * (int64_t)a.B + b) * a.n_seg;
    double wp = 1.0, wq = 0.0;
    const double* sw = sp;
    if (mode == kResidual) {
      if (sum_of(sr, a.n_seg, sh) > 0.0) {
        wp = st.wp;
        wq = st.wq;
        sw = sr;
      } else {
        mode = kFromP;                           // p == q everywhere: p itself
      }
    }
    // a thread's run of segments, the running sum over the threads, then over its run: the first
    // segment in which it passes u * total, or the last one with any weight if rounding
    // lets none pass
    const int run = (a.n_seg + kPassThreads - 1) / kPassThreads;
    const int s0 = min(a.n_seg, tid * run), s1 = min(a.n_seg, s0 + run);
    double mine = 0.0, total;
    int lastw = -1;
    for (int j = s0; j < s1; ++j) {
      mine += sw[j];
      if (sw[j] > 0.0) lastw = j;
    }
    const double upto = block_scan(mine, sh, total);
    const double want = a.u[(int64_t)b * a.n_q + k] * total;
    if (lastw >= 0) atomicMax(&last, lastw);
    int hit = INT_MAX;
    double left = 0.0;
    if (mine > 0.0 && upto > want) {
      double at = upto - mine;
      for (int j = s0; j < s1; ++j) {
        if (sw[j] > 0.0) {
          hit = j;
          left = want - at;
          if (at + sw[j] > want) break;
        }
        at += sw[j];
      }
      atomicMin(&seg_sh, hit);
    }
    __syncthreads();
    if (total > 0.0) {                           // else all of p is on the draft: st.token
      const int seg = seg_sh != INT_MAX ? seg_sh : last;
      if (seg_sh != INT_MAX ? hit == seg : tid == 0) left_sh = seg_sh != INT_MAX ? left : INFINITY;
      __syncthreads();
      if (tid == 0) last = -1;
      __syncthreads();
      const T* xp = target_row<T>(a, b, st.a);
      const T* xq = mode == kResidual ? draft_row<T>(a, b, st.a) : xp;
      const int skip = mode == kWithoutDraft ? st.token : -1;
      const Expo ep = expo_of(st.mp, st.inv_t), eq = expo_of(st.mq, st.inv_t);
      constexpr int N = kSeg / kPassThreads;
      const int j0 = seg * kSeg + tid * N;
      double wj[N], sum = 0.0, all;
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const int j = j0 + x;
        wj[x] = 0.0;
        if (j < a.V && j != skip) {
          wj[x] = weight64(to_f32(xp[j]), ep, table);
          if (mode == kResidual)
            wj[x] = residual_of(wj[x], wp, weight64(to_f32(xq[j]), eq, table), wq);
        }
        sum += wj[x];
      }
      double at = block_scan(sum, sh, all) - sum;
#pragma unroll
      for (int x = 0; x < N; ++x) {
        at += wj[x];
        if (wj[x] > 0.0) {
          if (at > left_sh) atomicMin(&found, j0 + x);
          atomicMax(&last, j0 + x);
        }
      }
      __syncthreads();
      token = found != INT_MAX ? found : last;
    }
  }
  const int n_a = st.a;
  for (int i = tid; i < a.n_q; i += kPassThreads)
    a.commit[(int64_t)b * a.n_q + i] = i < n_a ? a.drafts[(int64_t)b * k + i] : i == n_a ? token : -1;
  if (tid == 0) {
    a.accept_len[b] = n_a;
    a.n_commit[b] = n_a + 1;
    if (a.err_flag) a.err_flag[b] = st.err;
  }
}

// Kernels 2, 3 and 4, and the three in one for sequences that one block serves.
enum Part { kSumPart = 1, kResidualPart = 2, kPickPart = 4 };

template <typename T, int kParts>
__global__ void __launch_bounds__(kPassThreads, 2) sample_kernel(const SampleArgs a) {
  __shared__ double table[kTable];
  fill_table(table);
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int b = blockIdx.y, block = blockIdx.x, blocks = gridDim.x;
  if constexpr (kParts & kSumPart) sum_part<T>(a, b, block, blocks, table);
  if constexpr ((kParts & (kSumPart | kPickPart)) == (kSumPart | kPickPart)) __syncthreads();
  if constexpr (kParts & kResidualPart) residual_part<T>(a, b, block, blocks, table);
  if constexpr ((kParts & (kResidualPart | kPickPart)) == (kResidualPart | kPickPart)) __syncthreads();
  if constexpr (kParts & kPickPart) pick_part<T>(a, b, table);
}

struct SamplePlan {
  int splits, n_seg;
  size_t stat_off, sums_off, state_off, bytes;
};

// Slices of a row in kernel 1: two rounds of what the SMs hold at once, none under 1024 values
// (the whole call with one, two, four rounds: 8 x 65 fp32 rows of 128256 67.8, 65.9, 65.4 us,
// 64 x 4 bf16 rows 42.3, 41.5, 44.9 us).
SamplePlan sample_plan(int B, int n_q, int V, bool with_q) {
  SamplePlan p;
  const int64_t rows = (int64_t)B * (with_q ? 2 * n_q - 1 : n_q), sms = num_sms();
  const int64_t most = std::min<int64_t>(kMostSplits, std::max<int64_t>(1, V / 1024));
  p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, (2 * sms * kStatBlocks + rows - 1) / rows));
  p.n_seg = (V + kSeg - 1) / kSeg;
  p.stat_off = 0;
  p.sums_off = (size_t)rows * p.splits * sizeof(Stat);
  p.state_off = p.sums_off + (size_t)3 * B * p.n_seg * sizeof(double);
  p.bytes = p.state_off + (size_t)B * sizeof(State);
  return p;
}

template <typename T>
vc_status run_sample(const SampleArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.n_q + (a.draft_logits ? (int64_t)a.B * (a.n_q - 1) : 0);
  const int64_t y = std::min<int64_t>(rows, 32768);
  // kernels 2 and 3: the two blocks that an SM holds, over the B rows (64 rows, one, two, four
  // blocks an SM: 48.8, 41.5, 43.0 us for the call), a segment a warp at least
  const int blocks = (int)std::max<int64_t>(
      1, std::min<int64_t>((a.n_seg + kPassWarps - 1) / kPassWarps, (int64_t)num_sms() * 2 / a.B));
  VC_CUDA(launch_pdl(sample_stat_kernel<T>, dim3(a.splits, (unsigned)y, (unsigned)((rows + y - 1) / y)),
                     dim3(kStatThreads), 0, stream, 1, a));
  const dim3 grid(blocks, a.B), threads(kPassThreads);
  if (blocks == 1) {
    // one block a sequence: one launch instead of three (9 rows of 8192: 15.3 -> 13.0 us)
    VC_CUDA(launch_pdl(sample_kernel<T, kSumPart | kResidualPart | kPickPart>, grid, threads, 0, stream,
                       1, a));
    return VC_OK;
  }
  VC_CUDA(launch_pdl(sample_kernel<T, kSumPart>, grid, threads, 0, stream, 1, a));
  if (a.draft_logits)
    VC_CUDA(launch_pdl(sample_kernel<T, kResidualPart>, grid, threads, 0, stream, 1, a));
  VC_CUDA(launch_pdl(sample_kernel<T, kPickPart>, dim3(1, a.B), threads, 0, stream, 1, a));
  return VC_OK;
}

}  // namespace

size_t sample_workspace_bytes(int B, int n_q, int V) {
  return std::max(sample_plan(B, n_q, V, true).bytes, sample_plan(B, n_q, V, false).bytes);
}

vc_status launch_sample(const void* logits, const void* draft_logits, const int32_t* drafts,
                        const double* u, const float* temperature, const int32_t* n_drafts, int B,
                        int n_q, int V, int flags, int32_t* accept_len, int32_t* commit,
                        int32_t* n_commit, int32_t* err_flag, void* ws, cudaStream_t stream) {
  const SamplePlan p = sample_plan(B, n_q, V, draft_logits != nullptr && n_q > 1);
  char* w = static_cast<char*>(ws);
  SampleArgs a;
  a.logits = logits;
  a.draft_logits = n_q > 1 ? draft_logits : nullptr;
  a.drafts = drafts;
  a.u = u;
  a.temperature = temperature;
  a.n_drafts = n_drafts;
  a.B = B;
  a.n_q = n_q;
  a.V = V;
  a.splits = p.splits;
  a.n_seg = p.n_seg;
  a.stat = reinterpret_cast<Stat*>(w + p.stat_off);
  a.sums = reinterpret_cast<double*>(w + p.sums_off);
  a.state = reinterpret_cast<State*>(w + p.state_off);
  a.accept_len = accept_len;
  a.commit = commit;
  a.n_commit = n_commit;
  a.err_flag = err_flag;
  return flags & VC_LOGITS_BF16 ? run_sample<__nv_bfloat16>(a, stream)
                                : run_sample<float>(a, stream);
}

}  // namespace vc
