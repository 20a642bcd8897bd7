// swa_score.cuh -- what shapes the scores of an attention beyond the window:
// a tanh cap, a bias that grows with the distance, and documents (with
// prefixes) packed into one row of tokens.
//
//   u = scale q_i . k_j / cap,  s_ij = cap tanh(u) - slope_h |i - j|,
//   K(i) = [lo(i), hi(i)],  with [ds, de) the document of row i and pe = ds +
//   its prefix length:
//     lo(i) = max(ds, i - L),  hi(i) = min(de - 1, max(i + R, pe - 1)).
// Both bounds grow with the row (across documents too), so a tile of query
// rows still needs one contiguous run of key tiles, and the rows that see a
// key are an interval as well:
//     qlo(j) = ds if j < pe, else max(ds, j - R);  qhi(j) = min(de - 1, j + L).
#pragma once

#include <cstdint>

#include "swa_ptx.cuh"
#include "swa_sched.cuh"

namespace swa {

// The cap in log2 units as a function of the raw product s: cap log2(e) tanh(u)
// with u = s ci, ci = scale / cap.
//
// For |u| <= 1/2 (nearly always, with the caps that models use) it is u times a
// cubic in u^2: a degree-3 polynomial in z fitted to tanh(sqrt z) / sqrt z on
// [0, 1/4] by iterated weighted least squares (relative error 5.5e-7).  With
// ci^k folded into the coefficients on the host that is four operations on the
// FMA pipe, none on MUFU, which the exponentials already fill.  (Forming u first, a
// fifth one, took 8192 packed tokens from 157 to 169 us, a training step from
// 334 to 348.)
// A tanh from MUFU (error 2^-11) would be worth 2 % of a probability at a cap of
// 50.
// Elsewhere tanh u = 1 - 2 / (e^{2u} + 1) for either sign (absolute error
// about 5e-7, a like share of a tanh of at least 0.46; +-1 for infinite u, NaN
// for NaN), with two MUFU operations.  Nearer to 0 that error would count: the
// cap multiplies it.  So each score takes the form of its own u, and a warp
// only skips the second one when none of its scores needs it: a score's bits
// do not depend on its neighbours'.
// Where the folded coefficients would leave fp32's range (caps from 1e5 scale
// on, or below 1e-4 scale) u is formed first: pre = ci and plain coefficients.
// Then every score goes the way of both forms, which multiplies by pre; with
// folded coefficients pre is 1, and the bits are the short way's.
struct CapCoefs {
  float pre;
  float a0, a1, a2, a3;  // of (s pre)^1, ^3, ^5, ^7, in log2 units (the backward's: of tanh itself)
  float near;            // the cubic's range of |s|
  float vote;            // no score beyond it: the short way (-1: never)
  float far2;            // s pre far2 = 2 u log2 e
  float out;             // cap log2 e (0: no cap)
};

inline CapCoefs cap_coefs(float softcap, float scale, bool log2_units = true) {
  CapCoefs c{};
  if (!(softcap > 0.f)) return c;
  double ci = (double)scale / softcap, co = softcap * 1.4426950408889634;
  // ci and 1 / ci stay normal fp32 numbers.  A cap beyond 1e30 scale leaves every
  // product below 1e27 as it is (u^2 / 3 < 2^-24), and so does 1e30 scale in its
  // place; one below 1e-30 scale makes every product from 1e-29 on the cap itself.
  if (ci < 1e-30) {
    ci = 1e-30;
    co = scale * 1.4426950408889634 / ci;
  }
  if (ci > 1e30) ci = 1e30;
  const bool fold = ci > 1e-5 && ci < 1e4;
  const double unit = log2_units ? co : 1.0, f = fold ? ci : 1.0, z = f * f;
  c.pre = fold ? 1.f : (float)ci;
  c.a0 = (float)(0.99999945577 * f * unit);
  c.a1 = (float)(-0.33326318 * z * f * unit);
  c.a2 = (float)(0.13190297 * z * z * f * unit);
  c.a3 = (float)(-0.04440222 * z * z * z * f * unit);
  c.near = (float)(0.5 / ci);
  c.vote = fold ? c.near : -1.f;
  c.far2 = (float)(2.0 * f * 1.4426950408889634);
  c.out = (float)co;
  return c;
}

// The cubic of w = (s pre)^2 for a pair.
__device__ __forceinline__ float2 cap_cubic(const CapCoefs& c, float2 s) {
  const float2 w = mul2(s, s);
  float2 q = fma2(make_float2(c.a3, c.a3), w, make_float2(c.a2, c.a2));
  q = fma2(q, w, make_float2(c.a1, c.a1));
  return fma2(q, w, make_float2(c.a0, c.a0));
}
__device__ __forceinline__ float tanh_far(const CapCoefs& c, float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2_approx(s * c.far2) + 1.f));
  return fmaf(-2.f, r, 1.f);
}
// Capped scores of a pair of products plus add: with every |s| <= vote, or with any.
__device__ __forceinline__ float2 cap_small(const CapCoefs& c, float2 s, float2 add) {
  return fma2(s, cap_cubic(c, s), add);
}
__device__ __forceinline__ float2 cap_any(const CapCoefs& c, float2 s, float2 add) {
  const float2 v = mul2(s, make_float2(c.pre, c.pre)), near = cap_small(c, v, add);
  const float2 far = fma2(make_float2(tanh_far(c, v.x), tanh_far(c, v.y)),
                          make_float2(c.out, c.out), add);
  return make_float2(fabsf(s.x) <= c.near ? near.x : far.x, fabsf(s.y) <= c.near ? near.y : far.y);
}
// tanh of a pair (coefficients of tanh itself), likewise.
__device__ __forceinline__ float2 tanh_small(const CapCoefs& c, float2 s) {
  return mul2(s, cap_cubic(c, s));
}
__device__ __forceinline__ float2 tanh_any(const CapCoefs& c, float2 s) {
  const float2 v = mul2(s, make_float2(c.pre, c.pre)), near = tanh_small(c, v);
  return make_float2(fabsf(s.x) <= c.near ? near.x : tanh_far(c, v.x),
                     fabsf(s.y) <= c.near ? near.y : tanh_far(c, v.y));
}

// The documents of one row of tokens.
struct DocSpan {
  int start, end;  // positions [start, end); start >= end: none (padding)
  int pre;         // end of the prefix (<= start: none)
};

struct DocTiles;

struct DocMask {
  const int32_t* cu;   // [n + 1] boundaries (NULL: one document [0, N))
  const int32_t* pre;  // [n] prefix lengths (NULL: none)
  int n, N, L, R;

  __device__ __forceinline__ int clampN(int x) const { return x < 0 ? 0 : (x > N ? N : x); }
  __device__ __forceinline__ int first() const { return cu ? clampN(__ldg(cu)) : 0; }
  __device__ __forceinline__ int past() const { return cu ? clampN(__ldg(cu + n)) : N; }

  // The span of document m if it holds position i (m out of range: none).
  __device__ __forceinline__ DocSpan span(int m, int i) const {
    DocSpan s{0, 0, 0};
    if (m < 0 || m >= n) return s;
    const int a = clampN(__ldg(cu + m)), e = clampN(__ldg(cu + m + 1));
    if (i < a || i >= e) return s;
    s.start = a;
    s.end = e;
    s.pre = a;
    if (pre) {
      const int len = __ldg(pre + m);
      s.pre = len >= e - a ? e : a + (len < 0 ? 0 : len);
    }
    return s;
  }
  // Index of the last boundary <= i, searched by a whole converged warp for
  // the same i: 32 evenly spaced boundaries per step, one load latency each.
  __device__ __forceinline__ int find_warp(int i) const {
    const int lane = threadIdx.x & 31;
    int lo = 0, cnt = n + 1;
    while (cnt > 0) {
      const int step = (cnt + 31) / 32;
      const int idx = (lane + 1) * step - 1;
      const bool le = idx < cnt && __ldg(cu + lo + idx) <= i;
      const int c = __popc(__ballot_sync(0xffffffffu, le));
      lo += c * step;
      const int rest = cnt - c * step;
      cnt = rest < step - 1 ? rest : step - 1;
    }
    return lo - 1;
  }
  __device__ __forceinline__ DocSpan of_thread(const DocTiles& t, int i) const;
  // First and last key of row i of document s (none: 1, 0).
  __device__ __forceinline__ int key_first(const DocSpan& s, int i) const {
    if (s.start >= s.end) return 1;
    return (L < 0 || i - s.start <= L) ? s.start : i - L;
  }
  __device__ __forceinline__ int key_last(const DocSpan& s, int i) const {
    if (s.start >= s.end) return 0;
    const int h = (R < 0 || s.end - 1 - i <= R) ? s.end - 1 : i + R;
    return h > s.pre - 1 ? h : s.pre - 1;
  }
  // First and last row that sees key j of document s (none: 1, 0).
  __device__ __forceinline__ int query_first(const DocSpan& s, int j) const {
    if (s.start >= s.end) return 1;
    return (R < 0 || j < s.pre || j - s.start <= R) ? s.start : j - R;
  }
  __device__ __forceinline__ int query_last(const DocSpan& s, int j) const {
    if (s.start >= s.end) return 0;
    return (L < 0 || s.end - 1 - j <= L) ? s.end - 1 : j + L;
  }
};

// The key tiles of the query rows [m0, m1], and those of them that every row
// sees whole; or, transposed, the query tiles of the key rows [m0, m1].
struct DocTiles {
  int begin, end;        // tiles [begin, end)
  int int_lo, int_hi;    // tiles that need no element mask (lo > hi: none)
  int mlo, mhi;          // documents of the rows
  int c0, cn;            // rows outside [c0, cn) are padding
  // boundary base + lane and its document's prefix length, held by each lane
  int base, bound, pre;
};

// Makes span and of_thread of a warp's lanes (see DocTiles::bound).
__device__ __forceinline__ DocSpan span_of_lanes(const DocTiles& t, int n, int m, int i) {
  const int k = m - t.base;
  const int a = __shfl_sync(0xffffffffu, t.bound, k & 31);
  const int e = __shfl_sync(0xffffffffu, t.bound, (k + 1) & 31);
  const int len = __shfl_sync(0xffffffffu, t.pre, k & 31);
  DocSpan s{0, 0, 0};
  if (m < 0 || m >= n || i < a || i >= e) return s;
  s.start = a;
  s.end = e;
  s.pre = len >= e - a ? e : a + (len < 0 ? 0 : len);
  return s;
}

// By a whole converged warp (every warp of the block computes it for itself).
// With at most 31 documents all boundaries come in one load and the rest is
// warp votes and shuffles; otherwise the first row's document is searched
// for, and the 31 documents from there on are held (a tile's rows beyond
// them, tiny documents, are looked up in memory).
template <bool kQueriesOfKeys>
__device__ __forceinline__ DocTiles doc_tiles(const DocMask& dm, int m0, int m1) {
  const int lane = threadIdx.x & 31;
  DocTiles t;
  t.begin = t.end = 0;
  t.int_lo = 1;
  t.int_hi = 0;
  t.mlo = 0;
  t.mhi = -1;
  t.base = 0;
  t.bound = 0;
  t.pre = 0;
  DocSpan s0{0, dm.N, 0}, s1{0, dm.N, 0};
  int r0 = m0, r1 = m1;
  t.c0 = 0;
  t.cn = dm.N;
  if (dm.cu) {
    const bool few = dm.n <= 31;
    if (!few) {
      t.c0 = dm.first();
      t.cn = dm.past();
      t.base = dm.find_warp(m0 > t.c0 ? m0 : t.c0);
      t.base = t.base < 0 ? 0 : (t.base > dm.n ? dm.n : t.base);
    }
    const int at = t.base + lane;
    t.bound = at <= dm.n ? dm.clampN(__ldg(dm.cu + at)) : 0x7fffffff;
    if (dm.pre && at < dm.n) t.pre = __ldg(dm.pre + at);
    if (few) {
      t.c0 = __shfl_sync(0xffffffffu, t.bound, 0);
      t.cn = __shfl_sync(0xffffffffu, t.bound, dm.n);
    }
    r0 = m0 > t.c0 ? m0 : t.c0;
    r1 = m1 < t.cn - 1 ? m1 : t.cn - 1;
    if (r0 > r1) return t;
    t.mlo = t.base + __popc(__ballot_sync(0xffffffffu, t.bound <= r0)) - 1;
    t.mhi = t.base + __popc(__ballot_sync(0xffffffffu, t.bound <= r1)) - 1;
    s0 = span_of_lanes(t, dm.n, t.mlo, r0);
    if (t.mhi - t.base < 31) {
      s1 = span_of_lanes(t, dm.n, t.mhi, r1);
    } else {
      t.mhi = dm.find_warp(r1);
      s1 = dm.span(t.mhi, r1);
    }
  }
  if (r0 > r1) return t;
  const int a0 = kQueriesOfKeys ? dm.query_first(s0, r0) : dm.key_first(s0, r0);
  const int b1 = kQueriesOfKeys ? dm.query_last(s1, r1) : dm.key_last(s1, r1);
  if (a0 > b1) return t;
  t.begin = a0 / kTileN;
  t.end = b1 / kTileN + 1;
  if (r0 == m0 && r1 == m0 + kTileM - 1) {
    const int a = kQueriesOfKeys ? dm.query_first(s1, r1) : dm.key_first(s1, r1);
    const int b = kQueriesOfKeys ? dm.query_last(s0, r0) : dm.key_last(s0, r0);
    t.int_lo = (a + kTileN - 1) / kTileN;
    t.int_hi = (b + 1) / kTileN - 1;
  }
  return t;
}

// Longest walks first: of the 128-row tiles of a row of tokens (at most 32,
// lane k looks at tile k, and at most 31 documents), the one whose walk is the
// rank-th longest.  With packed documents the walks of the tiles differ widely
// and in no fixed order; started last, a long one is waited for.
template <bool kQueriesOfKeys>
__device__ __forceinline__ int tile_of_rank(const DocMask& dm, int rank) {
  const int lane = threadIdx.x & 31;
  const int tiles = (dm.N + kTileM - 1) / kTileM;
  DocTiles t{};
  t.bound = lane <= dm.n ? dm.clampN(__ldg(dm.cu + lane)) : 0x7fffffff;
  t.pre = dm.pre && lane < dm.n ? __ldg(dm.pre + lane) : 0;
  const int c0 = __shfl_sync(0xffffffffu, t.bound, 0);
  const int cn = __shfl_sync(0xffffffffu, t.bound, dm.n);
  const int m0 = lane * kTileM, m1 = m0 + kTileM - 1;
  const int r0 = m0 > c0 ? m0 : c0, r1 = m1 < cn - 1 ? m1 : cn - 1;
  int lo = -1, hi = -1;
  for (int k = 0; k <= dm.n; ++k) {
    const int b = __shfl_sync(0xffffffffu, t.bound, k);
    if (r0 >= b) lo = k;
    if (r1 >= b) hi = k;
  }
  const DocSpan s0 = span_of_lanes(t, dm.n, lo, r0), s1 = span_of_lanes(t, dm.n, hi, r1);
  const int a = kQueriesOfKeys ? dm.query_first(s0, r0) : dm.key_first(s0, r0);
  const int e = kQueriesOfKeys ? dm.query_last(s1, r1) : dm.key_last(s1, r1);
  const int n = lane >= tiles ? -1 : (r0 > r1 || a > e ? 0 : e / kTileN - a / kTileN + 1);
  int mine = 0;
  for (int k = 0; k < tiles; ++k) {
    const int other = __shfl_sync(0xffffffffu, n, k);
    mine += other > n || (other == n && k < lane) ? 1 : 0;
  }
  const unsigned at = __ballot_sync(0xffffffffu, lane < tiles && mine == rank);
  return at ? __ffs(at) - 1 : rank;
}

// The document of this thread's row i, one of the rows of t (a whole
// converged warp; other rows get none or a document that does not hold them).
__device__ __forceinline__ DocSpan DocMask::of_thread(const DocTiles& t, int i) const {
  if (!cu) return DocSpan{0, N, 0};
  int mlo = t.mlo < 0 ? 0 : t.mlo, mhi = t.mhi > n - 1 ? n - 1 : t.mhi;
  if (mhi - t.base < 31) {
    int m = mlo;
    for (int k = mlo + 1; k <= mhi; ++k)
      if (i >= __shfl_sync(0xffffffffu, t.bound, k - t.base)) m = k;
    return span_of_lanes(t, n, m, i);
  }
  while (mlo < mhi) {
    const int mid = (mlo + mhi + 1) >> 1;
    if (__ldg(cu + mid) <= i) mlo = mid;
    else mhi = mid - 1;
  }
  return span(mlo, i);
}

}  // namespace swa
