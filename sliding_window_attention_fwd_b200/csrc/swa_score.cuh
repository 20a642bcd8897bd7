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

// tanh(u) for a pair with |u| <= 1, on the FMA pipe: u times a degree-5
// polynomial in u^2, fitted to tanh(x)/x on [0, 1] by iterated weighted
// least squares (relative error 7e-7 evaluated in fp32).  A tanh from MUFU
// (error 2^-11) would be worth 2 % of a probability at a cap of 50, and the
// exact form below costs two MUFU operations an element, on the unit that the
// exponentials already fill.
__device__ __forceinline__ float2 tanh_poly2(float2 u) {
  constexpr float kT0 = 0.9999994039535522f, kT1 = -0.3332904279232025f,
                  kT2 = 0.13281433284282684f, kT3 = -0.051605675369501114f,
                  kT4 = 0.016743116080760956f, kT5 = -0.003067060373723507f;
  const float2 z = mul2(u, u);
  float2 q = fma2(make_float2(kT5, kT5), z, make_float2(kT4, kT4));
  q = fma2(q, z, make_float2(kT3, kT3));
  q = fma2(q, z, make_float2(kT2, kT2));
  q = fma2(q, z, make_float2(kT1, kT1));
  q = fma2(q, z, make_float2(kT0, kT0));
  return mul2(u, q);
}

// tanh(u) for any u: the polynomial, or past |u| = 1 the identity tanh |u| =
// 1 - 2 / (e^{2|u|} + 1) (absolute error about 2e-7 there; +-1 for infinite
// u, NaN for NaN).
__device__ __forceinline__ float tanh_any(float u) {
  if (fabsf(u) > 1.f) {
    const float e = ex2_approx(fabsf(u) * 2.8853900817779268f);
    return copysignf(1.f - __fdividef(2.f, e + 1.f), u);
  }
  return tanh_poly2(make_float2(u, u)).x;
}

// The documents of one row of tokens.
struct DocSpan {
  int start, end;  // positions [start, end); start >= end: none (padding)
  int pre;         // end of the prefix (<= start: none)
};

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
  // The document of row i, for a whole warp at once.
  __device__ __forceinline__ DocSpan of_warp(int i, int* m) const {
    if (!cu) {
      *m = 0;
      return DocSpan{0, N, 0};
    }
    *m = find_warp(i);
    return span(*m, i);
  }
  // The document of this thread's row i, known to be one of mlo..mhi.
  __device__ __forceinline__ DocSpan of_thread(int i, int mlo, int mhi) const {
    if (!cu) return DocSpan{0, N, 0};
    mlo = mlo < 0 ? 0 : mlo;
    mhi = mhi > n - 1 ? n - 1 : mhi;
    while (mlo < mhi) {
      const int mid = (mlo + mhi + 1) >> 1;
      if (__ldg(cu + mid) <= i) mlo = mid;
      else mhi = mid - 1;
    }
    return span(mlo, i);
  }
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
};

template <bool kQueriesOfKeys>
__device__ __forceinline__ DocTiles doc_tiles(const DocMask& dm, int m0, int m1) {
  DocTiles t;
  t.c0 = dm.first();
  t.cn = dm.past();
  t.begin = t.end = 0;
  t.int_lo = 1;
  t.int_hi = 0;
  t.mlo = 0;
  t.mhi = -1;
  const int r0 = m0 > t.c0 ? m0 : t.c0;
  const int r1 = m1 < t.cn - 1 ? m1 : t.cn - 1;
  if (r0 > r1) return t;
  const DocSpan s0 = dm.of_warp(r0, &t.mlo), s1 = dm.of_warp(r1, &t.mhi);
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

}  // namespace swa
