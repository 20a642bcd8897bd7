// swa_rope.cu -- rotary positions applied to a ragged batch of new tokens on
// their way into a paged KV cache.
//
// Token t of sequence b sits at position p = pos0[b] + t - cu[b].  With the
// angle a_i = p * inv_freq[i], each rotated pair (x1, x2) of a query or key
// head becomes (x1 cos a - x2 sin a, x2 cos a + x1 sin a); dimensions past
// the rotated ones, and the values, pass through.  Queries go to q_out, keys
// and values to row p % page_size of the sequence's page p / page_size.
//
// The work is a copy: every element is read and written once, so the bytes
// bound it, and for a decoding step the latency of the dependent reads
// (boundaries, position, page).  A block takes kTok tokens.  Its first
// elements are on their way into registers before their positions are looked
// up.  The angles of a token (the same for every head) are computed once, by
// one thread each, into shared memory: in fp64 up to the reduction to one
// turn (at position 131072 a fp32 product would be off by 2^-7 rad), then
// fp32 sin and cos.  Elements move as 16-byte vectors; one thread holds the
// two vectors whose elements pair up (or, for the adjacent-pair form, two
// neighbouring ones), eight angles for either form.
//
// Measured in a captured graph: 7564 tokens of 48 heads of 128 (186 MB) 37.3 us,
// 5.0 TB/s; one token of 64 sequences 3.8 us.  Two and three units in flight per thread, 1,
// 2 and 8 tokens a block, 128 to 512 threads and streaming loads and stores
// took 37 to 51 us for the former.
#include <cuda_runtime.h>

#include <cstdint>

#include "swa_internal.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kThreadsP = 256;

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride, qo_stride;  // elements between tokens
  const float* inv_freq;  // [rot / 2]
  const int32_t* cu;      // [B + 1]
  const int64_t* pos0;    // [B]
  const int32_t* table;   // [B, max_pages]
  uint16_t* q_out;
  uint16_t* k_pages;
  uint16_t* v_pages;
  int T, B, H, Hkv, rot, page_size, num_pages, max_pages;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Index of the last entry <= t of cu[0 .. n], by a whole warp.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, cnt = n + 1;
  while (cnt > 0) {
    const int step = (cnt + 31) / 32;
    const int idx = (lane + 1) * step - 1;
    const bool le = idx < cnt && __ldg(cu + lo + idx) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    const int rest = cnt - c * step;
    cnt = rest < step - 1 ? rest : step - 1;
  }
  return lo - 1;
}

// D: head size; kInter: rotated pairs are adjacent elements; kTok: tokens of
// a block; kU: units (pairs of vectors) a thread has in flight.
template <int D, bool kInter, int kTok, int kU>
__global__ void __launch_bounds__(kThreadsP) rope_append_kernel(const RopeParams p) {
  constexpr int kUnits = D / 16;  // pairs of 16-byte vectors per head
  __shared__ __align__(16) float2 cs[kTok][D / 2];  // (read as float4)
  __shared__ long long pos_s[kTok];   // position, or -1: not a token of any sequence
  __shared__ long long row_s[kTok];   // row of the page pool, or -1: not stored
  const int warp = threadIdx.x / 32;
  const int t0 = blockIdx.x * kTok;
  const int half = p.rot / 2;
  const int heads = p.H + 2 * p.Hkv;
  const int rot_units = p.rot / 16;
  const int n_tok = min(kTok, p.T - t0);
  // This thread's units: vectors u of the heads slot, slot + kSlots, ... of
  // the block's tokens one after another (no division on the way).
  constexpr int kSlots = kThreadsP / kUnits;
  const int u = threadIdx.x % kUnits;
  const int step_tk = kSlots / heads, step_hh = kSlots % heads;
  struct At {
    int tk, hh;
  };
  At at{(int)(threadIdx.x / kUnits) / heads, (int)(threadIdx.x / kUnits) % heads};
  auto next = [&]() -> At {
    const At r = at;
    at.tk += step_tk;
    at.hh += step_hh;
    if (at.hh >= heads) {
      at.hh -= heads;
      ++at.tk;
    }
    return r;
  };
  // a unit's two vectors: (u, u + rot / 16) in the half form's rotated part,
  // neighbours everywhere else
  auto turns_at = [&](int hh) { return hh < p.H + p.Hkv && u < rot_units; };
  auto second = [&](bool turn) { return (!kInter && turn) ? u + rot_units : 2 * u + 1; };
  auto first = [&](bool turn) { return (!kInter && turn) ? u : 2 * u; };
  struct Pair {
    uint4 a, b;
  };
  auto load = [&](const At& n) -> Pair {
    const long long t = t0 + n.tk;
    const uint16_t* src =
        n.hh < p.H ? p.q + t * p.q_stride + n.hh * D
                   : (n.hh < p.H + p.Hkv ? p.k + t * p.k_stride + (n.hh - p.H) * D
                                         : p.v + t * p.v_stride + (n.hh - p.H - p.Hkv) * D);
    const bool turn = turns_at(n.hh);
    return Pair{*reinterpret_cast<const uint4*>(src + first(turn) * 8),
                *reinterpret_cast<const uint4*>(src + second(turn) * 8)};
  };
  // What needs no position is on its way before the look-up: the frequency of
  // this thread's first angle and its first units.
  const float freq = threadIdx.x < kTok * half ? __ldg(p.inv_freq + threadIdx.x % half) : 0.f;
  At n[kU];
  Pair v[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    n[k] = next();
    if (n[k].tk < n_tok) v[k] = load(n[k]);
  }
  if (warp < kTok) {
    const int t = t0 + warp;
    long long pos = -1, row = -1;
    if (t < p.T) {
      const int b = find_seq(p.cu, p.B, t);
      if (b >= 0 && b < p.B) {
        const long long first = p.pos0[b];
        if (first >= 0) {
          pos = first + (t - __ldg(p.cu + b));
          if (pos < 0) pos = -1;  // (boundaries out of order)
          const long long lp = pos / p.page_size;
          if (pos >= 0 && lp < p.max_pages) {
            const int page = __ldg(p.table + (long long)b * p.max_pages + lp);
            if (page >= 0 && page < p.num_pages)
              row = (long long)page * p.page_size + pos % p.page_size;
          }
        }
      }
    }
    if ((threadIdx.x & 31) == 0) {
      pos_s[warp] = pos;
      row_s[warp] = row;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kTok * half; i += kThreadsP) {
    const int tk = i / half, f = i % half;
    const float w = i == (int)threadIdx.x ? freq : __ldg(p.inv_freq + f);
    const double turns = (double)pos_s[tk] * (double)w * 0.15915494309189535;
    float sn, cn;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &cn);
    cs[tk][f] = make_float2(cn, sn);
  }
  __syncthreads();
  while (n[0].tk < n_tok) {
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int tk = n[k].tk, hh = n[k].hh;
      if (tk >= n_tok || pos_s[tk] < 0) continue;
      const long long row = row_s[tk];
      if (hh >= p.H && row < 0) continue;
      const bool turn = turns_at(hh);
      uint32_t x[4] = {v[k].a.x, v[k].a.y, v[k].a.z, v[k].a.w};
      uint32_t y[4] = {v[k].b.x, v[k].b.y, v[k].b.z, v[k].b.w};
      if (turn) {
        const float4* c4 = reinterpret_cast<const float4*>(&cs[tk][8 * u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 w = c4[e];  // cos, sin of angles 2e and 2e + 1
          if (kInter) {
            // words 2e and 2e + 1 of the eight turn by those angles
            uint32_t* z = e < 2 ? x + 2 * e : y + 2 * (e - 2);
            const float l0 = lo16(z[0]), h0 = hi16(z[0]), l1 = lo16(z[1]), h1 = hi16(z[1]);
            z[0] = pack_bf16x2(l0 * w.x - h0 * w.y, h0 * w.x + l0 * w.y);
            z[1] = pack_bf16x2(l1 * w.z - h1 * w.w, h1 * w.z + l1 * w.w);
          } else {
            const float xl = lo16(x[e]), xh = hi16(x[e]), yl = lo16(y[e]), yh = hi16(y[e]);
            x[e] = pack_bf16x2(xl * w.x - yl * w.y, xh * w.z - yh * w.w);
            y[e] = pack_bf16x2(yl * w.x + xl * w.y, yh * w.z + xh * w.w);
          }
        }
      }
      uint16_t* dst = hh < p.H ? p.q_out + (t0 + tk) * p.qo_stride + hh * D
                               : (hh < p.H + p.Hkv ? p.k_pages + (row * p.Hkv + hh - p.H) * D
                                                   : p.v_pages +
                                                         (row * p.Hkv + hh - p.H - p.Hkv) * D);
      *reinterpret_cast<uint4*>(dst + first(turn) * 8) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(dst + second(turn) * 8) = make_uint4(y[0], y[1], y[2], y[3]);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      n[k] = next();
      if (n[k].tk < n_tok) v[k] = load(n[k]);
    }
  }
}

template <int D, bool kInter>
int launch(const RopeParams& p, cudaStream_t stream) {
  // Few tokens: one a block, so that a decoding step spreads over the SMs; more
  // share a block's look-ups and angles.  One / four a block with 48 heads of
  // 128: 4.9 / 6.4 us for 512 tokens, 7.8 / 7.7 for 768, 26 / 22 for 4096; 48
  // heads of 64: 3.7 / 4.2, 5.5 / 4.8, 16 / 10.5.
  if (p.T <= 512)
    rope_append_kernel<D, kInter, 1, 2><<<(unsigned)p.T, kThreadsP, 0, stream>>>(p);
  else
    rope_append_kernel<D, kInter, 4, 1><<<(unsigned)((p.T + 3) / 4), kThreadsP, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace

int launch_rope_append(const void* q, const void* k, const void* v, long long q_stride,
                       long long k_stride, long long v_stride, const float* inv_freq, int rot,
                       int interleaved, const int32_t* cu, const int64_t* pos0,
                       const int32_t* table, void* q_out, long long qo_stride, void* k_pages,
                       void* v_pages, int T, int B, int H, int Hkv, int D, int page_size,
                       int num_pages, int max_pages, cudaStream_t stream) {
  RopeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.qo_stride = qo_stride;
  p.inv_freq = inv_freq;
  p.cu = cu;
  p.pos0 = pos0;
  p.table = table;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pages = static_cast<uint16_t*>(k_pages);
  p.v_pages = static_cast<uint16_t*>(v_pages);
  p.T = T;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.rot = rot;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  if (D == 128)
    return interleaved ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  if (D == 64) return interleaved ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return SWA_ERR_UNSUPPORTED;
}

}  // namespace swa
