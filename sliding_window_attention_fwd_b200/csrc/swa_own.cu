// swa_own.cu -- the own keys of a decode behind a shared prefix: every
// sequence's positions past the prefix, read through its block table.
//
// One query vector per head meets the keys of one sequence, so the bytes of
// K and V bound it.  As in the ring decode (swa_decode_tc.cu) the keys take
// the MMA's M side:
//   S^T [128 keys x 16] = K_tile . Q^T,   O^T [D x 16] += V_tile^T . P^T
// with the GQA group's (up to 8) query vectors in the first columns.  The
// 16-row operands Q and P^T are stored as 8 rows only: the MMA reads the
// bytes behind them as rows 8-15, which fill columns that nobody reads.
//
// Tails are short (a few tiles), so a CTA per tail would spend most of its
// time filling and draining.  The CTAs stay (two per SM) and walk the items
// (part, kv head, sequence) i, i + grid, ...: the loads, the MMAs and the
// softmax run on across item borders (Q and O^T double buffered), and an
// item's result is written after the next one's first tile.
//
// Measured, with 8 kv heads of 128: 128 tails of 100 to 700 keys (210 MB) 54
// us, 3.9 TB/s (70 with a CTA per item and the ring decode's softmax; one CTA
// per SM with twice the ring 54); 64 tails of 1 to 256 keys (33 MB) 15 us (23;
// 18.5).  What is left is the chain of a tile (S^T, vote, exponentials, P^T, PV)
// and tails of uneven length.
//
// Warp roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer (and TMEM
// owner), warps 2-5 softmax (thread r: key r of a tile, dimension r of O^T).
// The softmax of a tile is the chain that bounds a CTA, so it is kept short: a
// tile is exponentiated against the running maximum unless some score exceeds
// it by 2^8 (one vote per tile, and only then a reduction over the four
// warps), and reductions of the group's values halve them at every shuffle.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "swa_internal.h"
#include "swa_ptx.cuh"
#include "swa_score.cuh"

namespace swa {
namespace {

constexpr int kTK = 128;                // keys per tile (MMA M)
constexpr int kQRows = 8;               // rows of the query and P^T operands
constexpr int kN = 16;                  // MMA N
constexpr int kSlice = kTK * 128;       // one 64-column slice of a 128-row tile (bytes)
constexpr float kLazy = 8.0f;           // log2 units

struct OwnParams {
  CUtensorMap tmQ;  // [B * H, D], boxes of 8 rows
  CUtensorMap tmK, tmV;
  const int64_t* pos;
  const int32_t* table;
  float* part_o;    // [parts, B, H, D]
  float* part_lse;  // [parts, B, H] natural log
  int* err;
  int B, H, Hkv, W, grp, parts, part_keys, items;
  int n_prefix, page_size, num_pages, max_pages;
  float scale_log2;
  CapCoefs cap;
  const float* slopes;
  int behind_prefix;  // launched while the prefix's kernel may still run
};

// At D = 64, O^T = V^T P^T keeps M = 128: rows 64-127 of its A operand are
// whatever follows the V tile in shared memory (the next ring slot, or the
// pad behind the last one), and nobody reads rows 64-127 of O^T.
template <int D>
struct OwnCfg {
  static constexpr int kTile = kTK * D * 2;            // one K or V tile
  static constexpr int kSlots = D == 128 ? 3 : 5;     // ring of tiles
  static constexpr int kPad = D == 128 ? 0 : kSlice;
  static constexpr int kQBytes = kQRows * D * 2;       // 8 rows, 1 KB per 64 columns
  static constexpr int kPBytes = kQRows * kTK * 2;     // P^T: 8 rows x 128 keys
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kSlots * kTile + kPad;
  static constexpr int kP = kQ + 2 * kQBytes;
  static constexpr int kBar = kP + 2 * kPBytes + 1024;  // (rows 8-15 of the last operand)
  // full[S], empty[S], s_full[2], p_full[2], o_done[2], q_full[2], q_free[2],
  // o_free[2], done
  static constexpr int kNumBars = 2 * kSlots + 13;
  static constexpr int kRed = kBar + kNumBars * 8;     // [2][warp][query] floats
  static constexpr int kMisc = kRed + 2 * 4 * kQRows * 4;
  static constexpr int kAlloc = kMisc + 16 + 1024;     // slack for 1024-byte alignment
  static constexpr int kThreads = 192;
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0, "operand alignment");
  static_assert(2 * (kAlloc + 1024) <= 233472, "two CTAs per SM");
};

// S^T buffers at columns 0 and 16, O^T at 32 and 48
constexpr uint32_t kTmemCols = 64;

// byte offset of (row, col) in an 8-row operand of 1 KB slices of 64 columns
__device__ __forceinline__ uint32_t off8(int row, int col) {
  const int c = col & 63;
  return (uint32_t)((col >> 6) * 1024 + row * 128 + (((c >> 3) ^ row) << 4) + ((c & 7) << 1));
}

// OR over the softmax threads, all of which get it.
__device__ __forceinline__ bool softmax_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Reduces kNQ values over the warp's 32 lanes: lane 16 b4 + 8 b3 + 4 b2 + ...
// gets the one numbered by its upper bits (kNQ = 8: 4 b4 + 2 b3 + b2).
template <int kNQ, class Op>
__device__ __forceinline__ float reduce_values(const float (&v)[kNQ], Op op) {
  static_assert(kNQ == 4 || kNQ == 8, "4 or 8 values");
  const int lane = threadIdx.x & 31;
  float a[kNQ];
#pragma unroll
  for (int n = 0; n < kNQ; ++n) a[n] = v[n];
  int o = 16;
#pragma unroll
  for (int w = kNQ / 2; w > 0; w >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int n = 0; n < w; ++n) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? a[n] : a[n + w], o);
      a[n] = op(up ? a[n + w] : a[n], other);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], o));
  return a[0];
}
// The value a lane gets, and whether it is the one to write it.
template <int kNQ>
__device__ __forceinline__ int reduced_index() {
  return (threadIdx.x & 31) / (32 / kNQ);
}
template <int kNQ>
__device__ __forceinline__ bool reduced_writer() {
  return (threadIdx.x & (32 / kNQ - 1)) == 0;
}

// One item: part `part` of the own keys of sequence b for kv head g.  Keys
// are counted from a64, the first seen position rounded down to 64 (so no
// 64-row box crosses a page): the part's are [s0, s1), those below lo masked.
struct Item {
  long long a64, pos;
  int b, g, part, lo, s0, s1, ntiles;
};

__device__ __forceinline__ Item item_of(const OwnParams& p, int i) {
  Item t;
  t.part = i % p.parts;
  i /= p.parts;
  t.g = i % p.Hkv;
  t.b = i / p.Hkv;
  t.pos = p.pos[t.b];
  long long a = t.pos - p.W + 1 > 0 ? t.pos - p.W + 1 : 0;
  if (a < p.n_prefix) a = p.n_prefix;
  t.a64 = a & ~63LL;
  t.lo = (int)(a - t.a64);
  // (of the positions the block table covers)
  const long long last = min(t.pos, (long long)p.max_pages * p.page_size - 1);
  const int n = last < a ? 0 : (int)(last - t.a64 + 1);
  t.s0 = t.part * p.part_keys;
  t.s1 = t.part == p.parts - 1 ? n : min(t.s0 + p.part_keys, n);
  t.ntiles = t.s1 > t.s0 ? (t.s1 - t.s0 + kTK - 1) / kTK : 0;
  return t;
}

// First key of tile k: from the last tile backwards, so that with a distance
// bias the nearest keys come first and the running maximum holds.
__device__ __forceinline__ int tile_key(const Item& t, int k) {
  return t.s0 + (t.ntiles - 1 - k) * kTK;
}

template <int D, int kNQ>
__global__ void __launch_bounds__(OwnCfg<D>::kThreads, 2)
    swa_own_kernel(const __grid_constant__ OwnParams p) {
  using C = OwnCfg<D>;
  constexpr int S_ = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);  // [slot]
  uint64_t* empty = full + S_;     // [slot]
  uint64_t* s_full = empty + S_;   // [tile & 1]: S^T ready
  uint64_t* p_full = s_full + 2;   // [tile & 1]: P^T written
  uint64_t* o_done = p_full + 2;   // [tile & 1]: its PV done
  uint64_t* q_full = o_done + 2;   // [item & 1]
  uint64_t* q_free = q_full + 2;   // [item & 1]: every S^T of the item computed
  uint64_t* o_free = q_free + 2;   // [item & 1]: O^T read out
  uint64_t* done = o_free + 2;     // every MMA done
  float* red = reinterpret_cast<float*>(smem + C::kRed);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

  // the merge may be scheduled once every CTA is here (it waits for the end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < S_; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&o_free[i], 128);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int step = gridDim.x;
  int n_items = 0;  // non-empty items of this CTA so far

  if (warp == 0) {
    // =========================== producer ===========================
    // ring load j: K of tile j / 2 (j even) or its V (j odd), tiles counted
    // over all items
    if (lane == 0) {
      prefetch_tensormap(&p.tmQ);
      prefetch_tensormap(&p.tmK);
      prefetch_tensormap(&p.tmV);
      int j = 0, last_q = -1;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < p.items; i += step) {
        const Item t = item_of(p, i);
        if (t.ntiles == 0) continue;
        const int qb = n_items & 1;
        if (n_items >= 2 &&
            !mbar_wait(&q_free[qb], (uint32_t)((n_items >> 1) - 1) & 1u, p.err, abort_flag))
          break;
        mbar_arrive_expect_tx(&q_full[qb], C::kQBytes);
        for (int cc = 0; cc < D / 64; ++cc)
          tma_load_4d(smem + C::kQ + qb * C::kQBytes + cc * 1024, &p.tmQ, &q_full[qb], cc * 64,
                      t.b * p.H + t.g * p.grp, 0, 0);
        last_q = n_items++;
        const int32_t* table = p.table + (long long)t.b * p.max_pages;
        // pages of tile k's two 64-row boxes (-1: read as zeros), looked up
        // one tile ahead
        auto page_at = [&](int k, int hh) -> int {
          const int idx0 = tile_key(t, k) + hh * 64;
          return k < t.ntiles && idx0 < t.s1 ? __ldg(table + (t.a64 + idx0) / p.page_size) : -1;
        };
        int ahead[2] = {page_at(0, 0), page_at(0, 1)};
        for (int k = 0; ok && k < t.ntiles; ++k) {
          int row[2];
          for (int hh = 0; hh < 2; ++hh) {
            row[hh] = ahead[hh] >= 0 && ahead[hh] < p.num_pages
                          ? ahead[hh] * p.page_size +
                                (int)((t.a64 + tile_key(t, k) + hh * 64) % p.page_size)
                          : -64;
            ahead[hh] = page_at(k + 1, hh);
          }
          for (int kv = 0; kv < 2; ++kv, ++j) {
            const int st = j % S_;
            if (j >= S_ &&
                !mbar_wait(&empty[st], (uint32_t)(j / S_ - 1) & 1u, p.err, abort_flag)) {
              ok = false;
              break;
            }
#ifdef SWA_TEST_WITHHOLD_TILE
            // failure-detection test build only: this K tile is never loaded,
            // so the issuer's bounded wait for it runs out
            if (j == 2 * SWA_TEST_WITHHOLD_TILE) continue;
#endif
            mbar_arrive_expect_tx(&full[st], C::kTile);
            for (int hh = 0; hh < 2; ++hh)
              for (int cc = 0; cc < D / 64; ++cc)
                tma_load_4d(smem + C::kRing + st * C::kTile + cc * kSlice + hh * (kSlice / 2),
                            kv ? &p.tmV : &p.tmK, &full[st], cc * 64, t.g, row[hh], 0);
          }
        }
      }
      if (*abort_flag) {  // leave no copy writing shared memory behind
#ifdef SWA_TEST_WITHHOLD_TILE
        const int skip = 2 * SWA_TEST_WITHHOLD_TILE;
#else
        const int skip = -1;
#endif
        drain_copies(full, S_, 0, j - 1, skip);
        drain_copies(q_full, 2, 0, last_q);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // =========================== MMA issuer ===========================
    // S^T of the next tile (the next item's first one, maybe) goes before PV
    // of this one: it reuses the S^T buffer of the tile before, whose P^T has
    // been waited for.
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kTK, kN, 0, 0);  // K-major A (K), K-major B (Q)
      const uint32_t idesc_o = idesc_bf16_f32(128, kN, 1, 0);  // MN-major A (V^T), K-major B (P^T)
      const uint32_t ring = smem_u32(smem + C::kRing);
      const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::kQ), 16, 1024);
      const uint64_t dp0 = sdesc_sw128(smem_u32(smem + C::kP), 16, 1024);
      const uint64_t dring_k = sdesc_sw128(ring, 16, 1024);
      const uint64_t dring_v = sdesc_sw128(ring, kSlice, 1024);
      constexpr uint64_t kSlotStep = C::kTile >> 4;
      // the walk over tiles: item `it` (its number among the non-empty ones
      // n), tile k of nt
      int it = blockIdx.x, n = 0, k = 0, nt = 0;
      auto seek = [&]() -> bool {  // to the first non-empty item from `it` on
        for (; it < p.items; it += step) {
          nt = item_of(p, it).ntiles;
          if (nt > 0) return true;
        }
        return false;
      };
      auto issue_s = [&](int tile) -> bool {  // of tile (n, k)
        const int j = 2 * tile, st = j % S_;
        if (k == 0 && !mbar_wait(&q_full[n & 1], (uint32_t)(n >> 1) & 1u, p.err, abort_flag))
          return false;
        if (!mbar_wait(&full[st], (uint32_t)(j / S_) & 1u, p.err, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dq = dq0 + (uint64_t)((n & 1) * C::kQBytes >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t ka = (uint64_t)(((s / 4) * kSlice + (s % 4) * 32) >> 4);
          const uint64_t kb = (uint64_t)(((s / 4) * 1024 + (s % 4) * 32) >> 4);
          mma_ss(tmem + 16u * (tile & 1), dring_k + st * kSlotStep + ka, dq + kb, idesc_s,
                 s > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[tile & 1]);
        tc_commit(&empty[st]);
        if (k == nt - 1) tc_commit(&q_free[n & 1]);
        return true;
      };
      bool more = seek();
      bool ok = more && issue_s(0);
      for (int tile = 0; ok && more; ++tile) {
        const int pn = n, pk = k;  // the tile whose PV is due
        if (++k == nt) {
          it += step;
          ++n;
          k = 0;
          more = seek();
        }
        if (more && !issue_s(tile + 1)) break;
        const int j = 2 * tile + 1, st = j % S_;
        if (!mbar_wait(&p_full[tile & 1], (uint32_t)(tile >> 1) & 1u, p.err, abort_flag) ||
            !mbar_wait(&full[st], (uint32_t)(j / S_) & 1u, p.err, abort_flag) ||
            (pk == 0 && pn >= 2 &&
             !mbar_wait(&o_free[pn & 1], (uint32_t)((pn >> 1) - 1) & 1u, p.err, abort_flag)))
          break;
        tc_fence_after();
        const uint64_t dp = dp0 + (uint64_t)((tile & 1) * C::kPBytes >> 4);
#pragma unroll
        for (int s = 0; s < kTK / 16; ++s) {
          const uint64_t ka = (uint64_t)((s * 2048) >> 4);  // 16 keys of the V tile
          const uint64_t kb = (uint64_t)(((s / 4) * 1024 + (s % 4) * 32) >> 4);
          mma_ss(tmem + 32u + 16u * (pn & 1), dring_v + st * kSlotStep + ka, dp + kb, idesc_o,
                 (pk > 0 || s > 0) ? 1u : 0u);
        }
        tc_commit(&o_done[tile & 1]);
        tc_commit(&empty[st]);
      }
      tc_commit(done);  // also on the abort path: TMEM quiescent before it is freed
    }
    __syncwarp();
  } else {
    // ============================ softmax ============================
    const int quad = warp & 3;       // TMEM lane quadrant
    const int r = quad * 32 + lane;  // key of the tile (S^T) / dimension (O^T)
    const int wi = warp - 2;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int nq = p.grp;
    const size_t rows = (size_t)p.B * p.H;
    const int my_n = reduced_index<kNQ>();
    bool ok = true;
    int tile = 0;  // over all items
    // the item whose result is still to be written: its sums, first row and
    // last tile
    float m_last[kNQ], l_last[kNQ];
    size_t row_last = 0;
    int tile_last = -1;
    // O / l and the lse of that item (the n-th): false when a wait gave up
    auto finish = [&](int n_item) -> bool {
      float* red_l = red + 4 * kNQ;
      const float mine = reduce_values<kNQ>(l_last, [](float x, float y) { return x + y; });
      if (reduced_writer<kNQ>()) red_l[wi * kNQ + my_n] = mine;
      const bool w = mbar_wait(&o_done[tile_last & 1], (uint32_t)(tile_last >> 1) & 1u, p.err,
                               abort_flag);
      if (!bar_red_and(1, 128, w)) return false;
      tc_fence_after();
      uint32_t ov[16];
      tmem_ld16(tmem + 32u + 16u * (n_item & 1) + lane_off, ov);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&o_free[n_item & 1]);
#pragma unroll
      for (int n = 0; n < kNQ; ++n) {
        if (n < nq) {
          const float l = red_l[n] + red_l[kNQ + n] + red_l[2 * kNQ + n] + red_l[3 * kNQ + n];
          if (D == 128 || r < D)
            p.part_o[(row_last + n) * D + r] =
                l == 0.f ? 0.f : __fdividef(__uint_as_float(ov[n]), l);
          if (r == 0)
            p.part_lse[row_last + n] = (m_last[n] + __log2f(l)) * 0.69314718055994531f;
        }
      }
      return true;
    };
    for (int i = blockIdx.x; ok && i < p.items; i += step) {
      const Item t = item_of(p, i);
      const size_t row0 = (size_t)t.part * rows + (size_t)t.b * p.H + (size_t)t.g * nq;
      if (t.ntiles == 0) {  // contributes nothing
        if (r < nq) p.part_lse[row0 + r] = -INFINITY;
        continue;
      }
      const uint32_t tO = tmem + 32u + 16u * (n_items & 1) + lane_off;
      float m_run[kNQ], lsum[kNQ], nslope2[kNQ];
#pragma unroll
      for (int n = 0; n < kNQ; ++n) {
        m_run[n] = -INFINITY;
        lsum[n] = 0.f;
        nslope2[n] = p.slopes && n < nq
                         ? -__ldg(p.slopes + t.g * nq + n) * 1.4426950408889634f
                         : 0.f;
      }
      for (int k = 0; k < t.ntiles; ++k, ++tile) {
        const int k0 = tile_key(t, k);  // the tile's first key
        const int idx = k0 + r;
        const bool valid = idx < t.s1 && idx >= t.lo;
        bool w_ok = true;
        if (k0 < t.lo || k0 + kTK > t.s1) {
          // rows of the pool that are not the sequence's may hold anything,
          // NaN included: their V rows become zeros before P = 0 meets them
          const int j = 2 * tile + 1, st = j % S_;
          w_ok = mbar_wait(&full[st], (uint32_t)(j / S_) & 1u, p.err, abort_flag);
          constexpr int kC16 = D / 8;
          const int below = t.lo > k0 ? t.lo - k0 : 0;
          const int past = t.s1 - k0 < kTK ? t.s1 - k0 : kTK;
          uint8_t* vt = smem + C::kRing + st * C::kTile;
          for (int u = r; w_ok && u < (below + kTK - past) * kC16; u += 128) {
            int row = u / kC16;
            row = row < below ? row : row - below + past;
            *reinterpret_cast<uint4*>(vt + (u % kC16 / 8) * kSlice + row * 128 + (u % 8) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        }
        w_ok = mbar_wait(&s_full[tile & 1], (uint32_t)(tile >> 1) & 1u, p.err, abort_flag) && w_ok;
        tc_fence_after();
        uint32_t sv[16];
        __syncwarp();
        tmem_ld16(tmem + 16u * (tile & 1) + lane_off, sv);
        tmem_wait_ld();
        float xs[kNQ];
        const float dist = (float)(t.pos - t.a64 - idx);
        if (p.cap.out > 0.f) {
          float big = 0.f;
#pragma unroll
          for (int n = 0; n < kNQ; ++n) big = fmaxf(big, fabsf(__uint_as_float(sv[n])));
          auto shape = [&](auto form) {
#pragma unroll
            for (int n = 0; n < kNQ; n += 2) {
              const float2 x =
                  form(p.cap, make_float2(__uint_as_float(sv[n]), __uint_as_float(sv[n + 1])),
                       make_float2(nslope2[n] * dist, nslope2[n + 1] * dist));
              xs[n] = x.x;
              xs[n + 1] = x.y;
            }
          };
          if (!__any_sync(0xffffffffu, valid && big > p.cap.vote))
            shape([](const CapCoefs& c, float2 s, float2 add) { return cap_small(c, s, add); });
          else
            shape([](const CapCoefs& c, float2 s, float2 add) { return cap_any(c, s, add); });
        } else {
#pragma unroll
          for (int n = 0; n < kNQ; ++n)
            xs[n] = fmaf(__uint_as_float(sv[n]), p.scale_log2, nslope2[n] * dist);
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
          xs[n] = valid && n < nq ? xs[n] : -INFINITY;
          grow = grow || xs[n] > m_run[n] + kLazy;
        }
        // one vote per tile: the running maxima hold, or not
        if (softmax_any(grow || !w_ok)) {
          const float mine = reduce_values<kNQ>(xs, [](float x, float y) { return fmaxf(x, y); });
          if (reduced_writer<kNQ>()) red[wi * kNQ + my_n] = mine;
          // (all four warps leave together when a wait of one gave up)
          if (!bar_red_and(1, 128, w_ok)) {
            ok = false;
            break;
          }
          float f[kNQ];
#pragma unroll
          for (int n = 0; n < kNQ; ++n) {
            const float m = fmaxf(fmaxf(red[n], red[kNQ + n]),
                                  fmaxf(red[2 * kNQ + n], red[3 * kNQ + n]));
            f[n] = 1.f;
            if (m > m_run[n] + kLazy) {
              f[n] = m_run[n] == -INFINITY ? 0.f : ex2_approx(m_run[n] - m);
              m_run[n] = m;
              lsum[n] *= f[n];
            }
          }
          if (k > 0) {  // O^T holds P V of the tiles before: complete, then scaled
            if (!__all_sync(0xffffffffu, mbar_wait(&o_done[(tile - 1) & 1],
                                                   (uint32_t)((tile - 1) >> 1) & 1u, p.err,
                                                   abort_flag)))
              ok = false;
            tc_fence_after();
            uint32_t ov[16];
            tmem_ld16(tO, ov);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < kNQ; ++n) ov[n] = __float_as_uint(__uint_as_float(ov[n]) * f[n]);
            tmem_st16(tO, ov);
            tmem_wait_st();
          }
        }
        // P^T buffer tile & 1 was last read by PV(tile - 2)
        if (tile >= 2 && !mbar_wait(&o_done[tile & 1], (uint32_t)((tile - 2) >> 1) & 1u, p.err,
                                    abort_flag))
          ok = false;
        uint8_t* pbuf = smem + C::kP + (tile & 1) * C::kPBytes;
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
          const float pr = ex2_approx(xs[n] - (m_run[n] == -INFINITY ? 0.f : m_run[n]));
          lsum[n] += pr;
          *reinterpret_cast<__nv_bfloat16*>(pbuf + off8(n, r)) = __float2bfloat16_rn(pr);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[tile & 1]);
        if (k == 0 && tile_last >= 0) {
          if (!finish(n_items - 1)) {
            ok = false;
            break;
          }
        }
      }
      ok = bar_red_and(1, 128, ok);  // (the warps go on, or leave, together)
      if (!ok) break;
#pragma unroll
      for (int n = 0; n < kNQ; ++n) {
        m_last[n] = m_run[n];
        l_last[n] = lsum[n];
      }
      row_last = row0;
      tile_last = tile - 1;
      ++n_items;
    }
    if (bar_red_and(1, 128, ok) && tile_last >= 0) finish(n_items - 1);
  }

  // ---- teardown: no MMA in flight, then free TMEM
  if (warp == 1 && lane == 0) {
    volatile int no_abort = 0;
    mbar_wait(done, 0, nullptr, &no_abort, 100000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // this grid's end is also the end of the prefix's (the merge waits for this
  // grid alone)
  if (blockIdx.x == 0 && p.behind_prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int kNQ>
int launch(const SharedArgs& a, const SharedPlan& pl, float* part_o, float* part_lse, bool behind,
           cudaStream_t stream) {
  using C = OwnCfg<D>;
  static std::atomic<unsigned long long> attr{0};
  if (!smem_attr_once(reinterpret_cast<const void*>(swa_own_kernel<D, kNQ>), C::kAlloc, attr))
    return SWA_ERR_CUDA;
  OwnParams p;
  std::memset(&p, 0, sizeof(p));
  p.tmK = *a.tmK;
  p.tmV = *a.tmV;
  const uint64_t rows = (uint64_t)a.B * a.H;
  const uint64_t dims[4] = {(uint64_t)D, rows, 1, 1};
  const uint64_t strides[3] = {(uint64_t)D * 2, rows * D * 2, rows * D * 2};
  const uint32_t box[4] = {64, kQRows, 1, 1};
  if (encode_tiled(&p.tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims,
                   strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return SWA_ERR_CUDA;
  p.pos = a.pos;
  p.table = a.table;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.err = device_error_word();
  if (!p.err) return SWA_ERR_CUDA;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.W = a.W;
  p.grp = a.H / a.Hkv;
  p.parts = pl.own_parts;
  p.part_keys = pl.part_keys;
  p.n_prefix = a.n_prefix;
  p.page_size = a.page_size;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.cap = cap_coefs(a.softcap, a.scale);
  p.slopes = a.slopes;
  p.behind_prefix = behind;
  const long long items = (long long)a.B * a.Hkv * pl.own_parts;
  if (items > 0x7fffffffLL - 4096) return SWA_ERR_UNSUPPORTED;
  p.items = (int)items;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 2 * pl.sms ? items : 2 * pl.sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, swa_own_kernel<D, kNQ>, p) == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace

int launch_own(const SharedArgs& a, const SharedPlan& pl, float* part_o, float* part_lse,
               bool behind, cudaStream_t stream) {
  // (groups of up to four take the form that carries four values)
  const bool four = a.H / a.Hkv <= 4;
  if (a.D == 128)
    return four ? launch<128, 4>(a, pl, part_o, part_lse, behind, stream)
                : launch<128, 8>(a, pl, part_o, part_lse, behind, stream);
  if (a.D == 64)
    return four ? launch<64, 4>(a, pl, part_o, part_lse, behind, stream)
                : launch<64, 8>(a, pl, part_o, part_lse, behind, stream);
  return SWA_ERR_UNSUPPORTED;
}

}  // namespace swa
