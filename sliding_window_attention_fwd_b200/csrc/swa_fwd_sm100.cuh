// swa_fwd_sm100.cuh -- the kernel of the fused bf16 sliding-window attention forward for B200.
//
// A CTA computes the same 128-row query tile of one (batch, residue class)
// for NSLOT (1 or 2) query heads.  Only the key tiles the band-aware
// scheduler lists are visited (page "别再只加Mask了", §1: out-of-window
// pairs are skipped, not masked; "空洞滑窗机制" §四: dilation handled on
// dense tiles of whole blocks), followed, when global tokens exist, by
// tiles of gathered global keys (aiqz.cc page, "全局注意力token").
//
// Two query heads per CTA let the tensor core alternate between them:
// while one softmax warpgroup turns S into P for head 0, the MMAs of head 1
// run, and the other way round.  The two heads share a kv head (GQA: one
// K/V stream; the kernel can also stream two kv heads, NSTREAM = 2).
// Without such a pair a CTA takes one head; at D = 64 two of those CTAs
// share an SM and alternate the same way.
//
// Warp roles (warpgroup 0 = warps 0-3; warpgroup 1 + s = softmax of slot s):
//   warp 0     producer: TMA loads of the Q tiles once and of the K/V tiles
//              into a shared-memory ring (128-byte swizzle); global keys are
//              gathered with plain 16-byte loads into the same layout;
//   warp 1 + s MMA issuer of slot s (warp 1 also owns the 512 TMEM columns):
//                S_s  = Q_s K^T     tcgen05.mma, operands in smem, fp32 in
//                                   TMEM, in two 64-key halves
//                O_s += P_s V       tcgen05.mma, P (bf16) read from TMEM where
//                                   it overwrote S_s, V from smem
//              Tile j's P is kept in the columns of its early half (j & 1);
//              the early half of tile j+1 goes to the other columns as soon
//              as the softmax has read them, so it is ready when the softmax
//              finishes tile j, and only the late half waits for PV(j).  PV
//              itself is issued in two key halves: the early half's share as
//              soon as its P is written, so only a quarter-tile of PV sits
//              between the end of tile j's softmax and S of tile j+1's late
//              half.  One issuer per slot, each on its own SM sub-partition:
//              a single issuer sharing a sub-partition with two busy softmax
//              warps gets too few issue slots to keep the tensor core fed;
//   softmax    thread t of warpgroup 1+s owns query row t of slot s: row max
//              and row sum are thread-local tree reductions, no shuffles.
//              Element masks only on tiles the scheduler marks as edges.
//              Scores are read from TMEM 64 columns at a time and turned into
//              P against the current running max while the half's max is
//              found (the max changes rarely); a max that grows by more than
//              2^8 is adopted before the next tile by rescaling O and l, one
//              that jumps by more than 2^64 at once (the half is redone), and
//              the final O / l is exact either way.  With two slots the
//              producer/issuer warpgroup gives registers to the softmax
//              warpgroups (setmaxnreg).  (A thread then spills at most 32 bytes,
//              but 260 to 400 in the forms that go from item to item.)
// Per row: out = O / l (bf16), lse = m + ln l (fp32).
//
// Two more forms share the roles, the pipeline and the tiles:
//  * shaped scores over packed documents (kind 3, swa_score.cuh): the key range
//    of a tile comes from the documents of its rows, and the softmax warps turn
//    raw products into capped and biased scores before the exponentials.  The
//    tensor core has to do 4 D operations a pair as before; the cap adds five
//    operations a score on the FMA pipe.  Tensor pipe and MUFU stay under half and
//    1.5 to 1.8 instructions of 4 issue a cycle: what bounds the form is the
//    latency of each phase of two softmax warps per sub-partition.  A cap alone
//    bounds the scores, and the running maximum falls away (kFixedRef).  Causal
//    window of 4096 at N = 8192, H 32 / Hkv 8, D = 128: 375 us plain, 435 to 460
//    with a document table, 440 to 455 capped at 50, 465 to 480 with a distance
//    bias, 530 to 560 with both; with many scores past half the cap (a cap of 3)
//    900 to 920: two more MUFU operations each, and both forms of the cap.
//  * the shared prefix of a decode (kind 4): the rows of an item are every
//    sequence's query vectors of one kv head, the keys the prefix's pages, and
//    the key walk is split until the SMs are full.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "swa_internal.h"
#include "swa_ptx.cuh"
#include "swa_sched.cuh"
#include "swa_score.cuh"

namespace swa {
namespace {

constexpr int kMaxClasses = 8;   // residue classes per launch (tensor maps in params)
constexpr int kChunkBytes = kTileM * 128;  // one 64-column slice of a 128-row tile
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// of the shaped forms, whose rows begin against 0 (P <= 2^32 is as good in bf16
// and fp32)
constexpr float kRescaleShaped = 32.0f;
// Scores that a cap holds within this many log2 units of 0 (a cap of 50 is 72.1)
// need no running maximum: every exponential is taken against 0, and P, l and O
// stay inside fp32 (and P in bf16, which has its exponents): of its 2^127, 2^73 for P
// leave 2^54 for the number of keys times the size of V.  That is the choice; a
// bound of 100 would leave 2^27, too little for a million keys.  Larger caps take
// the form with a bias, its slopes zero, at the price of one: a cap of
// 60 takes 525 us instead of 444 for the window above.
constexpr float kFixedRef = 73.0f;
struct FwdParams {
  CUtensorMap tmQ[kMaxClasses];
  CUtensorMap tmK[kMaxClasses];
  CUtensorMap tmV[kMaxClasses];
  CUtensorMap tmKf;  // K and V over the whole sequence (rows in position order):
  CUtensorMap tmVf;  // the keys of the global query rows
  uint16_t* out;
  float* lse;
  const int32_t* G;
  const uint16_t* q_raw;
  const uint16_t* k_raw;
  const uint16_t* v_raw;
  int* err;
  int n_global;
  int B, H, Hkv, N;
  int L, R, d, bs;
  int class0, nclass;
  // Global query rows: the first n_gitems CTAs of the grid each take up to
  // 128 global rows (a "global tile") of one (batch, head pair), n_gq_tiles
  // tiles per pair, and attend every key of the sequence (causal: up to the
  // row).  The band CTAs leave those rows to them.
  int n_gitems, n_gq_tiles;
  int qtile_prefix[kMaxClasses + 1];
  int qt_base;  // first query tile of the launch (a row-range launch of one class)
  int Mv[kMaxClasses];
  float scale_log2;
  // Query window (chunked append; pos0 == NULL otherwise): the Mq query
  // rows are local rows 0..Mq-1 of q / out / lse ([B, Mq, H, D] /
  // [B, H, Mq]) and sit at virtual rows q0.. of the key sequence, whose
  // row v holds position pos0[b] - (win - 1) + v; rows of negative
  // positions (v < win - 1 - pos0[b]) are masked.
  const int64_t* pos0;
  int q0, Mq, win;
  // In place (win % 64 == 0): the keys are read from the ring (tmK[0],
  // tmV[0]: [B, win, Hkv, D]) and the chunk (tmKf, tmVf: [B, Mq, Hkv, D])
  // without a staged copy.  Per batch, with s_first = (pos0 - win + 1) mod
  // win the slot of the window's oldest position and hs = s_first mod 64,
  // virtual key row v < cs reads ring slot (s_first - hs + v) mod win and
  // row v >= cs chunk row v - cs, where cs = the multiple of 64 at or above
  // hs + win - 1: every 64-row box then lies inside one source without
  // wrapping.  The history sits at rows [hs, hs + win - 1), the rows
  // [hs + win - 1, cs) between it and the chunk are masked, and chunk row c
  // (virtual row cs + c) sees rows [hs + c, cs + c].
  int inplace;
  // Stacked heads (query window, two slots, Mq <= 64, GQA group a multiple
  // of 4): a slot's 128-row tile holds two heads of the group, rows 0-63
  // the first one's tokens and rows 64-127 the second one's, so the four
  // heads of a CTA share one key walk with no empty query rows.
  int stack;
  // Split key walks (query window): each item's key tiles are cut into
  // nsplit contiguous parts, one CTA each, which write O / l (fp32) and
  // lse to part_o [nsplit, B, H, Mq, D] and part_lse [nsplit, B, H, Mq];
  // a merge kernel combines them.  nsplit == 1: the output is written
  // directly.
  int nsplit;
  float* part_o;
  float* part_lse;
  // Paired parts (nsplit == 2, launched as clusters of two CTAs whose rank
  // is the part): the two parts merge through distributed shared memory and
  // write out / lse themselves, with no partials and no merge kernel.
  // ring_store (paired, in place, one query tile, every head of the kv head
  // in one item, so the cluster holds every reader of the kv head's ring
  // rows): once both parts' MMAs are done, the chunk's keys (part 0) and
  // values (part 1) enter their ring slots (pos0 + c) % win.
  int pair;
  int ring_store;
  uint4* k_ring;
  uint4* v_ring;
  const uint4* kn_raw;
  const uint4* vn_raw;
  // Shaped scores (swa_score.cuh): the cap, the bias' slopes [H], documents.
  CapCoefs cap;
  const float* slopes;
  const int32_t* cu_docs;  // [B, n_docs + 1] (NULL: one document)
  const int32_t* doc_pre;  // [B, n_docs] (NULL: no prefixes)
  int n_docs;
  // Shared prefix (decode): the keys are the N = n_prefix positions in the
  // pages table[0 ..] of a pool (tmK[0] / tmV[0]: [pool rows, Hkv, D]); query
  // row R of a kv head is its head R % grp of sequence R / grp, at position
  // pos0[b]; it sees the prefix keys j <= pos0[b], and unless keep only those
  // of its window, j > pos0[b] - win.  Split into nsplit parts like a query
  // window, written to part_o [nsplit, B, H, D] / part_lse.
  const int32_t* table;
  int page_size, num_pages, keep;
};

template <int D, int NSLOT, int NSTREAM, int KIND, int SC = 0>
struct Cfg {
  static constexpr int kTile = D / 64 * kChunkBytes;        // 128 rows x D bf16
  static constexpr int kStageBytes = 2 * NSTREAM * kTile;   // K and V of every stream
  static constexpr int kQBytes = NSLOT * kTile;
  // one head at D = 64 is small enough for two CTAs per SM (shared memory,
  // TMEM and, with the register split below, registers), so one CTA's fill
  // and drain overlap the other's tiles
  static constexpr int kMinBlocks = (NSLOT == 1 && (D == 64 || KIND >= 3)) ? 2 : 1;
  static constexpr int kBudget = kMinBlocks == 2 ? 96 * 1024 : 224 * 1024;
  // TMEM: S/P of slot s at [128 s, 128 s + 128), O of slot s at kOcol + D s
  static constexpr uint32_t kOcol = 128u * NSLOT;
  static constexpr uint32_t kTmemCols = kOcol + NSLOT * D <= 256 ? 256u : 512u;
  static constexpr int kFit = (kBudget - kQBytes) / kStageBytes;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static_assert(kStages >= 1, "K/V ring");
  static constexpr int kThreads = 128 * (1 + NSLOT);
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQBytes;
  static constexpr int kBar = kRing + kStages * kStageBytes;
  // full_q, full_k[S], empty_k[S], full_v[S], empty_v[S],
  // se_full[2], sl_full[2], l_free[2], p_full[2], o_done[2], o_final[2],
  // pe_full[2], oe_done[2], peer_free, xfer
  // documents, two slots, no bias: one CTA per SM goes from item to item (kind 3 at
  // D = 128, per item and chained: 8192 tokens in 8 documents 134 and 110-122 us, in 7
  // ragged ones capped 156 and 150, window of 700 160 and 149; with a bias the loop
  // gets longer and a window of 4096 463 and 495.  With one slot two CTAs per SM
  // already overlap, D = 64 capped 133 and 148.)
  static constexpr bool kChain = KIND == 3 && NSLOT == 2 && SC < 2;
  // kChain: q_free, o_free[2], done[2], item_full[2], item_free[2], claimed
  static constexpr int kNumBars = 1 + 4 * kStages + 18 + (kChain ? 10 : 0);
  static constexpr int kMisc = kBar + kNumBars * 8;
  // kChain: the answer to a claim, and two items (kItemInts integers each)
  static constexpr int kClaim = (kMisc + 16 + 15) / 16 * 16;
  static constexpr int kItemInts = 16 + 64;
  static constexpr int kItems = kClaim + 16;
  static constexpr int kTotal = kChain ? kItems + 2 * kItemInts * 4 : kMisc + 16;
  static constexpr int kAlloc = kTotal + 1024;  // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "shared memory budget");
  // paired parts: the half of O the other part writes (fp32, NSLOT x 128
  // rows of D / 2) and its (m, l) per row land in the ring
  static constexpr int kRxO = NSLOT * 128 * (D / 2) * 4;
  static_assert(kRxO + NSLOT * 128 * 8 <= kStages * kStageBytes, "pair exchange area");
};

// KIND (compile-time, so each form carries only its own code): 0 band (and
// token/block dilation) only; 1 the query window of a chunked append; 2 the
// band plus global tokens (global-key tiles and global query rows); 3 the
// band with shaped scores and documents; 4 the shared prefix of a decode.
// SC (kinds 3 and 4): 1 a tanh cap, 2 a distance bias, 3 both.
template <int D, int NSLOT, int NSTREAM, int KIND, int SC = 0>
__global__ void __launch_bounds__(Cfg<D, NSLOT, NSTREAM, KIND, SC>::kThreads,
                                  Cfg<D, NSLOT, NSTREAM, KIND, SC>::kMinBlocks)
    swa_fwd_sm100_kernel(const __grid_constant__ FwdParams p) {
  using C = Cfg<D, NSLOT, NSTREAM, KIND, SC>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* full_q = bars;
  uint64_t* full_k = bars + 1;
  uint64_t* empty_k = full_k + kStages;
  uint64_t* full_v = empty_k + kStages;
  uint64_t* empty_v = full_v + kStages;
  uint64_t* se_full = empty_v + kStages;  // [slot]: early half of S ready
  uint64_t* sl_full = se_full + 2;        // [slot]: late half of S ready
  uint64_t* l_free = sl_full + 2;         // [slot]: late half of S read out
  uint64_t* p_full = l_free + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* o_final = o_done + 2;
  uint64_t* pe_full = o_final + 2;  // [slot]: P of the early half written
  uint64_t* oe_done = pe_full + 2;  // [slot]: PV of the early half done
  // paired parts: the other part's MMAs are done (its ring may be
  // written); the other part's half of O and (m, l) have landed here
  uint64_t* peer_free = oe_done + 2;
  uint64_t* xfer = peer_free + 1;
  // kChain: every QK of an item done; its O read out [slot]; every MMA done
  // [slot]; a further item described / read [item & 1]; the claim answered
  uint64_t* q_free = xfer + 1;
  uint64_t* o_free = q_free + 1;
  uint64_t* mma_done = o_free + 2;
  uint64_t* item_full = mma_done + 2;
  uint64_t* item_free = item_full + 2;
  uint64_t* claimed = item_free + 2;
  int* items = reinterpret_cast<int*>(smem + C::kItems);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  // ---- work item: the global tiles first (each walks the whole sequence),
  // then (class, q tile, batch, head pair) with heavy (late) tiles first
  constexpr bool qwin = KIND == 1;
  const bool stack = qwin && NSLOT == 2 && p.stack;
  const int npair = stack ? p.H / (2 * NSLOT) : (p.H + NSLOT - 1) / NSLOT;
  int x = blockIdx.x;
  constexpr bool glob = KIND == 2;
  constexpr bool docs = KIND == 3;
  constexpr bool chain = C::kChain;
  constexpr bool shared = KIND == 4;
  constexpr bool scored = docs || shared;
  // the own keys' kernel reads nothing of this one's: it may start with it
  if (shared) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool gitem = glob && x < p.n_gitems;
  if (glob && !gitem) x -= p.n_gitems;
  int sp = 0;  // part of a split key walk
  if (qwin || shared) {
    sp = x % p.nsplit;
    x /= p.nsplit;
  }
  int hp = shared ? 0 : x % npair;
  x /= shared ? 1 : npair;
  const int g_kv = shared ? x % p.Hkv : 0;
  x /= shared ? p.Hkv : 1;
  int b = shared ? 0 : x % p.B;
  x /= shared ? 1 : p.B;
  int cl = 0, qt = 0, gq0 = 0, gcnt = 0;
  const int sr0 = shared ? x * NSLOT * kTileM : 0;  // first query row of this item
  // the item's query rows (zeros past the last), all loads in flight at once
  // while the key range is found
  constexpr int kC16 = D / 8;  // 16-byte chunks per row; also chunks per thread
  uint4 q_val[shared ? kC16 : 1];
  if (shared && threadIdx.x >= 128) {
    const int grp_ = p.H / p.Hkv;
#pragma unroll
    for (int u = 0; u < kC16; ++u) {
      const int idx = (int)threadIdx.x - 128 + u * 128 * NSLOT;
      const int R = sr0 + idx / kC16, c16 = idx % kC16;
      q_val[shared ? u : 0] = make_uint4(0u, 0u, 0u, 0u);
      if (R < p.B * grp_)
        q_val[shared ? u : 0] = __ldg(reinterpret_cast<const uint4*>(
            p.q_raw + ((size_t)(R / grp_) * p.H + (size_t)g_kv * grp_ + R % grp_) * D + c16 * 8));
    }
  }
  if (shared) {
  } else if (gitem) {
    gq0 = x * kTileM;  // first global row of this tile
    gcnt = min(kTileM, p.n_global - gq0);
  } else {
    const int jt = p.qtile_prefix[p.nclass] - 1 - x;
    while (cl + 1 < p.nclass && p.qtile_prefix[cl + 1] <= jt) ++cl;
    qt = jt - p.qtile_prefix[cl] + p.qt_base;
  }
  const int c = p.class0 + cl;
  const int grp = p.H / p.Hkv;
  int head[NSLOT], kvh[NSLOT];
  bool slot_ok[NSLOT];
#pragma unroll
  for (int s = 0; s < NSLOT; ++s) {
    // stacked: slot s holds heads head[s] (rows 0-63) and head[s] + 1
    head[s] = stack ? hp * 2 * NSLOT + 2 * s : hp * NSLOT + s;
    slot_ok[s] = head[s] < p.H;
    if (!slot_ok[s]) head[s] = p.H - 1;
    kvh[s] = head[s] / grp;
    if (shared) {
      slot_ok[s] = sr0 + s * kTileM < p.B * grp;
      kvh[s] = g_kv;
    }
  }
  // in-place query window: per-batch key layout (see FwdParams::inplace)
  const bool inplace = qwin && p.inplace;
  int ip_hs = 0, ip_cs = 0, ip_base = 0;
  if (inplace) {
    const int W = p.win;
    long long sf = (p.pos0[b] - W + 1) % W;
    if (sf < 0) sf += W;
    ip_hs = (int)sf & 63;
    ip_cs = ip_hs <= 1 ? W : W + 64;
    ip_base = (int)sf - ip_hs;  // ring slot of virtual row 0, a multiple of 64
  }
  const Geometry g = inplace ? make_geometry(ip_cs + p.Mq, ip_cs - ip_hs, 0, 1, 0)
                             : make_geometry(p.N, p.L, p.R, p.d, p.bs);
  // a global tile's keys are the physical rows of the sequence
  const int Mv = gitem ? p.N : (inplace ? ip_cs + p.Mq : p.Mv[cl]);
  const int Mq = qwin ? p.Mq : (shared ? kTileM : Mv);  // query rows (local; stacked: tokens)
  const int q0 = qwin ? (inplace ? ip_cs : p.q0) : 0;  // virtual row of local query row 0
  const int qm0 = q0 + qt * kTileM;
  const int qm1 = q0 + min(qt * kTileM + kTileM - 1, Mq - 1);
  TileRange tr;
  DocTiles dt{};
  int seen_lo = 0, seen_hi = 0;  // shared prefix: the keys [lo, hi) that rows of the item see
  DocMask dm{docs && p.cu_docs ? p.cu_docs + (size_t)b * (p.n_docs + 1) : nullptr,
             docs && p.doc_pre ? p.doc_pre + (size_t)b * p.n_docs : nullptr, p.n_docs, p.N, p.L,
             p.R};
  if (docs) {
    dt = doc_tiles<false>(dm, qm0, qm1);
    tr.kv_begin = dt.begin;
    tr.kv_end = dt.end;
  } else if (shared) {
    // the tiles any of the item's rows sees: the sequences [b0, b1]
    const int b0 = sr0 / grp, b1 = min(sr0 + NSLOT * kTileM, p.B * grp) - 1;
    int lo = p.N, hi = -1;
    for (int bb = b0 + lane; bb <= b1 / grp; bb += 32) {
      const long long pb = p.pos0[bb];
      if (pb < 0) continue;
      const long long first = p.keep || pb < p.win ? 0 : pb - p.win + 1;
      lo = first < lo ? (int)first : lo;
      hi = max(hi, pb < p.N - 1 ? (int)pb : p.N - 1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    seen_lo = lo;
    seen_hi = hi + 1;
    tr.kv_begin = lo / kTileN;
    tr.kv_end = hi >= lo ? hi / kTileN + 1 : tr.kv_begin;
    const int n = tr.kv_end - tr.kv_begin;
    const int part = (n + p.nsplit - 1) / p.nsplit;
    const int a = tr.kv_begin + sp * part;
    const int z = tr.kv_end;
    tr.kv_begin = min(a, z);
    tr.kv_end = min(a + part, z);
  } else if (gitem) {
    // every key tile (causal: up to the tile's last, i.e. largest, global row)
    int last = __ldg(p.G + gq0 + gcnt - 1);
    last = last < 0 ? 0 : (last >= p.N ? p.N - 1 : last);
    tr.kv_begin = 0;
    tr.kv_end = p.R == 0 ? last / kTileN + 1 : (p.N + kTileN - 1) / kTileN;
  } else {
    tr = tile_range_rows(g, Mv, qm0, qm1);
    if (qwin && p.nsplit > 1) {
      // this CTA's part of the key walk
      const int n = tr.kv_end - tr.kv_begin;
      const int part = (n + p.nsplit - 1) / p.nsplit;
      const int a = tr.kv_begin + sp * part;
      tr.kv_begin = min(a, tr.kv_end);
      tr.kv_end = min(a + part, tr.kv_end);
    }
  }
  int lo_b = 0;  // first key row holding a real position (query window only)
  if (qwin) {
    const long long pb = p.pos0[b];
    const long long lb = (long long)(p.win - 1) - pb + ip_hs;
    lo_b = lb <= ip_hs ? ip_hs : (lb > Mv ? Mv : (int)lb);
  }
  // in place: the masked rows between the history and the chunk
  const int gap_lo = inplace ? ip_hs + p.win - 1 : 0, gap_hi = inplace ? ip_cs : 0;
  int n_band = tr.kv_end - tr.kv_begin;
  int n_gtiles = (!glob || gitem) ? 0 : (p.n_global + kTileN - 1) / kTileN;
  if (n_gtiles > 0 && p.d == 1 && p.bs <= 1 && p.L >= 0) {
    // token-level band: a global key g joins row i unless i - L <= g <= i +
    // R (in the band) or, causal, g > i.  If no row of the tile [qm0, qm1]
    // takes any global key (the smallest one lies inside or right of every
    // row's band, the largest inside or left of it), the global-key tiles
    // would be fully masked: skip them (attention sinks near the start of
    // the sequence, seen by the first W rows through the band anyway).
    const int qr0 = qt * kTileM, qr1 = min(qt * kTileM + kTileM - 1, Mv - 1);
    int g_first = __ldg(p.G), g_last = __ldg(p.G + p.n_global - 1);
    g_first = g_first < 0 ? 0 : (g_first >= p.N ? p.N - 1 : g_first);
    g_last = g_last < 0 ? 0 : (g_last >= p.N ? p.N - 1 : g_last);
    const bool left = g_first < qr1 - p.L;
    const bool right = p.R > 0 && g_last > qr0 + p.R;  // causal (R == 0) takes none right
    if (!left && !right) n_gtiles = 0;
  }
  int n_tiles = n_band + n_gtiles;
  const bool block_mode = p.bs > 1;
  const int map_idx = block_mode ? 0 : cl;

  // Key tile of step it.  With a distance bias the nearest keys come first
  // (the diagonal tile, those before it, then those behind): walked from far
  // to near, a steep bias would raise the running maximum on every tile.
  int near = tr.kv_end - 1;
  if (docs && (SC & 2)) near = min(near, max(tr.kv_begin, qt));
  // kChain: a CTA goes on with items of CTAs that have not started (see the
  // producer).  Makes item (qt_, hp_, b_) and its walk [begin, end) the current one.
  auto take_item = [&](int qt_, int hp_, int b_, int begin, int end) {
    qt = qt_;
    hp = hp_;
    b = b_;
    for (int s = 0; s < NSLOT; ++s) {
      head[s] = hp * NSLOT + s;
      kvh[s] = head[s] / grp;
    }
    if (p.cu_docs) dm.cu = p.cu_docs + (size_t)b * (p.n_docs + 1);
    if (p.doc_pre) dm.pre = p.doc_pre + (size_t)b * p.n_docs;
    tr.kv_begin = begin;
    tr.kv_end = end;
    n_tiles = n_band = end - begin;
    near = end - 1;
    if (SC & 2) near = min(near, max(begin, qt));
  };
  // Waits for the description of item n > 0 and takes it (false: there is none, or
  // a wait gave up).
  auto next_item = [&](int n) -> bool {
    if (!mbar_wait(&item_full[n & 1], (uint32_t)((n - 1) >> 1) & 1u, p.err, abort_flag))
      return false;
    const int* d = items + (n & 1) * C::kItemInts;
    const int at = d[0];
    if (at >= 0) take_item(at, d[1], d[2], d[3], d[4]);
    dt.int_lo = d[5];
    dt.int_hi = d[6];
    dt.mlo = d[7];
    dt.mhi = d[8];
    dt.c0 = d[9];
    dt.cn = d[10];
    dt.base = d[11];
    dt.bound = d[16 + lane];
    dt.pre = d[48 + lane];
    mbar_arrive(&item_free[n & 1]);
    return at >= 0;
  };
  auto kv_tile = [&](int it) -> int {
    if (!(SC & 2)) return tr.kv_begin + it;
    const int before = near - tr.kv_begin + 1;
    return it < before ? near - it : tr.kv_begin + it;
  };

  // virtual row -> TMA row coordinate of a 64-row box
  auto box_row = [&](int vrow) -> int {
    return block_mode ? (c + p.d * (vrow / kBlockRows)) * kBlockRows : vrow;
  };
  const CUtensorMap* mapK = gitem ? &p.tmKf : &p.tmK[map_idx];
  const CUtensorMap* mapV = gitem ? &p.tmVf : &p.tmV[map_idx];
  // the source of a 64-row key box at virtual row vrow (a multiple of 64):
  // its tensor map and row coordinate
  auto kv_box = [&](int kv, int vrow, int* row) -> const CUtensorMap* {
    if (shared) {
      // rows past the prefix, and pages outside the pool's, read as zeros
      const int lp = vrow / p.page_size;
      const int page = vrow < p.N ? __ldg(p.table + lp) : -1;
      *row = page < 0 || page >= p.num_pages ? -kBlockRows
                                             : page * p.page_size + vrow % p.page_size;
      return kv ? &p.tmV[0] : &p.tmK[0];
    }
    if (inplace) {
      if (vrow < ip_cs) {
        *row = (ip_base + vrow) % p.win;
        return kv ? &p.tmV[0] : &p.tmK[0];
      }
      *row = vrow - ip_cs;
      return kv ? &p.tmVf : &p.tmKf;
    }
    *row = gitem ? vrow : box_row(vrow);
    return kv ? mapV : mapK;
  };
  // TMA loads (one thread): the Q tiles, and K or V of band tile it
  auto load_q = [&]() {
    prefetch_tensormap(&p.tmQ[map_idx]);
    mbar_arrive_expect_tx(full_q, C::kQBytes);
    for (int s = 0; s < NSLOT; ++s)
      for (int cc = 0; cc < D / 64; ++cc)
        for (int hh = 0; hh < 2; ++hh)
          tma_load_4d(smem + C::kQ + s * C::kTile + cc * kChunkBytes + hh * (kChunkBytes / 2),
                      &p.tmQ[map_idx], full_q, cc * 64, head[s] + (stack ? hh : 0),
                      stack ? 0 : box_row(qt * kTileM + hh * 64), b);
  };
  // (base: tiles of the items before)
  auto load_kv = [&](int it, int kv, int base = 0) {
    const int st = (base + it) % kStages;
    uint64_t* ful = kv ? &full_v[st] : &full_k[st];
    uint8_t* dst = smem + C::kRing + st * C::kStageBytes + kv * NSTREAM * C::kTile;
    const int t = kv_tile(it);
    mbar_arrive_expect_tx(ful, NSTREAM * C::kTile);
    for (int hh = 0; hh < 2; ++hh) {
      int row;
      const CUtensorMap* m = kv_box(kv, t * kTileN + hh * 64, &row);
      for (int s = 0; s < NSTREAM; ++s)
        for (int cc = 0; cc < D / 64; ++cc)
          tma_load_4d(dst + s * C::kTile + cc * kChunkBytes + hh * (kChunkBytes / 2), m, ful,
                      cc * 64, kvh[s], row, b);
    }
  };
#ifdef SWA_TEST_WITHHOLD_TILE
  // failure-detection test build only: this K tile is never loaded, so the
  // MMA issuer's bounded wait for it runs out
  auto withheld = [](int it, int kv) { return kv == 0 && it == SWA_TEST_WITHHOLD_TILE; };
#else
  auto withheld = [](int, int) { return false; };
#endif
  // Thread 0 loads Q and the first K tile as soon as the barriers exist
  // (before TMEM allocation and the block barrier), the producer warp the
  // rest of the first ring pass after the block barrier: with every CTA of
  // a wave starting at once, a smaller first burst lands Q and K(0) sooner
  // (measured: append 57.3 -> 55.4 us, token / block dilation 152 -> 148 /
  // 154 -> 150 us, prefill within noise).  With global tokens the whole
  // first ring pass goes early (there one K tile only measured 2 % slower).
  const int n_early_k = gitem ? 0 : min(KIND == 2 ? kStages : 1, n_band);
  const int n_early_v = gitem ? 0 : min(KIND == 2 ? kStages : 0, n_band);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(full_q, 1);
    // every issuing slot releases each K/V stage once
    int n_issuers = 0;
    for (int s = 0; s < NSLOT; ++s) n_issuers += slot_ok[s] ? 1 : 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_k[s], 1);
      mbar_init(&empty_k[s], n_issuers);
      mbar_init(&full_v[s], 1);
      mbar_init(&empty_v[s], n_issuers);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&se_full[s], 1);
      mbar_init(&sl_full[s], 1);
      mbar_init(&l_free[s], 128);
      mbar_init(&p_full[s], 128);
      mbar_init(&o_done[s], 1);
      mbar_init(&o_final[s], 1);
      mbar_init(&pe_full[s], 128);
      mbar_init(&oe_done[s], 1);
    }
    mbar_init(peer_free, 128 * NSLOT);
    mbar_init(xfer, 128 * NSLOT);
    if (chain) {
      mbar_init(q_free, NSLOT);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&o_free[i], 128);
        mbar_init(&mma_done[i], 1);
        mbar_init(&item_full[i], 1);
        mbar_init(&item_free[i], NSLOT * 129);
      }
      mbar_init(claimed, 1);
    }
    fence_mbar_init();
    // (an empty part of a split key walk loads nothing: no copy may still
    // be landing in shared memory when the CTA exits)
    if (!gitem && n_tiles > 0) {
      prefetch_tensormap(mapK);
      prefetch_tensormap(mapV);
      if (inplace) {
        prefetch_tensormap(&p.tmKf);
        prefetch_tensormap(&p.tmVf);
      }
      if (!shared) load_q();
      for (int it = 0; it < n_early_k || it < n_early_v; ++it)
        for (int kv = 0; kv < 2; ++kv)
          if (it < (kv ? n_early_v : n_early_k) && !withheld(it, kv)) load_kv(it, kv);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (shared && n_tiles > 0 && threadIdx.x >= 128) {
    // the query rows in the swizzled layout of a TMA box
#pragma unroll
    for (int u = 0; u < kC16; ++u) {
      const int idx = (int)threadIdx.x - 128 + u * 128 * NSLOT;
      const int row = idx / kC16, c16 = idx % kC16;
      const int rr = row % kTileM;
      uint8_t* d8 = smem + C::kQ + (row / kTileM) * C::kTile + (c16 / 8) * kChunkBytes + rr * 128 +
                    (((c16 % 8) ^ (rr % 8)) * 16);
      *reinterpret_cast<uint4*>(d8) = q_val[shared ? u : 0];
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // paired parts: this CTA's barriers exist (the other part waits for this
  // arrival before its first access to them)
  const bool pair = qwin && p.pair;
  if (pair) cluster_arrive_relaxed();
  const uint32_t tmem = *tmem_holder;
  // TMEM columns: slot s has S/P at [128 s, 128 s + 128) and O at 256 + 128 s.
  const uint32_t q_addr = smem_u32(smem + C::kQ);
  const uint32_t ring_addr = smem_u32(smem + C::kRing);

  if (warp < 4) {
    // producer and issuers need few registers: hand the rest to the softmax
    // warpgroups (two slots: 128 x 56 + 256 x 208 = 60416 <= 384 x 168
    // launched; one slot, two CTAs per SM: 128 x 56 + 128 x 200 = 256 x 128)
    // (kChain: 128 x 80, its producer looks documents up)
    if (chain)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory");
    else if (NSLOT == 2 || C::kMinBlocks == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
    if (chain && warp == 0) {
      // ===================== producer (kChain) =====================
      // The walks of packed documents are short, and a CTA per item would spend a
      // third of its life starting and ending.  So a CTA claims the next item of
      // the grid that has not been started while it still works on its own, and
      // loads, MMAs and softmax run on across the border: the claims go in launch
      // order, which keeps the balance of the hardware's scheduling.
      int base = 0, claims = 0, last_k = n_early_k - 1, last_v = -1;
      int full = n_tiles > 0 ? 1 : 0;  // items whose Q is or was under way (the first's is)
      bool ok = true;
      auto all_wait = [&](uint64_t* bar, int phase) {
        return (bool)__all_sync(0xffffffffu,
                                mbar_wait(bar, (uint32_t)phase & 1u, p.err, abort_flag));
      };
      for (int n = 0; ok; ++n) {
        for (int it = 0; ok && it < n_tiles; ++it) {
          const int gt = base + it;
          for (int kv = 0; ok && kv < 2; ++kv) {  // 0: K, 1: V
            if (n == 0 && it < (kv ? n_early_v : n_early_k)) continue;
            uint64_t* emp = kv ? &empty_v[gt % kStages] : &empty_k[gt % kStages];
            if (gt >= kStages && !all_wait(emp, gt / kStages - 1)) {
              ok = false;
              break;
            }
            (kv ? last_v : last_k) = gt;
            if (!withheld(gt, kv) && lane == 0) load_kv(it, kv, base);
            if (n > 0 && it == 0 && kv == 0) {
              // Q of the item before has been read by every QK
              ok = full == 0 || all_wait(q_free, full - 1);
              if (ok && lane == 0) load_q();
              if (ok) ++full;
            }
          }
        }
        if (!ok) break;
        base += n_tiles;
        // claimed only now, so that a long walk does not hold a second item
        if (lane == 0) {
          mbar_arrive_expect_tx(claimed, 16);
          claim_next_cta(smem_u32(smem + C::kClaim), claimed);
        }
        ++claims;
        // the answer: another item, or none left
        if (!all_wait(claimed, n)) break;
        int y = claimed_cta(smem_u32(smem + C::kClaim));
        __syncwarp();
        fence_proxy_async_smem();  // (read, before the next claim writes it)
        int at = -1;
        if (y >= 0) {
          hp = y % npair;
          y /= npair;
          b = y % p.B;
          at = p.qtile_prefix[1] - 1 - y / p.B;
          take_item(at, hp, b, 0, 0);
          dt = doc_tiles<false>(dm, at * kTileM, min(at * kTileM + kTileM, p.N) - 1);
          take_item(at, hp, b, dt.begin, dt.end);
        }
        const int m = n + 1;
        if (m >= 3 && !all_wait(&item_free[m & 1], (m - 3) >> 1)) break;
        int* d = items + (m & 1) * C::kItemInts;
        if (lane == 0) {
          d[0] = at;
          d[1] = hp;
          d[2] = b;
          d[3] = dt.begin;
          d[4] = dt.end;
          d[5] = dt.int_lo;
          d[6] = dt.int_hi;
          d[7] = dt.mlo;
          d[8] = dt.mhi;
          d[9] = dt.c0;
          d[10] = dt.cn;
          d[11] = dt.base;
        }
        d[16 + lane] = dt.bound;
        d[48 + lane] = dt.pre;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_full[m & 1]);
        if (at < 0) break;
      }
      if (lane == 0 && *abort_flag) {
        // leave no copy and no answer writing shared memory behind
#ifdef SWA_TEST_WITHHOLD_TILE
        const int skip = SWA_TEST_WITHHOLD_TILE;
#else
        const int skip = -1;
#endif
        drain_copies(full_q, 1, 0, full - 1);
        drain_copies(full_k, kStages, 0, last_k, skip);
        drain_copies(full_v, kStages, 0, last_v);
        drain_copies(claimed, 1, 0, claims - 1);
      }
    } else if (warp == 0) {
      // =========================== producer ===========================
      if (gitem) {
        // gather the tile's global query rows (zeros past the last) with
        // plain 16-byte loads into the swizzled layout of a TMA box
        if (lane == 0) {
          prefetch_tensormap(mapK);
          prefetch_tensormap(mapV);
        }
        constexpr int kC16 = D / 8;  // 16-byte chunks per row
        for (int s = 0; s < NSLOT; ++s) {
          for (int idx = lane; idx < kTileM * kC16; idx += 32) {
            const int row = idx / kC16, c16 = idx % kC16;
            uint4 val = make_uint4(0u, 0u, 0u, 0u);
            if (row < gcnt) {
              int gv = __ldg(p.G + gq0 + row);
              gv = gv < 0 ? 0 : (gv >= p.N ? p.N - 1 : gv);
              val = __ldg(reinterpret_cast<const uint4*>(
                  p.q_raw + (((size_t)b * p.N + gv) * p.H + head[s]) * D + c16 * 8));
            }
            uint8_t* d8 = smem + C::kQ + s * C::kTile + (c16 / 8) * kChunkBytes + row * 128 +
                          (((c16 % 8) ^ (row % 8)) * 16);
            *reinterpret_cast<uint4*>(d8) = val;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_q);
      }
      // last tiles whose loads were issued (the first n_early_k / n_early_v
      // already are)
      int last_k = n_early_k - 1, last_v = n_early_v - 1;
      for (int it = min(n_early_k, n_early_v); it < n_tiles; ++it) {
        const int st = it % kStages;
        const uint32_t ph = (uint32_t)(it / kStages) & 1u;
        for (int kv = 0; kv < 2; ++kv) {  // 0: K, 1: V
          if (it < (kv ? n_early_v : n_early_k)) continue;
          uint64_t* emp = kv ? &empty_v[st] : &empty_k[st];
          uint64_t* ful = kv ? &full_v[st] : &full_k[st];
          uint8_t* dst = smem + C::kRing + st * C::kStageBytes + kv * NSTREAM * C::kTile;
          if (it >= kStages && !mbar_wait(emp, ph ^ 1u, p.err, abort_flag)) goto producer_done;
          (kv ? last_v : last_k) = it;
          if (withheld(it, kv)) continue;
          if (!glob || it < n_band) {
            if (lane == 0) load_kv(it, kv);
          } else {
            // gather global-key rows with plain 16-byte loads into the
            // swizzled layout the MMA expects
            const int g0 = (it - n_band) * kTileN;
            const int cnt = min(kTileN, p.n_global - g0);
            const uint16_t* src_base = kv ? p.v_raw : p.k_raw;
            constexpr int kC16 = D / 8;  // 16-byte chunks per row
            for (int s = 0; s < NSTREAM; ++s) {
              for (int idx = lane; idx < kTileN * kC16; idx += 32) {
                const int row = idx / kC16, c16 = idx % kC16;
                uint4 val = make_uint4(0u, 0u, 0u, 0u);
                if (row < cnt) {
                  int gv = __ldg(p.G + g0 + row);
                  gv = gv < 0 ? 0 : (gv >= p.N ? p.N - 1 : gv);
                  const uint16_t* src =
                      src_base + (((size_t)b * p.N + gv) * p.Hkv + kvh[s]) * D + c16 * 8;
                  val = __ldg(reinterpret_cast<const uint4*>(src));
                }
                uint8_t* d8 = dst + s * C::kTile + (c16 / 8) * kChunkBytes + row * 128 +
                              (((c16 % 8) ^ (row % 8)) * 16);
                *reinterpret_cast<uint4*>(d8) = val;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ful);
          }
        }
      }
    producer_done:
      if (lane == 0 && *abort_flag) {
        // leave no copy writing shared memory behind
#ifdef SWA_TEST_WITHHOLD_TILE
        const int skip = SWA_TEST_WITHHOLD_TILE;
#else
        const int skip = -1;
#endif
        if (!shared) drain_copies(full_q, 1, 0, 0);
        drain_copies(full_k, kStages, 0, last_k, skip);
        drain_copies(full_v, kStages, 0, last_v);
      }
    } else if (warp <= NSLOT) {
      // =========================== MMA issuers ===========================
      // Warp 1 + s issues the MMAs of slot s (lane 0; the rest of the warp
      // idles at __syncwarp).  Each issuer sits on its own SM sub-partition:
      // a single issuer sharing its sub-partition with two busy softmax
      // warps gets too few issue slots to keep the tensor core fed, two of
      // them together do.  A wait of one issuer leaves the tensor core to
      // the other's MMAs.
      //
      // S of a slot is computed in two 64-key halves.  Tile j's P lives in
      // the TMEM columns of its early half E(j) = j & 1, so the other half's
      // columns are free as soon as the softmax has read them: the early
      // half of tile j+1 (same columns) is issued then, while the softmax
      // is still busy with tile j, and only the late half waits for PV(j).
      const int s = warp - 1;
      if ((chain || n_tiles > 0) && slot_ok[s] && lane == 0) {
        const uint32_t idesc_qk = idesc_bf16_f32(kTileM, kTileN / 2, 0, 0);
        const uint32_t idesc_pv = idesc_bf16_f32(kTileM, D, 0, 1);
        // Descriptors are built once; every MMA then only adds a compile-time
        // offset (start address field, 16-byte units) to a base descriptor.
        const uint64_t dq0 = sdesc_sw128(q_addr, 16, 1024) + (uint64_t)s * (C::kTile >> 4);
        const uint64_t dk0 = sdesc_sw128(ring_addr, 16, 1024) +
                             (NSTREAM == 2 ? (uint64_t)s * (C::kTile >> 4) : 0ull);
        const uint64_t dv0 = sdesc_sw128(ring_addr + NSTREAM * C::kTile, kChunkBytes, 1024) +
                             (NSTREAM == 2 ? (uint64_t)s * (C::kTile >> 4) : 0ull);
        constexpr uint64_t kStageStep = C::kStageBytes >> 4;
        constexpr uint64_t kHalfRows = (64 * 128) >> 4;  // 64 K rows inside a 64-column chunk
        const uint32_t tslot = tmem + 128u * s;
        // S[:, 64 hf : 64 hf + 64] = Q_s K[64 hf : 64 hf + 64]^T of tile it
        auto qk_half = [&](int it, int hf, uint64_t* done) {
          const uint64_t dq = chain ? sdesc_fresh(dq0) : dq0;
          const uint64_t dk = (chain ? sdesc_fresh(dk0) : dk0) +
                              (uint64_t)(it % kStages) * kStageStep + (uint64_t)hf * kHalfRows;
          const uint32_t ts = tslot + 64u * hf;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)(((k / 4) * kChunkBytes + (k % 4) * 32) >> 4);
            mma_ss(ts, dq + off, dk + off, idesc_qk, k > 0 ? 1u : 0u);
          }
          tc_commit(done);
        };
        // O_s += P_s V over the keys of one half of tile it.  P (bf16 pairs)
        // sits in the columns of the tile's early half e = it & 1: the early
        // keys' P at [64 e, 64 e + 32), the late keys' at [64 e + 32, 64 e + 64).
        // The early half's share is issued as soon as its P is written, so
        // after the softmax finishes a tile only a quarter-tile of PV stands
        // between it and the late half of the next tile's S.
        auto pv_half = [&](int it, int e, bool first, bool early) {
          const uint64_t dv =
              (chain ? sdesc_fresh(dv0) : dv0) + (uint64_t)(it % kStages) * kStageStep;
          const uint32_t to = tmem + C::kOcol + (uint32_t)D * s;
          const uint32_t tp = tslot + 64u * (uint32_t)e + (early ? 0u : 32u);
          const int kh = early ? e : (e ^ 1);  // key half
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int k = kh * 4 + kk;
            mma_ts(to, tp + 8u * kk, dv + (uint64_t)((k * 2048) >> 4), idesc_pv,
                   (!first || kk > 0) ? 1u : 0u);
          }
        };
        // base: tiles of the items before; full: items with tiles so far (kChain)
        int base = 0, full = 0;
        int nt = n_tiles;
        for (int n = 0;; ++n) {
          if (chain && n > 0) {
            if (!mbar_wait(&item_full[n & 1], (uint32_t)((n - 1) >> 1) & 1u, p.err, abort_flag))
              break;
            const int* d = items + (n & 1) * C::kItemInts;
            const int at = d[0];
            nt = d[4] - d[3];
            mbar_arrive(&item_free[n & 1]);
            if (at < 0) break;
          }
          if (chain && nt == 0) continue;
          // (a shared prefix's query rows were in place at the block barrier)
          bool ok = (shared || mbar_wait(full_q, (uint32_t)full & 1u, p.err, abort_flag)) &&
                    mbar_wait(&full_k[base % kStages], (uint32_t)(base / kStages) & 1u, p.err,
                              abort_flag);
          tc_fence_after();
          if (ok) {
            // (an item begins with half 0 wherever it runs, so that its bits do not
            // depend on the items before; the PV before has been issued)
            qk_half(base, 0, &se_full[s]);
            qk_half(base, 1, &sl_full[s]);
            tc_commit(&empty_k[base % kStages]);
            if (chain && nt == 1) tc_commit(q_free);
          }
          // (O of the item before has been read out)
          if (chain && ok && full > 0)
            ok = mbar_wait(&o_free[s], (uint32_t)(full - 1) & 1u, p.err, abort_flag);
          for (int it = 0; ok && it < nt; ++it) {
            const int gt = base + it, st = gt % kStages;
            const bool more = it + 1 < nt;
            const int e_next = (it + 1) & 1;  // early half of tile it + 1
            ok = false;
            // the early half's P is in TMEM: its share of PV goes first
            if (!mbar_wait(&pe_full[s], (uint32_t)gt & 1u, p.err, abort_flag)) break;
            if (!mbar_wait(&full_v[st], (uint32_t)(gt / kStages) & 1u, p.err, abort_flag)) break;
            tc_fence_after();
            pv_half(gt, it & 1, it == 0, true);
            tc_commit(&oe_done[s]);
            if (more) {
              // the softmax has read the late half of tile it; K of tile it + 1
              if (!mbar_wait(&l_free[s], (uint32_t)gt & 1u, p.err, abort_flag)) break;
              if (!mbar_wait(&full_k[(gt + 1) % kStages], (uint32_t)((gt + 1) / kStages) & 1u,
                             p.err, abort_flag))
                break;
              tc_fence_after();
              qk_half(gt + 1, e_next, &se_full[s]);
            }
            // P of tile it is in TMEM; V of tile it
            if (!mbar_wait(&p_full[s], (uint32_t)gt & 1u, p.err, abort_flag)) break;
            tc_fence_after();
            pv_half(gt, it & 1, false, false);
            tc_commit(&o_done[s]);
            tc_commit(&empty_v[st]);
            if (more) {
              qk_half(gt + 1, e_next ^ 1, &sl_full[s]);
              tc_commit(&empty_k[(gt + 1) % kStages]);
              if (chain && it + 2 == nt) tc_commit(q_free);
            }
            ok = true;
          }
          // o_final completes once every MMA issued above has finished (also on
          // the abort path, so TMEM is quiescent before it is freed).
          tc_commit(&o_final[s]);
          base += nt;
          ++full;
          if (!chain || !ok) break;
        }
        if (chain) tc_commit(&mma_done[s]);
      }
      __syncwarp();
    }
  } else {
    if (NSLOT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    if (NSLOT == 1 && C::kMinBlocks == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;" ::: "memory");
    // ============================ softmax ============================
    const int slot = warp / 4 - 1;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + 128u * slot + lane_off;
    const uint32_t tO = tmem + C::kOcol + (uint32_t)D * slot + lane_off;
    // stacked: lanes 64-127 are the slot's second head, same tokens
    int base = 0, full = 0, n_item = 0;  // (kChain: as the issuers')
  another_item:
    const int sR = sr0 + slot * kTileM + r;  // shared prefix: row among the kv head's queries
    const int h = shared ? g_kv * grp + sR % grp : head[slot] + (stack ? (r >> 6) : 0);
    const int m_row = stack ? (r & 63) : qt * kTileM + r;  // local query row
    const int m_v = q0 + m_row;         // its virtual row among the keys
    bool row_valid;
    int klo, khi, i_phys;
    long long pos_q = 0;  // position of the row's query (shared prefix)
    if (shared) {
      row_valid = sR < p.B * grp;
      pos_q = row_valid ? p.pos0[sR / grp] : -1;
      klo = p.keep || pos_q < p.win ? 0 : (int)min(pos_q - p.win + 1, (long long)p.N);
      khi = pos_q < 0 ? -1 : (pos_q < p.N - 1 ? (int)pos_q : p.N - 1);
      i_phys = 0;
    } else if (docs) {
      row_valid = m_row < Mq && slot_ok[slot];
      const DocSpan ds = dm.of_thread(dt, m_v);
      klo = dm.key_first(ds, m_v);
      khi = row_valid ? dm.key_last(ds, m_v) : -1;
      i_phys = m_v;
    } else if (gitem) {
      // global row: every key of the sequence (causal: up to the row)
      row_valid = r < gcnt && slot_ok[slot];
      int gv = r < gcnt ? __ldg(p.G + gq0 + r) : 0;
      gv = gv < 0 ? 0 : (gv >= p.N ? p.N - 1 : gv);
      i_phys = gv;
      klo = 0;
      khi = r < gcnt ? (p.R == 0 ? gv : p.N - 1) : -1;
    } else {
      row_valid = m_row < Mq && slot_ok[slot];
      klo = max(key_lo(g, m_v), lo_b);
      // in place: a window that starts past the history starts in the
      // chunk, beyond the masked rows between the two
      if (inplace && klo >= gap_lo) klo += gap_hi - gap_lo;
      khi = key_hi(g, m_v, Mv);
      i_phys = (int)phys_row(g, c, m_v);
      // a global row is written by its global tile, not by the band
      if (glob && row_valid) {
        int lo = 0, hi = p.n_global - 1;
        while (lo <= hi) {
          const int mid = (lo + hi) >> 1;
          const int gv = __ldg(p.G + mid);
          if (gv == i_phys) {
            row_valid = false;
            break;
          }
          if (gv < i_phys) lo = mid + 1;
          else hi = mid - 1;
        }
      }
    }
    // a warp of a global tile whose 32 rows are all past the tile's last
    // global row only keeps the barriers going
    const bool warp_idle = gitem && quad * 32 >= gcnt;
    const bool causal = p.R == 0;
    // band of the row in physical positions, for the global-key test
    const int glo = p.L < 0 ? -0x40000000
                            : (block_mode ? (i_phys / p.bs - (p.L / p.bs) * p.d) * p.bs
                                          : i_phys - p.L * p.d);
    const int ghi = p.R < 0 ? 0x40000000
                            : (block_mode ? (i_phys / p.bs + (p.R / p.bs) * p.d + 1) * p.bs - 1
                                          : i_phys + p.R * p.d);
    constexpr bool cap_on = (SC & 1) != 0, bias_on = (SC & 2) != 0;
    constexpr bool fixed_ref = SC == 1;
    const float nslope2 = bias_on && p.slopes ? -__ldg(p.slopes + h) * 1.4426950408889634f : 0.f;
    const float sl2 = p.scale_log2;
    float m_used = -INFINITY;  // running max, scaled log2 units
    float l = 0.f;
    bool ok = slot_ok[slot];

    float m_pend = -INFINITY;  // max seen but not yet adopted (adopted next tile)
    int int_lo, int_hi;        // key tiles that need no element mask
    // (stacked: from the tokens' rows, conservatively as if they were the
    // last 128 rows below the last token)
    interior_tiles_rows(g, Mv, stack ? q0 + Mq - kTileM : qm0, &int_lo, &int_hi);
    const int last_row = stack ? Mq - 1 : qt * kTileM + kTileM - 1;  // local
    if (docs) {
      int_lo = dt.int_lo;
      int_hi = dt.int_hi;
    } else if (shared) {
      // (klo differs between the rows: the warp's mask test sorts it out)
      int_lo = (klo + kTileN - 1) / kTileN;
      int_hi = (khi + 1) / kTileN - 1;
    }
    // mask every tile: global tiles, rows of negative positions, partial
    // query tiles, and in-place windows that start in the chunk
    if (gitem || lo_b > ip_hs || (!shared && (stack ? Mq < 64 : qt * kTileM + kTileM > Mq)) ||
        (inplace && last_row >= p.win - 1))
      int_hi = int_lo - 1;

    // the 64 score columns of key half hf (TMEM -> registers)
    auto read_half = [&](int hf, float (&sv)[64]) {
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t v[32];
        tmem_ld32(tS + hf * 64 + jj * 32, v);
#pragma unroll
        for (int e = 0; e < 32; ++e) sv[jj * 32 + e] = __uint_as_float(v[e]);
      }
      tmem_wait_ld();
    };
    // Shaped scores: the raw products of a key half become score - m_ref in
    // log2 units.  The cap is s * q(s^2), so its last multiplication takes the
    // subtraction of m_ref (and the bias) with it.  The bias is linear in the
    // key while a half lies on one side of every row of the warp; only halves
    // on the diagonal need |i - j| per key.
    struct HalfShape {
      float add, k1, base;  // addend of key j: add + k1 j, or -m_ref + nslope2 |base - j|
      bool diag, small;
    };
    auto half_shape = [&](int it, int hf, const float (&sv)[64], float m_ref) -> HalfShape {
      HalfShape q;
      q.add = -m_ref;
      q.k1 = q.base = 0.f;
      q.diag = false;
      q.small = true;
      if (bias_on) {
        const int n0 = kv_tile(it) * kTileN + hf * 64;
        // rows of the warp relative to the half's first key (keys of a shared
        // prefix never lie behind a row that sees them)
        const int lo = shared ? 64 : m_v - lane - n0, hi = lo + 31;
        q.base = shared ? (float)(pos_q - n0) : (float)(m_v - n0);
        q.diag = lo < 63 && hi > 0;
        q.k1 = lo >= 63 ? -nslope2 : nslope2;
        if (!q.diag) q.add = fmaf(-q.k1, q.base, -m_ref);
      }
      if (cap_on) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = max3f(fabsf(sv[e]), fabsf(sv[4 + e]), fabsf(sv[8 + e]));
#pragma unroll
        for (int j = 12; j < 60; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = max3f(t[e], fabsf(sv[j + e]), fabsf(sv[j + 4 + e]));
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = fmaxf(t[e], fabsf(sv[60 + e]));
        const float big = max3f(t[0], t[1], fmaxf(t[2], t[3]));
        q.small = !__any_sync(0xffffffffu, big > p.cap.vote);
      }
      return q;
    };
    // Addends of the keys 2e and 2e + 1 counted from the half's key `from` (a
    // multiple of 16), for e in order: bias and -m_ref.  Off the diagonal they are
    // stepped through, afresh every eight pairs, so that at most seven roundings add
    // up.
    auto next_addend = [&](const HalfShape& q, float from, int e, auto is_linear, float2& add) {
      const float k0 = from + (float)(2 * e), k1 = from + (float)(2 * e + 1);
      if (!bias_on) {
        add = make_float2(q.add, q.add);
      } else if (!decltype(is_linear)::value) {
        add = make_float2(fmaf(nslope2, fabsf(q.base - k0), q.add),
                          fmaf(nslope2, fabsf(q.base - k1), q.add));
      } else if ((e & 7) == 0) {
        add.x = fmaf(q.k1, k0, q.add);
        add.y = fmaf(q.k1, k1, q.add);
      } else {
        add = add2(add, make_float2(2.f * q.k1, 2.f * q.k1));
      }
    };
    // (without a cap, or with every product in the cubic's range)
    auto shape_pair = [&](float2 s, float2 add) -> float2 {
      return cap_on ? cap_small(p.cap, s, add) : fma2(s, make_float2(sl2, sl2), add);
    };
    auto shape_half = [&](const HalfShape& q, float (&sv)[64]) {
      auto run = [&](auto is_linear) {
        float2 add;
        if (q.small) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            next_addend(q, 0.f, e, is_linear, add);
            const float2 x = shape_pair(make_float2(sv[2 * e], sv[2 * e + 1]), add);
            sv[2 * e] = x.x;
            sv[2 * e + 1] = x.y;
          }
          return;
        }
        // Rarely taken, so kept small: 16 keys at a time, the half turned by as
        // many in between (unrolled, its 700 instructions cost the usual path 2 %).
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          float done[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            next_addend(q, (float)c, e, is_linear, add);
            const float2 x = cap_any(p.cap, make_float2(sv[2 * e], sv[2 * e + 1]), add);
            done[2 * e] = x.x;
            done[2 * e + 1] = x.y;
          }
#pragma unroll
          for (int j = 0; j < 48; ++j) sv[j] = sv[j + 16];
#pragma unroll
          for (int j = 0; j < 16; ++j) sv[48 + j] = done[j];
        }
      };
      if (bias_on && q.diag) run(std::false_type());
      else run(std::true_type());
    };
    // zeros over the V rows of tile it outside [z0, z1) (thread r: row r), so
    // that whatever lies there, NaN included, adds nothing through P = 0.  After
    // se_full of the tile: its QK was issued once V of the tile before had landed, so
    // the stage's barrier is in the phase of this V or just past it (the next needs
    // the P that this warp still owes), and the parity says which.  Earlier, with
    // one stage, the barrier may be two phases away, and no wait tells those apart.
    auto clear_v_rows = [&](int it, int z0, int z1) -> bool {
      const int gt = base + it, st = gt % kStages;
      if (!mbar_wait(&full_v[st], (uint32_t)(gt / kStages) & 1u, p.err, abort_flag)) return false;
      const int j = kv_tile(it) * kTileN + r;
      if (j < z0 || j >= z1) {
        uint8_t* vt = smem + C::kRing + st * C::kStageBytes + NSTREAM * C::kTile;
#pragma unroll 1
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint4*>(vt + (i / 8) * kChunkBytes + r * 128 + (i % 8) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      return true;
    };
    // -inf outside the row's key set, on edge and global tiles: a keep-mask
    // of the half's 64 keys (bit j: key j is in the set) applied by one
    // shared select loop
    auto mask_half = [&](int it, int hf, bool edge, float (&sv)[64]) {
      uint64_t keep = ~0ull;
      if (!glob || it < n_band) {
        if (edge) {
          const int n0 = kv_tile(it) * kTileN + hf * 64;
          const int lo = max(klo - n0, 0);
          const int hi = min(min(khi, Mv - 1) - n0, 63);  // inclusive
          keep = hi < lo ? 0ull : ((~0ull >> (63 - hi)) & (~0ull << lo));
          if (inplace) {
            const int a = max(gap_lo - n0, 0), z = min(gap_hi - n0, 64);  // [a, z)
            if (a < z) keep &= ~((z >= 64 ? ~0ull : ((1ull << z) - 1ull)) & (~0ull << a));
          }
        }
      } else {
        // a global key joins the row unless it is already in the row's band
        // (same residue class and inside [glo, ghi]) or, causal, after it
        const int g0 = (it - n_band) * kTileN + hf * 64;
        keep = 0ull;
#pragma unroll 1
        for (int j = 0; j < 64 && g0 + j < p.n_global; ++j) {
          int gv = __ldg(p.G + g0 + j);
          gv = gv < 0 ? 0 : (gv >= p.N ? p.N - 1 : gv);
          bool same = true;
          if (p.d > 1) same = ((block_mode ? gv / p.bs : gv) % p.d) == c;
          const bool inband = same && gv >= glo && gv <= ghi;
          if (!inband && (!causal || gv <= i_phys)) keep |= 1ull << j;
        }
      }
      if (__any_sync(0xffffffffu, keep != ~0ull)) {
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (!((keep >> j) & 1ull)) sv[j] = -INFINITY;
      }
    };
    // Edge tiles, for one warp's rows and one key half: whether some row misses a
    // key (returned), and whether no row sees any (none: P = 0, no scores to
    // read).  Of the halves that an edge crosses a quarter is of either kind.
    auto half_edge = [&](int it, int hf, bool edge, bool& none) -> bool {
      none = false;
      if (!__any_sync(0xffffffffu, edge)) return false;
      const int n0 = kv_tile(it) * kTileN + hf * 64, last = min(khi, Mv - 1);
      none = !__any_sync(0xffffffffu, klo <= last && klo < n0 + 64 && last >= n0);
      return __any_sync(0xffffffffu, klo > n0 || last < n0 + 63);
    };
    auto half_max = [&](const float (&sv)[64]) -> float {
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = max3f(sv[e], sv[8 + e], sv[16 + e]);
#pragma unroll
      for (int j = 24; j < 56; j += 16)
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = max3f(t[e], sv[j + e], sv[j + 8 + e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = fmaxf(t[e], sv[56 + e]);
      return max3f(max3f(t[0], t[1], t[2]), max3f(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
    };
    // P = 2^(s * scale * log2 e - m_ref) for one key half, stored as 32
    // columns of bf16 pairs from TMEM column pcol.  At D = 128 seven of
    // every eight column pairs go to the MUFU ex2 unit and one to the FMA
    // pipe (polynomial), which takes some load off MUFU (measured best of 0,
    // 1/8, 1/4 and 1/2 on the FMA pipe with the split PV and the register
    // split); at D = 64 all go to MUFU (1/8 and 1/4 measured 1-4 % slower
    // on the one-head form).
    auto exp_half = [&](int pcol, const float (&sv)[64], float m_ref, float2 (&ls)[4]) {
      const float2 sl2_2 = make_float2(sl2, sl2), negm2 = make_float2(-m_ref, -m_ref);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 xa =
              fma2(make_float2(sv[jj * 32 + 2 * e], sv[jj * 32 + 2 * e + 1]), sl2_2, negm2);
          float2 pr;
          if (D != 64 && (e & 7) == 7) {
            pr = exp2_poly2(xa);
          } else {
            pr.x = ex2_approx(xa.x);
            pr.y = ex2_approx(xa.y);
          }
          ls[e & 3] = add2(ls[e & 3], pr);
          pk[e] = pack_bf16x2(pr.x, pr.y);
        }
        tmem_st16(tS + pcol + jj * 16, pk);
      }
    };
    // The same for shaped scores, whose maximum is already taken off.  raw: sv
    // holds the raw products still (linear bias, cap in its usual range) and
    // is shaped on the way, so that the FMA pipe works on some keys while MUFU
    // works on others.  (All exponentials go to MUFU: 1/8 on the FMA pipe measured no
    // faster.)
    auto exp_shaped = [&](int pcol, float (&sv)[64], float2 (&ls)[4], const HalfShape& q,
                          auto raw) {
      float2 add;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c = jj * 16 + e;
          float2 xa = make_float2(sv[2 * c], sv[2 * c + 1]);
          if (decltype(raw)::value) {
            next_addend(q, 0.f, c, std::true_type(), add);
            xa = shape_pair(xa, add);
            sv[2 * c] = xa.x;
            sv[2 * c + 1] = xa.y;
          }
          const float2 pr = make_float2(ex2_approx(xa.x), ex2_approx(xa.y));
          ls[e & 3] = add2(ls[e & 3], pr);
          pk[e] = pack_bf16x2(pr.x, pr.y);
        }
        tmem_st16(tS + pcol + jj * 16, pk);
      }
    };
    // zeros as the P of a key half (32 columns of bf16 pairs from pcol)
    auto zero_p = [&](int pcol) {
      uint32_t z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0u;
      tmem_st16(tS + pcol, z);
      tmem_st16(tS + pcol + 16, z);
    };
    // Multiplies O (and l) by 2^(m_from - m_to) and adopts m_to; O holds
    // P_0..P_{it-1} V, whose MMAs are complete once o_done says so.
    auto rescale_o = [&](int it, bool mine, float m_to) -> bool {
      const bool o_ok = mbar_wait(&o_done[slot], (uint32_t)(base + it - 1) & 1u, p.err, abort_flag);
      if (!__all_sync(0xffffffffu, o_ok)) return false;
      tc_fence_after();
      const float f = mine ? ex2_approx(m_used - m_to) : 1.f;
      l *= f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t v[32];
        tmem_ld32(tO + j * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
        tmem_st32(tO + j * 32, v);
      }
      tmem_wait_st();
      if (mine) m_used = m_to;
      return true;
    };

    // Scores are exponentiated against the running max as it stands (a row
    // without keys so far adopts the max of the half at hand; its O and l
    // are still zero), and the tile max is tracked on the way.  Scores
    // above the running max only enlarge P, by at most 2^64 (safe in fp32
    // and bf16); a larger jump is adopted at once by rescaling O, l, the
    // partial sums and the P already written.
    for (int it = 0; ok && warp_idle && it < n_tiles; ++it) {
      // rows without a query: no scores to read and no P to write (the PV
      // MMA reads whatever these TMEM lanes hold; those O rows are never
      // stored), but the arrivals keep the phases of the barriers in step
      const uint32_t ph = (uint32_t)it & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&sl_full[slot], ph, p.err, abort_flag))) {
        ok = false;
        break;
      }
      mbar_arrive(&pe_full[slot]);
      mbar_arrive(&l_free[slot]);
      mbar_arrive(&p_full[slot]);
    }
    for (int it = 0; ok && !warp_idle && it < n_tiles; ++it) {
      const int e = it & 1;  // early key half; P of the tile lives in its columns
      const uint32_t ph = (uint32_t)(base + it) & 1u;
      const int t_kv = kv_tile(it);
      const bool edge = ((!glob || it < n_band) && !(t_kv >= int_lo && t_kv <= int_hi)) ||
                        (inplace && t_kv * kTileN < gap_hi && t_kv * kTileN + kTileN > gap_lo);

      // padding rows, and pool rows that no query sees, may hold anything
      const int z0 = docs ? dt.c0 : seen_lo, z1 = docs ? dt.cn : seen_hi;
      const bool v_pad = scored && (t_kv * kTileN < z0 || t_kv * kTileN + kTileN > z1);

      // adopt a larger max seen on the previous tile (rare after the start)
      const bool pend = !fixed_ref && m_pend > m_used;
      if (!fixed_ref && __any_sync(0xffffffffu, pend)) {
        if (!rescale_o(it, pend, m_pend)) { ok = false; break; }
      }

      float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                      make_float2(0.f, 0.f)};
      float sv[64];

      if constexpr (fixed_ref) {
        // exponentials against 0: no maximum to find, none to adopt
#pragma unroll 1
        for (int late = 0; late < 2; ++late) {
          const int hf = e ^ late, pcol = 64 * e + 32 * late;
          const bool w_ok =
              mbar_wait(late ? &sl_full[slot] : &se_full[slot], ph, p.err, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          tc_fence_after();
          if (v_pad && !late && !__all_sync(0xffffffffu, clear_v_rows(it, z0, z1))) {
            ok = false;
            break;
          }
          bool none;
          const bool h_edge = half_edge(it, hf, edge, none);
          if (!none) read_half(hf, sv);
          if (late) {
            // these columns now belong to the early half of the next tile
            tc_fence_before();
            mbar_arrive(&l_free[slot]);
          }
          if (none) {
            zero_p(pcol);
          } else {
            const HalfShape q = half_shape(it, hf, sv, 0.f);
            if (q.small && !h_edge) {
              exp_shaped(pcol, sv, ls, q, std::true_type());
            } else {
              shape_half(q, sv);
              mask_half(it, hf, h_edge, sv);
              exp_shaped(pcol, sv, ls, q, std::false_type());
            }
          }
          tmem_wait_st();
          tc_fence_before();
          if (!late) mbar_arrive(&pe_full[slot]);
        }
        if (!ok) break;
        const float2 a2 = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l += a2.x + a2.y;
        mbar_arrive(&p_full[slot]);
        continue;
      } else if constexpr (scored) {
        // The early half, then the late one (one body, so that the loop stays
        // small): scores against the running maximum m_used (0 while the row
        // has no key), P, and the half's maximum.
        float tmax = -INFINITY;  // of the tile
#pragma unroll 1
        for (int late = 0; late < 2; ++late) {
          const int hf = e ^ late, pcol = 64 * e + 32 * late;
          const bool w_ok =
              mbar_wait(late ? &sl_full[slot] : &se_full[slot], ph, p.err, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          tc_fence_after();
          if (v_pad && !late && !__all_sync(0xffffffffu, clear_v_rows(it, z0, z1))) {
            ok = false;
            break;
          }
          // (Windows of 700 / 4096, 64-wide heads, bias alone: 160 / 432 us without
          // the skip of halves that no row sees, 155 / 443 with it; with the cap
          // besides 186 / 503 and 187 / 563; neither: whole tiles 132 / 360, halves
          // 138 / 396.)
          bool none = false, h_edge = false;
          if (SC == 2) h_edge = half_edge(it, hf, edge, none);
          if (SC != 2 || !none) read_half(hf, sv);
          if (late) {
            // these columns now belong to the early half of the next tile
            tc_fence_before();
            mbar_arrive(&l_free[slot]);
          }
          if (SC == 2 && none) {
            zero_p(pcol);
            tmem_wait_st();
            tc_fence_before();
            if (!late) mbar_arrive(&pe_full[slot]);
            continue;
          }
          // (votes in front of the reads cost the others up to a tenth)
          if (SC == 0) h_edge = __any_sync(0xffffffffu, edge);
          if (SC == 3) h_edge = half_edge(it, hf, edge, none);
          const float m_ref = m_used == -INFINITY ? 0.f : m_used;
          const HalfShape q = half_shape(it, hf, sv, m_ref);
          float2 lh[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
          // the usual half, with no key to mask: P is formed while the half's
          // maximum is found (a row's first against 0, which holds for any
          // maximum in [-20, 64]); otherwise the maximum comes first (and the
          // reference is the same: a row's bits do not depend on which way the
          // other rows of the warp need)
          const bool usual = !q.diag && q.small && !h_edge;
          if (usual) {
            exp_shaped(pcol, sv, lh, q, std::true_type());
          } else {
            shape_half(q, sv);
            mask_half(it, hf, h_edge, sv);
          }
          const float hmax = half_max(sv);  // above m_ref
          tmax = fmaxf(tmax, m_ref + hmax);
          const bool adopt = m_used == -INFINITY;
          const bool jump = !adopt && hmax > 64.f;
          const bool holds = hmax <= 64.f && hmax >= -20.f;
          if (adopt) m_used = holds ? 0.f : hmax;
          const bool redo = __any_sync(0xffffffffu, jump || (adopt && !holds)) || !usual;
          if (__any_sync(0xffffffffu, jump)) {
            const float m_old = m_used;
            if (late) {
              // O must hold the early half's PV before it is scaled
              const bool oe_ok = mbar_wait(&oe_done[slot], ph, p.err, abort_flag);
              if (!__all_sync(0xffffffffu, oe_ok)) { ok = false; break; }
            }
            if (!rescale_o(it, jump, m_ref + hmax)) { ok = false; break; }
            const float f = jump ? ex2_approx(m_old - m_used) : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) ls[j] = make_float2(ls[j].x * f, ls[j].y * f);
          }
          if (redo) {
            const float d = m_used == -INFINITY ? 0.f : m_ref - m_used;
#pragma unroll
            for (int j = 0; j < 64; ++j) sv[j] += d;
#pragma unroll
            for (int j = 0; j < 4; ++j) lh[j] = make_float2(0.f, 0.f);
            tmem_wait_st();
            exp_shaped(pcol, sv, lh, q, std::false_type());
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) ls[j] = add2(ls[j], lh[j]);
          tmem_wait_st();
          tc_fence_before();
          if (!late) mbar_arrive(&pe_full[slot]);
        }
        if (!ok) break;
        const float2 a2 = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l += a2.x + a2.y;
        if (tmax > m_used + kRescaleShaped) m_pend = tmax;
        mbar_arrive(&p_full[slot]);
        continue;
      }

      // ---- early half
      bool w_ok = mbar_wait(&se_full[slot], ph, p.err, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      tc_fence_after();
      // key halves of a global-key tile past the last global key hold no
      // key of any row: no scores to read, P = 0 (the same for every row)
      const bool gskip_e = glob && it >= n_band && (it - n_band) * kTileN + 64 * e >= p.n_global;
      float tmax = -INFINITY;
      if (gskip_e) {
        zero_p(64 * e);
      } else {
      read_half(e, sv);
      mask_half(it, e, edge, sv);
      if (!__any_sync(0xffffffffu, m_used == -INFINITY)) {
        // optimistic: exponentiate against the running max while the half's
        // max is found (no dependence between the two); a jump (rare)
        // rescales O and l and redoes the half against the new max
        exp_half(64 * e, sv, m_used, ls);
        tmax = half_max(sv);
        const bool jump = tmax * sl2 > m_used + 64.f;
        if (__any_sync(0xffffffffu, jump)) {
          if (!rescale_o(it, jump, fmaxf(m_used, tmax * sl2))) { ok = false; break; }
#pragma unroll
          for (int j = 0; j < 4; ++j) ls[j] = make_float2(0.f, 0.f);
          tmem_wait_st();
          exp_half(64 * e, sv, m_used, ls);
        }
      } else {
        // some row of the warp meets its first keys: find the max first
        tmax = half_max(sv);
        const bool adopt = m_used == -INFINITY;
        const bool jump = !adopt && tmax * sl2 > m_used + 64.f;
        if (adopt) m_used = tmax * sl2;
        if (__any_sync(0xffffffffu, jump)) {
          if (!rescale_o(it, jump, fmaxf(m_used, tmax * sl2))) { ok = false; break; }
        }
        exp_half(64 * e, sv, m_used == -INFINITY ? 0.f : m_used, ls);
      }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&pe_full[slot]);

      // ---- late half
      w_ok = mbar_wait(&sl_full[slot], ph, p.err, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      tc_fence_after();
      const bool gskip_l =
          glob && it >= n_band && (it - n_band) * kTileN + 64 * (e ^ 1) >= p.n_global;
      if (gskip_l) {
        tc_fence_before();
        mbar_arrive(&l_free[slot]);
        zero_p(64 * e + 32);
      } else {
      read_half(e ^ 1, sv);
      // these columns now belong to the early half of the next tile
      tc_fence_before();
      mbar_arrive(&l_free[slot]);
      mask_half(it, e ^ 1, edge, sv);
      if (!__any_sync(0xffffffffu, m_used == -INFINITY)) {
        // optimistic as above; on a jump O must also hold the early half's
        // PV (issued once its P was written) before it is scaled
        float2 lh[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        exp_half(64 * e + 32, sv, m_used, lh);
        const float tmax1 = half_max(sv);
        tmax = fmaxf(tmax, tmax1);
        const bool jump = tmax1 * sl2 > m_used + 64.f;
        if (__any_sync(0xffffffffu, jump)) {
          const float m_old = m_used;
          const bool oe_ok = mbar_wait(&oe_done[slot], ph, p.err, abort_flag);
          if (!__all_sync(0xffffffffu, oe_ok)) { ok = false; break; }
          if (!rescale_o(it, jump, fmaxf(m_used, tmax1 * sl2))) { ok = false; break; }
          const float f = jump ? ex2_approx(m_old - m_used) : 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ls[j] = make_float2(ls[j].x * f, ls[j].y * f);
            lh[j] = make_float2(0.f, 0.f);
          }
          tmem_wait_st();
          exp_half(64 * e + 32, sv, m_used, lh);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) ls[j] = add2(ls[j], lh[j]);
      } else {
        const float tmax1 = half_max(sv);
        tmax = fmaxf(tmax, tmax1);
        const bool adopt = m_used == -INFINITY;
        const bool jump = !adopt && tmax1 * sl2 > m_used + 64.f;
        if (adopt) m_used = tmax1 * sl2;
        if (__any_sync(0xffffffffu, jump)) {
          const float m_old = m_used;
          const bool oe_ok = mbar_wait(&oe_done[slot], ph, p.err, abort_flag);
          if (!__all_sync(0xffffffffu, oe_ok)) { ok = false; break; }
          if (!rescale_o(it, jump, fmaxf(m_used, tmax1 * sl2))) { ok = false; break; }
          const float f = jump ? ex2_approx(m_old - m_used) : 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) ls[j] = make_float2(ls[j].x * f, ls[j].y * f);
        }
        exp_half(64 * e + 32, sv, m_used == -INFINITY ? 0.f : m_used, ls);
      }
      }
      {
        const float2 a2 = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l += a2.x + a2.y;
      }
      // a max that grew by more than 2^8 is adopted before the next tile
      if (tmax * sl2 > m_used + kRescaleThreshold) m_pend = tmax * sl2;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[slot]);
    }

    // (any key's P is at least 2^-kFixedRef)
    if (fixed_ref && l != 0.f) m_used = 0.f;

    // split key walk: this CTA's part goes to the partials (fp32 O / l and
    // lse); an empty part contributes nothing (lse = -inf)
    const bool split = p.nsplit > (shared ? 0 : 1) && (shared || (qwin && !pair));
    const size_t prow = shared ? ((size_t)sp * p.B + sR / grp) * p.H + h
                               : (((size_t)sp * p.B + b) * p.H + h) * (size_t)Mq + m_row;
    if (split && ok && n_tiles == 0 && row_valid && !warp_idle) {
      float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D);
      for (int e = 0; e < D / 4; ++e) dst[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      p.part_lse[prow] = -INFINITY;
    }
    if (docs && ok && n_tiles == 0 && row_valid) {
      // a tile of padding rows
      uint4* dst = reinterpret_cast<uint4*>(p.out + (((size_t)b * p.N + m_row) * p.H + h) * D);
      for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse) p.lse[((size_t)b * p.H + h) * p.N + m_row] = -INFINITY;
    }
    bool fin = ok && n_tiles > 0 && !warp_idle;
    if (fin) fin = mbar_wait(&o_final[slot], (uint32_t)full & 1u, p.err, abort_flag);
    if (pair) {
      // The two parts of the key walk merge through distributed shared
      // memory.  Once both have finished their MMAs (each tells the other
      // on peer_free), each sends the other the half of its O columns that
      // the other writes, with its (m, l), and merges the half it keeps:
      // with M = max(m_0, m_1) and a_i = 2^(m_i - M), out = (a_0 O_0 + a_1
      // O_1) / (a_0 l_0 + a_1 l_1) (the split softmax's lse identity).
      constexpr int kHalf = D / 2;  // columns a part writes
      constexpr int kV4 = kHalf / 4;
      const uint32_t peer = (uint32_t)(sp ^ 1);
      const int rrow = slot * 128 + r;
      // receive area (the ring, free once this CTA's MMAs are done): row
      // rrow's kV4 float4, XOR-swizzled by the row against bank conflicts,
      // then (m, l) per row
      const uint32_t rx_o = smem_u32(smem + C::kRing) + (uint32_t)(rrow * kV4 * 16);
      const uint32_t rx_ml = smem_u32(smem + C::kRing) + (uint32_t)(C::kRxO + rrow * 8);
      // O in TMEM is complete (an empty part, or one that gave up, sends
      // zeros with m = -inf)
      const bool have = __all_sync(0xffffffffu, fin);
      const float m_me = have ? m_used : -INFINITY, l_me = have ? l : 0.f;
      __syncwarp();
      cluster_wait();  // the other part's barriers exist
      mbar_arrive_cluster(map_shared_rank(smem_u32(peer_free), peer));
      const bool go = __all_sync(0xffffffffu, mbar_wait<true>(peer_free, 0, p.err, abort_flag));
      if (go) {
        const uint32_t dst = map_shared_rank(rx_o, peer);
#pragma unroll
        for (int j = 0; j < kHalf / 32; ++j) {
          uint32_t v[32];
          if (have) {
            tmem_ld32(tO + (uint32_t)(peer * kHalf + 32 * j), v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4)
            st_cluster_f4(dst + (uint32_t)(((j * 8 + e4) ^ (r & 7)) * 16),
                          __uint_as_float(v[4 * e4]), __uint_as_float(v[4 * e4 + 1]),
                          __uint_as_float(v[4 * e4 + 2]), __uint_as_float(v[4 * e4 + 3]));
        }
        st_cluster_f2(map_shared_rank(rx_ml, peer), m_me, l_me);
      }
      mbar_arrive_cluster(map_shared_rank(smem_u32(xfer), peer));
      // both parts' MMAs are done, so every read of this kv head's ring rows
      // is: the chunk enters the ring (keys from part 0, values from part 1)
      if (p.ring_store && go && (have || n_tiles == 0)) {
        const long long p0 = p.pos0[b];
        constexpr int kRv = D / 8;  // 16-byte vectors per row
        const int c_first = Mq > p.win ? Mq - p.win : 0;
        const uint4* src = sp == 0 ? p.kn_raw : p.vn_raw;
        uint4* dst = sp == 0 ? p.k_ring : p.v_ring;
        const int kv = kvh[0];
        if (p0 >= 0) {
          for (int t = (int)threadIdx.x - 128; t < (Mq - c_first) * kRv; t += 128 * NSLOT) {
            const int cc = c_first + t / kRv, i = t % kRv;
            const long long slot_r = (p0 + cc) % p.win;
            dst[(((long long)b * p.win + slot_r) * p.Hkv + kv) * kRv + i] =
                __ldg(src + (((long long)b * Mq + cc) * p.Hkv + kv) * kRv + i);
          }
        }
      }
      const bool got = __all_sync(0xffffffffu, mbar_wait<true>(xfer, 0, p.err, abort_flag));
      if (got) {
        const float2 mlp = ld_shared_f2(rx_ml);
        const float M = fmaxf(m_me, mlp.x);
        const float a_me = m_me == -INFINITY ? 0.f : ex2_approx(m_me - M);
        const float a_pe = mlp.x == -INFINITY ? 0.f : ex2_approx(mlp.x - M);
        const float L_ = a_me * l_me + a_pe * mlp.y;
        const float inv = L_ > 0.f ? 1.f / L_ : 0.f;
        const float c_me = a_me * inv, c_pe = a_pe * inv;
        uint16_t* orow = p.out + (((size_t)b * Mq + m_row) * p.H + h) * D + sp * kHalf;
#pragma unroll
        for (int j = 0; j < kHalf / 32; ++j) {
          uint32_t v[32];
          if (have) {
            tmem_ld32(tO + (uint32_t)(sp * kHalf + 32 * j), v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          uint32_t pk[16];
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 o = ld_shared_f4(rx_o + (uint32_t)(((j * 8 + e4) ^ (r & 7)) * 16));
            pk[2 * e4] = pack_bf16x2(__uint_as_float(v[4 * e4]) * c_me + o.x * c_pe,
                                     __uint_as_float(v[4 * e4 + 1]) * c_me + o.y * c_pe);
            pk[2 * e4 + 1] = pack_bf16x2(__uint_as_float(v[4 * e4 + 2]) * c_me + o.z * c_pe,
                                         __uint_as_float(v[4 * e4 + 3]) * c_me + o.w * c_pe);
          }
          if (row_valid) {
            uint4* dst = reinterpret_cast<uint4*>(orow + 32 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          }
        }
        if (row_valid && sp == 0 && p.lse)
          p.lse[((size_t)b * p.H + h) * Mq + m_row] = (M + __log2f(L_)) * 0.69314718055994531f;
      }
    } else if (__all_sync(0xffffffffu, fin)) {
      tc_fence_after();
      // (l == 0: a part of a split walk with none of the row's keys, whose
      // lse is -inf and which the merge skips, or a padding row: zeros)
      // (a row without keys: nothing was added to its sum.  Its maximum would not say so:
      // one over NaN scores and masked ones is -inf too.)
      const bool none = scored && l == 0.f;
      const float inv = l > 0.f && !none ? 1.f / l : 0.f;
      const size_t orow_i = qwin ? (size_t)b * Mq + m_row : (size_t)b * p.N + i_phys;
      uint16_t* orow = p.out + (orow_i * p.H + h) * D;
      // rows start on 128-byte multiples from out: 32-byte stores when out
      // itself is 32-byte aligned
      const bool out_v8 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
      // 64 columns of O per TMEM round trip (two loads, one wait)
#pragma unroll
      for (int j2 = 0; j2 < D / 64; ++j2) {
        uint32_t v[2][32];
        __syncwarp();
        tmem_ld32(tO + j2 * 64, v[0]);
        tmem_ld32(tO + j2 * 64 + 32, v[1]);
        tmem_wait_ld();
        if (none) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[0][e] = v[1][e] = 0u;
        }
        if (split) {
          if (shared && row_valid && (reinterpret_cast<uintptr_t>(p.part_o) & 31u) == 0) {
            // (whole 32-byte sectors)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              v[0][e] = __float_as_uint(__uint_as_float(v[0][e]) * inv);
              v[1][e] = __float_as_uint(__uint_as_float(v[1][e]) * inv);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_global_v8(p.part_o + prow * D + j2 * 64 + e * 8, &v[e >> 2][(e & 3) * 8]);
          } else if (row_valid) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + j2 * 64);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              dst[e] = make_float4(__uint_as_float(v[e >> 3][(e & 7) * 4]) * inv,
                                   __uint_as_float(v[e >> 3][(e & 7) * 4 + 1]) * inv,
                                   __uint_as_float(v[e >> 3][(e & 7) * 4 + 2]) * inv,
                                   __uint_as_float(v[e >> 3][(e & 7) * 4 + 3]) * inv);
          }
          continue;
        }
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = pack_bf16x2(__uint_as_float(v[jj][2 * e]) * inv,
                                __uint_as_float(v[jj][2 * e + 1]) * inv);
          if (row_valid) {
            if (out_v8) {
              // two full 32-byte sectors per lane
              st_global_v8(orow + j2 * 64 + jj * 32, pk);
              st_global_v8(orow + j2 * 64 + jj * 32 + 16, pk + 8);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + j2 * 64 + jj * 32);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            }
          }
        }
      }
      const float lse_v = none ? -INFINITY
                               : (m_used + (fixed_ref ? log2f(l) : __log2f(l))) *
                                     0.69314718055994531f;
      if (row_valid && split)
        p.part_lse[prow] = lse_v;
      else if (row_valid && p.lse)
        p.lse[((size_t)b * p.H + h) * (qwin ? Mq : p.N) + (qwin ? m_row : i_phys)] = lse_v;
    }
    if (chain && __all_sync(0xffffffffu, fin || (ok && n_tiles == 0))) {
      if (n_tiles > 0) {
        // O and the whole of S are read out
        tc_fence_before();
        mbar_arrive(&o_free[slot]);
        base += n_tiles;
        ++full;
      }
      if (__all_sync(0xffffffffu, next_item(++n_item))) goto another_item;
    }
  }

  // ---- teardown: make sure no MMA is in flight, then free TMEM.
  if (chain && warp >= 1 && warp <= NSLOT && lane == 0) {
    volatile int no_abort = 0;
    mbar_wait(&mma_done[warp - 1], 0, nullptr, &no_abort, 100000000ull);
  }
  if (!chain && warp >= 1 && warp <= NSLOT && lane == 0 && n_tiles > 0 && slot_ok[warp - 1] &&
      *abort_flag) {
    // abort path: o_final was committed after the last MMA this issuer
    // issued; give it a bounded chance to land before TMEM is released.
    volatile int no_abort = 0;
    mbar_wait(&o_final[warp - 1], 0, nullptr, &no_abort, 100000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // paired parts: neither CTA exits while the other may still write its
  // shared memory (the softmax warps waited on the first cluster barrier
  // in their epilogue, the others do here)
  if (pair) {
    if (warp < 4) cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
}
// The register split of the forms that use setmaxnreg (warpgroup 0: 56 per
// thread, each softmax warpgroup: 208 with two slots, 200 with one) must fit
// in what the block is launched with, or setmaxnreg.inc would never return:
// checked once per kernel form.
template <int D, int NSLOT, int NSTREAM, int KIND, int SC>
bool fwd_regs_fit() {
  using C = Cfg<D, NSLOT, NSTREAM, KIND, SC>;
  if (!(NSLOT == 2 || C::kMinBlocks == 2)) return true;
  const long need = (C::kChain ? 128L * 80 : 128L * 56) + (NSLOT == 2 ? 256L * 208 : 128L * 200);
  static std::atomic<int> known{0};
  if (known.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, KIND, SC>) !=
        cudaSuccess)
      return false;
    known.store((long)fa.numRegs * C::kThreads >= need ? 1 : -1, std::memory_order_release);
  }
  return known.load(std::memory_order_acquire) > 0;
}

// The kernel's SC for these scores (see kFixedRef).
inline int score_form(const ScoreArgs& sc) {
  return sc.kind() == 1 && sc.softcap * 1.4426950408889634f > kFixedRef ? 3 : sc.kind();
}

// Fills in what shapes the scores.
inline void set_score(FwdParams& p, const ScoreArgs& sc, float scale) {
  p.cap = cap_coefs(sc.softcap, scale);
  p.slopes = sc.slopes;
  p.cu_docs = sc.cu_docs;
  p.doc_pre = sc.prefix;
  p.n_docs = sc.n_docs;
}

}  // namespace
}  // namespace swa
