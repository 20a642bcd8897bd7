// swa_fwd_sm100.cu -- launches of the fused bf16 forward (swa_fwd_sm100.cuh):
// the band with token or block dilation, the band plus global tokens, and the
// query window of a chunked append.
#include "swa_fwd_sm100.cuh"

namespace swa {
namespace {

// Whether the device can place clusters of two CTAs of the query-window
// form (paired parts); asked once per form.
template <int D, int NSLOT, int NSTREAM>
bool pair_clusters_fit() {
  using C = Cfg<D, NSLOT, NSTREAM, 1>;
  static std::atomic<int> known{0};  // 0 not asked, 1 yes, -1 no
  int k = known.load(std::memory_order_acquire);
  if (k == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kAlloc;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(
        &n, reinterpret_cast<const void*>(swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 1>), &cfg);
    if (e != cudaSuccess) cudaGetLastError();
    k = (e == cudaSuccess && n > 0) ? 1 : -1;
    known.store(k, std::memory_order_release);
  }
  return k > 0;
}

template <int D, int NSLOT, int NSTREAM>
int launch_impl(const void* q, const void* k, const void* v, void* out, float* lse, int B, int H,
                int Hkv, int N, int L, int R, int d, int bs, const int32_t* G, int ng,
                float scale, cudaStream_t stream, const QueryWindow* qw, int qt_lo, int qt_hi) {
  using C = Cfg<D, NSLOT, NSTREAM, 0>;  // (the same for kinds 0 to 2)
  static std::atomic<unsigned long long> attr_kind[3] = {{0}, {0}, {0}};
  const int kind = qw ? 1 : (ng > 0 ? 2 : 0);
  const void* kfn[3] = {reinterpret_cast<const void*>(swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 0>),
                        reinterpret_cast<const void*>(swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 1>),
                        reinterpret_cast<const void*>(swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 2>)};
  if (!smem_attr_once(kfn[kind], C::kAlloc, attr_kind[kind])) return SWA_ERR_CUDA;
  if (NSLOT == 2 || C::kMinBlocks == 2) {
    // The register split (warpgroup 0: 56 per thread, each softmax
    // warpgroup: 208 with two slots, 200 with one) must fit in what the
    // block is launched with, or setmaxnreg.inc would never return: checked
    // once per kernel form.
    const long need = NSLOT == 2 ? 128L * 56 + 256L * 208 : 128L * 56 + 128L * 200;
    static std::atomic<int> regs_ok[3] = {{0}, {0}, {0}};
    if (regs_ok[kind].load(std::memory_order_acquire) == 0) {
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kfn[kind]) != cudaSuccess) return SWA_ERR_CUDA;
      regs_ok[kind].store((long)fa.numRegs * C::kThreads >= need ? 1 : -1,
                          std::memory_order_release);
    }
    if (regs_ok[kind].load(std::memory_order_acquire) < 0) return SWA_ERR_UNSUPPORTED;
  }
  int* err = device_error_word();
  if (!err) return SWA_ERR_CUDA;
  const Geometry geo = make_geometry(N, L, R, d, bs);
  const bool block_mode = geo.bs > 1;
  for (int c0 = 0; c0 < geo.nclass; c0 += kMaxClasses) {
    FwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.nclass = geo.nclass - c0 < kMaxClasses ? geo.nclass - c0 : kMaxClasses;
    p.class0 = c0;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.G = G;
    p.q_raw = static_cast<const uint16_t*>(q);
    p.k_raw = static_cast<const uint16_t*>(k);
    p.v_raw = static_cast<const uint16_t*>(v);
    p.err = err;
    p.n_global = ng;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.N = N;
    p.L = L;
    p.R = R;
    p.d = d;
    p.bs = geo.bs;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.qtile_prefix[0] = 0;
    for (int cl = 0; cl < p.nclass; ++cl) {
      p.Mv[cl] = class_valid_rows(geo, c0 + cl);
      const int rows_q = qw ? qw->Mq : p.Mv[cl];
      p.qtile_prefix[cl + 1] = p.qtile_prefix[cl] + (rows_q + kTileM - 1) / kTileM;
    }
    if (qt_hi >= 0) {
      // a row-range launch (one class): only query tiles [qt_lo, qt_hi)
      if (geo.nclass != 1 || qw) return SWA_ERR_UNSUPPORTED;
      const int all = p.qtile_prefix[1];
      const int lo = qt_lo < 0 ? 0 : (qt_lo > all ? all : qt_lo);
      const int hi = qt_hi > all ? all : (qt_hi < lo ? lo : qt_hi);
      p.qt_base = lo;
      p.qtile_prefix[1] = hi - lo;
    }
    const bool inplace = qw && qw->kn;
    if (qw) {
      p.pos0 = qw->pos0;
      p.q0 = qw->q0;
      p.Mq = qw->Mq;
      p.win = qw->win;
      p.inplace = inplace ? 1 : 0;
      p.stack = (NSLOT == 2 && qw->stack) ? 1 : 0;
      p.nsplit = qw->nsplit > 1 ? qw->nsplit : 1;
      p.pair = (p.nsplit == 2 && qw->pair && pair_clusters_fit<D, NSLOT, NSTREAM>()) ? 1 : 0;
      if (p.nsplit > 1 && !p.pair) {
        if (!qw->part) return SWA_ERR_ARG;
        p.part_o = qw->part;
        p.part_lse = qw->part + (size_t)p.nsplit * B * H * qw->Mq * D;
      }
      // the chunk enters the rings inside the launch when each cluster holds
      // every reader of its kv head's ring rows: one query tile and all the
      // kv head's query heads in one item
      const int heads_per_item = p.stack ? 2 * NSLOT : NSLOT;
      if (p.pair && inplace && qw->ring_k && qw->ring_v && p.nclass == 1 &&
          p.qtile_prefix[1] == 1 && heads_per_item == H / Hkv) {
        p.ring_store = 1;
        p.k_ring = static_cast<uint4*>(qw->ring_k);
        p.v_ring = static_cast<uint4*>(qw->ring_v);
        p.kn_raw = static_cast<const uint4*>(qw->kn);
        p.vn_raw = static_cast<const uint4*>(qw->vn);
      }
      if (qw->done) *qw->done = p.pair | (p.ring_store << 1);
    }
    const uint32_t box[4] = {64, 1, (uint32_t)kBlockRows, 1};
    const int nmaps = block_mode ? 1 : p.nclass;
    for (int cl = 0; cl < nmaps; ++cl) {
      const int cc = c0 + cl;
      const uint64_t rows = block_mode ? (uint64_t)N : (uint64_t)class_rows(geo, cc);
      const uint64_t rstep = block_mode ? 1 : (uint64_t)d;
      const size_t qoff = block_mode ? 0 : (size_t)cc * H * D;
      const size_t kvoff = block_mode ? 0 : (size_t)cc * Hkv * D;
      const uint64_t qrows = qw ? (uint64_t)qw->Mq : rows;
      const uint64_t qN = qw ? (uint64_t)qw->Mq : (uint64_t)N;
      const uint64_t dq[4] = {(uint64_t)D, (uint64_t)H, qrows, (uint64_t)B};
      const uint64_t sq[3] = {(uint64_t)D * 2, rstep * H * D * 2, qN * H * D * 2};
      // in place: K / V are the rings, win rows per batch
      const uint64_t krows = inplace ? (uint64_t)qw->win : rows;
      const uint64_t kN = inplace ? (uint64_t)qw->win : (uint64_t)N;
      const uint64_t dk[4] = {(uint64_t)D, (uint64_t)Hkv, krows, (uint64_t)B};
      const uint64_t sk[3] = {(uint64_t)D * 2, rstep * Hkv * D * 2, kN * Hkv * D * 2};
      void* qb = (void*)(static_cast<const uint16_t*>(q) + qoff);
      void* kb = (void*)(static_cast<const uint16_t*>(k) + kvoff);
      void* vb = (void*)(static_cast<const uint16_t*>(v) + kvoff);
      if (encode_tiled(&p.tmQ[cl], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, qb, dq, sq, box,
                       CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
          encode_tiled(&p.tmK[cl], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, kb, dk, sk, box,
                       CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
          encode_tiled(&p.tmV[cl], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, vb, dk, sk, box,
                       CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return SWA_ERR_CUDA;
    }
    if (inplace) {
      // the chunk's keys and values, [B, Mq, Hkv, D]
      const uint64_t dn[4] = {(uint64_t)D, (uint64_t)Hkv, (uint64_t)qw->Mq, (uint64_t)B};
      const uint64_t sn[3] = {(uint64_t)D * 2, (uint64_t)Hkv * D * 2,
                              (uint64_t)qw->Mq * Hkv * D * 2};
      if (encode_tiled(&p.tmKf, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(qw->kn),
                       dn, sn, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
          encode_tiled(&p.tmVf, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(qw->vn),
                       dn, sn, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return SWA_ERR_CUDA;
    }
    // the global tiles ride with the first launch
    if (c0 == 0 && kind == 2) {
      p.n_gq_tiles = (ng + kTileM - 1) / kTileM;
      p.n_gitems = p.n_gq_tiles * B * ((H + NSLOT - 1) / NSLOT);
      const uint64_t df[4] = {(uint64_t)D, (uint64_t)Hkv, (uint64_t)N, (uint64_t)B};
      const uint64_t sf[3] = {(uint64_t)D * 2, (uint64_t)Hkv * D * 2,
                              (uint64_t)N * Hkv * D * 2};
      if (encode_tiled(&p.tmKf, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(k), df, sf,
                       box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
          encode_tiled(&p.tmVf, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v), df, sf,
                       box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return SWA_ERR_CUDA;
    }
    const long heads_per_item = p.stack ? 2 * NSLOT : NSLOT;
    const long grid = (long)p.n_gitems + (long)p.qtile_prefix[p.nclass] * B *
                                             ((H + heads_per_item - 1) / heads_per_item) *
                                             (qw ? p.nsplit : 1);
    if (grid <= 0) continue;
    if (grid > 0x7fffffffL) return SWA_ERR_UNSUPPORTED;
    if (kind == 1 && p.pair) {
      // clusters of two: the two parts of an item are consecutive CTAs
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)grid);
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kAlloc;
      cfg.stream = stream;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2;
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 1>, p) != cudaSuccess)
        return SWA_ERR_CUDA;
    } else if (kind == 1)
      swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 1><<<(unsigned)grid, C::kThreads, C::kAlloc,
                                                   stream>>>(p);
    else if (kind == 2)
      swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 2><<<(unsigned)grid, C::kThreads, C::kAlloc,
                                                   stream>>>(p);
    else
      swa_fwd_sm100_kernel<D, NSLOT, NSTREAM, 0><<<(unsigned)grid, C::kThreads, C::kAlloc,
                                                   stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SWA_ERR_CUDA;
  }
  return SWA_OK;
}

}  // namespace

bool fwd_qwin_stacks(int H, int Hkv, int Mq) {
  const int grp = H / Hkv;
  return grp % 4 == 0 && Mq <= 64;  // two slots (even group), four heads per CTA
}

// Two query heads per CTA when they share a kv head (GQA group of even
// size); otherwise one head per CTA, two CTAs per SM at D = 64 (measured on
// the D = 64 MHA workloads against two heads with two K/V streams per CTA:
// Longformer 133 -> 125 us, token dilation 172 -> 155, block 169 -> 156).
int launch_fwd_sm100(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                     int H, int Hkv, int N, int D, int L, int R, int d, int bs, const int32_t* G,
                     int ng, float scale, cudaStream_t stream, const QueryWindow* qw, int qt_lo,
                     int qt_hi) {
  const bool gqa_pair = (H / Hkv) % 2 == 0;
  if (D == 128) {
    if (gqa_pair)
      return launch_impl<128, 2, 1>(q, k, v, out, lse, B, H, Hkv, N, L, R, d, bs, G, ng, scale,
                                    stream, qw, qt_lo, qt_hi);
    return launch_impl<128, 1, 1>(q, k, v, out, lse, B, H, Hkv, N, L, R, d, bs, G, ng, scale,
                                  stream, qw, qt_lo, qt_hi);
  }
  if (D == 64) {
    if (gqa_pair)
      return launch_impl<64, 2, 1>(q, k, v, out, lse, B, H, Hkv, N, L, R, d, bs, G, ng, scale,
                                   stream, qw, qt_lo, qt_hi);
    return launch_impl<64, 1, 1>(q, k, v, out, lse, B, H, Hkv, N, L, R, d, bs, G, ng, scale,
                                 stream, qw, qt_lo, qt_hi);
  }
  return SWA_ERR_UNSUPPORTED;
}

}  // namespace swa
