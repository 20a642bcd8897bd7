// swa_prefix.cu -- launch of the shared prefix's part of a decode: the kernel of
// the fused forward (swa_fwd_sm100.cuh) with every sequence's queries of a kv
// head as its rows and the prefix's pages as its keys.
#include "swa_fwd_sm100.cuh"

namespace swa {
namespace {

template <int D, int NSLOT, int SC>
int launch(const SharedArgs& a, int nsplit, float* part_o, float* part_lse,
           cudaStream_t stream) {
  using C = Cfg<D, NSLOT, 1, 4, SC>;
  const auto kernel = swa_fwd_sm100_kernel<D, NSLOT, 1, 4, SC>;
  static std::atomic<unsigned long long> attr{0};
  if (!smem_attr_once(reinterpret_cast<const void*>(kernel), C::kAlloc, attr)) return SWA_ERR_CUDA;
  if (!fwd_regs_fit<D, NSLOT, 1, 4, SC>()) return SWA_ERR_UNSUPPORTED;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.err = device_error_word();
  if (!p.err) return SWA_ERR_CUDA;
  p.q_raw = static_cast<const uint16_t*>(a.q);
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.N = a.n_prefix;
  p.L = -1;
  p.R = -1;
  p.d = 1;
  p.nclass = 1;
  p.Mv[0] = a.n_prefix;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  ScoreArgs sc;
  sc.softcap = a.softcap;
  sc.slopes = a.slopes;
  set_score(p, sc, a.scale);
  p.pos0 = a.pos;
  p.win = a.W;
  p.keep = a.keep;
  p.table = a.prefix_table;
  p.page_size = a.page_size;
  p.num_pages = a.num_pages;
  p.nsplit = nsplit;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.tmK[0] = *a.tmK;
  p.tmV[0] = *a.tmV;
  const long long rows = (long long)a.B * (a.H / a.Hkv);
  const long long grid = (rows + NSLOT * kTileM - 1) / (NSLOT * kTileM) * a.Hkv * nsplit;
  if (grid > 0x7fffffffLL) return SWA_ERR_UNSUPPORTED;
  kernel<<<(unsigned)grid, C::kThreads, C::kAlloc, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace

int launch_prefix(const SharedArgs& a, const SharedPlan& pl, float* part_o, float* part_lse,
                  cudaStream_t stream) {
  const int nsplit = pl.prefix_parts;
  ScoreArgs sc;
  sc.softcap = a.softcap;
  sc.slopes = a.slopes;
  auto go = [&](auto d, auto ns) -> int {
    constexpr int kD = decltype(d)::value, kS = decltype(ns)::value;
    switch (score_form(sc)) {
      case 0: return launch<kD, kS, 0>(a, nsplit, part_o, part_lse, stream);
      case 1: return launch<kD, kS, 1>(a, nsplit, part_o, part_lse, stream);
      case 2: return launch<kD, kS, 2>(a, nsplit, part_o, part_lse, stream);
      default: return launch<kD, kS, 3>(a, nsplit, part_o, part_lse, stream);
    }
  };
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  if (a.D == 128) {
    using D128 = std::integral_constant<int, 128>;
    return pl.two ? go(D128(), I2()) : go(D128(), I1());
  }
  if (a.D == 64) {
    using D64 = std::integral_constant<int, 64>;
    return pl.two ? go(D64(), I2()) : go(D64(), I1());
  }
  return SWA_ERR_UNSUPPORTED;
}

}  // namespace swa
