// swa_scored.cu -- launches of the forward with shaped scores: the kernel of
// the fused forward (swa_fwd_sm100.cuh) in its form for documents, with the
// cap and the bias compiled in or left out (swa_score.cuh).
#include "swa_fwd_sm100.cuh"

namespace swa {
namespace {

template <int D, int NSLOT, int SC>
int launch(const void* q, const void* k, const void* v, void* out, float* lse, int B, int H,
           int Hkv, int N, int L, int R, const ScoreArgs& sc, float scale, cudaStream_t stream) {
  using C = Cfg<D, NSLOT, 1, 3, SC>;
  const auto kernel = swa_fwd_sm100_kernel<D, NSLOT, 1, 3, SC>;
  static std::atomic<unsigned long long> attr{0};
  if (!smem_attr_once(reinterpret_cast<const void*>(kernel), C::kAlloc, attr)) return SWA_ERR_CUDA;
  if (!fwd_regs_fit<D, NSLOT, 1, 3, SC>()) return SWA_ERR_UNSUPPORTED;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.err = device_error_word();
  if (!p.err) return SWA_ERR_CUDA;
  p.nclass = 1;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.N = N;
  p.L = L;
  p.R = R;
  p.d = 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.Mv[0] = N;
  p.qtile_prefix[1] = (N + kTileM - 1) / kTileM;
  set_score(p, sc, scale);
  if (encode_kv_map(&p.tmQ[0], q, D, H, N, B) != SWA_OK ||
      encode_kv_map(&p.tmK[0], k, D, Hkv, N, B) != SWA_OK ||
      encode_kv_map(&p.tmV[0], v, D, Hkv, N, B) != SWA_OK)
    return SWA_ERR_CUDA;
  const long long grid = (long long)p.qtile_prefix[1] * B * ((H + NSLOT - 1) / NSLOT);
  if (grid > 0x7fffffffLL) return SWA_ERR_UNSUPPORTED;
  kernel<<<(unsigned)grid, C::kThreads, C::kAlloc, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace

int launch_fwd_scored(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                      int H, int Hkv, int N, int D, int L, int R, const ScoreArgs& sc, float scale,
                      cudaStream_t stream) {
  if (sc.plain())
    return launch_fwd_sm100(q, k, v, out, lse, B, H, Hkv, N, D, L, R, 1, 0, nullptr, 0, scale,
                            stream);
  auto go = [&](auto d, auto ns) -> int {
    constexpr int kD = decltype(d)::value, kS = decltype(ns)::value;
    switch (score_form(sc)) {
      case 0: return launch<kD, kS, 0>(q, k, v, out, lse, B, H, Hkv, N, L, R, sc, scale, stream);
      case 1: return launch<kD, kS, 1>(q, k, v, out, lse, B, H, Hkv, N, L, R, sc, scale, stream);
      case 2: return launch<kD, kS, 2>(q, k, v, out, lse, B, H, Hkv, N, L, R, sc, scale, stream);
      default: return launch<kD, kS, 3>(q, k, v, out, lse, B, H, Hkv, N, L, R, sc, scale, stream);
    }
  };
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  // Two heads of a GQA group per CTA where the group pairs up, as the forward;
  // one head while that leaves SMs idle (two sequences of 517 tokens with 8
  // heads: 13.1 -> 10.9 us; 8192 tokens with 32 heads, where it does not: 175
  // against 190 us with one).
  const long long items = (long long)((N + kTileM - 1) / kTileM) * B * H / 2;
  const bool pairs = (H / Hkv) % 2 == 0 && items > sm_count();
  if (D == 128) {
    using D128 = std::integral_constant<int, 128>;
    return pairs ? go(D128(), I2()) : go(D128(), I1());
  }
  if (D == 64) {
    using D64 = std::integral_constant<int, 64>;
    return pairs ? go(D64(), I2()) : go(D64(), I1());
  }
  return SWA_ERR_UNSUPPORTED;
}

}  // namespace swa
