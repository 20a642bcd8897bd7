// swa_shared.cu -- decode of a batch whose sequences begin with the same
// prefix: how the keys are split over the SMs, the launches, and the merge.
//
// The prefix's keys and values are the same for every sequence, so they are
// read once: all B * H / Hkv query vectors of a kv head form the rows of a
// matrix product against them (the fused forward's kernel in its prefix form,
// swa_fwd_sm100.cuh).  The keys behind the prefix belong to one sequence each
// (swa_own.cu).  Both write partial results (O / l, lse), and
//   out = sum_i e^(lse_i - lse) O_i / l_i,   lse = ln sum_i e^lse_i
// joins them.  The three launches depend on one another only through the
// partial results, so each is scheduled while the one before runs.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "swa_internal.h"
#include "swa_ptx.cuh"
#include "swa_sched.cuh"

namespace swa {
namespace {

// (a NaN among a part's scores makes the row NaN, as in one softmax over all keys)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// One warp per row (sequence, head): the parts' weights e^(lse_i - lse), 32 at
// a time, one per lane, then the weighted sum of the parts, eight loads in
// flight per lane.
template <int D>
__global__ void __launch_bounds__(256)
    merge_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                 uint16_t* __restrict__ out, float* __restrict__ lse, int parts, int rows) {
  constexpr int kPer = D / 32;  // elements per lane
  using Vec = typename std::conditional<D == 128, float4, float2>::type;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long row = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32) m = max_nan(m, part_lse[(long long)i * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[kPer] = {};
  float wsum = 0.f;
  for (int i0 = 0; i0 < parts && m != -INFINITY; i0 += 32) {
    const float w = i0 + lane < parts
                        ? __expf(part_lse[(long long)(i0 + lane) * rows + row] - m)
                        : 0.f;
    wsum += w;
    const int n = parts - i0 < 32 ? parts - i0 : 32;
    for (int b0 = 0; b0 < n; b0 += 8) {
      Vec o[8];
      float wi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wi[i] = __shfl_sync(0xffffffffu, w, (b0 + i) & 31);
        if (b0 + i >= n) wi[i] = 0.f;
        // (a part without keys of the row has weight 0, and its O may be
        // anything)
        if (wi[i] != 0.f)
          o[i] = reinterpret_cast<const Vec*>(part_o + ((long long)(i0 + b0 + i) * rows + row) *
                                                           D)[lane];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (wi[i] == 0.f) continue;
        const float* f = reinterpret_cast<const float*>(&o[i]);
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] += wi[i] * f[e];
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint16_t* dst = out + row * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lse && lane == 0) lse[row] = wsum == 0.f ? -INFINITY : m + __logf(wsum);
}

int merge(const float* part_o, const float* part_lse, void* out, float* lse, int parts, int rows,
          int D, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e =
      D == 128 ? cudaLaunchKernelEx(&cfg, merge_kernel<128>, part_o, part_lse,
                                    static_cast<uint16_t*>(out), lse, parts, rows)
               : cudaLaunchKernelEx(&cfg, merge_kernel<64>, part_o, part_lse,
                                    static_cast<uint16_t*>(out), lse, parts, rows);
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace

int sm_count() {
  constexpr int kMax = 64;
  static std::atomic<int> known[kMax];  // by device, 0: not asked
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
    cudaGetLastError();
    return 148;
  }
  if (dev < kMax && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  if (dev < kMax) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

SharedPlan shared_plan(int B, int H, int Hkv, int D, int n_prefix, int W, int max_tail) {
  SharedPlan pl;
  pl.sms = sm_count();
  const long long sms = pl.sms;
  // prefix: query tiles x kv heads, each walk split until the SMs are full
  const long long rows = (long long)B * (H / Hkv);
  const long long tiles = ((long long)n_prefix + kTileN - 1) / kTileN;
  auto parts_of = [&](int per_item, int per_sm) -> long long {
    if (tiles == 0) return 0;
    const long long items = (rows + per_item - 1) / per_item * Hkv;
    const long long parts = sms * per_sm / items;
    return parts < 1 ? 1 : (parts < tiles ? parts : tiles);
  };
  // (measured with 256 rows of 128 against one tile per CTA, two CTAs per SM:
  // 44.8 and 46.6 us for 64 sequences behind 8192 tokens, 154 and 178 us for
  // 128 behind 32741)
  pl.two = rows > kTileM;
  pl.prefix_parts = (int)(pl.two ? parts_of(2 * kTileM, 1) : parts_of(kTileM, 2));
  // own keys: at most about 1024 per part; fewer, down to 256, while the
  // sequences do not fill two CTAs per SM
  const long long tail = (max_tail < W ? max_tail : W) + (long long)kBlockRows - 1;
  long long own = (tail + 1023) / 1024;
  const long long fill = (2 * sms + (long long)B * Hkv - 1) / ((long long)B * Hkv);
  const long long most = (tail + 255) / 256;
  if (own < fill) own = fill < most ? fill : most;
  // (and no more than four items per CTA need: the rest would only be merged)
  if (own > 4 * fill) own = 4 * fill;
  pl.own_parts = (int)(own < 1 ? 1 : own);
  const long long keys = (tail + pl.own_parts - 1) / pl.own_parts;
  pl.part_keys = (int)((keys + kTileN - 1) / kTileN * kTileN);
  pl.bytes = (size_t)(pl.prefix_parts + pl.own_parts) * B * H * (D + 1) * sizeof(float);
  return pl;
}

int launch_decode_shared(SharedArgs a, const SharedPlan& pl, void* workspace,
                         cudaStream_t stream) {
  const int parts = pl.prefix_parts + pl.own_parts;
  const size_t rows = (size_t)a.B * a.H;
  float* part_o = static_cast<float*>(workspace);
  float* part_lse = part_o + (size_t)parts * rows * a.D;
  CUtensorMap tm[2];
  const int pool_rows = a.num_pages * a.page_size;
  if (encode_kv_map(&tm[0], a.k_pages, a.D, a.Hkv, pool_rows, 1) != SWA_OK ||
      encode_kv_map(&tm[1], a.v_pages, a.D, a.Hkv, pool_rows, 1) != SWA_OK)
    return SWA_ERR_CUDA;
  a.tmK = &tm[0];
  a.tmV = &tm[1];
  if (pl.prefix_parts > 0) {
    const int st = launch_prefix(a, pl, part_o, part_lse, stream);
    if (st != SWA_OK) return st;
  }
  const int st = launch_own(a, pl, part_o + (size_t)pl.prefix_parts * rows * a.D,
                            part_lse + (size_t)pl.prefix_parts * rows, pl.prefix_parts > 0, stream);
  if (st != SWA_OK) return st;
  return merge(part_o, part_lse, a.out, a.lse, parts, (int)rows, a.D, stream);
}

}  // namespace swa
