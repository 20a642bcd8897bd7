// swa_shared.cu -- decode of a batch whose sequences begin with the same
// prefix: how the keys are split over the SMs, and the three launches.
//
// The prefix's keys and values are the same for every sequence, so they are
// read once: all B * H / Hkv query vectors of a kv head form the rows of a
// matrix product against them (the fused forward's kernel in its prefix
// form, swa_fwd_sm100.cu).  The keys behind the prefix belong to one sequence
// each (the decode kernel in its own-keys form, swa_decode_tc.cu).  Both write
// partial results (O / l, lse), and
//   out = sum_i e^(lse_i - lse) O_i / l_i,   lse = ln sum_i e^lse_i
// joins them.
#include <cuda_runtime.h>

#include "swa_internal.h"
#include "swa_sched.cuh"

namespace swa {
namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

}  // namespace

SharedPlan shared_plan(int B, int H, int Hkv, int D, int n_prefix, int W, int max_tail) {
  SharedPlan pl;
  const long long sms = sm_count();
  // prefix: query tiles x kv heads, each walk split until the SMs are full
  const long long rows = (long long)B * (H / Hkv);
  const long long per_item = rows > kTileM ? 2 * kTileM : kTileM;
  const long long items = (rows + per_item - 1) / per_item * Hkv;
  const long long tiles = ((long long)n_prefix + kTileN - 1) / kTileN;
  long long parts = sms / items;
  parts = parts < 1 ? 1 : parts;
  pl.prefix_parts = (int)(parts < tiles ? parts : tiles);
  // own keys: about 1024 per part, as many as the longest tail needs
  const long long tail = (max_tail < W ? max_tail : W) + (long long)kBlockRows - 1;
  const long long own = (tail + 1023) / 1024;
  pl.own_parts = (int)(own < 1 ? 1 : own);
  const long long keys = (tail + pl.own_parts - 1) / pl.own_parts;
  pl.part_keys = (int)((keys + kTileN - 1) / kTileN * kTileN);
  pl.bytes = (size_t)(pl.prefix_parts + pl.own_parts) * B * H * (D + 1) * sizeof(float);
  return pl;
}

int launch_decode_shared(const SharedArgs& a, const SharedPlan& pl, void* workspace,
                         cudaStream_t stream) {
  const int parts = pl.prefix_parts + pl.own_parts;
  const size_t rows = (size_t)a.B * a.H;
  float* part_o = static_cast<float*>(workspace);
  float* part_lse = part_o + (size_t)parts * rows * a.D;
  if (pl.prefix_parts > 0) {
    const int st = launch_prefix(a, pl.prefix_parts, part_o, part_lse, stream);
    if (st != SWA_OK) return st;
  }
  const int st = launch_own(a, pl, part_o + (size_t)pl.prefix_parts * rows * a.D,
                            part_lse + (size_t)pl.prefix_parts * rows, stream);
  if (st != SWA_OK) return st;
  return split_merge(part_o, a.out, a.lse, parts, a.B, 1, a.H, a.D, stream);
}

}  // namespace swa
