// attention_split.cu — attention over the paged cache, the split kernel: one
// CTA per SM, each on one of two sides.  Parts that many query rows share run on
// tcgen05 (attention_tc.cuh), parts of at most 16 rows on warp MMAs
// (attention_warp.cuh); a batch behind a prefix has both, one bound by the
// tensor cores and the other by HBM, and the plan gives each side as many CTAs
// as its units need, so that they end together.  As two kernels after one
// another, each with the whole chip, their start-up and tails added up: when the
// two were joined, 64 sequences of up to 2,047 tokens behind 8,192 (56 query, 8
// key heads of 128) went from 99 us in all to 86.  They take 88 to 91 with what
// the kernel does today.
#include "attention_tc.cuh"
#include "attention_warp.cuh"

namespace moe {
namespace {

union SplitShared {
  TcShared tc;
  WarpShared warp;
};

template <int D>
constexpr int split_smem() {
  return TcCfg<D>::kSmem > WarpCfg<D>::kSmem ? TcCfg<D>::kSmem : WarpCfg<D>::kSmem;
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    k_attn_split(const AttnParams p, const __grid_constant__ CUtensorMap warp_k, const __grid_constant__ CUtensorMap warp_v,
                 const __grid_constant__ CUtensorMap tc_k, const __grid_constant__ CUtensorMap tc_v) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ AttnPlan plan;
  __shared__ SplitShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  attn_plan(p, plan);
  if ((int)blockIdx.x < plan.ctas[1]) {
    attn_tc_role<D>(p, tc_k, tc_v, plan, sh.tc, dyn);
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if (warp < kAttnWarpWorkers) {
      if (lane == 0) {
        for (int s = 0; s < WarpCfg<D>::kStages; ++s) mbar_init(&sh.warp.full[warp][s], 1);
        mbar_init_fence();
      }
      __syncwarp();
      attn_warp_role<D>(p, warp_k, warp_v, plan, sh.warp, dyn);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  }
}

// The warp side alone, for calls that have nothing for the other: the smaller
// kernel starts faster (24 sequences of up to 32,771 tokens, 4 key heads of 64,
// with the join: 79 us, 87 us on the split kernel).
template <int D>
__global__ void __launch_bounds__(kAttnWarpWorkers * 32, 1)
    k_attn_warp(const AttnParams p, const __grid_constant__ CUtensorMap warp_k, const __grid_constant__ CUtensorMap warp_v) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ AttnPlan plan;
  __shared__ WarpShared sh;
  if ((threadIdx.x & 31) == 0) {
    for (int s = 0; s < WarpCfg<D>::kStages; ++s) mbar_init(&sh.full[threadIdx.x >> 5][s], 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  attn_plan(p, plan);
  attn_warp_role<D>(p, warp_k, warp_v, plan, sh, dyn);
}

template <int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap (&m)[4], cudaStream_t s) {
  cudaError_t err;
  if (!p.side[1].own && !p.side[1].prefix) {
    constexpr int kSmem = WarpCfg<D>::kSmem;
    if ((err = ensure_smem_attr((const void*)k_attn_warp<D>, kSmem)) != cudaSuccess) return err;
    return launch_pdl(k_attn_warp<D>, dim3(kAttnCtas), dim3(kAttnWarpWorkers * 32), kSmem, s, p, m[0], m[1]);
  }
  if ((err = ensure_smem_attr((const void*)k_attn_split<D>, split_smem<D>())) != cudaSuccess) return err;
  return launch_pdl(k_attn_split<D>, dim3(kAttnCtas), dim3(kAttnThreads), split_smem<D>(), s, p, m[0], m[1], m[2], m[3]);
}

}  // namespace

cudaError_t launch_attn_split(const AttnParams& p, const CUtensorMap (&maps)[4], cudaStream_t s) {
  return p.head_dim == 128 ? launch<128>(p, maps, s) : launch<64>(p, maps, s);
}

}  // namespace moe
