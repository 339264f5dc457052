// rms_norm.cu — residual sum and root-mean-square norm of rows, the result in
// fp32, bf16 or as an MX matrix.
//
//   h = x + residual,  y = h weight / sqrt(mean(h^2) + eps)
//
// A CTA takes a row and keeps h in registers between the sum of squares and the
// result, so that every value crosses HBM once: bound by HBM for many rows, by
// the launch, one load and two barriers for a few.  The sum of squares has a
// fixed order (eights of a thread, lanes, warps).
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;

struct NormShared {
  float warp[2][32];
};

// Sum (or maximum) of v over the CTA, in a fixed order; `side` alternates
// between calls, so that one barrier a call is enough.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float (&warp)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if (lane == 0) warp[w] = v;
  __syncthreads();
  v = lane < n ? warp[lane] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

// XB, RB: x, the residual in bf16; R: there is a residual; OUT: MOE_DT_F32,
// MOE_DT_BF16, or 2 + MX type; C: eights of values a thread holds.
template <bool XB, bool R, bool RB, int OUT, int C>
__global__ void __launch_bounds__(kMaxThreads) k_rms_norm(const NormParams p) {
  __shared__ NormShared sh;
  const int r = blockIdx.x, per_row = p.cols / 8;
  pdl_trigger();
  pdl_wait();
  const uint8_t* x = (const uint8_t*)p.x + r * p.x_stride;
  const uint8_t* res = (const uint8_t*)p.res + r * p.res_stride;
  Eight<XB> ex[C];
  Eight<RB> er[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = threadIdx.x + j * blockDim.x;
    if (c8 < per_row) {
      ex[j].load(x, c8);
      if (R) er[j].load(res, c8);
    }
  }
  float h[C][8];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = threadIdx.x + j * blockDim.x;
    if (c8 < per_row) {
      ex[j].get(h[j]);
      if (R) {
        float q[8];
        er[j].get(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += q[i];
        Eight<RB>::store((uint8_t*)p.res_out + r * p.res_stride, c8, h[j]);
      }
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(h[j][i], h[j][i], s);
      sum += s;
    }
  }
  sum = cta_reduce<false>(sum, sh.warp[0]);
  float factor = rsqrtf(sum / (float)p.cols + p.eps), up = 1.f;
  if (sum > 3.0e38f) {
    // Squares past fp32's range (uniform over the CTA): again with the row's
    // largest magnitude brought to 1.  (A row with an infinity or a NaN keeps it.)
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if ((int)(threadIdx.x + j * blockDim.x) < per_row)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(h[j][i]));
    m = cta_reduce<true>(m, sh.warp[1]);
    if (m < INFINITY) {
      const uint32_t e = __float_as_uint(m) >> 23;  // of m > 2^50: at least 177
      up = __uint_as_float((e < 253u ? 254u - e : 1u) << 23);
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if ((int)(threadIdx.x + j * blockDim.x) < per_row)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(h[j][i] * up, h[j][i] * up, sum);
      sum = cta_reduce<false>(sum, sh.warp[0]);
      factor = rsqrtf(sum / (float)p.cols + p.eps * up * up);
    } else {
      factor = 0.f;  // 1 / sqrt(infinity): NaN where h is infinite, 0 elsewhere
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = threadIdx.x + j * blockDim.x;
    if (c8 < per_row) {
      if (p.weight) {
        float w[8];
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.weight) + 2 * c8);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.weight) + 2 * c8 + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * up * factor * w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * up * factor;
      }
      if (OUT == MOE_DT_F32)
        Eight<false>::store((uint8_t*)p.out + r * p.out_stride, c8, h[j]);
      else if (OUT == MOE_DT_BF16)
        Eight<true>::store((uint8_t*)p.out + r * p.out_stride, c8, h[j]);
      else
        mx_store8<OUT == 2 + MOE_MX_E4M3>(h[j], p.mx.q + r * p.mx.q_stride, p.mx.s + r * p.mx.s_stride, c8);
    }
  }
}

template <bool XB, bool R, bool RB, int OUT>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
  const int per_row = p.cols / 8;
  const int c = per_row <= kMaxThreads ? 1 : 2;
  // Whole warps; the lanes of a block are a group of four of one warp.
  const int threads = ((per_row + c - 1) / c + 31) & ~31;
  const dim3 grid((unsigned)p.rows), block((unsigned)threads);
  return c == 1 ? launch_pdl(k_rms_norm<XB, R, RB, OUT, 1>, grid, block, 0, s, p)
                : launch_pdl(k_rms_norm<XB, R, RB, OUT, 2>, grid, block, 0, s, p);
}
template <bool XB, bool R, bool RB>
cudaError_t launch_out(const NormParams& p, int out, cudaStream_t s) {
  switch (out) {
    case MOE_DT_F32: return launch<XB, R, RB, MOE_DT_F32>(p, s);
    case MOE_DT_BF16: return launch<XB, R, RB, MOE_DT_BF16>(p, s);
    case 2 + MOE_MX_E2M1: return launch<XB, R, RB, 2 + MOE_MX_E2M1>(p, s);
    default: return launch<XB, R, RB, 2 + MOE_MX_E4M3>(p, s);
  }
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams& p, int x_dtype, int res_dtype, int out, cudaStream_t s) {
  const bool xb = x_dtype == MOE_DT_BF16, rb = res_dtype == MOE_DT_BF16;
  if (!p.res) return xb ? launch_out<true, false, false>(p, out, s) : launch_out<false, false, false>(p, out, s);
  if (xb) return rb ? launch_out<true, true, true>(p, out, s) : launch_out<true, true, false>(p, out, s);
  return rb ? launch_out<false, true, true>(p, out, s) : launch_out<false, true, false>(p, out, s);
}

}  // namespace moe
