// rms_norm.cu — residual sum and root-mean-square norm of rows, the result in
// fp32, bf16 or as an MX matrix.
//
//   h = x + residual,  y = h weight / sqrt(mean(h^2) + eps)
//
// A CTA, or for narrow rows a warp, takes a row and keeps h in registers between
// the sum of squares and the result, so that every value crosses HBM once: bound by
// HBM for many rows (4,096 x 7,168, bf16 into an fp32 residual, MXFP8 out: 52 us,
// 6.2 TB/s), by the launch, one load and two barriers for a few (1 row: 2.6 us).
//
// The sum of squares has a fixed order (eights of a thread, lanes, warps); the
// reciprocal root is rsqrtf's with one Newton step, since its error is common to a
// row.  An MX result is rounded to 2 or 4 significant bits, where a difference of the
// last place of y moves values next to a border by a step: some 10 of 29 million.
// (Sums and products in pairs of floats left about as many and took 64 us.)
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpRows = 8;         // rows of a CTA where a warp takes a row
constexpr int kWarpEights = 3;       // eights of values a lane holds there: rows of up to 768

struct NormShared {
  float sum[32], most[32];
};

// Sum over the row's threads.
template <bool WARP>
__device__ __forceinline__ float row_add(float v, NormShared& sh) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (WARP) return v;
  const int lane = threadIdx.x & 31, n = (blockDim.x + 31) >> 5;
  if (lane == 0) sh.sum[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < n ? sh.sum[lane] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <bool WARP>
__device__ __forceinline__ float row_max(float v, NormShared& sh) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if (WARP) return v;
  const int lane = threadIdx.x & 31, n = (blockDim.x + 31) >> 5;
  if (lane == 0) sh.most[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < n ? sh.most[lane] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// 1 / sqrt(sum / cols + eps).
__device__ __forceinline__ float factor_of(float sum, float cols, float eps) {
  const float x = sum / cols + eps, r = rsqrtf(x);
  const float t = x * r, e = fmaf(-fmaf(x, r, -t), r, fmaf(-t, r, 1.f));  // 1 - x r^2
  return fmaf(0.5f * r, e, r);
}

// XB, RB: x, the residual in bf16; R: there is a residual; OUT: MOE_DT_F32,
// MOE_DT_BF16, or 2 + MX type; C: eights of values a thread holds; WARP: a warp
// takes a row, else a CTA.
template <bool XB, bool R, bool RB, int OUT, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpRows * 32 : kMaxThreads) k_rms_norm(const NormParams p) {
  __shared__ NormShared sh;
  const int r = WARP ? blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x, per_row = p.cols / 8;
  const int first = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
  pdl_trigger();
  pdl_wait();
  if (WARP && r >= p.rows) return;
  const uint8_t* x = (const uint8_t*)p.x + r * p.x_stride;
  const uint8_t* res = (const uint8_t*)p.res + r * p.res_stride;
  Eight<XB> ex[C];
  Eight<RB> er[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = first + j * step;
    if (c8 < per_row) {
      ex[j].load(x, c8);
      if (R) er[j].load(res, c8);
    }
  }
  float h[C][8];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = first + j * step;
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
  sum = row_add<WARP>(sum, sh);
  float factor = factor_of(sum, (float)p.cols, p.eps);
  if (!(sum < p.most)) {
    // Squares, or their mean and eps, past fp32's range, an infinity or a NaN (uniform
    // over the row): again with the row's largest magnitude brought near 1, if it is a
    // number.
    float m = 0.f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (first + j * step < per_row)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(h[j][i])), nan |= h[j][i] != h[j][i];
    // A maximum leaves NaN out: as infinity, told apart below.
    m = row_max<WARP>(nan ? INFINITY : m, sh);
    if (m < INFINITY) {
      const uint32_t e = __float_as_uint(m) >> 23;  // of m > 2^50
      const float up = __uint_as_float((e < 253u ? 254u - e : 1u) << 23);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (first + j * step < per_row)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[j][i] *= up;
            s = fmaf(h[j][i], h[j][i], s);
          }
      factor = factor_of(row_add<WARP>(s, sh), (float)p.cols, p.eps * up * up);
    } else {
      // 1 / sqrt(infinity): NaN where h is infinite, 0 elsewhere; a NaN anywhere makes
      // the mean one.
      float any = nan ? 1.f : 0.f;
      if (!WARP) __syncthreads();  // sh.most is used again
      any = row_max<WARP>(any, sh);
      factor = any != 0.f ? __int_as_float(0x7FC00000) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c8 = first + j * step;
    if (c8 < per_row) {
      if (p.weight) {
        const float4 a = reinterpret_cast<const float4*>(p.weight)[2 * c8];
        const float4 b = reinterpret_cast<const float4*>(p.weight)[2 * c8 + 1];
        const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * factor * w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] *= factor;
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
  const int per_row = p.cols / 8, eights = (per_row + 31) / 32;
  if (eights <= kWarpEights) {
    const dim3 grid(((unsigned)p.rows + kWarpRows - 1) / kWarpRows), block(kWarpRows * 32);
    if (eights <= 1) return launch_pdl(k_rms_norm<XB, R, RB, OUT, 1, true>, grid, block, 0, s, p);
    return launch_pdl(k_rms_norm<XB, R, RB, OUT, kWarpEights, true>, grid, block, 0, s, p);
  }
  const int c = per_row <= kMaxThreads ? 1 : 2;
  // Whole warps; the lanes of a block are a group of four of one warp.
  const int threads = ((per_row + c - 1) / c + 31) & ~31;
  const dim3 grid((unsigned)p.rows), block((unsigned)threads);
  return c == 1 ? launch_pdl(k_rms_norm<XB, R, RB, OUT, 1, false>, grid, block, 0, s, p)
                : launch_pdl(k_rms_norm<XB, R, RB, OUT, 2, false>, grid, block, 0, s, p);
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
