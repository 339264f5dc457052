// mx.cu — rows of fp32 or bf16 to MX matrices (MXFP4, MXFP8) and back.
//
// A block of 32 gets the scale 2^(floor(log2 M) - emax), M its largest
// magnitude: an exponent field less a constant, and multiplying by its inverse is
// exact, so that the only rounding is the conversion's.  Each element is read
// and written once; bound by HBM for matrices, by the launch and one memory
// latency for a few rows.
//
// A lane takes eight neighbouring values (16-byte loads of bf16), four lanes a
// block (two shuffles for M), so that a warp's loads, codes and scales are
// contiguous.
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Unit u of eight values: row and place in the row.
__device__ __forceinline__ void place(uint32_t u, uint32_t per_row, uint32_t& row, uint32_t& c8) {
  row = u / per_row;
  c8 = u - row * per_row;
}

template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kThreads) k_mx_quantize(const QuantizeParams p, uint32_t units, uint32_t per_row) {
  pdl_trigger();
  pdl_wait();
  // units is a multiple of 4: groups of four lanes stay whole.
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  uint32_t row, c8;
  place(u, per_row, row, c8);
  Eight<BF16> e;
  e.load((const uint8_t*)p.x + row * p.stride, c8);
  float v[8];
  e.get(v);
  mx_store8<E4M3>(v, p.mx.q + row * p.mx.q_stride, p.mx.s + row * p.mx.s_stride, c8);
}

template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(const QuantizeParams p, uint32_t units, uint32_t per_row) {
  pdl_trigger();
  pdl_wait();
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  uint32_t row, c8;
  place(u, per_row, row, c8);
  const uint8_t* q = p.mx.q + row * p.mx.q_stride;
  const float scale = e8m0_f32(p.mx.s[row * p.mx.s_stride + (c8 >> 2)]);
  float v[8];
  if (E4M3) {
    const uint2 c = reinterpret_cast<const uint2*>(q)[c8];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      const uint16_t two = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
      const float2 f = f16x2_f32x2(h);
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  } else {
    const uint32_t c = reinterpret_cast<const uint32_t*>(q)[c8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f16x2_f32x2(e2m1x2_f16x2(c, i));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
  Eight<BF16>::store((uint8_t*)p.out + row * p.stride, c8, v);
}

template <typename Kernel>
cudaError_t launch(Kernel k, const QuantizeParams& p, cudaStream_t s) {
  const uint32_t per_row = p.cols / 8;
  const uint64_t units = (uint64_t)p.rows * per_row;
  return launch_pdl(k, dim3((unsigned)((units + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, p, (uint32_t)units, per_row);
}

}  // namespace

cudaError_t launch_mx_quantize(const QuantizeParams& p, int x_dtype, int type, cudaStream_t s) {
  if (x_dtype == MOE_DT_F32)
    return type == MOE_MX_E4M3 ? launch(k_mx_quantize<false, true>, p, s) : launch(k_mx_quantize<false, false>, p, s);
  return type == MOE_MX_E4M3 ? launch(k_mx_quantize<true, true>, p, s) : launch(k_mx_quantize<true, false>, p, s);
}

cudaError_t launch_mx_dequantize(const QuantizeParams& p, int out_dtype, int type, cudaStream_t s) {
  if (out_dtype == MOE_DT_F32)
    return type == MOE_MX_E4M3 ? launch(k_mx_dequantize<false, true>, p, s) : launch(k_mx_dequantize<false, false>, p, s);
  return type == MOE_MX_E4M3 ? launch(k_mx_dequantize<true, true>, p, s) : launch(k_mx_dequantize<true, false>, p, s);
}

}  // namespace moe
