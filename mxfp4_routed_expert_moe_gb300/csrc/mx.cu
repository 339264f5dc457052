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
// contiguous; kPer such eights a lane, all loaded first (9,216 x 7,168 bf16 to MXFP4:
// 38 us with one, 27 with four, 6.2 TB/s; back: 34 and 26), or one where that
// leaves too few CTAs (61 x 7,168: 1.3 and 1.8 us).
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Unit u of eight values: row and place in the row.  WHOLE: rows follow one another
// without gaps in all operands, and count as one (of less than 2^34 values: a place
// in it counts 16-byte vectors, two an eight, in 32 bits).
template <bool WHOLE>
__device__ __forceinline__ void place(uint32_t u, uint32_t per_row, uint32_t& row, uint32_t& c8) {
  row = WHOLE ? 0u : u / per_row;
  c8 = WHOLE ? u : u - row * per_row;
}

template <bool BF16, bool E4M3, bool WHOLE, int kPer>
__global__ void __launch_bounds__(kThreads) k_mx_quantize(const QuantizeParams p, uint32_t units, uint32_t per_row) {
  pdl_trigger();
  pdl_wait();
  const uint32_t u0 = blockIdx.x * (kThreads * kPer) + threadIdx.x;
  Eight<BF16> e[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t u = u0 + j * kThreads;
    uint32_t row, c8;
    place<WHOLE>(u, per_row, row, c8);
    if (u < units) e[j].load((const uint8_t*)p.x + row * p.stride, c8);
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    // units is a multiple of 4: groups of four lanes stay whole.
    const uint32_t u = u0 + j * kThreads;
    if (u >= units) break;
    uint32_t row, c8;
    place<WHOLE>(u, per_row, row, c8);
    float v[8];
    e[j].get(v);
    mx_store8<E4M3>(v, p.mx.q + row * p.mx.q_stride, p.mx.s + row * p.mx.s_stride, c8);
  }
}

// Eight codes as they are held, and what they stand for times a scale.
template <bool E4M3>
struct Codes;
template <>
struct Codes<true> {
  uint2 c;
  __device__ __forceinline__ void load(const uint8_t* q, uint32_t c8) { c = reinterpret_cast<const uint2*>(q)[c8]; }
  __device__ __forceinline__ void get(float scale, float (&v)[8]) const {
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
  }
};
template <>
struct Codes<false> {
  uint32_t c;
  __device__ __forceinline__ void load(const uint8_t* q, uint32_t c8) { c = reinterpret_cast<const uint32_t*>(q)[c8]; }
  __device__ __forceinline__ void get(float scale, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f16x2_f32x2(e2m1x2_f16x2(c, i));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
};

template <bool BF16, bool E4M3, bool WHOLE, int kPer>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(const QuantizeParams p, uint32_t units, uint32_t per_row) {
  pdl_trigger();
  pdl_wait();
  const uint32_t u0 = blockIdx.x * (kThreads * kPer) + threadIdx.x;
  Codes<E4M3> c[kPer];
  uint32_t s[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t u = u0 + j * kThreads;
    uint32_t row, c8;
    place<WHOLE>(u, per_row, row, c8);
    if (u < units) {
      c[j].load(p.mx.q + row * p.mx.q_stride, c8);
      s[j] = p.mx.s[row * p.mx.s_stride + (c8 >> 2)];
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t u = u0 + j * kThreads;
    if (u >= units) break;
    uint32_t row, c8;
    place<WHOLE>(u, per_row, row, c8);
    float v[8];
    c[j].get(e8m0_f32(s[j]), v);
    Eight<BF16>::store((uint8_t*)p.out + row * p.stride, c8, v);
  }
}

struct Quantize {
  template <bool BF16, bool E4M3, bool WHOLE, int PER>
  static auto kernel() { return k_mx_quantize<BF16, E4M3, WHOLE, PER>; }
};
struct Dequantize {
  template <bool BF16, bool E4M3, bool WHOLE, int PER>
  static auto kernel() { return k_mx_dequantize<BF16, E4M3, WHOLE, PER>; }
};
template <typename D, bool BF16, bool E4M3>
cudaError_t launch(const QuantizeParams& p, cudaStream_t s) {
  const uint32_t per_row = p.cols / 8;
  const uint32_t units = (uint32_t)((uint64_t)p.rows * per_row);
  const bool whole = units < 1u << 31 &&
                     (p.rows == 1 || (p.stride == (int64_t)p.cols * (BF16 ? 2 : 4) &&
                                      p.mx.q_stride == (E4M3 ? p.cols : p.cols / 2) && p.mx.s_stride == p.cols / 32));
  const int per = units > 4u * kThreads * 4 * kNumSMs ? 4 : 1;
  auto kern = whole ? (per == 4 ? D::template kernel<BF16, E4M3, true, 4>() : D::template kernel<BF16, E4M3, true, 1>())
                    : (per == 4 ? D::template kernel<BF16, E4M3, false, 4>() : D::template kernel<BF16, E4M3, false, 1>());
  return launch_pdl(kern, dim3((units + (uint64_t)kThreads * per - 1) / (kThreads * per)), dim3(kThreads), 0, s, p, units, per_row);
}
template <typename D>
cudaError_t launch(const QuantizeParams& p, int dtype, int type, cudaStream_t s) {
  if (dtype == MOE_DT_F32) return type == MOE_MX_E4M3 ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
  return type == MOE_MX_E4M3 ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
}

}  // namespace

cudaError_t launch_mx_quantize(const QuantizeParams& p, int x_dtype, int type, cudaStream_t s) {
  return launch<Quantize>(p, x_dtype, type, s);
}
cudaError_t launch_mx_dequantize(const QuantizeParams& p, int out_dtype, int type, cudaStream_t s) {
  return launch<Dequantize>(p, out_dtype, type, s);
}

}  // namespace moe
