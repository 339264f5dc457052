// dense.cuh — parameters of the kernels behind moe_dense.h and the MX block
// arithmetic that they share.
//
// These kernels read operands by plain loads behind pdl_wait(): what the kernel before
// writes while this one has started already is not read-only for it, as the
// non-coherent path (ld.global.nc, __ldg) requires.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "moe_dense.h"

namespace moe {

// ------------------------------------------------------------- MX rounding --
// A block's scale from the bits of its largest magnitude (an integer maximum of
// magnitudes' bits: NaN above infinity above all numbers): the biased exponent
// less emax, not below 0; 255 where the block holds an infinity or a NaN.
template <bool E4M3>
__device__ __forceinline__ uint32_t mx_scale(uint32_t most_bits) {
  const int e = (int)(most_bits >> 23) - (E4M3 ? 8 : 2);
  return most_bits >= 0x7F800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}
// 2^(127 - s), by which elements are multiplied before rounding (exact); 0 for
// a block that reads as NaN.
__device__ __forceinline__ float mx_inverse(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }

// Eight values times `inv` as codes: 8 bytes of E4M3, or 4 bytes of E2M1.  The
// hardware's conversions round to nearest even and saturate; a block that reads
// as NaN (inv 0) has codes 0.
__device__ __forceinline__ uint32_t mx_pack_e2m1(const float (&v)[8], float inv) {
  if (inv == 0.f) return 0u;
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv), "f"(v[5] * inv),
        "f"(v[6] * inv), "f"(v[7] * inv));
  return r;
}
__device__ __forceinline__ uint32_t mx_pack4_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 h0, h1;\n cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n"
      " mov.b32 %0, {h0, h1};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint2 mx_pack_e4m3(const float (&v)[8], float inv) {
  if (inv == 0.f) return make_uint2(0u, 0u);
  return make_uint2(mx_pack4_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    mx_pack4_e4m3(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

__device__ __forceinline__ uint32_t most_bits8(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  return m;
}

// Eight values of a block whose 32 lie in four neighbouring lanes: codes and
// scale to row pointers q and s, c8 the index of the eight in the row.  All
// lanes of a group of four call it.
template <bool E4M3>
__device__ __forceinline__ void mx_store8(const float (&v)[8], uint8_t* q, uint8_t* s, uint32_t c8) {
  uint32_t m = most_bits8(v);
  const uint32_t group = 0xFu << (threadIdx.x & 28);
  uint32_t o = __shfl_xor_sync(group, m, 1);
  m = o > m ? o : m;
  o = __shfl_xor_sync(group, m, 2);
  m = o > m ? o : m;
  const uint32_t sc = mx_scale<E4M3>(m);
  const float inv = mx_inverse(sc);
  if (E4M3)
    reinterpret_cast<uint2*>(q)[c8] = mx_pack_e4m3(v, inv);
  else
    reinterpret_cast<uint32_t*>(q)[c8] = mx_pack_e2m1(v, inv);
  if ((c8 & 3u) == 0u) s[c8 >> 2] = (uint8_t)sc;
}

// ------------------------------------------------------------ rows of eight --
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
}
// Eight elements of a row of bf16 or fp32, as they are held.
template <bool BF16>
struct Eight;
template <>
struct Eight<true> {
  uint4 v;
  __device__ __forceinline__ void load(const void* row, uint32_t c8) { v = __ldcs(reinterpret_cast<const uint4*>(row) + c8); }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack8(v, x); }
  __device__ __forceinline__ static void store(void* row, uint32_t c8, const float (&x)[8]) {
    reinterpret_cast<uint4*>(row)[c8] = pack8(x);
  }
};
template <>
struct Eight<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* row, uint32_t c8) {
    a = __ldcs(reinterpret_cast<const float4*>(row) + 2 * c8);
    b = __ldcs(reinterpret_cast<const float4*>(row) + 2 * c8 + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ static void store(void* row, uint32_t c8, const float (&x)[8]) {
    reinterpret_cast<float4*>(row)[2 * c8] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(row)[2 * c8 + 1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// ------------------------------------------------------------------ launches --
struct MxRows {  // rows of an MX matrix
  uint8_t* q;
  uint8_t* s;
  int64_t q_stride, s_stride;
};

struct QuantizeParams {  // either direction
  uint32_t rows, cols;
  const void* x;
  void* out;
  int64_t stride;  // bytes between rows of x or out
  MxRows mx;
};
cudaError_t launch_mx_quantize(const QuantizeParams& p, int x_dtype, int type, cudaStream_t s);
cudaError_t launch_mx_dequantize(const QuantizeParams& p, int out_dtype, int type, cudaStream_t s);

struct NormParams {
  int rows, cols;
  const void *x, *res;
  void *res_out, *out;
  int64_t x_stride, res_stride, out_stride;  // bytes
  const float* weight;
  float eps;
  float most;  // a sum of squares below it is taken as it is
  MxRows mx;
};
// out: MOE_DT_F32, MOE_DT_BF16, or 2 + moe_mx_type.
cudaError_t launch_rms_norm(const NormParams& p, int x_dtype, int res_dtype, int out, cudaStream_t s);

struct LinearParams {
  int T, N, K;
  const uint8_t *xs, *ws;  // scales
  int64_t xs_stride, ws_stride;
  const void* add;
  void* out;
  int64_t add_stride, out_stride;  // elements
  int32_t* status;
  long long wait_limit;
};
cudaError_t launch_mx_linear(const LinearParams& p, const moe_mx& x, const moe_mx& w, int out_dtype, cudaStream_t s);

struct LogprobParams {
  int rows, vocab, top, chunk;
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
};
cudaError_t launch_token_logprobs(const LogprobParams& p, int dtype, cudaStream_t s);

}  // namespace moe
