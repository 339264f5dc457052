// kv_append.cu — new keys and values into the paged cache, rotary positions
// applied on the way.
//
//   value pair (a, b) of a rotated head, angle theta = position * frequency:
//   a' = a cos - b sin,  b' = b cos + a sin   (fp32, one rounding to bf16)
//
// Each projection value is read once and written once, 16 bytes at a time, with
// no reuse and nothing to tile: bound by HBM for large batches (16,384 tokens of
// 56 + 8 + 8 heads of 128: 104 us, 5.9 TB/s), by launch and load latency for a
// decode step (8 tokens: 2.6 us).
#include "serve.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct V8 {
  float f[8];
};

template <typename T>
__device__ __forceinline__ V8 load8(const T* p);
template <>
__device__ __forceinline__ V8 load8<float>(const float* p) {
  V8 v;
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v.f[0] = a.x, v.f[1] = a.y, v.f[2] = a.z, v.f[3] = a.w, v.f[4] = b.x, v.f[5] = b.y, v.f[6] = b.z, v.f[7] = b.w;
  return v;
}
template <>
__device__ __forceinline__ V8 load8<uint16_t>(const uint16_t* p) {
  V8 v;
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v.f[2 * i] = __uint_as_float(w[i] << 16), v.f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  return v;
}

__device__ __forceinline__ void store8(uint16_t* p, const V8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v.f[0], v.f[1]), pack_bf16(v.f[2], v.f[3]),
                                            pack_bf16(v.f[4], v.f[5]), pack_bf16(v.f[6], v.f[7]));
}

// One CTA (or, for few tokens, several) per token; a thread takes 16 values
// of a head: two groups of 8 that are rotated together (values i and i +
// rot / 2, or neighbours), or two groups that are only converted.  All of a
// pair is read before any of it is written, so q_out may be q.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) k_kv_append(AppendParams p) {
  pdl_trigger();
  pdl_wait();
  const int n = blockIdx.x;
  int seq = n, i = 0, ql = 1;
  bool ok = true;
  if (p.b.q_start) {
    seq = find_sequence(p.b.q_start, p.b.batch, n);
    const int q0 = __ldg(&p.b.q_start[seq]), q1 = __ldg(&p.b.q_start[seq + 1]);
    i = n - q0;
    ql = q1 - q0;
    ok = q0 >= 0 && i >= 0 && i < ql && ql <= p.b.max_q;
  }
  const int len = __ldg(&p.b.kv_len[seq]);
  const long long j = (long long)len - ql + i;
  const long long pos = p.b.prefix_len + j;
  const int ps = p.c.page_size;
  ok = ok && j >= 0 && len <= (long long)p.b.table_pages * ps && (p.rot == 0 || pos < p.rope_rows);
  int page = -1;
  if (ok) page = __ldg(&p.b.table[(int64_t)seq * p.b.table_stride + j / ps]);
  if (!ok || page < 0 || page >= p.c.num_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  const int D = p.c.head_dim, units = D / 16, rot = p.rot;
  const int hq = p.q ? p.q_heads : 0, hk = p.c.kv_heads;
  const int items = (hq + 2 * hk) * units;
  const int64_t at = page * p.c.page_stride + (j % ps) * p.c.token_stride;
  const float* angle = p.rope + pos * rot;
  for (int it = blockIdx.y * kThreads + threadIdx.x; it < items; it += gridDim.y * kThreads) {
    const int head = it / units, u = it - head * units;
    const T* src;
    uint16_t* dst;
    bool turn = true;
    if (head < hq) {
      src = (const T*)p.q + n * p.q_stride + head * D;
      dst = p.q_out + n * p.q_out_stride + head * D;
    } else if (head < hq + hk) {
      src = (const T*)p.k + n * p.k_stride + (head - hq) * D;
      dst = (uint16_t*)p.c.k + at + (head - hq) * p.c.head_stride;
    } else {
      src = (const T*)p.v + n * p.v_stride + (head - hq - hk) * D;
      dst = (uint16_t*)p.c.v + at + (head - hq - hk) * p.c.head_stride;
      turn = false;
    }
    // The unit's two groups of 8: unit u < rot / 16 is rotated.
    const bool rotated = u < rot / 16;
    const int a = INTER || !rotated ? 16 * u : 8 * u;
    const int b = INTER || !rotated ? a + 8 : a + rot / 2;
    V8 x = load8<T>(src + a), y = load8<T>(src + b);
    if (turn && rotated) {
      const float4* c4 = reinterpret_cast<const float4*>(angle + 8 * u);
      const float4* s4 = reinterpret_cast<const float4*>(angle + rot / 2 + 8 * u);
      const float4 c0 = __ldg(c4), c1 = __ldg(c4 + 1), s0 = __ldg(s4), s1 = __ldg(s4 + 1);
      const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // Pair e: (x[e], y[e]), or neighbours 2e, 2e + 1 of the 16 values.
        float& va = INTER ? (e < 4 ? x.f[(2 * e) & 7] : y.f[(2 * e) & 7]) : x.f[e];
        float& vb = INTER ? (e < 4 ? x.f[(2 * e + 1) & 7] : y.f[(2 * e + 1) & 7]) : y.f[e];
        const float ra = va * c[e] - vb * s[e], rb = vb * c[e] + va * s[e];
        va = ra;
        vb = rb;
      }
    }
    store8(dst + a, x);
    store8(dst + b, y);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int x_dtype, bool interleaved, cudaStream_t s) {
  const int items = ((p.q ? p.q_heads : 0) + 2 * p.c.kv_heads) * (p.c.head_dim / 16);
  // A few tokens: one pass per thread, so that a step is one load latency deep.
  int ny = 1;
  if (p.b.tokens < 4 * kNumSMs) ny = (items + kThreads - 1) / kThreads;
  const dim3 grid(p.b.tokens, ny), block(kThreads);
  if (x_dtype == MOE_DT_F32)
    return interleaved ? launch_pdl(k_kv_append<float, true>, grid, block, 0, s, p)
                       : launch_pdl(k_kv_append<float, false>, grid, block, 0, s, p);
  return interleaved ? launch_pdl(k_kv_append<uint16_t, true>, grid, block, 0, s, p)
                     : launch_pdl(k_kv_append<uint16_t, false>, grid, block, 0, s, p);
}

}  // namespace moe
