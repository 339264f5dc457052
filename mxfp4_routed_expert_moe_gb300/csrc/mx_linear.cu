// mx_linear.cu — product of MX activations x [T][K] (MXFP8 or MXFP4) with MXFP4
// weights w [N][K], added to an addend.
//
// The tensor core takes both operands as they are stored: tcgen05.mma with block
// scales, A = 128 weight rows, B = up to 256 activation rows, fp32 accumulators in
// Tensor Memory (row i of the weights in lane i, activation row t in column t).
//   x E4M3: kind::mxf8f6f4, K = 32 an MMA; the copy engine spreads the weights'
//           4-bit codes to bytes on their way to shared memory;
//   x E2M1: kind::mxf4, K = 64 an MMA, both operands packed.
// Either way a slice of the inner size is 128 bytes of each operand row in shared
// memory (128 or 256 elements), four MMAs, and one or two 4-byte scale words a row.
//
// A CTA's warps: one copies operand tiles by tensor maps, one issues the MMAs, four
// bring scale words from global memory into the 32 x 4 word blocks that tcgen05.cp
// spreads to Tensor Memory, and write the result in the end.
#include <cooperative_groups.h>

#include "dense.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kRows = 128;           // weight rows of a tile
constexpr int kTileBytes = kRows * 128;
constexpr int kMaxNt = 256;          // activation rows of a tile
constexpr int kMaxStages = 8;
constexpr int kMaxCl = 8;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kSfWarp0 = 2, kSfWarps = 4;
constexpr int kThreads = (kSfWarp0 + kSfWarps) * 32;

// MX instruction descriptor of kind::mxf4 (E2M1 both, UE8M0 scales, K = 64): a_sf,
// b_sf are 0 or 2, the first of the two scale bytes.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t a_sf, uint32_t b_sf) {
  return (b_sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
         (a_sf << 29);
}
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes from shared memory to 32 lanes x 4 columns, in each of the
// four lane quarters.  In order with the MMAs that the same thread issues.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128u >> 4) << 32;  // eight rows of 16 bytes
  d |= (uint64_t)1u << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

struct LinShared {
  uint64_t full[kMaxStages];   // stage filled: the copies' bytes and the scale warps
  uint64_t empty[kMaxStages];  // stage consumed: tcgen05.commit
  uint64_t done;               // all MMAs of the tile
  uint32_t tmem_base;
  int abort_flag;
};

// What the launch fixes.
struct LinTile {
  int nt;            // activation rows of a tile, a multiple of 16
  int stages;
  uint32_t stage_bytes;
  int slices;        // of the whole inner size
  int per;           // of a CTA
  uint32_t tmem_cols;
};

struct LinCtx {
  LinShared* sh;
  int32_t* status;
  long long wait_limit;
};

__device__ __forceinline__ bool lin_wait(const LinCtx& c, uint64_t* bar, uint32_t parity) {
  LinShared& sh = *c.sh;
  const bool diag = c.wait_limit < kWaitCycles;
  if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&sh.abort_flag) return false;
    if (clock64() - t0 > c.wait_limit) {
      if (c.status) atomicCAS((unsigned*)c.status, 0u, (unsigned)MOE_ERR_TIMEOUT);
      *(volatile int*)&sh.abort_flag = 1;
      return false;
    }
  }
}

// Scale words of one row: 16 bytes (four words) a step.
struct ScaleRow {
  const uint32_t* p;  // word 0, or null: a row past the end reads as scale 1
  int words;
  bool wide;
  __device__ __forceinline__ uint4 load(int w) const {
    const uint32_t one = 0x7F7F7F7Fu;
    if (!p || w >= words) return make_uint4(one, one, one, one);
    if (wide && w + 4 <= words) return __ldg(reinterpret_cast<const uint4*>(p + w));
    uint4 v = make_uint4(one, one, one, one);
    v.x = __ldg(p + w);
    if (w + 1 < words) v.y = __ldg(p + w + 1);
    if (w + 2 < words) v.z = __ldg(p + w + 2);
    if (w + 3 < words) v.w = __ldg(p + w + 3);
    return v;
  }
};

template <bool F4>
struct LinCfg {
  static constexpr int kWords = F4 ? 2 : 1;  // scale words of a row in a slice
  static constexpr int kSfBytes = 512 * kWords;  // of 128 rows
};

// Scale bytes and Tensor Memory columns of a stage.
template <bool F4>
__host__ __device__ constexpr uint32_t sf_bytes(int nt) { return LinCfg<F4>::kSfBytes * (1 + (nt + 127) / 128); }
template <bool F4>
__host__ __device__ constexpr uint32_t sf_cols(int nt) { return 4 * LinCfg<F4>::kWords * (1 + (nt + 127) / 128); }

// One tile, its inner size cut among the CTAs of a cluster, which add their sums in
// rank order through distributed shared memory.
template <bool F4, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads) k_linear(const LinearParams p, const LinTile t,
                                                     const __grid_constant__ CUtensorMap wmap,
                                                     const __grid_constant__ CUtensorMap xmap) {
  using C = LinCfg<F4>;
  extern __shared__ uint8_t lin_dyn[];
  __shared__ LinShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_dyn) + 1023) & ~(uintptr_t)1023);
  const int n0 = (blockIdx.x / cl) * kRows, t0 = blockIdx.y * t.nt;
  const int s0 = rank * t.per, s1 = min(s0 + t.per, t.slices);
  const int ns = s1 > s0 ? s1 - s0 : 0;
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, t.tmem_cols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < t.stages; ++i) {
      mbar_init(&sh.full[i], 1 + kSfWarps);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  LinCtx c = {&sh, p.status, p.wait_limit};
  // Not before Tensor Memory is held: a CTA of the next kernel that took it would
  // wait for this one to end.
  pdl_trigger();
  const uint32_t x_off = kTileBytes, sf_off = x_off + t.nt * 128;
  pdl_wait();

  if (warp == kTmaWarp) {
    if (lane == 0) {
      const uint32_t tx = (F4 ? kTileBytes : kTileBytes / 2) + (uint32_t)t.nt * 128;
      for (int i = 0; i < ns; ++i) {
        const int st = i % t.stages, use = i / t.stages;
        if (use > 0 && !lin_wait(c, &sh.empty[st], (use - 1) & 1)) break;
        uint8_t* sb = ring + (size_t)st * t.stage_bytes;
        mbar_arrive_expect_tx(&sh.full[st], tx);
        tma_load_2d(sb, &wmap, (s0 + i) * 128, n0, &sh.full[st]);
        tma_load_2d(sb + x_off, &xmap, (s0 + i) * 128, t0, &sh.full[st]);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < ns; ++i) {
        const int st = i % t.stages;
        if (!lin_wait(c, &sh.full[st], (i / t.stages) & 1)) break;
        tc_fence_after();
        const uint32_t sbase = smem_u32(ring + (size_t)st * t.stage_bytes);
        const uint32_t sfa = tmem + (uint32_t)t.nt + (uint32_t)st * sf_cols<F4>(t.nt);
        const uint32_t sfb = sfa + 4 * C::kWords;
        const int nb = (t.nt + 127) / 128;
#pragma unroll
        for (int w = 0; w < C::kWords; ++w) {
          tmem_cp_scales(sfa + 4 * w, sbase + sf_off + 512 * w);
          for (int b = 0; b < nb; ++b)
            tmem_cp_scales(sfb + 4 * (w * nb + b), sbase + sf_off + C::kSfBytes + 512 * (w * nb + b));
        }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          const uint64_t ad = sdesc_sw128(sbase + 32 * kb), bd = sdesc_sw128(sbase + x_off + 32 * kb);
          const uint32_t acc = (i > 0 || kb > 0) ? 1u : 0u;
          if (F4) {
            const uint32_t id = 2 * (kb & 1);
            umma_mxf4(tmem, ad, bd, idesc_mxf4(kRows, t.nt, id, id), sfa + 4 * (kb >> 1), sfb + 4 * nb * (kb >> 1), acc);
          } else {
            umma_mx(tmem, ad, bd, idesc_mx_f32(kRows, t.nt, kMxE2M1, kMxE4M3, kb, kb), sfa, sfb, acc);
          }
        }
        umma_commit(&sh.empty[st]);
      }
      umma_commit(&sh.done);
      // Everything issued has finished before Tensor Memory is released.
      if (!mbar_wait(&sh.done, 0) && p.status) atomicCAS((unsigned*)p.status, 0u, (unsigned)MOE_ERR_TIMEOUT);
    }
  } else {
    const int i = tid - kSfWarp0 * 32;  // weight row; activation rows i and i + 128
    const int words = p.K / 128, w0 = s0 * C::kWords;
    const int nb = (t.nt + 127) / 128;
    auto row = [&](const uint8_t* base, int64_t stride, int at, int rows) {
      ScaleRow s;
      s.p = at < rows ? reinterpret_cast<const uint32_t*>(base + at * stride) + w0 : nullptr;
      s.words = words - w0;
      s.wide = (((uintptr_t)base | (uintptr_t)stride | (uintptr_t)(4 * w0)) & 15) == 0;
      return s;
    };
    const ScaleRow rw = row(p.ws, p.ws_stride, n0 + i, p.N);
    const ScaleRow rx0 = row(p.xs, p.xs_stride, t0 + i, i < t.nt ? p.T : 0);
    const ScaleRow rx1 = row(p.xs, p.xs_stride, t0 + 128 + i, 128 + i < t.nt ? p.T : 0);
    constexpr int PER = 4 / C::kWords;  // slices of a step of four words
    uint4 vw = rw.load(0), va = rx0.load(0), vb = rx1.load(0);
    bool ok = true;
    for (int g = 0; g < ns && ok; g += PER) {
      const int next = (g + PER) * C::kWords;
      const bool more = g + PER < ns;
      const uint4 nw = more ? rw.load(next) : vw, na = more ? rx0.load(next) : va, nbv = more && nb > 1 ? rx1.load(next) : vb;
      const uint32_t a[4] = {vw.x, vw.y, vw.z, vw.w}, b0[4] = {va.x, va.y, va.z, va.w}, b1[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int sl = g + j;
        if (sl >= ns) break;
        const int st = sl % t.stages, use = sl / t.stages;
        ok = use == 0 || lin_wait(c, &sh.empty[st], (use - 1) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint32_t* sf = reinterpret_cast<uint32_t*>(ring + (size_t)st * t.stage_bytes + sf_off) + (i & 31) * 4 + (i >> 5);
#pragma unroll
        for (int w = 0; w < C::kWords; ++w) {
          sf[128 * w] = a[j * C::kWords + w];
          sf[128 * (C::kWords + w * nb)] = b0[j * C::kWords + w];
          if (nb > 1) sf[128 * (C::kWords + w * nb + 1)] = b1[j * C::kWords + w];
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[st]);
      }
      vw = nw, va = na, vb = nbv;
    }
    // The sums, by way of shared memory (the ring is free) where others add to
    // them: token t's 128 in a row.
    const int q = warp & 3;
    const int valid = min(t.nt, p.T - t0);
    const bool fine = __all_sync(0xFFFFFFFFu, lin_wait(c, &sh.done, 0));
    tc_fence_after();
    const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
    float* stage = reinterpret_cast<float*>(ring);
    const int n = n0 + q * 32 + lane;
    for (int c0 = 0; c0 < valid; c0 += 16) {
      uint32_t v[16];
      if (ns > 0 && fine) {
        tmem_ld16(tbase + (uint32_t)c0, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0u;
      }
      if (cl > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < valid) stage[(c0 + e) * kRows + q * 32 + lane] = __uint_as_float(v[e]);
      } else if (n < p.N) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < valid) {
            const int64_t tt = t0 + c0 + e;
            float y = __uint_as_float(v[e]);
            if (OUT_BF16) {
              if (p.add) y += bf16_f32(((const uint16_t*)p.add)[tt * p.add_stride + n]);
              ((uint16_t*)p.out)[tt * p.out_stride + n] = (uint16_t)(bf16x2_rn(y, 0.f) & 0xFFFFu);
            } else {
              if (p.add) y += ((const float*)p.add)[tt * p.add_stride + n];
              ((float*)p.out)[tt * p.out_stride + n] = y;
            }
          }
      }
    }
    tc_fence_before();
  }
  if (cl > 1) {
    cluster.sync();
    // This CTA's share of the rows: kRows / cl of each token's.
    const float* stage = reinterpret_cast<const float*>(ring);
    const int valid = min(t.nt, p.T - t0), share = kRows / cl;
    const float* from[kMaxCl];
#pragma unroll
    for (int j = 0; j < kMaxCl; ++j) from[j] = j < cl ? cluster.map_shared_rank(stage, j) : nullptr;
    for (int i = tid; i < valid * share; i += kThreads) {
      const int tt = i / share, rr = rank * share + i % share, n = n0 + rr;
      float y = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxCl; ++j)
        if (j < cl) y += from[j][tt * kRows + rr];
      if (n < p.N) {
        const int64_t at = t0 + tt;
        if (OUT_BF16) {
          if (p.add) y += bf16_f32(((const uint16_t*)p.add)[at * p.add_stride + n]);
          ((uint16_t*)p.out)[at * p.out_stride + n] = (uint16_t)(bf16x2_rn(y, 0.f) & 0xFFFFu);
        } else {
          if (p.add) y += ((const float*)p.add)[at * p.add_stride + n];
          ((float*)p.out)[at * p.out_stride + n] = y;
        }
      }
    }
    cluster.sync();  // no CTA leaves while its sums are read
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort_flag) {
    // A wait gave up: copies may be in flight, and have to land before the CTA may
    // exit.  Their barriers miss other arrivals, so a time is waited that covers any.
    const long long w0 = clock64();
    while (clock64() - w0 < 20000000) __nanosleep(1000);
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, t.tmem_cols);
  }
}

// Tensor map of an operand: rows of `row_bytes` bytes of codes, boxes of 128 bytes
// of shared memory by `rows` rows, 128-byte swizzle.  spread: 4-bit codes that take
// a byte each in shared memory.  Rows and columns past the end read as zero.
cudaError_t operand_map(CUtensorMap* m, const moe_mx& a, bool spread, int rows) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t row_elems = spread ? a.cols : (a.type == MOE_MX_E4M3 ? a.cols : a.cols / 2);
  const cuuint64_t dims[2] = {row_elems, (cuuint64_t)a.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)a.q_stride};
  const cuuint32_t box[2] = {128, (cuuint32_t)rows};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = enc(m, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.q, dims,
                         strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool F4, bool OUT_BF16>
cudaError_t launch(const LinearParams& p, const moe_mx& x, const moe_mx& w, cudaStream_t s) {
  LinTile t;
  const int tiles_t = (p.T + kMaxNt - 1) / kMaxNt;
  t.nt = ((p.T + tiles_t - 1) / tiles_t + 15) & ~15;
  t.slices = (p.K + (F4 ? 255 : 127)) / (F4 ? 256 : 128);
  const int tiles_n = (p.N + kRows - 1) / kRows;
  // CTAs of a tile: while all run at once and each has four slices.
  int cl = 1;
  while (cl < kMaxCl && (long long)tiles_n * tiles_t * cl * 2 <= kNumSMs && t.slices >= 8 * cl) cl *= 2;
  t.per = (t.slices + cl - 1) / cl;
  t.stage_bytes = (uint32_t)align_up(kTileBytes + t.nt * 128 + sf_bytes<F4>(t.nt), 1024);
  t.stages = (int)(220 * 1024 / t.stage_bytes);
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  const uint32_t cols = t.nt + t.stages * sf_cols<F4>(t.nt);
  t.tmem_cols = 32;
  while (t.tmem_cols < cols) t.tmem_cols *= 2;
  const size_t smem = (size_t)t.stages * t.stage_bytes + 1024;
  CUtensorMap wmap, xmap;
  cudaError_t err;
  if ((err = operand_map(&wmap, w, !F4, kRows)) != cudaSuccess || (err = operand_map(&xmap, x, false, t.nt)) != cudaSuccess)
    return err;
  auto kern = k_linear<F4, OUT_BF16>;
  if ((err = ensure_smem_attr((const void*)kern, smem)) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles_n * cl), (unsigned)tiles_t);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, t, wmap, xmap);
}

}  // namespace

cudaError_t launch_mx_linear(const LinearParams& p, const moe_mx& x, const moe_mx& w, int out_dtype, cudaStream_t s) {
  if (x.type == MOE_MX_E2M1)
    return out_dtype == MOE_DT_BF16 ? launch<true, true>(p, x, w, s) : launch<true, false>(p, x, w, s);
  return out_dtype == MOE_DT_BF16 ? launch<false, true>(p, x, w, s) : launch<false, false>(p, x, w, s);
}

}  // namespace moe
