// attention_warp.cuh — the warp side of attention: 16 query rows a warp on
// m16n8k16 MMAs (attention_split.cu, and the tile kernel of attention.cu).
#pragma once

#include "serve.cuh"
#include "tcgen05.cuh"

namespace moe {

// For parts of at most 16 query rows per key head: decode.  Bound by HBM: 4 *
// head_dim bytes per token and key head against 4 * head_dim * rows
// operations, so warp MMAs (m16n8k16) keep up, and 16 rows waste less than a
// Tensor Memory tile of 128.  Every warp is a worker of its own: it copies the
// K and V of its next units (16 KB: 32 tokens of 128, 64 of 64) into its own ring of shared memory
// with tensor-map boxes and takes them in turn, so that no warp waits for
// another and short sequences cost no CTA-wide joins (four warps that shared
// each unit spent 1.0 us of a 3.2 us one-unit segment on joining).  48 sequences
// of up to 32,768 tokens, with the join: 6.6 TB/s with 8 key heads of 128 (492
// us), 6.0 TB/s with 4 of 64 and 16 query heads each (135 us).
constexpr int kWorkers = kAttnWarpWorkers;

template <int D>
struct WarpCfg {
  static constexpr int kUnit = attn_warp_unit(D);
  static constexpr int kHalf = kUnit * 128;            // bytes of a unit's tokens x 64 dims
  static constexpr int kMat = kHalf * (D / 64);        // K or V of a stage
  static constexpr int kStage = 2 * kMat;              // 16 KB
  static constexpr int kStages = 2;
  static constexpr int kSmem = kWorkers * kStages * kStage;
};

constexpr int kWarpSegs = 4;
struct WarpShared {
  uint64_t full[kWorkers][2];
  AttnSeg seg[kWorkers][kWarpSegs];  // segments between the loads and the sums
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a (16 x 16, row) * b (16 x 8, col), bf16 in, fp32 out.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The rows of a 16-row tile as one warp holds them: lane l has rows l / 4 and
// l / 4 + 8 in MMA fragments.
template <int D>
struct WarpRows {
  static constexpr int NT = D / 8, kUnit = WarpCfg<D>::kUnit;
  uint32_t qf[D / 16][4];
  float o[NT][4];
  float m[2], l[2];

  // Rows row0 .. row0 + rows - 1 of a set whose first token is tok0.
  __device__ __forceinline__ void load(const AttnParams& p, int tok0, int kvh, int row0, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      const bool in = r < rows;
      const int rr = row0 + (in ? r : 0), i = rr / p.group;
      const uint16_t* src = p.q + (int64_t)(tok0 + i) * p.q_stride + (int64_t)(kvh * p.group + rr - i * p.group) * D +
                            2 * (lane & 3);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][h] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk)) : 0u;
        qf[kk][h + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8)) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.f;
  }

  // One unit: its tokens of K and V in a stage of the warp's ring.  Every row
  // of the tile sees the first `all` tokens (all, if that is kUnit or more), row
  // h the first see[h], and the V rows from n on are not to be used.  True if
  // values were taken out (clear_odd_values).
  __device__ __forceinline__ bool unit(uint8_t* stage, float scale_log2, int all, const int (&see)[2], int n) {
    using C = WarpCfg<D>;
    constexpr int kHalf = C::kHalf;
    const int lane = threadIdx.x & 31;
    const uint32_t kb = smem_u32(stage), vb = kb + C::kMat;
    const bool edge = all < kUnit;
    bool odd = false;
    if (edge) {
      // Rows of V past the length may hold anything, and 0 * NaN is NaN.
      for (int i = n * 8 + lane; i < kUnit * 8; i += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<uint4*>(stage + C::kMat + h * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
      odd = all < n && clear_odd_values<D / 64>(stage + C::kMat, kHalf, all < 0 ? 0 : all, n < kUnit ? n : kUnit);
      // Before the tensor-map copy that refills the stage (the async proxy).
      fence_async_smem();
      __syncwarp();
    }
    float sc[kUnit / 8][4];
#pragma unroll
    for (int i = 0; i < kUnit / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int j = 0; j < kUnit / 16; ++j) {
        const int tok = 16 * j + (lane & 7) + ((lane >> 4) << 3);
        const int c = (kk & 3) * 2 + ((lane >> 3) & 1);
        uint32_t b[4];
        ldsm4(kb + (kk >> 2) * kHalf + tok * 128 + ((c ^ (tok & 7)) << 4), b);
        mma_bf16(sc[2 * j], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b[0], b[1]);
        mma_bf16(sc[2 * j + 1], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b[2], b[3]);
      }
    }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int i = 0; i < kUnit / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float t = sc[i][e] * scale_log2;
        if (edge && 8 * i + 2 * (lane & 3) + (e & 1) >= see[e >> 1]) t = -CUDART_INF_F;
        sc[i][e] = t;
        mx[e >> 1] = fmaxf(mx[e >> 1], t);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
    }
    if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = mx[h] > m[h] ? ex2(m[h] - mx[h]) : 1.f;
        m[h] = mx[h];
        l[h] *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][2 * h] *= f, o[i][2 * h + 1] *= f;
      }
    }
    const float ms[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
#pragma unroll
    for (int j = 0; j < kUnit / 16; ++j) {
      uint32_t a[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* s4 = sc[2 * j + i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s4[e] = ex2(s4[e] - ms[e >> 1]);
          l[e >> 1] += s4[e];
        }
        // bf16 weights: at most 2^-8 relative each, averaged over the sum,
        // below the rounding of the bf16 output.
        a[2 * i] = pack_bf16(s4[0], s4[1]);
        a[2 * i + 1] = pack_bf16(s4[2], s4[3]);
      }
#pragma unroll
      for (int t = 0; t < NT; t += 2) {
        const int tok = 16 * j + (lane & 15);
        const int c = (t & 7) + (lane >> 4);
        uint32_t b[4];
        ldsm4t(vb + (t >> 3) * kHalf + tok * 128 + ((c ^ (tok & 7)) << 4), b);
        mma_bf16(o[t], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma_bf16(o[t + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
      }
    }
    return odd;
  }

  // The four lanes of a row add up its sum.
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
    }
  }

  // o to rows of D at `dst`, m and l to ml[row], ml[16 + row].
  __device__ __forceinline__ void store(float* dst, float* ml, int rows) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if (r >= rows) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(dst + r * D + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
      if ((lane & 3) == 0) {
        ml[r] = m[h];
        ml[kAttnWarpRows + r] = l[h];
      }
    }
  }
};

// The warp side of the split kernel: warp `warp` of the CTA is a worker.  Its
// barriers (sh.full[warp]) are initialised; the plan is made.
//
template <int D>
__device__ __forceinline__ void attn_warp_role(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                               const AttnPlan& plan, WarpShared& sh, uint8_t* dyn) {
  using C = WarpCfg<D>;
  constexpr int kUnit = C::kUnit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnSide& sd = p.side[0];
  AttnWalk w;
  if (!attn_begin(p, plan, 0, warp, w)) return;
  uint8_t* ring = dyn + warp * (C::kStages * C::kStage);
  uint64_t* full = sh.full[warp];
  AttnSeg* segs = sh.seg[warp];
  // ------------------------------------------------------------------ loads --
  // A stage holds min(page, unit)-token boxes of K and V: lane i issues box i / 4
  // of matrix i % 2, half (i / 2) % 2 of the dims.  Page ids are read one unit
  // ahead.
  const int box = attn_box(p.page_size, kUnit);
  const int my_box = lane >> 2, my_half = (lane >> 1) & 1, my_v = lane & 1;
  const bool my_lane = my_half < D / 64 && my_box * box < kUnit;
  AttnSeg lg = {};
  int lkv = 0, lpage = 0;
  bool lready = false, lmore = true;         // a unit to load is known; there may be more segments
  uint32_t ln = 0, seg_in = 0, seg_out = 0;  // units loaded; segments passed on, taken
  uint32_t un = 0;                           // units taken
  auto fetch_page = [&] {
    const int tok = lkv + my_box * box;
    lpage = my_lane && tok < lg.kv1 ? __ldg(&attn_table(p, lg.set)[tok >> p.page_shift]) : 0;
  };
  // Find the next unit to load.  Segments are passed on as they come (an empty
  // one has no unit), as far as the queue has room.
  auto advance = [&] {
    while (!lready && lmore && seg_in - seg_out < (uint32_t)kWarpSegs) {
      lmore = attn_next<false>(p, plan, sd, w, lg);
      if (!lmore) break;
      if (lane == 0) segs[seg_in % kWarpSegs] = lg;
      ++seg_in;
      lkv = lg.kv0;
      lready = lkv < lg.kv1;
      if (lready) fetch_page();
    }
  };
  // Load units while there are units and free stages (`issue` false: only look
  // for the first one).
  auto fill = [&](bool issue) {
    advance();
    while (issue && lready && ln - un < (uint32_t)C::kStages) {
      const int st = ln % C::kStages;
      const int left = lg.kv1 - lkv < kUnit ? lg.kv1 - lkv : kUnit;
      const int nb = (left + box - 1) / box;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nb * box * D * 4));
      __syncwarp();
      if (my_lane && my_box < nb) {
        int page = lpage;
        if (page < 0 || page >= p.num_pages) {
          set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
          page = p.num_pages;  // past the map: the box is filled with zeros
        }
        tma_load_4d(ring + st * C::kStage + my_v * C::kMat + my_half * C::kHalf + my_box * box * 128,
                    my_v ? &vmap : &kmap, my_half * 64, (lkv + my_box * box) & (p.page_size - 1), lg.kvh, page, &full[st]);
      }
      ++ln;
      lkv += kUnit;
      lready = lkv < lg.kv1;
      if (lready) fetch_page();
      else advance();
    }
    __syncwarp();
  };
  // ------------------------------------------------------------------- sums --
  // The first segment's queries are asked for before the first keys: all
  // workers' first loads together keep HBM busy for 5 us, and what is asked for
  // after them waits that long.
  WarpRows<D> rows;
  AttnSeg g;
  int kv = 0, vis[2] = {0, 0}, vis_min = 0;
  bool issue = false, in_seg = false;
  const float scale = p.scale_log2;
  for (;;) {
    fill(issue);
    if (!in_seg) {
      if (seg_out == seg_in) break;
      g = segs[seg_out % kWarpSegs];
      rows.load(p, g.tok0, g.kvh, g.row0, g.rows);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (lane >> 2) + 8 * h;
        vis[h] = r < g.rows ? attn_visible(p, g, (g.row0 + r) / p.group) : 0;
      }
      // Units that end above the first row's tokens need the mask.
      vis_min = attn_visible(p, g, g.row0 / p.group);
      kv = g.kv0;
      in_seg = true;
      if (!issue) {
        issue = true;
        continue;
      }
    }
    if (kv < g.kv1) {
      const int st = un % C::kStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_for(&full[st], (un / C::kStages) & 1, p.wait_limit))) {
        set_status_word(p.status, MOE_ERR_TIMEOUT);
        break;
      }
      const int see[2] = {vis[0] - kv, vis[1] - kv};
      if (rows.unit(ring + st * C::kStage, scale, vis_min - kv, see, g.kv1 - kv)) segs[seg_out % kWarpSegs].odd = 1;
      ++un;
      kv += kUnit;
      __syncwarp();  // every lane has read the stage
    }
    if (kv >= g.kv1) {
      rows.close();
      float* slot = sd.slots + (int64_t)g.slot * kAttnWarpRows * (D + 2);
      rows.store(slot, slot + kAttnWarpRows * D, g.rows);
      const AttnSeg& whole = segs[seg_out % kWarpSegs];
      if (__builtin_expect(whole.odd, 0)) add_odd_values<D>(p, whole, 0, whole.rows, slot);
      ++seg_out;
      in_seg = false;
    }
  }
  // No copy may be in flight when the warp leaves its ring.
  for (uint32_t i = ln > (uint32_t)C::kStages ? ln - C::kStages : 0u; i < ln; ++i)
    if (!mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1)) set_status_word(p.status, MOE_ERR_TIMEOUT);
}

}  // namespace moe
