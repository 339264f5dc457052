// attention_tc.cuh — the Tensor Memory side of attention (attention_split.cu),
// for parts that many query rows share: the prefix of a batch, and long new
// parts (prompts).
//
// Bound by the tensor cores from about 280 rows per key head on (2 * rows
// operations per cache byte against the chip's ratio of the two rates), by HBM
// below.  One CTA per SM takes a contiguous range of (row tile of 256, unit of
// 128 tokens) work.  Roles:
//   * a producer warp copies K and V units (128 tokens x head_dim) into a ring
//     of shared-memory buffers with tensor-map boxes, one per page;
//   * one thread issues the MMAs: S_t = Q_t K^T and O_t += P_t V for the two
//     128-row halves t of the tile, S and O in Tensor Memory (S_0, S_1, O_0,
//     O_1: 128 columns each, all 512 at head_dim 128);
//   * a warp walks the CTA's range and hands its segments on through shared
//     memory, so that the others hold no walk state (with it the softmax
//     spilled, and its spills went past the 28 KB that L1 has left);
//   * a warp prepares the values of units that not every row sees whole: what
//     lies past the end is cleared, and so are infinities and NaN of tokens that
//     only some rows see (0 * NaN is NaN), which the softmax warps add to the
//     sums of those rows;
//   * warpgroup t turns S_t into P_t = 2^(S_t scale - m) in bf16, written over
//     S_t, one row per thread, so that row sums and maxima need no exchange.
// While one half's softmax runs, the other half's MMAs do.  The reference m of
// a row moves only when its maximum grew by more than 2^8 (then the warpgroup
// rescales O_t in Tensor Memory): any reference gives the same quotient, and
// 2^8 keeps every partial sum far inside fp32.
//
// A unit takes 1.48 us with all SMs at work, 1.34 at the chip's measured tensor
// rate: 256 sequences of 56 query and 8 key heads over a shared prefix alone take
// 172 us for 32,768 tokens and 312 for 65,536, start-up and join included, 1.72
// PFLOP/s between the two.
#pragma once

#include "serve.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kHalfRows = 128;           // rows of an MMA tile
constexpr int kAttnThreads = 12 * 32;    // 2 x 4 softmax warps, producer, MMA, walk, edge values
constexpr int kBufs = 5;
constexpr int kSegs = 4;                 // segments handed from the walking warp to the others
constexpr uint32_t kTmemCols = 512;
// Registers: 168 a thread at launch (384 * 168 = 64,512); the softmax
// warpgroups take 224 each, which holds a row of 128 scores, and the third
// keeps 56: 128 * (224 + 224 + 56) = 64,512.
constexpr int kRegsSoftmax = 224, kRegsRest = 56;
constexpr float kGrow = 8.f;             // log2 of the growth a stale reference may see

template <int D>
struct TcCfg {
  static constexpr int kSub = kAttnTcUnit * 128;           // 128 rows x 64 values
  static constexpr int kMat = kSub * (D / 64);       // one operand tile
  static constexpr int kSmem = (2 + kBufs) * kMat;   // Q_0, Q_1, ring
};

struct TcShared {
  uint64_t full[kBufs], empty[kBufs];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t raw[kBufs];        // an edge unit's values have landed; `full` when they are prepared
  uint64_t odd_known[kSegs];
  AttnSeg seg[kSegs];
  uint64_t q_ready[2], s_full[2], p_ready[2][2], o_done[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ bool tc_wait(TcShared& sh, uint64_t* bar, uint32_t parity, const AttnParams& p) {
  const bool diag = p.wait_limit < kWaitCycles;
  if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&sh.abort_flag) return false;
    if (clock64() - t0 > p.wait_limit) {
      set_status_word(p.status, MOE_ERR_TIMEOUT);
      *(volatile int*)&sh.abort_flag = 1;
      return false;
    }
  }
}

// The MMAs are issued by converged code of the whole warp with a predicate
// that is true in one lane: in a divergent branch each operand goes through a
// vector-to-uniform move of its own, which measured 125 cycles an MMA.
// Descriptors are given by their low words (address >> 4, and the leading
// offset above it).
//
// High words: stride offset 1024 bytes, fixed bit, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// Low word of a K-major operand (leading offset unused).
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
// V as B operand [N = values][K = tokens]: N contiguous (128-byte swizzle
// atoms of 64 values x 8 tokens); 8-token groups 1024 bytes apart, the halves
// of 64 values (leading offset) one sub-tile apart.
template <int D>
__device__ __forceinline__ uint32_t desc_v(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)(TcCfg<D>::kSub >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " mov.b64 da, {%1, %6};\n mov.b64 db, {%2, %6};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " mov.b64 db, {%2, %6};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}

// Two fp32 values in one register pair, for the packed FMA and add.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The Tensor Memory side of the split kernel, for all kAttnThreads threads.
template <int D>
__device__ __forceinline__ void attn_tc_role(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                             const AttnPlan& plan, TcShared& sh, uint8_t* dyn) {
  using C = TcCfg<D>;
  constexpr int kUnit = kAttnTcUnit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnSide& sd = p.side[1];
  if (warp == 9) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.raw[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.q_ready[t], 4);
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_ready[t][0], 4);
      mbar_init(&sh.p_ready[t][1], 4);
      mbar_init(&sh.o_done[t], 1);
    }
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], 11);
      mbar_init(&sh.odd_known[i], 1);
    }
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  uint8_t* ring = dyn + 2 * C::kMat;
  // The n-th segment of the range, null past the last one or when a wait gave
  // up; release it when it is no longer read.
  uint32_t nseg = 0;
  auto take_seg = [&]() -> const AttnSeg* {
    const bool got = tc_wait(sh, &sh.seg_full[nseg % kSegs], (nseg / kSegs) & 1, p);
    const AttnSeg* g = &sh.seg[nseg % kSegs];
    return __all_sync(0xFFFFFFFFu, got) && g->slot >= 0 ? g : nullptr;
  };
  auto drop_seg = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.seg_empty[nseg % kSegs]);
    ++nseg;
  };
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 8) {
    // ------------------------------------------------------------ producer --
    const int box = attn_box(p.page_size, kUnit);
    int bi = 0, use = 0;
    uint32_t raw = 0, nraw = 0;  // by buffer: whether it was last used for edge values; how often, modulo 2
    bool ok = true;
    while (ok) {
      const AttnSeg* sg = take_seg();
      if (!sg) break;
      const AttnSeg g = *sg;
      const int common = attn_visible(p, g, g.row0 / p.group);  // tokens that every row sees
      drop_seg();
      const int32_t* table = attn_table(p, g.set);
      int kv = attn_first(p, g) - kUnit;
      for (int n = (g.kv1 - g.kv0 + kUnit - 1) / kUnit; n > 0 && ok; --n) {
        kv = kv + kUnit < g.kv1 ? kv + kUnit : g.kv0;
        const int left = g.kv1 - kv < kUnit ? g.kv1 - kv : kUnit;
        const int nb = (left + box - 1) / box;
        int page = 0, y = 0;
        if (lane < nb) {
          const int tok = kv + lane * box;
          page = __ldg(&table[tok >> p.page_shift]);
          if (page < 0 || page >= p.num_pages) {
            set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
            page = p.num_pages;  // past the map: the box is filled with zeros
          }
          y = tok & (p.page_size - 1);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          bool got = true;
          if (use > 0 && lane == 0) got = tc_wait(sh, &sh.empty[bi], (use - 1) & 1, p);
          if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
            ok = false;
            break;
          }
          const bool edge = m && common - kv < kUnit;
          raw = edge ? raw | 1u << bi : raw & ~(1u << bi);
          if (edge) nraw ^= 1u << bi;
          uint64_t* bar = edge ? &sh.raw[bi] : &sh.full[bi];
          if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(nb * box * D * 2));
          __syncwarp();
          if (lane < nb) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(ring + bi * C::kMat + h * C::kSub + lane * box * 128, m ? &vmap : &kmap, h * 64, y, g.kvh,
                          page, bar);
          }
          __syncwarp();
          if (++bi == kBufs) bi = 0, ++use;
        }
      }
    }
    // No copy may be in flight when the CTA exits.
    if (lane == 0)
      for (int i = 0; i < kBufs; ++i) {
        const int n = use + (i < bi ? 1 : 0);
        if (n > 0 && !(raw >> i & 1 ? mbar_wait(&sh.raw[i], (nraw >> i & 1) ^ 1) : mbar_wait(&sh.full[i], (n - 1) & 1)))
          set_status_word(p.status, MOE_ERR_TIMEOUT);
      }
    } else if (warp == 9) {
    // ----------------------------------------------------------------- MMA --
    const uint32_t id_s = idesc_bf16_f32(128, kUnit);
    const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // B: N contiguous
    const uint32_t qb = smem_u32(dyn), rb = smem_u32(ring);
    const uint32_t one = elect_one();  // commits track the electing lane's MMAs
    int bi = 0, use = 0;         // next ring buffer
    uint32_t nq = 0, np = 0;     // parities by half: of the segments, of the P tiles taken
    bool ok = true;
    auto all = [](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };
    auto take = [&](int& b) {    // the next ring buffer, filled
      b = bi;
      ok = ok && all(tc_wait(sh, &sh.full[bi], use & 1, p));
      if (++bi == kBufs) bi = 0, ++use;
    };
    auto scores = [&](int t, int b) {
      const uint32_t qa = desc_k(qb + t * C::kMat), ka = desc_k(rb + b * C::kMat);
#pragma unroll
      for (int kb = 0; kb < D / 16; ++kb) {
        const uint32_t off = ((kb >> 2) * C::kSub + 32 * (kb & 3)) >> 4;
        mma_ss(tmem + 128 * t, qa + off, ka + off, id_s, kb > 0, one);
      }
      commit_one(&sh.s_full[t], one);
    };
    // P_t V of one half: the two parts of 64 tokens as their weights arrive.
    auto values = [&](int t, int b, bool first) {
      const uint32_t va = desc_v<D>(rb + b * C::kMat);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ok = ok && all(tc_wait(sh, &sh.p_ready[t][k], np >> t & 1, p));
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int kb = 4 * k; kb < 4 * k + 4; ++kb)
          mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * kb, va + kb * (2048 >> 4), id_o, !first || kb > 0, one);
      }
      np ^= 1u << t;
    };
    // The buffers of the next unit are waited for while MMAs are queued: the
    // time between the last scores of a unit and the next P V is tensor idle.
    while (ok) {
      const AttnSeg* sg = take_seg();
      if (!sg) break;
      const int kv0 = sg->kv0, kv1 = sg->kv1;
      const bool two = sg->rows > kHalfRows;
      drop_seg();
      const int nt = (kv1 - kv0 + kUnit - 1) / kUnit;
      if (nt == 0) continue;
      int kbuf, vbuf;
      take(kbuf);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t == 1 && !two) break;
        ok = ok && all(tc_wait(sh, &sh.q_ready[t], nq >> t & 1, p));
        nq ^= 1u << t;
        if (!ok) break;
        tc_fence_after();
        scores(t, kbuf);
      }
      if (!ok) break;
      commit_one(&sh.empty[kbuf], one);
      take(vbuf);
      if (nt > 1) take(kbuf);
      for (int j = 0; j < nt && ok; ++j) {
        const bool more = j + 1 < nt;
        int vnext = 0, knext = 0;
        values(0, vbuf, j == 0);
        if (!ok) break;
        if (more) scores(0, kbuf);
        else commit_one(&sh.o_done[0], one);
        if (two) {
          values(1, vbuf, j == 0);
          if (!ok) break;
        }
        commit_one(&sh.empty[vbuf], one);
        if (more) {
          take(vnext);
          if (two) scores(1, kbuf);
          commit_one(&sh.empty[kbuf], one);
          if (j + 2 < nt) take(knext);
        } else if (two) {
          commit_one(&sh.o_done[1], one);
        }
        vbuf = vnext;
        kbuf = knext;
      }
    }
    // No MMA may be in flight when Tensor Memory is released.
    commit_one(&sh.drain, one);
    if (!mbar_wait(&sh.drain, 0)) set_status_word(p.status, MOE_ERR_TIMEOUT);
    } else if (warp == 10) {
      // -------------------------------------------------------------- walk --
      AttnWalk w;
      bool more = attn_begin(p, plan, 1, 0, w);
      for (;; ++nseg) {
        if (nseg >= (uint32_t)kSegs &&
            !__all_sync(0xFFFFFFFFu, tc_wait(sh, &sh.seg_empty[nseg % kSegs], (nseg / kSegs - 1) & 1, p)))
          break;
        AttnSeg g;
        g.slot = -1;
        more = more && attn_next<true>(p, plan, sd, w, g);
        if (!more) g.slot = -1;
        if (lane == 0) {
          sh.seg[nseg % kSegs] = g;
          mbar_arrive(&sh.seg_full[nseg % kSegs]);
        }
        __syncwarp();
        if (!more) break;
      }
    } else {
      // ------------------------------------------------------- edge values --
      uint32_t unit = 0, nraw = 0;  // units of all segments so far; by buffer: its edge values so far, modulo 2
      bool ok = true;
      for (;;) {
        if (!take_seg()) break;
        AttnSeg* sg = &sh.seg[nseg % kSegs];
        const int kv0 = sg->kv0, kv1 = sg->kv1, common = attn_visible(p, *sg, sg->row0 / p.group);
        bool odd = false;
        int kv = attn_first(p, *sg);
        for (int n = (kv1 - kv0 + kUnit - 1) / kUnit; n > 0; --n, ++unit, kv = kv + kUnit < kv1 ? kv + kUnit : kv0) {
          if (common - kv >= kUnit) continue;
          const uint32_t b = (2 * unit + 1) % kBufs;  // a unit's values follow its keys
          ok = __all_sync(0xFFFFFFFFu, tc_wait(sh, &sh.raw[b], nraw >> b & 1, p));
          if (!ok) break;
          nraw ^= 1u << b;
          uint8_t* v = ring + b * C::kMat;
          const int t0 = common > kv ? common - kv : 0, t1 = kv1 - kv < kUnit ? kv1 - kv : kUnit;
          odd |= clear_odd_values<D / 64>(v, C::kSub, t0, t1);
#pragma unroll 1
          for (int h = 0; h < D / 64; ++h) {
            for (int i = t1 * 8 + lane; i < kUnit * 8; i += 32)
              *reinterpret_cast<uint4*>(v + h * C::kSub + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[b]);
        }
        if (!ok) break;
        if (lane == 0) {
          sg->odd = odd;
          mbar_arrive(&sh.odd_known[nseg % kSegs]);
        }
        drop_seg();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax --
    const int t = warp >> 2, q = warp & 3;
    const int r = t * kHalfRows + q * 32 + lane;  // row of the tile
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
    const float c = p.scale_log2;
    uint32_t ns = 0, no = 0;
    bool ok = true;
    uint8_t* qd = dyn + t * C::kMat;
    for (;;) {
      const AttnSeg* sg = take_seg();
      if (!sg) break;
      if (t == 1 && sg->rows <= kHalfRows) {
        drop_seg();
        continue;
      }
      const int kv0 = sg->kv0, kv1 = sg->kv1;
      const int vis = r < sg->rows ? attn_visible(p, *sg, (sg->row0 + r) / p.group) : 0;
      const int vis_min = attn_visible(p, *sg, (sg->row0 + t * kHalfRows) / p.group);
      if (kv0 < kv1) {
        const int row0 = sg->row0, row_end = row0 + sg->rows, tok0 = sg->tok0, head0 = sg->kvh * p.group;
        // The warp's 32 query rows into the swizzled A tile, whole rows at a
        // time (one row per thread would take 32 lines per load).  The MMAs
        // that read the previous ones are complete: their scores came back.
        constexpr int L = D / 8, R = 32 / L;  // lanes of a row, rows of a pass
        const int rl = q * 32 + lane / L, ch = lane % L;
#pragma unroll 1
        for (int b = 0; b < 32 / R; b += 8) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = row0 + t * kHalfRows + rl + (b + k) * R;
            const int ii = rr / p.group;
            v[k] = rr < row_end
                       ? __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)(tok0 + ii) * p.q_stride +
                                                              (int64_t)(head0 + rr - ii * p.group) * D + 8 * ch))
                       : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(qd + (ch >> 3) * C::kSub + sw128_offset(rl + (b + k) * R, ch & 7)) = v[k];
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_ready[t]);
      }
      float m = -CUDART_INF_F, l = 0.f;
      int kv = attn_first(p, *sg);
      for (int n = (kv1 - kv0 + kUnit - 1) / kUnit; n > 0; --n) {
        ok = __all_sync(0xFFFFFFFFu, tc_wait(sh, &sh.s_full[t], ns++ & 1, p));
        if (!ok) break;
        tc_fence_after();
        if (kv + kUnit > vis_min) {
          // The few units with an edge: mask the scores where they are.
#pragma unroll 1
          for (int k = 0; k < kUnit; k += 32) {
            uint32_t x[32];
            tmem_ld32(ts + k, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kv + k + e >= vis) x[e] = 0xFF800000u;
            tmem_st32(ts + k, x);
          }
          tmem_st_wait();
        }
        uint32_t s[kUnit];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(ts + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * k));
        tmem_ld_wait();
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mx[k] = __uint_as_float(s[32 * k]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(s[32 * k + e])), __uint_as_float(s[32 * k + e + 1]));
          mx[k] = fmaxf(mx[k], __uint_as_float(s[32 * k + 31]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        // Weights of 64 tokens against the row's reference m.
        const uint64_t c2 = pack2(c, c);
        uint64_t sum[2] = {0, 0};
        auto weights = [&](const uint32_t* x, uint32_t* v, float ref) {
          const uint64_t r2 = pack2(-ref, -ref);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, r2), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[e & 1] = add2(sum[e & 1], pack2(a, b));
            v[e] = pack_bf16(a, b);
          }
        };
        auto give = [&](uint32_t* v, int k) {
          tmem_st32(ts + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_ready[t][k]);
        };
        uint32_t v[32];
        // The first half's weights against the old reference, while the
        // maximum is still being found; taken again if the reference moves.
        for (;;) {
          sum[0] = sum[1] = 0;
          weights(s, v, m == -CUDART_INF_F ? 0.f : m);
          if (!__any_sync(0xFFFFFFFFu, top > m + kGrow)) break;
          const float mn = top > m + kGrow ? top : m;
          if (__any_sync(0xFFFFFFFFu, m != -CUDART_INF_F)) {
            // O_t is complete up to the previous unit: its MMAs were issued
            // before the scores that just arrived.  Without a maximum in any
            // row it holds nothing yet, or zeros.
            const float f = m == mn ? 1.f : ex2(m - mn);
            l *= f;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              tmem_ld32(to + 32 * k, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
              tmem_st32(to + 32 * k, v);
            }
          }
          m = mn;
        }
        give(v, 0);
        weights(s + 64, v, m == -CUDART_INF_F ? 0.f : m);
        give(v, 1);
        float sa, sb;
        unpack2(add2(sum[0], sum[1]), sa, sb);
        l += sa + sb;
        kv += kUnit;
        if (kv >= sg->kv1) kv = sg->kv0;
      }
      if (!ok) break;
      float* slot = sd.slots + (int64_t)sg->slot * kAttnTcRows * (D + 2);
      const int rows = sg->rows;
      if (kv0 < kv1) {
        ok = __all_sync(0xFFFFFFFFu, tc_wait(sh, &sh.o_done[t], no++ & 1, p) && (sg->set == p.b.batch ||  // all rows see all of a prefix
                                         tc_wait(sh, &sh.odd_known[nseg % kSegs], (nseg / kSegs) & 1, p)));
        if (!ok) break;
        tc_fence_after();
        // Through this warp's part of the query tile, so that whole lines
        // leave: row = lane in, 8 lanes of a row out.
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t v[32];
          tmem_ld32(to + 32 * k, v);
          tmem_ld_wait();
          uint8_t* st = qd + q * 4096;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(st + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int rr = 4 * e + (lane >> 3), ro = t * kHalfRows + q * 32 + rr;
            const uint4 x = *reinterpret_cast<const uint4*>(st + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (ro < rows) *reinterpret_cast<uint4*>(slot + (int64_t)ro * D + 32 * k + 4 * (lane & 7)) = x;
          }
          __syncwarp();
        }
        tc_fence_before();
        const int w0 = t * kHalfRows + q * 32;
        if (__builtin_expect(sg->odd, 0)) add_odd_values<D>(p, *sg, w0, rows < w0 + 32 ? rows : w0 + 32, slot);
      }
      if (r < rows) {
        slot[kAttnTcRows * D + r] = m;
        slot[kAttnTcRows * (D + 1) + r] = l;
      }
      drop_seg();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace moe
