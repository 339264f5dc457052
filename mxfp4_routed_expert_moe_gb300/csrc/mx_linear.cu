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
// bring the scales to Tensor Memory, the epilogue's warps write the results.
//
// Scales lie in rows as stored, 16 bytes (four words) a row at a time; the MMA
// wants the words of rows l, l + 32, l + 64, l + 96 side by side in lane l, in each
// of the four lane quarters.  The four warps read a row a thread, several steps
// ahead, exchange the words through shared memory and store them with tcgen05.st,
// four words (two or four slices) a step.  (By tcgen05.cp from shared memory, with a
// proxy fence after the writes of each slice and releases of the cluster's scope, a
// slice took 1 us: fences wait for the thread's loads in flight as well.)
#include <type_traits>

#include "dense.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;           // weight rows of a tile
constexpr int kTileBytes = kRows * 128;
constexpr int kMaxNt = 256;          // activation rows of a tile
constexpr int kMaxStages = 8;
constexpr int kMaxCl = 8;
constexpr int kSfRing = 3;           // steps of scales in Tensor Memory
constexpr int kTmaWarp = 0, kMmaWarp = 1, kSfWarp0 = 2, kSfWarps = 4;
constexpr int kThreads = (kSfWarp0 + kSfWarps) * 32;
constexpr int kSfBarrier = 1;        // named barrier of the scale warps

// Instruction descriptor of kind::mxf4 (E2M1 both, UE8M0 scales, K = 64): a_sf,
// b_sf are 0 or 2, the first of the two scale bytes.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t a_sf, uint32_t b_sf) {
  return (b_sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
         (a_sf << 29);
}

// ------------------------------------------- instructions of one CTA or a pair --
// G = 1: one CTA's tile; G = 2: a pair's, issued by its first CTA for both.  The
// whole warp runs the issuing code with a predicate (`one`) that is true in one lane:
// in a divergent branch every operand goes through a vector-to-uniform move of its
// own (an MMA took 90 cycles).  Descriptors of operands are given by their low words.
//
// High words: stride offset 1024 bytes, fixed bit, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}
template <int G>
__device__ __forceinline__ void mma_mx(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, bool acc,
                                       uint32_t one) {
  if (G == 1)
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n mov.b64 da, {%1, %8};\n"
        " mov.b64 db, {%2, %8};\n"
        " @e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)acc), "r"(one), "n"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n mov.b64 da, {%1, %8};\n"
        " mov.b64 db, {%2, %8};\n"
        " @e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)acc), "r"(one), "n"(kDescHigh)
        : "memory");
}
template <int G>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, bool acc,
                                         uint32_t one) {
  if (G == 1)
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n mov.b64 da, {%1, %8};\n"
        " mov.b64 db, {%2, %8};\n"
        " @e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)acc), "r"(one), "n"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n mov.b64 da, {%1, %8};\n"
        " mov.b64 db, {%2, %8};\n"
        " @e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)acc), "r"(one), "n"(kDescHigh)
        : "memory");
}
// Arrive on the barrier (of both CTAs of a pair) when all that the elected lane
// issued has completed.
template <int G>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t one) {
  if (G == 1)
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3), "r"(one)
        : "memory");
}
template <int G>
__device__ __forceinline__ void lin_alloc(uint32_t* dst, uint32_t cols) {
  if (G == 1) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ __forceinline__ void lin_dealloc(uint32_t taddr, uint32_t cols) {
  if (G == 1)
    tmem_dealloc(taddr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Address of rank's copy of a shared-memory place of this CTA.
__device__ __forceinline__ uint32_t remote_smem(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// Without waiting for this thread's stores (1 to 2 us behind results).
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Tensor-map load into this CTA's shared memory, its bytes counted on a barrier of
// the pair's first CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
// Shared memory of this CTA to another's, completing on a barrier there.
__device__ __forceinline__ void bulk_s2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// What these arrivals order lies in Tensor Memory, by tcgen05's own fences: a release
// of the cluster's scope would wait for the thread's loads in flight (0.5 us a slice).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// ------------------------------------------------------------------ common parts --
struct LinShared {
  uint64_t full[kMaxStages];    // operands landed (a pair: the first CTA's, for both)
  uint64_t empty[kMaxStages];   // consumed: commit
  uint64_t sf_full[kSfRing];    // scales stored: scale warps (a pair: the first CTA's)
  uint64_t sf_empty[kSfRing];   // used: commit
  uint64_t sums;                // a tile's MMAs have finished: commit
  uint64_t ended;               // MMAs that a wait cut short have finished: commit
  uint64_t drained;             // pairs: the sums have been read
  uint64_t recv;                // clusters: the others' sums have arrived
  uint32_t tmem_base;
  int abort_flag;
};

// What the launch fixes.
struct LinTile {
  int nt;            // activation rows of a tile
  int xrows;         // of them in one CTA's shared memory
  int nb;            // blocks of 128 in nt, rounded up
  int stages;
  uint32_t stage_bytes;
  int slices;        // of the inner size
  int per;           // of a CTA
  int tiles_n, tiles;
  uint32_t tmem_cols, sf_col;
  uint32_t recv_off;  // of the others' sums, behind the ring and this CTA's own
};

struct LinCtx {
  LinShared* sh;
  int32_t* status;
  long long wait_limit;
};

__device__ __forceinline__ void report(int32_t* status) {
  if (status) atomicCAS((unsigned*)status, 0u, (unsigned)MOE_ERR_TIMEOUT);
}
__device__ __forceinline__ bool lin_wait(const LinCtx& c, uint64_t* bar, uint32_t parity) {
  LinShared& sh = *c.sh;
  const bool diag = c.wait_limit < kWaitCycles;
  if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&sh.abort_flag) return false;
    if (clock64() - t0 > c.wait_limit) {
      report(c.status);
      *(volatile int*)&sh.abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool lin_warp_wait(const LinCtx& c, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, lin_wait(c, bar, parity));
}

// Barrier of the scale warps, and whether all their threads have `own`.
__device__ __forceinline__ bool sync_all_of(bool own) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.and.pred b, %2, %3, a;\n selp.u32 %0, 1, 0, b;\n}"
      : "=r"(all)
      : "r"((uint32_t)own), "n"(kSfBarrier), "n"(kSfWarps * 32)
      : "memory");
  return all;
}

// To a pair's second CTA, which does not see this one's flag.
__device__ __forceinline__ void tell_abort(const LinShared& sh, uint32_t one) {
  if (one)
    asm volatile("st.shared::cluster.u32 [%0], 1;\n fence.acq_rel.cluster;" ::"r"(remote_smem(&sh.abort_flag, 1)) : "memory");
  __syncwarp();
}

// Place in a ring: index, and the parity of its current round.
struct Ring {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) i = 0, ++round;
  }
  // Parity of the phase that frees the place for this round (rounds from 1).
  __device__ __forceinline__ uint32_t freed() const { return (round - 1) & 1; }
  __device__ __forceinline__ uint32_t filled() const { return round & 1; }
};

template <bool F4>
struct LinCfg {
  static constexpr int kWords = F4 ? 2 : 1;       // scale words of a row in a slice
  static constexpr int kStep = 4 / kWords;        // slices of a step of scales
};

// Scale words of one row, four a step; past the end, and in rows past the end, scale
// 1.  WIDE: by 16-byte loads (aligned rows of a multiple of four words).  Predicated
// loads into the registers that keep the words: with branches the compiler moves
// them there where paths join, and waits for each load on the spot (0.3 us a slice).
template <bool WIDE>
struct ScaleRow {
  const uint32_t* p;
  int words;
  __device__ __forceinline__ ScaleRow(const uint8_t* base, int64_t stride, int row, int rows, int w0, int count)
      : p(reinterpret_cast<const uint32_t*>(base + (row < rows ? row : 0) * stride) + w0), words(row < rows ? count - w0 : 0) {}
  __device__ __forceinline__ void load(uint4& v, int w) const {
    constexpr uint32_t one = 0x7F7F7F7Fu;
    if (WIDE) {
      asm volatile(
          "{\n .reg .pred q;\n setp.lt.s32 q, %5, %6;\n mov.b32 %0, %7;\n mov.b32 %1, %7;\n mov.b32 %2, %7;\n mov.b32 %3, %7;\n"
          " @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
          : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
          : "l"(p + w), "r"(w), "r"(words), "n"(one));
    } else {
      asm volatile(
          "{\n .reg .pred q0, q1, q2, q3;\n setp.lt.s32 q0, %5, %6;\n setp.lt.s32 q1, %7, %6;\n setp.lt.s32 q2, %8, %6;\n"
          " setp.lt.s32 q3, %9, %6;\n mov.b32 %0, %10;\n mov.b32 %1, %10;\n mov.b32 %2, %10;\n mov.b32 %3, %10;\n"
          " @q0 ld.global.u32 %0, [%4];\n @q1 ld.global.u32 %1, [%4 + 4];\n @q2 ld.global.u32 %2, [%4 + 8];\n"
          " @q3 ld.global.u32 %3, [%4 + 12];\n}"
          : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
          : "l"(p + w), "r"(w), "r"(words), "r"(w + 1), "r"(w + 2), "r"(w + 3), "n"(one));
    }
  }
};
// Whether all scale rows of both operands, from word w0 on, take 16-byte loads.
__device__ __forceinline__ bool wide_scales(const LinearParams& p, int w0) {
  return (((uintptr_t)p.ws | (uintptr_t)p.xs | (uintptr_t)p.ws_stride | (uintptr_t)p.xs_stride | (uintptr_t)(4 * w0) |
           (uintptr_t)(p.K / 32)) & 15) == 0;
}

// One tile's scales by the four scale warps: `steps` steps of words from w0 on, of
// weight rows n0.. and activation rows t0...  ok turns false where a wait gave up;
// the steps are walked all the same, since the warps meet at each.
constexpr int kSfAhead = 4;  // steps in flight: more than HBM's latency
constexpr uint32_t kSwapWords = 4 * 3 * kRows;  // of one exchange buffer (there are two)
template <int G, int WARP0, bool WIDE>
__device__ __forceinline__ void scales_of_tile(const LinearParams& p, const LinTile& t, const LinCtx& c, uint32_t* swap,
                                               uint32_t tmem, int n0, int t0, int w0, int steps, Ring& ring, int& step,
                                               bool& ok) {
  const int tid = threadIdx.x - WARP0 * 32, lane = tid & 31, q = (threadIdx.x >> 5) & 3;
  // Thread tid reads row tid / 4 + 32 (tid % 4) of each block: the word's place
  // among the blocks of four is tid.
  const int r = (tid >> 2) + 32 * (tid & 3), words = p.K / 128;
  const ScaleRow<WIDE> rw(p.ws, p.ws_stride, n0 + r, p.N, w0, words);
  const ScaleRow<WIDE> rx0(p.xs, p.xs_stride, t0 + r, r < t.nt ? p.T : 0, w0, words);
  const ScaleRow<WIDE> rx1(p.xs, p.xs_stride, t0 + 128 + r, 128 + r < t.nt ? p.T : 0, w0, words);
  const int nb = t.nb, blocks = 1 + nb;
  uint4 vw[kSfAhead], va[kSfAhead], vb[kSfAhead];
#pragma unroll
  for (int d = 0; d < kSfAhead; ++d) {
    rw.load(vw[d], 4 * d);
    rx0.load(va[d], 4 * d);
    rx1.load(vb[d], 4 * d);
  }
  const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + t.sf_col;
  for (int g0 = 0; g0 < steps; g0 += kSfAhead) {
#pragma unroll
    for (int d = 0; d < kSfAhead; ++d) {
      if (g0 + d >= steps) break;
      uint32_t* buf = swap + (step & 1) * kSwapWords;
      const uint32_t a[4] = {vw[d].x, vw[d].y, vw[d].z, vw[d].w}, b0[4] = {va[d].x, va[d].y, va[d].z, va[d].w},
                     b1[4] = {vb[d].x, vb[d].y, vb[d].z, vb[d].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        buf[(3 * w + 0) * kRows + tid] = a[w];
        buf[(3 * w + 1) * kRows + tid] = b0[w];
        if (nb > 1) buf[(3 * w + 2) * kRows + tid] = b1[w];
      }
      // Everyone has read the other buffer, too, before it is written again.
      named_sync(kSfBarrier, kSfWarps * 32);
      // (Words of another CTA's part are read in vain at the end.)
      const int w = 4 * (g0 + d + kSfAhead);
      rw.load(vw[d], w);
      rx0.load(va[d], w);
      rx1.load(vb[d], w);
      if (ok && ring.round > 0) ok = lin_warp_wait(c, &c.sh->sf_empty[ring.i], ring.freed());
      if (!ok) {
        ++step;
        continue;
      }
      tc_fence_after();
      const uint32_t col = lanes + (uint32_t)(ring.i * 16 * blocks);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 x = *reinterpret_cast<const uint4*>(&buf[(3 * w + 0) * kRows + 4 * lane]);
        const uint4 y = *reinterpret_cast<const uint4*>(&buf[(3 * w + 1) * kRows + 4 * lane]);
        tmem_st4(col + (uint32_t)(4 * blocks * w), x.x, x.y, x.z, x.w);
        tmem_st4(col + (uint32_t)(4 * blocks * w + 4), y.x, y.y, y.z, y.w);
        if (nb > 1) {
          const uint4 z = *reinterpret_cast<const uint4*>(&buf[(3 * w + 2) * kRows + 4 * lane]);
          tmem_st4(col + (uint32_t)(4 * blocks * w + 8), z.x, z.y, z.z, z.w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (G == 1)
          mbar_arrive(&c.sh->sf_full[ring.i]);
        else
          mbar_arrive_cluster(remote_smem(&c.sh->sf_full[ring.i], 0));
      }
      ring.next(kSfRing);
      ++step;
    }
  }
}

// One tile's MMAs, `count` slices, by one warp.
template <bool F4, int G>
__device__ __forceinline__ bool mmas_of_tile(const LinTile& t, const LinCtx& c, uint32_t ring0, uint32_t tmem, int count,
                                             Ring& ring, Ring& sf, uint32_t one) {
  using C = LinCfg<F4>;
  const uint32_t blocks4 = 4 * (1 + t.nb);
  const uint32_t id0 = F4 ? idesc_mxf4(G * kRows, t.nt, 0, 0) : idesc_mx_f32(G * kRows, t.nt, kMxE2M1, kMxE4M3, 0, 0);
  for (int s0 = 0; s0 < count; s0 += C::kStep) {
    if (!lin_warp_wait(c, &c.sh->sf_full[sf.i], sf.filled())) return false;
    const uint32_t col = tmem + t.sf_col + (uint32_t)sf.i * 4 * blocks4;
#pragma unroll
    for (int j = 0; j < C::kStep; ++j) {
      if (s0 + j >= count) break;
      if (!lin_warp_wait(c, &c.sh->full[ring.i], ring.filled())) return false;
      tc_fence_after();
      const uint32_t a0 = desc_low(ring0 + (uint32_t)ring.i * t.stage_bytes), b0 = a0 + (kTileBytes >> 4);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const uint32_t w = F4 ? 2 * j + (kb >> 1) : j, id = F4 ? 2 * (kb & 1) : kb;
        const uint32_t sfa = col + blocks4 * w, idesc = id0 | (id << 4) | (id << 29);
        if (F4)
          mma_mxf4<G>(tmem, a0 + 2 * kb, b0 + 2 * kb, idesc, sfa, sfa + 4, s0 + j > 0 || kb > 0, one);
        else
          mma_mx<G>(tmem, a0 + 2 * kb, b0 + 2 * kb, idesc, sfa, sfa + 4, s0 + j > 0 || kb > 0, one);
      }
      commit<G>(&c.sh->empty[ring.i], one);
      ring.next(t.stages);
    }
    commit<G>(&c.sh->sf_empty[sf.i], one);
    sf.next(kSfRing);
  }
  return true;
}

// After the last __syncthreads of a CTA in which a wait gave up: copies may be in
// flight, and have to land before the CTA may exit.  Their barriers miss other
// arrivals, so a time is waited that covers any.
__device__ __forceinline__ void let_copies_land(const LinShared& sh) {
  if (sh.abort_flag) {
    const long long w0 = clock64();
    while (clock64() - w0 < 20000000) __nanosleep(1000);
  }
}

// Four neighbouring addends, or results, as they are held.
template <bool OUT_BF16>
struct Four;
template <>
struct Four<true> {
  typedef uint2 Raw;
  typedef uint16_t One;
  static __device__ __forceinline__ float4 get(const uint2& a) {
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint2 put(const float4& y) { return make_uint2(bf16x2_rn(y.x, y.y), bf16x2_rn(y.z, y.w)); }
  static __device__ __forceinline__ float get1(uint16_t a) { return bf16_f32(a); }
  static __device__ __forceinline__ uint16_t put1(float y) { return (uint16_t)(bf16x2_rn(y, 0.f) & 0xFFFFu); }
};
template <>
struct Four<false> {
  typedef float4 Raw;
  typedef float One;
  static __device__ __forceinline__ float4 get(const float4& a) { return a; }
  static __device__ __forceinline__ float4 put(const float4& y) { return y; }
  static __device__ __forceinline__ float get1(float a) { return a; }
  static __device__ __forceinline__ float put1(float y) { return y; }
};
// One column's results of up to 32 rows from row t on.
template <bool OUT_BF16>
__device__ __forceinline__ void put_column(const LinearParams& p, int64_t t, int n, const uint32_t (&v)[32], int count) {
  typedef typename Four<OUT_BF16>::One T;
  T* o = (T*)p.out + t * p.out_stride + n;
  auto put = [&](int e, float y) { o[e * p.out_stride] = Four<OUT_BF16>::put1(y); };
  if (!p.add) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (e < count) put(e, __uint_as_float(v[e]));
    return;
  }
  const T* ad = (const T*)p.add + t * p.add_stride + n;
  // Addends 16 at a time, all before the first store, which may be to the same place
  // (4,096 x 7,168 x 1,408, fp32: 70 us by 8, 61 by 16).
#pragma unroll
  for (int e0 = 0; e0 < 32; e0 += 16) {
    float a[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      a[e] = 0.f;
      if (e0 + e < count) a[e] = Four<OUT_BF16>::get1(ad[(e0 + e) * p.add_stride]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e0 + e < count) put(e0 + e, __uint_as_float(v[e0 + e]) + a[e]);
  }
}
// The same rows where a wait gave up and there is no sum.
template <bool OUT_BF16>
__device__ __forceinline__ void put_nan(const LinearParams& p, int64_t t, int n, int count) {
  typedef typename Four<OUT_BF16>::One T;
  T* o = (T*)p.out + t * p.out_stride + n;
#pragma unroll 1
  for (int e = 0; e < count; ++e) o[e * p.out_stride] = Four<OUT_BF16>::put1(__int_as_float(0x7FC00000));
}
// Whether rows of out and the addend are whole groups of four, all aligned.
template <bool OUT_BF16>
__device__ __forceinline__ bool wide_rows(const LinearParams& p) {
  const uintptr_t size = OUT_BF16 ? 2 : 4;
  const uintptr_t bits = (uintptr_t)p.out | (uintptr_t)(p.out_stride * size) | (p.add ? (uintptr_t)p.add | (uintptr_t)(p.add_stride * size) : 0);
  return (bits & (4 * size - 1)) == 0 && p.N % 4 == 0;
}

// --------------------------------------------------------------------- clusters --
// Small products, bound by the weights' bytes: a tile's inner size is cut among the
// CTAs of a cluster, so that all SMs stream weights.  Each CTA owns some of the
// tile's activation rows; the others send it their sums (one bulk copy between
// shared memories each: remote stores and loads of single words took 4 cycles a
// word), and it adds them in rank order.
template <bool F4, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads) k_linear(const LinearParams p, const LinTile t,
                                                     const __grid_constant__ CUtensorMap wmap,
                                                     const __grid_constant__ CUtensorMap xmap) {
  using C = LinCfg<F4>;
  extern __shared__ uint8_t lin_dyn[];
  __shared__ LinShared sh;
  __shared__ __align__(16) uint32_t swap[2 * kSwapWords];
  const int cl = (int)cluster_size(), rank = (int)cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_dyn) + 1023) & ~(uintptr_t)1023);
  const int n0 = (blockIdx.x / cl) * kRows, t0 = blockIdx.y * t.nt;
  const int s0 = rank * t.per, ns = max(min(s0 + t.per, t.slices) - s0, 0);
  // Rows of the tile that this CTA owns.
  const int valid = min(t.nt, p.T - t0), own = (valid + cl - 1) / cl;
  const int own0 = min(rank * own, valid), mine = min(own, valid - own0);
  if (warp == kMmaWarp) lin_alloc<1>(&sh.tmem_base, t.tmem_cols);
  if (tid == 0) {
    for (int i = 0; i < t.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kSfRing; ++i) {
      mbar_init(&sh.sf_full[i], kSfWarps);
      mbar_init(&sh.sf_empty[i], 1);
    }
    mbar_init(&sh.sums, 1);
    mbar_init(&sh.ended, 1);
    mbar_init(&sh.recv, 1);
    sh.abort_flag = 0;
    mbar_init_fence();
    if (cl > 1) mbar_arrive_expect_tx(&sh.recv, (uint32_t)((cl - 1) * mine * kRows * 4));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (cl > 1) cluster_arrive();
  const uint32_t tmem = sh.tmem_base;
  const LinCtx c = {&sh, p.status, p.wait_limit};
  // Not before Tensor Memory is held: a CTA of the next kernel that took it would
  // wait for this one to end.
  pdl_trigger();
  if (warp == kTmaWarp && lane == 0) {
    // Maps, and the first weights as far as L2, while the kernel before ends (L2 holds
    // what it may still write).
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int i = 0; i < min(ns, t.stages); ++i) tma_prefetch_2d(&wmap, (s0 + i) * 128, n0);
  }
  pdl_wait();

  // Results: a thread takes four neighbouring columns of rows 4 apart, kUnits rows at a
  // time; their addends are read before the sums are waited for, and all before the
  // first store, which may be to the same place.
  typedef Four<OUT_BF16> F;
  typedef typename F::Raw Raw;
  constexpr int kUnits = 8, kApart = kSfWarps * 32 * 4 / kRows;
  const int tt0 = (tid - kSfWarp0 * 32) / (kRows / 4), col4 = tid % (kRows / 4) * 4;
  const bool wide = wide_rows<OUT_BF16>(p), live = n0 + col4 < p.N;
  Raw add[kUnits];
  auto addends = [&](int tb) {
    const Raw* from = (const Raw*)((const typename F::One*)p.add + (int64_t)(t0 + own0 + tb) * p.add_stride + n0 + col4);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      add[k] = Raw();
      if (p.add && wide && live && tb + kApart * k < mine)
        add[k] = *(const Raw*)((const typename F::One*)from + (int64_t)(kApart * k) * p.add_stride);
    }
  };
  bool fine = false;
  if (warp == kTmaWarp) {
    if (lane == 0) {
      const uint32_t tx = (F4 ? kTileBytes : kTileBytes / 2) + (uint32_t)t.nt * 128;
      Ring r;
      for (int i = 0; i < ns; ++i, r.next(t.stages)) {
        if (r.round > 0 && !lin_wait(c, &sh.empty[r.i], r.freed())) break;
        uint8_t* sb = ring + (size_t)r.i * t.stage_bytes;
        mbar_arrive_expect_tx(&sh.full[r.i], tx);
        tma_load_2d(sb, &wmap, (s0 + i) * 128, n0, &sh.full[r.i]);
        tma_load_2d(sb + kTileBytes, &xmap, (s0 + i) * 128, t0, &sh.full[r.i]);
      }
    }
  } else if (warp == kMmaWarp) {
    Ring r, sf;
    const uint32_t one = elect_one();  // commits track the elected lane's MMAs
    uint64_t* end = mmas_of_tile<F4, 1>(t, c, smem_u32(ring), tmem, ns, r, sf, one) ? &sh.sums : &sh.ended;
    commit<1>(end, one);
    // Everything issued has finished before Tensor Memory is released.
    if (!mbar_wait(end, 0)) report(p.status);
  } else {
    Ring sf;
    int step = 0;
    bool ok = true;
    const int w0 = s0 * C::kWords, steps = (ns + C::kStep - 1) / C::kStep;
    if (wide_scales(p, w0))
      scales_of_tile<1, kSfWarp0, true>(p, t, c, swap, tmem, n0, t0, w0, steps, sf, step, ok);
    else
      scales_of_tile<1, kSfWarp0, false>(p, t, c, swap, tmem, n0, t0, w0, steps, sf, step, ok);
    addends(tt0);
    fine = lin_warp_wait(c, &sh.sums, 0) && ns > 0;
    tc_fence_after();
  }
  __syncwarp();
  if (cl > 1) cluster_wait();  // every CTA has started
  if (warp >= kSfWarp0) {
    // Sums to shared memory (the ring is free), an activation row's 128 in a row.
    const int q = warp & 3, etid = tid - kSfWarp0 * 32;
    const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
    float* stage = reinterpret_cast<float*>(ring);
    float* recv = reinterpret_cast<float*>(ring + t.recv_off);
    for (int c0 = 0; c0 < valid; c0 += 32) {
      uint32_t v[32];
      tmem_ld32(tbase + (uint32_t)c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (c0 + e < valid) stage[(c0 + e) * kRows + q * 32 + lane] = fine ? __uint_as_float(v[e]) : 0.f;
    }
    tc_fence_before();
    if (cl > 1) fence_async_smem();
    const bool whole = sync_all_of(fine || ns == 0);
    if (cl > 1) {
      // Where a wait gave up nothing is sent, and the others' waits give up as well.
      if (etid < cl && etid != rank && whole) {
        const int o0 = min(etid * own, valid), n = min(own, valid - o0);
        if (n > 0)
          bulk_s2s(remote_smem(recv + (size_t)(rank < etid ? rank : rank - 1) * own * kRows, etid), stage + o0 * kRows,
                   (uint32_t)(n * kRows * 4), remote_smem(&sh.recv, etid));
      }
      // No CTA leaves before all sums have arrived: told as soon as they have.
      if (!lin_warp_wait(c, &sh.recv, 0)) let_copies_land(sh);
      __syncwarp();
      cluster_arrive_relaxed();
    }
    // In rank order.
    auto part = [&](int j) { return j == rank ? stage + own0 * kRows : recv + (size_t)(j < rank ? j : j - 1) * own * kRows; };
    auto results = [&](auto units) {
      constexpr int U = decltype(units)::value;
      for (int tb = tt0; live && tb < mine; tb += U * kApart) {
        if (tb != tt0) addends(tb);
        float4 y[U];
#pragma unroll
        for (int k = 0; k < U; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int j = 0; j < cl; ++j) {
          const float* from = part(j) + tb * kRows + col4;
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (tb + kApart * k < mine) {
              const float4 a = *reinterpret_cast<const float4*>(from + kApart * k * kRows);
              y[k].x += a.x, y[k].y += a.y, y[k].z += a.z, y[k].w += a.w;
            }
        }
        typename F::One* to = (typename F::One*)p.out + (int64_t)(t0 + own0 + tb) * p.out_stride + n0 + col4;
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (tb + kApart * k < mine) {
            const float4 a = F::get(add[k]);
            y[k].x += a.x, y[k].y += a.y, y[k].z += a.z, y[k].w += a.w;
            *(Raw*)(to + (int64_t)(kApart * k) * p.out_stride) = F::put(y[k]);
          }
      }
    };
    if (wide) {
      if (mine <= kApart)
        results(std::integral_constant<int, 1>());
      else
        results(std::integral_constant<int, kUnits>());
    } else if (n0 + etid < p.N) {  // a column a thread
#pragma unroll 1
      for (int tt = 0; tt < mine; ++tt) {
        const int64_t t1 = t0 + own0 + tt;
        float y = 0.f;
        for (int j = 0; j < cl; ++j) y += part(j)[tt * kRows + etid];
        if (p.add) y += F::get1(((const typename F::One*)p.add)[t1 * p.add_stride + n0 + etid]);
        ((typename F::One*)p.out)[t1 * p.out_stride + n0 + etid] = F::put1(y);
      }
    }
  } else if (cl > 1) {
    cluster_arrive_relaxed();
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort_flag) {
    let_copies_land(sh);
    if (tid < kRows && n0 + tid < p.N) put_nan<OUT_BF16>(p, t0 + own0, n0 + tid, mine);
  }
  __syncwarp();
  if (cl > 1) cluster_wait();
  if (warp == kMmaWarp) {
    tc_fence_after();
    lin_dealloc<1>(tmem, t.tmem_cols);
  }
}

// ------------------------------------------------------------------------ pairs --
// Large products: a pair of CTAs on neighbouring SMs takes 256 weight rows by up to
// 256 activation rows, one MMA for both (cta_group::2).  Each CTA holds its 128
// weight rows and half of the activation rows in shared memory, and the sums of its
// weight rows in its Tensor Memory, so that a byte from L2 or shared memory feeds up
// to twice the products of a tile of one CTA.  Scales of all activation rows go to
// both.  The first CTA's thread issues the MMAs of both; barriers of full stages, of
// stored scales and of drained sums are the first CTA's, those of consumed stages and
// finished sums are signalled in both.  Pairs walk the tiles in turn.
//
// Eight epilogue warps take a tile's sums to registers at once (128 a thread) and
// give Tensor Memory back; addends and stores go on beside the next tile's MMAs
// (4,096 x 9,216 x 7,168: 206 -> 176 us, MXFP4 activations 146 -> 112).  The
// registers come from the other warpgroups.  That product now takes 148 to 155 us in
// some hundred calls (3.5 PFLOP/s; the tensor pipe 79 % busy) and 174 to 179 in
// thousands, which the power limit holds at 1.53 GHz; with MXFP4 activations 98 to 101
// (5.4 PFLOP/s, 56 %) either way.
constexpr int kPairSfWarp0 = 4, kPairEpWarp0 = 8, kPairEpWarps = 8;
constexpr int kPairThreads = (kPairEpWarp0 + kPairEpWarps) * 32;
constexpr int kRegsLaunch = 128, kRegsCopy = 56, kRegsScale = 120, kRegsEpilogue = 168;
static_assert(kRegsCopy + kRegsScale + 2 * kRegsEpilogue <= 4 * kRegsLaunch, "warpgroups share the launch's registers");
static_assert(kPairThreads * kRegsLaunch <= 65536, "registers of an SM");

template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr int kPairs = kNumSMs / 2;

template <bool F4, bool OUT_BF16>
__global__ void __launch_bounds__(kPairThreads, 1) k_linear_pair(const LinearParams p, const LinTile t,
                                                                 const __grid_constant__ CUtensorMap wmap,
                                                                 const __grid_constant__ CUtensorMap xmap) {
  using C = LinCfg<F4>;
  extern __shared__ uint8_t lin_dyn[];
  __shared__ LinShared sh;
  __shared__ __align__(16) uint32_t swap[2 * kSwapWords];
  const int rank = (int)cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_dyn) + 1023) & ~(uintptr_t)1023);
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (warp == kMmaWarp) lin_alloc<2>(&sh.tmem_base, t.tmem_cols);
  if (tid == 0) {
    for (int i = 0; i < t.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kSfRing; ++i) {
      mbar_init(&sh.sf_full[i], 2 * kSfWarps);
      mbar_init(&sh.sf_empty[i], 1);
    }
    mbar_init(&sh.sums, 1);
    mbar_init(&sh.ended, 1);
    mbar_init(&sh.drained, 2 * kPairEpWarps);
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();
  const uint32_t tmem = sh.tmem_base;
  const LinCtx c = {&sh, p.status, p.wait_limit};
  cluster_wait();  // both CTAs' barriers are ready, both hold Tensor Memory
  pdl_trigger();
  if (warp == kTmaWarp && lane == 0) {  // as in k_linear
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int i = 0; i < min(t.slices, t.stages); ++i) tma_prefetch_2d(&wmap, i * 128, ((pair % t.tiles_n) * 2 + rank) * kRows);
  }
  pdl_wait();

  if (warp < kPairSfWarp0) {
    regs_dec<kRegsCopy>();
    if (warp == kTmaWarp && lane == 0) {
      const uint32_t tx = (F4 ? kTileBytes : kTileBytes / 2) + (uint32_t)t.xrows * 128;
      Ring r;
      bool ok = true;
      for (int tile = pair; tile < t.tiles && ok; tile += pairs) {
        const int n0 = ((tile % t.tiles_n) * 2 + rank) * kRows, t0 = (tile / t.tiles_n) * t.nt + rank * t.xrows;
        for (int i = 0; i < t.slices; ++i, r.next(t.stages)) {
          ok = r.round == 0 || lin_wait(c, &sh.empty[r.i], r.freed());
          if (!ok) break;
          uint8_t* sb = ring + (size_t)r.i * t.stage_bytes;
          // The first CTA's barrier counts both CTAs' bytes.
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[r.i], 2 * tx);
          const uint32_t bar = remote_smem(&sh.full[r.i], 0);
          tma_load_2d_pair(sb, &wmap, i * 128, n0, bar);
          tma_load_2d_pair(sb + kTileBytes, &xmap, i * 128, t0, bar);
        }
      }
    }
    if (warp == kMmaWarp && rank == 0) {
      Ring r, sf;
      const uint32_t one = elect_one();
      int ti = 0;
      bool ok = true;
      for (int tile = pair; tile < t.tiles; tile += pairs, ++ti) {
        ok = ti == 0 || lin_warp_wait(c, &sh.drained, (ti - 1) & 1);
        tc_fence_after();
        ok = ok && mmas_of_tile<F4, 2>(t, c, smem_u32(ring), tmem, t.slices, r, sf, one);
        if (!ok) break;
        commit<2>(&sh.sums, one);
      }
      if (!ok) {
        tell_abort(sh, one);
        commit<2>(&sh.ended, one);
      }
      // Everything issued has finished before Tensor Memory is released.
      if (!(ok ? mbar_wait(&sh.sums, (ti - 1) & 1) : mbar_wait(&sh.ended, 0))) report(p.status);
    }
  } else if (warp < kPairEpWarp0) {
    regs_dec<kRegsScale>();
    Ring sf;
    int step = 0;
    bool ok = true;
    const int steps = (t.slices + C::kStep - 1) / C::kStep;
    const bool wide = wide_scales(p, 0);
    for (int tile = pair; tile < t.tiles; tile += pairs) {
      const int n0 = ((tile % t.tiles_n) * 2 + rank) * kRows, t0 = (tile / t.tiles_n) * t.nt;
      if (wide)
        scales_of_tile<2, kPairSfWarp0, true>(p, t, c, swap, tmem, n0, t0, 0, steps, sf, step, ok);
      else
        scales_of_tile<2, kPairSfWarp0, false>(p, t, c, swap, tmem, n0, t0, 0, steps, sf, step, ok);
    }
  } else {
    regs_inc<kRegsEpilogue>();
    const int q = warp & 3, part = (warp - kPairEpWarp0) >> 2;  // lanes 32 q ..; half of the columns
    const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(part * t.xrows);
    int ti = 0, tile = pair;
    for (; tile < t.tiles; tile += pairs, ++ti) {
      const int n = ((tile % t.tiles_n) * 2 + rank) * kRows + q * 32 + lane;
      const int64_t tt = (int64_t)(tile / t.tiles_n) * t.nt + part * t.xrows;
      const int count0 = n - lane < p.N ? (int)min((int64_t)t.xrows, p.T - tt) : 0, count = n < p.N ? count0 : 0;
      if (p.add) {  // on their way to L2 while the MMAs run
        const uint8_t* ad = (const uint8_t*)p.add + (tt * p.add_stride + n) * (OUT_BF16 ? 2 : 4);
        for (int e = lane; e < count0; e += 32) prefetch_l2_line(ad + (int64_t)e * p.add_stride * (OUT_BF16 ? 2 : 4) - lane * (OUT_BF16 ? 2 : 4));
      }
      if (!lin_warp_wait(c, &sh.sums, ti & 1)) break;
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * j < t.xrows) tmem_ld32(tbase + 32 * j, v[j]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(remote_smem(&sh.drained, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * j < count) put_column<OUT_BF16>(p, tt + 32 * j, n, v[j], count - 32 * j);
    }
#pragma unroll 1
    for (; tile < t.tiles; tile += pairs) {  // without sums
      const int n = ((tile % t.tiles_n) * 2 + rank) * kRows + q * 32 + lane;
      const int64_t tt = (int64_t)(tile / t.tiles_n) * t.nt + part * t.xrows;
      if (n < p.N) put_nan<OUT_BF16>(p, tt, n, (int)min((int64_t)t.xrows, p.T - tt));
    }
  }
  tc_fence_before();
  __syncthreads();
  let_copies_land(sh);
  __syncwarp();
  cluster_arrive();
  cluster_wait();  // neither CTA leaves while the other may reach its shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    lin_dealloc<2>(tmem, t.tmem_cols);
  }
}

// ----------------------------------------------------------------------- launch --
// Tensor map of an operand: rows of codes, boxes of 128 bytes of shared memory by
// `rows` rows, 128-byte swizzle.  spread: 4-bit codes that take a byte each in
// shared memory.  Rows and columns past the end read as zero.
cudaError_t operand_map(CUtensorMap* m, const moe_mx& a, bool spread, int rows) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t width = spread || a.type == MOE_MX_E4M3 ? a.cols : a.cols / 2;
  const cuuint64_t dims[2] = {width, (cuuint64_t)a.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)a.q_stride};
  const cuuint32_t box[2] = {128, (cuuint32_t)rows};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = enc(m, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.q, dims,
                         strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename Kernel>
cudaError_t start(Kernel kern, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t s, const LinearParams& p,
                  const LinTile& t, const moe_mx& x, const moe_mx& w) {
  CUtensorMap wmap, xmap;
  cudaError_t err;
  if ((err = operand_map(&wmap, w, x.type == MOE_MX_E4M3, kRows)) != cudaSuccess ||
      (err = operand_map(&xmap, x, false, t.xrows)) != cudaSuccess ||
      (err = ensure_smem_attr((const void*)kern, smem)) != cudaSuccess)
    return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, t, wmap, xmap);
}

int up(int a, int b) { return (a + b - 1) / b; }

template <bool F4, bool OUT_BF16>
cudaError_t launch(const LinearParams& p, const moe_mx& x, const moe_mx& w, cudaStream_t s) {
  LinTile t = {};
  const size_t most = (size_t)214 * 1024;  // dynamic shared memory, beside 13 KB of static
  t.slices = up(p.K, F4 ? 256 : 128);
  auto shape = [&](int nt, int granule, int share) {
    const int tiles_t = up(p.T, nt);
    t.nt = up(up(p.T, tiles_t), granule) * granule;
    t.xrows = t.nt / share;  // a multiple of 16: the operand's 1024-byte atoms stay whole
    t.nb = up(t.nt, 128);
    t.stage_bytes = (uint32_t)(kTileBytes + t.xrows * 128);
    t.sf_col = (uint32_t)t.nt;
    t.tmem_cols = 32;
    while (t.tmem_cols < t.nt + (uint32_t)(kSfRing * 16 * (1 + t.nb))) t.tmem_cols *= 2;
    return tiles_t;
  };
  // Clusters, of one CTA where the inner size is not cut, while all tiles of up to 64
  // activation rows are on the chip at once (two an SM of up to 32 rows); pairs
  // otherwise, in the smallest tiles that still make one round of the chip, and for
  // MXFP4 activations of more than 32 rows where clusters would not cut.  Up to 32 rows
  // of MXFP8 take several rounds of the chip that way, too, if the inner size is long:
  // a pair's MMAs do not get faster with fewer rows (1 x 163,840: 106 us, pairs 126;
  // inner size 1,408, 30 x 262,144: 53 and 46).  Measured,
  // inner size 7,168, MXFP8 activations (us, clusters / pairs): 16 x 9,216: 10.2 / 16.5;
  // 64 x 7,168: 10.8 / 18.3; 256 x 1,408: 9.6 / 17.1; uncut, 1 x 16,384: 15.6 / 17.8;
  // 64 x 19,456: 18.6 / 19.5; 128 x 9,216: 17.4 / 18.6.  MXFP4 activations: 64 x 9,216:
  // 10.1 / 12.0; uncut, 1 x 16,384: 12.1 / 13.2; 64 x 19,456: 16.2 / 15.6.
  const int rows = up(p.N, kRows), pair_rows = up(p.N, 2 * kRows);
  const long long tiles = (long long)rows * up(p.T, 64);
  const bool few = p.T <= 32, cut = 2 * tiles <= kNumSMs;
  if (!(cut || (!F4 && tiles <= kNumSMs) || (few && (tiles <= 2 * kNumSMs || (!F4 && t.slices >= 16))))) {
    int nt = 32;
    while (nt < kMaxNt && (long long)pair_rows * up(p.T, nt) > kPairs) nt *= 2;
    const int tiles_t = shape(nt, 32, 2);
    t.tmem_cols = 512;
    t.per = t.slices;
    t.tiles_n = pair_rows;
    t.tiles = pair_rows * tiles_t;
    t.stages = (int)((most - 1024) / t.stage_bytes);
    if (t.stages > kMaxStages) t.stages = kMaxStages;
    return start(k_linear_pair<F4, OUT_BF16>, dim3((unsigned)(2 * (t.tiles < kPairs ? t.tiles : kPairs))), kPairThreads, 2,
                 (size_t)t.stages * t.stage_bytes + 1024, s, p, t, x, w);
  }
  const int tiles_t = shape(64, 16, 1);
  t.tiles_n = rows;
  t.tiles = (int)tiles;
  // CTAs of a tile: as many as fit with one CTA an SM, or two where that leaves fewer
  // SMs idle and the rings are small (1 x 7,168: 112 CTAs 8.9 us, 280 CTAs 8.3;
  // 64 x 7,168: 10.9 and 14.3); two slices each at least.
  auto fit = [&](int ctas) {
    int c = (int)(ctas / tiles);
    c = c < kMaxCl ? c : kMaxCl;
    c = c < t.slices / 2 ? c : t.slices / 2;
    return c > 1 ? c : 1;
  };
  const int one = fit(kNumSMs), both = fit(2 * kNumSMs);
  const bool two = few && (tiles > kNumSMs || tiles * both * 10 > tiles * one * 20 + kNumSMs);
  const int cl = two ? both : one;
  t.per = up(t.slices, cl);
  // The CTA's sums lie in the ring, those that it receives behind.
  const int valid = p.T < t.nt ? p.T : t.nt;
  const size_t recv = cl > 1 ? (size_t)(cl - 1) * up(valid, cl) * kRows * 4 : 0;
  // Two CTAs share an SM's Tensor Memory as they share its shared memory; no other
  // may join them and wait for some.
  const size_t space = two ? (size_t)98 * 1024 : most;
  t.stages = (int)((space - recv - 1024) / t.stage_bytes);
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  const size_t sums = align_up((size_t)valid * kRows * 4, 1024), ring = (size_t)t.stages * t.stage_bytes;
  t.recv_off = (uint32_t)(ring > sums ? ring : sums);
  size_t smem = t.recv_off + recv + 1024;
  const size_t least = two ? space : (size_t)110 * 1024;
  if (smem < least) smem = least;
  return start(k_linear<F4, OUT_BF16>, dim3((unsigned)(t.tiles_n * cl), (unsigned)tiles_t), kThreads, cl, smem, s, p, t, x, w);
}

}  // namespace

cudaError_t launch_mx_linear(const LinearParams& p, const moe_mx& x, const moe_mx& w, int out_dtype, cudaStream_t s) {
  if (x.type == MOE_MX_E2M1)
    return out_dtype == MOE_DT_BF16 ? launch<true, true>(p, x, w, s) : launch<true, false>(p, x, w, s);
  return out_dtype == MOE_DT_BF16 ? launch<false, true>(p, x, w, s) : launch<false, false>(p, x, w, s);
}

}  // namespace moe
