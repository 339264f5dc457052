// sample.cu — sampling from logits: temperature, top-k, top-p, min-p and a
// draw by a given uniform number.
//
// With z = logit / T and m = max z, every token has an integer weight
// W = rint(exp(z - m) 2^31).  Sums of integers are exact, so neither the split
// of a row over CTAs nor the order of atomics changes a result.  Top-k, top-p
// and min-p each keep a prefix of the ranking by (z descending, index
// ascending), so the kept set is one bound K* on the 50-bit key
//   K = (descending order bits of z) * 2^18 + index,
// and the drawn token is found by a running sum in index order.
//
// A cluster of 1 to 8 CTAs takes a row; its scores are read from HBM once and
// stay in shared memory.  K* comes from histograms (count or sum of W per bin)
// that the CTAs of the cluster add up over distributed shared memory: the
// first by m - z in some 1,000 equal bins (a monotone function of z); if the
// bin that holds the bound has more than kList tokens (ties), the next by equal
// pieces of the range of its keys.  A bin of at most kList tokens goes to the
// first CTA as a list, which it searches alone, in the same way.  Top-k is searched
// first, by counts alone (no exponentials); what it drops, later passes skip.
// When all tokens down to the end of the first bin found number at most kList
// (small top-k, peaked rows), the first CTA gets them all and finishes alone.
// Bound by latency (cluster barriers of 0.8 us) for few rows, by the
// instructions of the passes and the barriers for many: shared memory holds
// some 38 rows of 128,000 scores on the chip at a time.  Reading the scores
// again from L2 for each pass instead, with more CTAs resident, was slower
// (512 rows of 128,000 with all filters and probabilities: 391 against 377 us
// then; 64 rows of 163,840: 74 against 64 us).  They take 259 and 49 us now, one
// row of 100,003 10.7.
#include <cooperative_groups.h>

#include <cuda/std/type_traits>

#include "serve.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 1024;             // tokens that one CTA searches or finishes alone
constexpr int kDirect = 128;            // tokens that are ranked pair by pair
constexpr int kIdxBits = 18;             // MOE_SAMPLE_MAX_VOCAB = 2^18
constexpr int kPiece = (1 << kIdxBits) / kBins;  // indices of one of kBins pieces of the longest row
constexpr int kMaxCl = 8;
constexpr int kMostScores = 65536;       // of a CTA
constexpr int kMostBytes = 84 << 10;
constexpr float kFix = 2147483648.f;     // 2^31
constexpr float kBinScale = 45.9f;       // times kCut: below kBins - 1
constexpr uint32_t kSureBins = 700;      // weights of 2^31 exp(-15) and more
constexpr float kCut = 22.25f;           // below m - kCut every W is 0
constexpr unsigned long long kKeyAll = ~0ull;

struct SampleShared {
  union {
    // Histogram of this CTA: count, low and high 16 bits of W (native 32-bit
    // shared-memory atomics; at most kMostScores tokens a CTA keep all three
    // within 32 bits, even if they share a bin).
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];
    };
    // After the cluster has added them up: the keys of some tokens, and
    // cursors of the bins.
    struct {
      unsigned long long list[kList];
      uint32_t cursor[kBins];
    };
  };
  unsigned long long tsum[kBins];  // the cluster's totals
  uint32_t tcnt[kBins];
  uint32_t list_n;  // rank 0's is the cluster's
  unsigned long long end_total, end_key;  // of a row that rank 0 finished
  union {
    struct {  // the tokens of the list that are left
      unsigned long long key[kDirect];
      uint32_t w[kDirect];
    } few;
    uint32_t piece_w[kPiece];  // weights of the kept tokens of a piece, by index
  };
  uint32_t few_n, list_at;
  unsigned long long warp_low[kWarps], cl_low[kMaxCl];
  unsigned long long warp_best[kWarps];
  unsigned long long warp_sum[kWarps];
  uint32_t warp_cnt[kWarps];
  unsigned long long cl_best[kMaxCl];
  unsigned long long cl_sum[kMaxCl];
  uint32_t cl_cnt[kMaxCl], cl_kept[kMaxCl];
  // Where a search ended.
  uint32_t f_bin, f_cnt, f_before_cnt;
  uint32_t f_w;
  unsigned long long f_before_sum, f_key;
  unsigned long long limit, target;
};
static_assert(MOE_SAMPLE_MAX_VOCAB <= kMostScores * kMaxCl, "a cluster takes the longest row");
static_assert(MOE_SAMPLE_MAX_VOCAB == 1 << kIdxBits, "index bits of the key");

__device__ __forceinline__ float order_float(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }
// Order-preserving bits of a float (ascending), -0 excluded.
__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t b = __float_as_uint(z);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long rank_key(float z, uint32_t idx) {
  return ((unsigned long long)(~order_bits(z)) << kIdxBits) | idx;
}

struct Row {
  float m;       // largest scaled score
  float least;   // scores below have W = 0 or rank past K*
  float min_p;   // 0: off
  bool bounded;  // K* is set: score z_max, index i_max
  float z_max;
  uint32_t i_max;

  // exp(z - m).  expf, not an approximation: the weights are part of the
  // definition, and the same function gives the same integers everywhere.
  __device__ __forceinline__ float w(float z) const { return expf(z - m); }
  __device__ __forceinline__ static uint32_t fixed(float w) { return __float2uint_rn(w * kFix); }
  __device__ __forceinline__ uint32_t weight(unsigned long long key) const {
    return fixed(w(order_float(~(uint32_t)(key >> kIdxBits))));
  }
  // Bin of a score with m - z <= kCut: adding 2^23 leaves the rounded
  // product in the low bits (monotone in z; cheaper than a conversion).
  __device__ __forceinline__ int bin(float z) const {
    return (int)(__float_as_uint(fmaf(m - z, kBinScale, 8388608.f)) & (kBins - 1));
  }
  // Not dropped by the bound found so far (for z >= least).
  __device__ __forceinline__ bool within(float z, uint32_t idx) const {
    return !bounded || z > z_max || (z == z_max && idx <= i_max);
  }
  __device__ __forceinline__ void set_max(unsigned long long key) {
    bounded = true;
    z_max = order_float(~(uint32_t)(key >> kIdxBits));
    i_max = (uint32_t)key & ((1u << kIdxBits) - 1);
    least = fmaxf(least, z_max);
  }
  // Weight of a kept token, 0 for the others.
  __device__ __forceinline__ uint32_t kept(float z, uint32_t idx) const {
    if (!(z >= least)) return 0u;
    const float e = w(z);
    if (min_p > 0.f && !(e >= min_p)) return 0u;
    return within(z, idx) ? fixed(e) : 0u;
  }
};

// Over a warp, on the 32-bit reduction instruction.
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(v >> 32));
  return (unsigned long long)hi << 32 | __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
// For v whose sum over the warp is below 2^57 (weights: below 2^50).
__device__ __forceinline__ unsigned long long warp_add(unsigned long long v) {
  const uint32_t lo = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)v & 0x3FFFFFFu);
  return ((unsigned long long)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 26)) << 26) + lo;
}

// What a search looks for: the token of a given rank (its limit is the rank + 1),
// or the last one whose better ranks weigh less than the limit.  A bound p * S
// in double becomes a limit by rounding up: sums of integers are below the one
// exactly when they are below the other, and the double arithmetic, which is
// slow on this chip, is done once.
struct Target {
  unsigned long long limit;
  template <bool SUMS>
  __device__ __forceinline__ bool holds(uint32_t before_cnt, uint32_t cnt, unsigned long long before,
                                        unsigned long long sum) const {
    return SUMS ? before < limit && before + sum >= limit : before_cnt < limit && before_cnt + cnt >= limit;
  }
};
__device__ __forceinline__ unsigned long long share_limit(float p, unsigned long long sum) {
  return __double2ull_ru((double)p * (double)sum);
}

// Tokens that match the search so far: level -1 those down to bin b0, 0 all, 1
// those of bin b0, 2 those of them with a key in [lo, hi].
struct Match {
  int level, b0;
  unsigned long long lo, hi;
};

// 1,024 equal pieces of a range of keys.
struct Pieces {
  unsigned long long lo;
  int shift;
  __device__ __forceinline__ Pieces(unsigned long long low, unsigned long long high) : lo(low), shift(0) {
    const int bits = 64 - __clzll((long long)(high - low));
    if (bits > 10) shift = bits - 10;
  }
  __device__ __forceinline__ int piece(unsigned long long key) const { return (int)((key - lo) >> shift); }
  __device__ __forceinline__ void narrow(int piece, unsigned long long& l, unsigned long long& h) const {
    l = lo + ((unsigned long long)piece << shift);
    h = l + (1ull << shift) - 1;
  }
};

// NaN stays NaN: it is below every bound and never the largest.
__device__ __forceinline__ float scaled(float x, float inv) {
  return fmaf(x, inv, 0.f);  // + 0: no negative zeros
}

// A CTA's scores in shared memory, in groups of four, -inf around them: fp32
// ones scaled, bf16 ones as they came (half the space; scaled when read).
template <typename T>
struct Scores;
template <>
struct Scores<float> {
  const float4* g;
  float inv;
  __device__ __forceinline__ float4 get(int v) const { return g[v]; }
};
template <>
struct Scores<uint16_t> {
  const uint2* g;
  float inv;
  __device__ __forceinline__ float4 get(int v) const {
    const uint2 x = g[v];
    return make_float4(scaled(__uint_as_float(x.x << 16), inv), scaled(__uint_as_float(x.x & 0xFFFF0000u), inv),
                       scaled(__uint_as_float(x.y << 16), inv), scaled(__uint_as_float(x.y & 0xFFFF0000u), inv));
  }
};

template <typename T>
class Sampler {
 public:
  SampleShared& sh;
  Scores<T> sc;
  int n4;          // groups
  uint32_t first;  // index in the row of the first entry
  int cl, rank;
  Row row;
  cg::cluster_group cluster;
  // What this CTA's tokens add to the bins of the last histogram by sums, bins
  // kBins / kThreads * tid and on; and the tokens that it gave to the list.
  unsigned long long own_sum[kBins / kThreads];
  uint32_t own_cnt[kBins / kThreads], own_listed;

  __device__ Sampler(SampleShared& s, const Scores<T>& scores, int n, uint32_t f)
      : sh(s), sc(scores), n4((n + 3) / 4), first(f), cluster(cg::this_cluster()) {
    cl = (int)cluster.num_blocks();
    rank = (int)cluster.block_rank();
  }

  template <typename U>
  __device__ __forceinline__ U* remote(U* p, int r) {
    return cluster.map_shared_rank(p, r);
  }

  // f(score, index) for the CTA's scores from `cut` to `top`, eight per thread
  // and step; FEW: most steps are expected to have none.
  template <bool FEW = false, typename F>
  __device__ __forceinline__ void each(float cut, float top, F f) const {
    const float kNone = -CUDART_INF_F;
    for (int v = threadIdx.x; v < n4; v += 2 * kThreads) {
      const float4 a = sc.get(v);
      const float4 b = v + kThreads < n4 ? sc.get(v + kThreads) : make_float4(kNone, kNone, kNone, kNone);
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (FEW) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) any |= x[e] >= cut && x[e] <= top;
        if (!any) continue;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (x[e] >= cut && x[e] <= top) f(x[e], first + 4 * (v + (e >> 2) * kThreads) + (e & 3));
    }
  }
  // No score of a bin up to b0 is below this.
  __device__ __forceinline__ float bin_cut(int b0) const {
    return fmaxf(row.least, row.m - ((float)b0 + 1.f) / kBinScale);
  }
  // No score that matches is above this.
  __device__ __forceinline__ float bin_top(const Match& mt) const {
    return mt.level < 1 ? CUDART_INF_F : row.m - ((float)mt.b0 - 1.f) / kBinScale;
  }

  __device__ __forceinline__ bool matches(const Match& mt, float zi, uint32_t idx) const {
    if (!row.within(zi, idx)) return false;
    if (mt.level == 0) return true;
    if (mt.level < 0) return row.bin(zi) <= mt.b0;
    if (row.bin(zi) != mt.b0) return false;
    if (mt.level == 1) return true;
    const unsigned long long k = rank_key(zi, idx);
    return k >= mt.lo && k <= mt.hi;
  }

  // Histogram of the matching tokens over the cluster into tcnt / tsum, by
  // the next level's bins; of counts alone where no sums are needed.  Tokens
  // whose weight rounds to 0 count too: they rank last.
  template <bool SUMS>
  __device__ void histogram(const Match& mt, const Pieces& pc) {
    const int tid = threadIdx.x;
    for (int b = tid; b < kBins; b += kThreads) {
      sh.cnt[b] = 0u;
      if (SUMS) sh.lo[b] = sh.hi[b] = 0u;
    }
    __syncthreads();
    auto add = [&](int b, uint32_t w) {
      atomicAdd(&sh.cnt[b], 1u);
      if (SUMS) {
        atomicAdd(&sh.lo[b], w & 0xFFFFu);
        atomicAdd(&sh.hi[b], w >> 16);
      }
    };
    if (mt.level == 0) {
      // Weights of a whole group at once: in one branch per score, the latency
      // of the exponential would not overlap.
      for (int v = threadIdx.x; v < n4; v += kThreads) {
        const float4 a = sc.get(v);
        const float x[4] = {a.x, a.y, a.z, a.w};
        if (!(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)) >= row.least)) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = SUMS ? Row::fixed(row.w(x[e])) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] >= row.least && row.within(x[e], first + 4 * v + e)) add(row.bin(x[e]), w[e]);
      }
    } else {
      each(bin_cut(mt.b0), bin_top(mt), [&](float zi, uint32_t idx) {
        if (matches(mt, zi, idx)) add(pc.piece(rank_key(zi, idx)), SUMS ? Row::fixed(row.w(zi)) : 0u);
      });
    }
    cluster.sync();
    // Each CTA adds up its share of the bins and gives every CTA the totals.
    const int share = kBins / cl;
    for (int b = rank * share + tid; b < (rank + 1) * share; b += kThreads) {
      uint32_t c = 0;
      unsigned long long s = 0;
#pragma unroll
      for (int r = 0; r < kMaxCl; ++r) {
        if (r < cl) {
          const SampleShared* o = remote(&sh, r);
          c += o->cnt[b];
          if (SUMS) s += o->lo[b] + ((unsigned long long)o->hi[b] << 16);
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCl; ++r) {
        if (r < cl) {
          SampleShared* o = remote(&sh, r);
          o->tcnt[b] = c;
          if (SUMS) o->tsum[b] = s;
        }
      }
    }
    if (SUMS) {
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        const int b = tid * (kBins / kThreads) + i;
        own_cnt[i] = sh.cnt[b];
        own_sum[i] = sh.lo[b] + ((unsigned long long)sh.hi[b] << 16);
      }
    }
    if (tid == 0) sh.list_n = 0;
    cluster.sync();
  }

  // Least and greatest key of the CTA's matching tokens (f visits them).
  template <typename F>
  __device__ void key_range(F visit, unsigned long long& low, unsigned long long& high) {
    low = kKeyAll;
    high = 0;
    visit([&](unsigned long long k) {
      low = k < low ? k : low;
      high = k > high ? k : high;
    });
    low = ~warp_max(~low);
    high = warp_max(high);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_low[threadIdx.x >> 5] = low, sh.warp_best[threadIdx.x >> 5] = high;
    __syncthreads();
    low = ~warp_max(~sh.warp_low[threadIdx.x & (kWarps - 1)]);
    high = warp_max(sh.warp_best[threadIdx.x & (kWarps - 1)]);
  }

  // Sums of weights by bin within a CTA: the halves are added apart, on native
  // atomics, and joined by the thread that reads the bin in find_bin.
  __device__ __forceinline__ void add_weight(int b, uint32_t w) {
    uint32_t* half = reinterpret_cast<uint32_t*>(&sh.tsum[b]);
    atomicAdd(half, w & 0xFFFFu);
    atomicAdd(half + 1, w >> 16);
  }
  __device__ __forceinline__ void join_weights() {
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      const unsigned long long x = sh.tsum[threadIdx.x * (kBins / kThreads) + i];
      sh.tsum[threadIdx.x * (kBins / kThreads) + i] = (x & 0xFFFFFFFFull) + ((x >> 32) << 16);
    }
  }

  // The bin that holds the target, given what ranks before this histogram;
  // false (uniform): there is none.  By sums, with p >= 0 the limit is first set
  // to that share of the histogram's total.  `offsets`: tcnt becomes the number
  // of tokens in better bins.
  template <bool SUMS>
  __device__ bool find_bin(Target& tg, uint32_t before_cnt, unsigned long long before_sum, float p,
                           bool offsets = false) {
    constexpr int P = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t xc[P], c = 0;
    unsigned long long xs[P], s = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      xc[i] = sh.tcnt[tid * P + i];
      xs[i] = SUMS ? sh.tsum[tid * P + i] : 0ull;
      c += xc[i];
      s += xs[i];
    }
    const uint32_t wc = __reduce_add_sync(0xFFFFFFFFu, c);
    const unsigned long long ws = SUMS ? warp_add(s) : 0ull;
    if (lane == 0) {
      sh.warp_cnt[warp] = wc;
      if (SUMS) sh.warp_sum[warp] = ws;
    }
    if (tid == 0) sh.f_bin = kBins;
    __syncthreads();
    if (SUMS && p >= 0.f) {
      if (warp == 0) {
        const unsigned long long all = warp_add(lane < kWarps ? sh.warp_sum[lane] : 0ull);
        if (lane == 0) sh.limit = share_limit(p, all);
      }
      __syncthreads();
      tg.limit = sh.limit;
    }
    uint32_t bc = before_cnt + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.warp_cnt[lane] : 0u);
    unsigned long long bs = before_sum + (SUMS ? warp_add(lane < warp ? sh.warp_sum[lane] : 0ull) : 0ull);
    const bool here = tg.template holds<SUMS>(bc, wc, bs, ws);  // one warp at most
    if (here || offsets) {
      uint32_t ic = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t oc = __shfl_up_sync(0xFFFFFFFFu, ic, o);
        if (lane >= o) ic += oc;
      }
      bc += ic - c;
    }
    if (here) {
      uint32_t at = bc;
      if (SUMS) {
        unsigned long long is = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long os = __shfl_up_sync(0xFFFFFFFFu, is, o);
          if (lane >= o) is += os;
        }
        bs += is - s;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (tg.template holds<SUMS>(at, xc[i], bs, xs[i])) {
          sh.f_bin = tid * P + i;
          sh.f_cnt = xc[i];
          sh.f_before_cnt = at;
          sh.f_before_sum = bs;
        }
        at += xc[i];
        bs += xs[i];
      }
    }
    if (offsets) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        sh.tcnt[tid * P + i] = bc;
        bc += xc[i];
      }
    }
    __syncthreads();
    return sh.f_bin < kBins;
  }

  // Hand the first CTA the list of the matching tokens (in any order).  A
  // CTA collects its own first, where the totals of the histogram were, and then
  // takes its place in the lists with one remote atomic: one per token cost a
  // round trip each, in turn for the tokens of a warp.  No CTA still reads the
  // list of an earlier search: two cluster barriers of a histogram lie between.
  __device__ void gather(const Match& mt) {
    if (threadIdx.x == 0) sh.few_n = 0;
    for (int b = threadIdx.x; b < kBins; b += kThreads) sh.cursor[b] = 0u;
    __syncthreads();
    each<true>(bin_cut(mt.b0), bin_top(mt), [&](float zi, uint32_t idx) {
      if (!matches(mt, zi, idx)) return;
      const uint32_t at = atomicAdd(&sh.few_n, 1u);
      if (at < kList) sh.tsum[at] = rank_key(zi, idx);
    });
    __syncthreads();
    const uint32_t n = own_listed = sh.few_n;
    if (threadIdx.x == 0) sh.list_at = n ? atomicAdd(remote(&sh.list_n, 0), n) : 0u;
    __syncthreads();
    const uint32_t at = sh.list_at;
    SampleShared* o = remote(&sh, 0);
    for (uint32_t i = threadIdx.x; i < n && at + i < kList; i += kThreads) o->list[at + i] = sh.tsum[i];
    cluster.sync();
  }

  // After find_bin on the first histogram: the key of the target.
  template <bool SUMS>
  __device__ unsigned long long resolve(Target& tg) {
    Match mt;
    mt.level = 1;
    mt.b0 = (int)sh.f_bin;
    mt.lo = 0;
    mt.hi = kKeyAll;
    uint32_t before_cnt = sh.f_before_cnt, cnt = sh.f_cnt;
    unsigned long long before_sum = sh.f_before_sum;
    while (cnt > kList) {  // uniform: every CTA of the cluster has the same totals
      unsigned long long low, high;
      key_range([&](auto f) {
        each(bin_cut(mt.b0), bin_top(mt), [&](float zi, uint32_t idx) { if (matches(mt, zi, idx)) f(rank_key(zi, idx)); });
      }, low, high);
      if ((int)threadIdx.x < cl) {
        SampleShared* o = remote(&sh, threadIdx.x);
        o->cl_low[rank] = low;
        o->cl_best[rank] = high;
      }
      cluster.sync();
      for (int r = 0; r < cl; ++r) {
        low = sh.cl_low[r] < low ? sh.cl_low[r] : low;
        high = sh.cl_best[r] > high ? sh.cl_best[r] : high;
      }
      const Pieces pc(low, high);
      histogram<SUMS>(mt, pc);
      find_bin<SUMS>(tg, before_cnt, before_sum, -1.f);
      pc.narrow((int)sh.f_bin, mt.lo, mt.hi);
      mt.level = 2;
      before_cnt = sh.f_before_cnt;
      before_sum = sh.f_before_sum;
      cnt = sh.f_cnt;
    }
    gather(mt);
    if (rank == 0) {
      const unsigned long long key = in_list<SUMS>(tg, cnt, before_cnt, before_sum);
      if ((int)threadIdx.x < cl) remote(&sh, threadIdx.x)->end_key = key;
    }
    cluster.sync();
    return sh.end_key;
  }

  // The key of the target among the cnt tokens of the list (one CTA).
  template <bool SUMS>
  __device__ unsigned long long in_list(Target& tg, uint32_t cnt, uint32_t before_cnt, unsigned long long before_sum) {
    const int n = (int)cnt;
    unsigned long long lo = 0, hi = kKeyAll;
    auto left = [&](auto f) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long k = sh.list[i];
        if (k >= lo && k <= hi) f(k);
      }
    };
    while (cnt > kDirect) {
      unsigned long long low, high;
      key_range([&](auto f) { left(f); }, low, high);
      const Pieces pc(low, high);
      for (int b = threadIdx.x; b < kBins; b += kThreads) {
        sh.tcnt[b] = 0u;
        sh.tsum[b] = 0ull;
      }
      __syncthreads();
      left([&](unsigned long long k) {
        const int b = pc.piece(k);
        atomicAdd(&sh.tcnt[b], 1u);
        if (SUMS) add_weight(b, row.weight(k));
      });
      __syncthreads();
      if (SUMS) join_weights();
      find_bin<SUMS>(tg, before_cnt, before_sum, -1.f);
      pc.narrow((int)sh.f_bin, lo, hi);
      before_cnt = sh.f_before_cnt;
      before_sum = sh.f_before_sum;
      cnt = sh.f_cnt;
    }
    if (threadIdx.x == 0) sh.few_n = 0;
    __syncthreads();
    left([&](unsigned long long k) {
      const uint32_t at = atomicAdd(&sh.few_n, 1u);
      sh.few.key[at] = k;
      sh.few.w[at] = row.weight(k);
    });
    __syncthreads();
    pick<SUMS>(tg, cnt, before_cnt, before_sum);
    return sh.f_key;
  }

  // The target among sh.few, by comparing all pairs: f_key, f_w.
  template <bool SUMS>
  __device__ void pick(const Target& tg, uint32_t cnt, uint32_t before_cnt, unsigned long long before_sum) {
    constexpr uint32_t kEach = kThreads / kDirect;  // threads of a token
    static_assert(kEach * kDirect == kThreads && kEach <= 32, "neighbouring lanes share a token");
    const uint32_t mine = threadIdx.x / kEach;
    const unsigned long long k = mine < cnt ? sh.few.key[mine] : 0ull;
    uint32_t c = 0;
    unsigned long long s = 0;
#pragma unroll 4
    for (uint32_t j = threadIdx.x % kEach; j < cnt; j += kEach) {
      const bool better = sh.few.key[j] < k;
      c += better;
      s += better ? sh.few.w[j] : 0u;
    }
#pragma unroll
    for (uint32_t o = 1; o < kEach; o *= 2) {
      c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    }
    if (mine < cnt && tg.template holds<SUMS>(before_cnt + c, 1u, before_sum + s, sh.few.w[mine])) {
      sh.f_key = k;
      sh.f_w = sh.few.w[mine];
    }
    __syncthreads();
  }

  // All candidates are the cnt <= kList tokens of the list, those of the first
  // bins of the histogram (tcnt: tokens in better bins): rank them, apply the
  // filters and draw (one CTA, no cluster barrier).  The filters are top-k (k >
  // 0), then top-p as a limit on the sum of better ranks: that of the search by
  // sums, or (`own_limit`) the share tp of what top-k keeps.  f_key and f_w are
  // the drawn token's index and weight.  `probs` (or null) is the row's, all
  // zero (the CTAs stored the zeros before a cluster barrier).
  __device__ void finish(uint32_t cnt, int k, float tp, bool own_limit, float u, unsigned long long& total,
                         uint32_t& kept, float* probs) {
    constexpr int E = kList / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t kIdxMask = (1u << kIdxBits) - 1;
    // Grouped by bin, then placed by comparing within the bin.
    auto bin_of = [&](unsigned long long key) { return row.bin(order_float(~(uint32_t)(key >> kIdxBits))); };
    for (uint32_t i = tid; i < cnt; i += kThreads) {
      const unsigned long long x = sh.list[i];
      const int b = bin_of(x);
      sh.tsum[sh.tcnt[b] + atomicAdd(&sh.cursor[b], 1u)] = x;
    }
    __syncthreads();
    for (uint32_t i = tid; i < cnt; i += kThreads) {
      const unsigned long long x = sh.tsum[i];
      const int b = bin_of(x);
      const uint32_t from = sh.tcnt[b], to = from + sh.cursor[b];
      uint32_t at = from;
#pragma unroll 4
      for (uint32_t j = from; j < to; ++j) at += sh.tsum[j] < x;
      sh.list[at] = x;
    }
    __syncthreads();
    // Running sum by rank; a thread has ranks E * tid, ...
    unsigned long long key[E], inc[E], sum = 0;
    uint32_t w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool is = E * tid + i < (int)cnt;
      key[i] = is ? sh.list[E * tid + i] : kKeyAll;
      w[i] = is ? row.weight(key[i]) : 0u;
      sum += w[i];
    }
    unsigned long long run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xFFFFFFFFu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) sh.warp_sum[warp] = run;
    __syncthreads();
    run += warp_add(lane < warp ? sh.warp_sum[lane] : 0ull) - sum;
#pragma unroll
    for (int i = 0; i < E; ++i) inc[i] = run += w[i];
    if (own_limit && tp < 1.f) {
      const int last = (k > 0 && k < (int)cnt ? k : (int)cnt) - 1;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (E * tid + i == last) sh.limit = share_limit(tp, inc[i]);
      __syncthreads();
    }
    bool in[E];
    kept = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = E * tid + i;
      in[i] = e < (int)cnt && (k <= 0 || e < k) && w[i] > 0u;
      if (tp < 1.f) in[i] = in[i] && (inc[i] - w[i] < sh.limit || e == 0);
      if (row.min_p > 0.f) in[i] = in[i] && row.w(order_float(~(uint32_t)(key[i] >> kIdxBits))) >= row.min_p;
      kept += (uint32_t)__syncthreads_count(in[i]);  // each filter keeps a prefix of the ranking
    }
    const bool direct = kept <= kDirect;
    if (!direct) {
      for (int b = tid; b < kBins; b += kThreads) sh.tsum[b] = 0ull;
      if (tid < kPiece) sh.piece_w[tid] = 0u;
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = E * tid + i;
      if (e == (int)kept - 1) {
        sh.end_total = inc[i];
        sh.end_key = key[i];
        sh.target = draw(u, inc[i]);
      }
      if (!in[i]) continue;
      const uint32_t idx = (uint32_t)key[i] & kIdxMask;
      if (direct) {
        sh.few.key[e] = idx;
        sh.few.w[e] = w[i];
      } else {
        add_weight(idx / kPiece, w[i]);
      }
    }
    __syncthreads();
    total = sh.end_total;
    if (probs) {
      const float scale = 1.f / __ull2float_rn(total);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (in[i]) probs[(uint32_t)key[i] & kIdxMask] = __uint2float_rn(w[i]) * scale;
    }
    // The first token in index order at which the running sum exceeds the target.
    Target tg;
    tg.limit = sh.target + 1;
    if (direct) {
      pick<true>(tg, kept, 0u, 0ull);
      return;
    }
    // Of many: first the piece of the index range, then the token in it.
    join_weights();
    find_bin<true>(tg, 0u, 0ull, -1.f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t idx = (uint32_t)key[i] & kIdxMask;
      if (in[i] && idx / kPiece == sh.f_bin) sh.piece_w[idx % kPiece] = w[i];
    }
    __syncthreads();
    if (warp == 0) {
      constexpr int kEach = kPiece / 32;
      uint32_t x[kEach];
      sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[i] = sh.piece_w[lane * kEach + i], sum += x[i];
      run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += y;
      }
      run += sh.f_before_sum - sum;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (run < tg.limit && run + x[i] >= tg.limit) {
          sh.f_key = sh.f_bin * kPiece + lane * kEach + i;
          sh.f_w = x[i];
        }
        run += x[i];
      }
    }
    __syncthreads();
  }

  // floor(u * total), in [0, total).
  __device__ static unsigned long long draw(float u, unsigned long long total) {
    const unsigned long long t = u > 0.f ? (unsigned long long)((double)fminf(u, 1.f) * (double)total) : 0ull;
    return t >= total ? total - 1 : t;
  }
};

// A CTA's shared memory may be accessed by the others of its cluster once it has
// started: all arrive on entry and wait before the first remote access, which
// the loads between have long covered.  No data is passed on by this one.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// How scores of a type are read and kept.
template <typename T>
struct Loader;
template <>
struct Loader<float> {
  static constexpr int kVec = 4;
  using Vec = float4;
  __device__ static float one(const float* p) { return __ldcs(p); }
  __device__ static void unpack(const float4& v, float (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ static float store(float z, float) { return z; }
  __device__ static void store_vec(float* d, const float (&z)[4], const float4&) {
    *reinterpret_cast<float4*>(d) = make_float4(z[0], z[1], z[2], z[3]);
  }
  static constexpr bool kScaled = true;  // kept as scaled scores
  __device__ static float value(float x) { return x; }
  __device__ static float none() { return -CUDART_INF_F; }
  __device__ static float zero() { return 0.f; }
};
template <>
struct Loader<uint16_t> {
  static constexpr int kVec = 8;
  using Vec = uint4;
  __device__ static float one(const uint16_t* p) { return __uint_as_float((uint32_t)__ldcs(p) << 16); }
  __device__ static void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  __device__ static uint16_t store(float, uint16_t x) { return x; }
  __device__ static void store_vec(uint16_t* d, const float (&)[8], const uint4& x) { *reinterpret_cast<uint4*>(d) = x; }
  static constexpr bool kScaled = false;
  __device__ static float value(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  __device__ static uint16_t none() { return 0xFF80u; }
  __device__ static uint16_t zero() { return 0u; }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleParams p) {
  using L = Loader<T>;
  extern __shared__ __align__(32) uint8_t smp_dyn[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smp_dyn);
  cluster_arrive();
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cl;
  const int start = rank * p.chunk;
  const int n = start < p.vocab ? (p.vocab - start < p.chunk ? p.vocab - start : p.chunk) : 0;
  const float temp = p.temperature ? __ldg(&p.temperature[r]) : 1.f;
  const int k = p.top_k ? __ldg(&p.top_k[r]) : 0;
  const float tp = p.top_p ? __ldg(&p.top_p[r]) : 1.f;
  const float mp = p.min_p ? __ldg(&p.min_p[r]) : 0.f;
  const float u = __ldg(&p.u[r]);
  const bool greedy = temp == 0.f;
  const bool valid = temp >= 0.f;
  const float inv = greedy ? 1.f : 1.f / temp;
  const T* src = (const T*)p.logits + r * p.stride + start;
  float best = -CUDART_INF_F;
  auto put = [&](float v) {
    best = fmaxf(best, v);
    return v;
  };
  const int mis = (int)(((uintptr_t)src / sizeof(T)) & (L::kVec - 1));  // entries before the first score
  T* zbuf = reinterpret_cast<T*>(smp_dyn + ((sizeof(SampleShared) + 31) & ~(size_t)31));
  Scores<T> sc;
  sc.g = reinterpret_cast<decltype(sc.g)>(zbuf);
  sc.inv = inv;
  {
    // Shared memory takes the scores at the global address's offset within 16
    // bytes, so that both sides of a vector are aligned.
    T* z = zbuf + mis;
    const int head = n < ((L::kVec - mis) & (L::kVec - 1)) ? n : ((L::kVec - mis) & (L::kVec - 1));
    const int nvec = (n - head) / L::kVec;
    auto one = [&](int i) { z[i] = L::store(put(scaled(L::one(src + i), inv)), src[i]); };
    if (tid < head) one(tid);
    const typename L::Vec* v = reinterpret_cast<const typename L::Vec*>(src + head);
    constexpr int U = 4;
    for (int i0 = tid; i0 < nvec; i0 += kThreads * U) {
      typename L::Vec x[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kThreads < nvec) x[j] = __ldcs(v + i0 + j * kThreads);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i < nvec) {
          float f[L::kVec];
          L::unpack(x[j], f);
#pragma unroll
          for (int e = 0; e < L::kVec; ++e) f[e] = put(scaled(f[e], inv));
          L::store_vec(z + head + i * L::kVec, f, x[j]);
        }
      }
    }
    const int i = head + nvec * L::kVec + tid;
    if (i < n) one(i);
    // -inf around the scores: the passes take whole groups of four.
    if (tid < mis) zbuf[tid] = L::none();
    if (tid < 4) z[n + tid] = L::none();
  }
  // Where few tokens will be kept, the zeros of the probabilities go out now,
  // while there is other work; the kept ones follow when they are known.
  const bool single = greedy || tp <= 0.f;  // only the best token passes
  float* probs = p.probs ? p.probs + (int64_t)r * p.vocab + start : nullptr;
  const bool zero_first = probs && (single || (k > 0 && k <= kList));
  const bool aligned4 = (((uintptr_t)(probs - mis)) & 15) == 0;
  if (zero_first) {
    for (int v = tid; v < (mis + n + 3) / 4; v += kThreads) {
      const int i = 4 * v - mis;
      if (aligned4 && i >= 0 && i + 4 <= n) {
        __stcs(reinterpret_cast<float4*>(probs + i), make_float4(0.f, 0.f, 0.f, 0.f));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e >= 0 && i + e < n) __stcs(&probs[i + e], 0.f);
      }
    }
  }
  // Largest score of the row.
  const uint32_t warp_most = __reduce_max_sync(0xFFFFFFFFu, order_bits(best));
  if (lane == 0) sh.warp_cnt[warp] = warp_most;
  __syncthreads();
  cluster_wait();  // the first remote access follows
  if (warp == 0) {
    const uint32_t b = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? sh.warp_cnt[lane] : 0u);
    if (lane < cl) cluster.map_shared_rank(&sh, lane)->cl_cnt[rank] = b;
  }
  cluster.sync();
  float m = order_float(__reduce_max_sync(0xFFFFFFFFu, lane < cl ? sh.cl_cnt[lane] : 0u));
  const bool empty = !valid || m == -CUDART_INF_F;
  if (empty) {  // uniform over the cluster; no remote access follows
    if (rank == 0 && tid == 0) {
      p.token[r] = -1;
      if (p.logprob) p.logprob[r] = -CUDART_INF_F;
      if (p.kept) p.kept[r] = 0;
    }
    if (probs && !zero_first)
      for (int i = tid; i < n; i += kThreads) probs[i] = 0.f;
    return;
  }
  if (m == CUDART_INF_F) {
    // Only the infinite ones count, all alike: make them 0 and the rest -inf.
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      zbuf[mis + i] = scaled(L::value(zbuf[mis + i]), L::kScaled ? 1.f : inv) == CUDART_INF_F ? L::zero() : L::none();
    sc.inv = 1.f;
    m = 0.f;
    __syncthreads();
  }
  Sampler<T> s(sh, sc, mis + n, (uint32_t)(start - mis));
  s.row.m = m;
  // Rounded up: a large m has no float at m - kCut, and one below it would be
  // past the last bin (every W between is 0 all the same).
  s.row.least = __fsub_ru(m, kCut);
  s.row.min_p = mp > 0.f ? fminf(mp, 1.f) : 0.f;  // the best token passes
  s.row.bounded = false;
  if (single) {
    // The lowest index among equals: the least key.
    unsigned long long low, high;
    s.key_range([&](auto f) { s.each(m, m, [&](float zi, uint32_t idx) { f(rank_key(zi, idx)); }); }, low, high);
    if (tid == 0) cluster.map_shared_rank(&sh, 0)->cl_low[rank] = low;
    cluster.sync();  // no remote access follows
    if (rank == 0 && warp == 0) {
      low = ~warp_max(lane < cl ? ~sh.cl_low[lane] : 0ull);
      if (lane == 0) {
        const int idx = (int)((uint32_t)low & ((1u << kIdxBits) - 1));
        p.token[r] = idx;
        if (p.logprob) p.logprob[r] = 0.f;
        if (p.kept) p.kept[r] = 1;
        if (p.probs) p.probs[(int64_t)r * p.vocab + idx] = 1.f;
      }
    }
    return;
  }
  Match all;
  all.level = all.b0 = 0;
  all.lo = all.hi = 0;
  bool short_list = false, by_bins = false;
  unsigned long long sum = 0;  // by_bins: of this thread's share of the CTA's kept tokens
  uint32_t count = 0;
  unsigned long long total = 0;
  uint32_t kept = 0;
  const bool use_k = k > 0 && k < p.vocab, use_p = tp < 1.f;
  // Top-k, then top-p of what it left.  A short list of candidates ends the row.
  auto search = [&](auto by_sum, Target tg, float share) {
    constexpr bool SUMS = decltype(by_sum)::value;
    s.template histogram<SUMS>(all, Pieces(0, 0));
    if (!s.template find_bin<SUMS>(tg, 0u, 0ull, share, rank == 0)) return;
    const uint32_t upto = sh.f_before_cnt + sh.f_cnt;
    if (upto > kList) {
      const uint32_t bin = sh.f_bin, cnt = sh.f_cnt;
      const unsigned long long key = s.template resolve<SUMS>(tg);
      s.row.set_max(key);
      // With the bin's tokens listed one by one, each CTA knows what its kept
      // tokens weigh without another pass.  (In the bins up to kSureBins no
      // weight rounds to 0, so that tokens counted are tokens kept.)
      if (SUMS && s.row.min_p == 0.f && cnt <= kList && bin < kSureBins) {
        by_bins = true;
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i)
          if (tid * (kBins / kThreads) + i < (int)bin) sum += s.own_sum[i], count += s.own_cnt[i];
        // The first CTA's own copy is gone, but it has the list.
        const unsigned long long* list = rank == 0 ? sh.list : sh.tsum;
        const uint32_t listed = rank == 0 ? cnt : s.own_listed;
        for (uint32_t i = tid; i < listed; i += kThreads) {
          const unsigned long long x = list[i];
          if (x <= key && (rank != 0 || ((uint32_t)x & ((1u << kIdxBits) - 1)) < (uint32_t)n)) {
            sum += s.row.weight(x);
            ++count;
          }
        }
      }
      return;
    }
    short_list = true;
    Match to;
    to.level = -1;
    to.b0 = (int)sh.f_bin;
    s.gather(to);
    if (rank == 0) {
      s.finish(upto, SUMS ? 0 : k, tp, !SUMS, u, total, kept, zero_first ? p.probs + (int64_t)r * p.vocab : nullptr);
      if (tid == 0) {
        p.token[r] = (int)sh.f_key;
        if (p.logprob) p.logprob[r] = logf(__uint2float_rn(sh.f_w) / __ull2float_rn(total));
      }
      if (probs && !zero_first && tid > 0 && tid < cl) {
        SampleShared* o = cluster.map_shared_rank(&sh, tid);
        o->end_total = sh.end_total;
        o->end_key = sh.end_key;
      }
    }
    if (probs && !zero_first) {  // the others need the bound; no remote access follows
      cluster.sync();
      total = sh.end_total;
      s.row.set_max(sh.end_key);
    }
  };
  if (use_k) {
    Target tg;
    tg.limit = (unsigned long long)k;
    search(cuda::std::false_type{}, tg, -1.f);
  }
  if (use_p && !short_list) {
    Target tg;
    tg.limit = 0;
    search(cuda::std::true_type{}, tg, tp);
  }
  // Kept weight by warp: warp w owns a contiguous piece of the CTA's groups
  // of four.
  const Row row = s.row;
  const int base = start - mis;  // index in the row of the first entry
  const int piece = (((s.n4 + kWarps - 1) / kWarps) + 31) & ~31;
  const int p0 = warp * piece < s.n4 ? warp * piece : s.n4, p1 = p0 + piece < s.n4 ? p0 + piece : s.n4;
  auto kept4 = [&](int v, uint32_t (&w)[4]) {
    const float4 x = sc.get(v);
    w[0] = row.kept(x.x, (uint32_t)(base + 4 * v));
    w[1] = row.kept(x.y, (uint32_t)(base + 4 * v + 1));
    w[2] = row.kept(x.z, (uint32_t)(base + 4 * v + 2));
    w[3] = row.kept(x.w, (uint32_t)(base + 4 * v + 3));
  };
  if (!short_list) {
    auto pass = [&] {
      if (!row.bounded && row.min_p == 0.f) {  // no filter: exp and add
#pragma unroll 2
        for (int v = p0 + lane; v < p1; v += 32) {
          const float4 x = sc.get(v);
          const float z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = Row::fixed(row.w(z[e]));
            sum += w;
            count += w != 0u;
          }
        }
      } else {
#pragma unroll 2
        for (int v = p0 + lane; v < p1; v += 32) {
          uint32_t w[4];
          kept4(v, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += w[e], count += w[e] != 0u;
        }
      }
    };
    if (!by_bins) pass();
    sum = warp_add(sum);
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    __syncthreads();  // warp_sum, warp_cnt are also find_bin's
    if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_cnt[warp] = count;
    __syncthreads();
    if (warp == 0) {
      const unsigned long long a = warp_add(lane < kWarps ? sh.warp_sum[lane] : 0ull);
      const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.warp_cnt[lane] : 0u);
      if (lane < cl) {
        SampleShared* o = cluster.map_shared_rank(&sh, lane);
        o->cl_sum[rank] = a;
        o->cl_kept[rank] = c;
      }
    }
    cluster.sync();  // no remote access follows
    const unsigned long long of_cta = lane < cl ? sh.cl_sum[lane] : 0ull;
    total = warp_add(of_cta);
    kept = __reduce_add_sync(0xFFFFFFFFu, lane < cl ? sh.cl_kept[lane] : 0u);
    unsigned long long before = warp_add(lane < rank ? of_cta : 0ull);
    if (tid == 0) sh.target = Sampler<T>::draw(u, total);
    __syncthreads();
    const unsigned long long target = sh.target;
    if (by_bins) {
      // Only the CTA of the target looks where it is.
      sum = 0;
      if (target >= before && target < before + sh.cl_sum[rank]) {
        pass();
        sum = warp_add(sum);
        if (lane == 0) sh.warp_sum[warp] = sum;
        __syncthreads();
      }
    }
    before += warp_add(lane < warp ? sh.warp_sum[lane] : 0ull);
    if (target >= before && target < before + sum) {  // one warp of the cluster
      unsigned long long run = before;
      for (int v0 = p0; v0 < p1; v0 += 32) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (v0 + lane < p1) kept4(v0 + lane, w);
        const unsigned long long mine = (unsigned long long)w[0] + w[1] + w[2] + w[3];
        unsigned long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
          if (lane >= o) inc += x;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, target < run + inc);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            unsigned long long at = run + inc - mine;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (target >= at && target < at + w[e]) {
                p.token[r] = base + 4 * (v0 + lane) + e;
                if (p.logprob) p.logprob[r] = logf(__uint2float_rn(w[e]) / __ull2float_rn(total));
              }
              at += w[e];
            }
          }
          break;
        }
        run += __shfl_sync(0xFFFFFFFFu, inc, 31);
      }
    }
  }
  if (rank == 0 && tid == 0 && p.kept) p.kept[r] = (int)kept;
  if (probs && !(short_list && zero_first)) {
    const float scale = 1.f / __ull2float_rn(total);
    for (int v = tid; v < s.n4; v += kThreads) {
      uint32_t w[4];
      kept4(v, w);
      const int i = 4 * v - mis;
      if (aligned4 && i >= 0 && i + 4 <= n) {
        __stcs(reinterpret_cast<float4*>(probs + i), make_float4(__uint2float_rn(w[0]) * scale, __uint2float_rn(w[1]) * scale,
                                                                 __uint2float_rn(w[2]) * scale, __uint2float_rn(w[3]) * scale));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e >= 0 && i + e < n) __stcs(&probs[i + e], __uint2float_rn(w[e]) * scale);
      }
    }
  }
}

template <typename T>
cudaError_t launch(SampleParams p, cudaStream_t s) {
  // CTAs of a row: few enough scores that two CTAs fit an SM (kMostBytes); more
  // a row while all of them still run at once, down to 2,048 scores each.
  int cl = 1;
  auto piece = [&](int c) { return (p.vocab + c - 1) / c; };
  while (cl < kMaxCl && (piece(cl) > kMostScores || piece(cl) * (int)sizeof(T) > kMostBytes ||
                         (2ll * cl * p.rows <= 2 * kNumSMs && piece(cl) > 4096)))
    cl *= 2;
  p.chunk = (piece(cl) + 7) & ~7;
  const size_t smem = ((sizeof(SampleShared) + 31) & ~(size_t)31) + (size_t)(p.chunk + 16) * sizeof(T);
  auto kern = k_sample<T>;
  cudaError_t err = ensure_smem_attr((const void*)kern, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.rows * cl));
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
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DT_F32 ? launch<float>(p, s) : launch<uint16_t>(p, s);
}

}  // namespace moe
