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
// stay in shared memory.  K* comes from histograms (count and sum of W per
// bin) that the CTAs of the cluster add up over distributed shared memory: the
// first by m - z in 1,024 equal bins (a monotone function of z), then, only
// if the bin that holds the bound has more than kList tokens, by 10 bits of K
// at a time; a bin of at most kList tokens is ranked directly.
// Bound by latency (a handful of cluster barriers) for few rows, by the passes
// over shared memory and HBM for many.
#include <cooperative_groups.h>

#include "serve.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 1024;
constexpr int kIdxBits = 18;             // MOE_SAMPLE_MAX_VOCAB = 2^18
constexpr int kMaxCl = 8;
constexpr float kFix = 2147483648.f;     // 2^31
constexpr float kBinScale = 46.f;        // W > 0 needs m - z < 22.2: bins 0 .. 1021
constexpr unsigned long long kKeyAll = ~0ull;

struct SampleShared {
  // Histogram of this CTA (count, low and high 16 bits of W: native 32-bit
  // shared-memory atomics; at most 2^15 tokens a CTA keep all three below
  // 2^31), and, once the cluster has added them up, the list of one bin.
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];
    } h;
    struct {
      unsigned long long key[kList];
      uint32_t w[kList];
    } list;
  };
  unsigned long long tsum[kBins];  // the cluster's totals
  uint32_t tcnt[kBins];
  unsigned long long warp_best[kWarps];
  unsigned long long warp_sum[kWarps];
  uint32_t warp_cnt[kWarps];
  unsigned long long cl_best[kMaxCl];
  unsigned long long cl_sum[kMaxCl];
  uint32_t cl_cnt[kMaxCl];
  uint32_t list_n;  // rank 0's is the cluster's
  // Where a search ended.
  uint32_t f_bin, f_cnt, f_before_cnt;
  unsigned long long f_before_sum, f_key, f_sum;
};
static_assert(MOE_SAMPLE_MAX_VOCAB == 1 << kIdxBits, "index bits of the key");

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
  bool inf;      // m = +inf
  float min_p;   // 0: off
  unsigned long long key_max;  // K*

  // exp(z - m).  expf, not an approximation: the weights are part of the
  // definition, and the same function gives the same integers everywhere.
  __device__ __forceinline__ float w(float z) const { return inf ? (z == m ? 1.f : 0.f) : expf(z - m); }
  __device__ __forceinline__ static uint32_t fixed(float w) { return __float2uint_rn(w * kFix); }
  __device__ __forceinline__ int bin(float z) const {
    if (inf) return 0;
    const int b = (int)((m - z) * kBinScale);
    return b < kBins - 1 ? b : kBins - 1;
  }
  // Weight of a kept token, 0 for the others.
  __device__ __forceinline__ uint32_t kept(float z, uint32_t idx) const {
    const float e = w(z);
    if (min_p > 0.f && !(e >= min_p)) return 0u;
    if (key_max != kKeyAll && rank_key(z, idx) > key_max) return 0u;
    return fixed(e);
  }
};

__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long x = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = x > v ? x : v;
  }
  return v;
}

// What a search looks for: the token of a given rank, or the last one whose
// better ranks weigh less than a bound.
struct Target {
  bool by_count;
  uint32_t count;   // >= 1: rank count - 1
  double bound;
  __device__ __forceinline__ bool holds(uint32_t before_cnt, uint32_t cnt, unsigned long long before,
                                        unsigned long long sum) const {
    if (cnt == 0) return false;
    return by_count ? before_cnt < count && before_cnt + cnt >= count
                    : (double)before < bound && (double)(before + sum) >= bound;
  }
};

// Tokens of the CTA that match the search so far: bin b0 of the first
// histogram (-1: all), and the key's upper bits.
struct Match {
  int b0;
  int shift;                  // bits below the ones fixed so far
  unsigned long long prefix;  // key >> shift of the fixed bits
};

class Sampler {
 public:
  SampleShared& sh;
  const float* z;  // this CTA's scaled scores
  int n;           // how many
  uint32_t first;  // index of the first in the row
  int cl, rank;
  Row row;
  cg::cluster_group cluster;

  __device__ Sampler(SampleShared& s, const float* zs, int n_, uint32_t f)
      : sh(s), z(zs), n(n_), first(f), cluster(cg::this_cluster()) {
    cl = (int)cluster.num_blocks();
    rank = (int)cluster.block_rank();
  }

  template <typename T>
  __device__ __forceinline__ T* remote(T* p, int r) {
    return cluster.map_shared_rank(p, r);
  }

  __device__ __forceinline__ bool matches(const Match& mt, float zi, uint32_t idx) const {
    if (mt.b0 >= 0 && row.bin(zi) != mt.b0) return false;
    return (rank_key(zi, idx) >> mt.shift) == mt.prefix;
  }

  // Histogram of the matching tokens over the cluster into tcnt / tsum: by
  // m - z (mt.b0 < 0), else by the 10 key bits below mt.shift.
  __device__ void histogram(const Match& mt) {
    const int tid = threadIdx.x;
    for (int b = tid; b < kBins; b += kThreads) sh.h.cnt[b] = sh.h.lo[b] = sh.h.hi[b] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float zi = z[i];
      const uint32_t w = Row::fixed(row.w(zi));
      if (w == 0u) continue;
      int b;
      if (mt.b0 < 0) {
        b = row.bin(zi);
      } else {
        if (!matches(mt, zi, first + i)) continue;
        b = (int)(rank_key(zi, first + i) >> (mt.shift - 10)) & (kBins - 1);
      }
      atomicAdd(&sh.h.cnt[b], 1u);
      atomicAdd(&sh.h.lo[b], w & 0xFFFFu);
      atomicAdd(&sh.h.hi[b], w >> 16);
    }
    cluster.sync();
    // Each CTA adds up its share of the bins and gives every CTA the totals.
    const int share = kBins / cl;
    for (int b = rank * share + tid; b < (rank + 1) * share; b += kThreads) {
      uint32_t c = 0;
      unsigned long long s = 0;
      for (int r = 0; r < cl; ++r) {
        const SampleShared* o = remote(&sh, r);
        c += o->h.cnt[b];
        s += o->h.lo[b] + ((unsigned long long)o->h.hi[b] << 16);
      }
      for (int r = 0; r < cl; ++r) {
        SampleShared* o = remote(&sh, r);
        o->tcnt[b] = c;
        o->tsum[b] = s;
      }
    }
    if (tid == 0 && rank == 0) sh.list_n = 0;
    cluster.sync();
  }

  // The bin that holds the target, given what ranks before this histogram;
  // false (uniform): there is none.  Also returns the histogram's totals.
  __device__ bool find_bin(const Target& tg, uint32_t before_cnt, unsigned long long before_sum, uint32_t& all_cnt,
                           unsigned long long& all_sum) {
    constexpr int P = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t c = 0;
    unsigned long long s = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c += sh.tcnt[tid * P + i];
      s += sh.tsum[tid * P + i];
    }
    uint32_t ic = c;
    unsigned long long is = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t oc = __shfl_up_sync(0xFFFFFFFFu, ic, o);
      const unsigned long long os = __shfl_up_sync(0xFFFFFFFFu, is, o);
      if (lane >= o) ic += oc, is += os;
    }
    if (lane == 31) sh.warp_cnt[warp] = ic, sh.warp_sum[warp] = is;
    if (tid == 0) sh.f_bin = kBins;
    __syncthreads();
    all_cnt = 0;
    all_sum = 0;
    uint32_t bc = before_cnt;
    unsigned long long bs = before_sum;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) bc += sh.warp_cnt[i], bs += sh.warp_sum[i];
      all_cnt += sh.warp_cnt[i];
      all_sum += sh.warp_sum[i];
    }
    bc += ic - c;
    bs += is - s;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t xc = sh.tcnt[tid * P + i];
      const unsigned long long xs = sh.tsum[tid * P + i];
      if (tg.holds(bc, xc, bs, xs)) {
        sh.f_bin = tid * P + i;
        sh.f_cnt = xc;
        sh.f_before_cnt = bc;
        sh.f_before_sum = bs;
      }
      bc += xc;
      bs += xs;
    }
    __syncthreads();
    return sh.f_bin < kBins;
  }

  // After find_bin on the first histogram: the key of the target and the sum
  // of W up to and including it.  `fresh` becomes false if the first
  // histogram's totals were overwritten.
  __device__ void resolve(const Target& tg, unsigned long long& key, unsigned long long& sum, bool& fresh) {
    Match mt;
    mt.b0 = (int)sh.f_bin;
    mt.shift = 50;
    mt.prefix = 0;
    uint32_t before_cnt = sh.f_before_cnt;
    unsigned long long before_sum = sh.f_before_sum;
    while (sh.f_cnt > kList) {  // uniform: every CTA of the cluster has the same totals
      __syncthreads();
      fresh = false;
      histogram(mt);
      uint32_t ac;
      unsigned long long as;
      find_bin(tg, before_cnt, before_sum, ac, as);
      mt.shift -= 10;
      mt.prefix = (mt.prefix << 10) | sh.f_bin;
      before_cnt = sh.f_before_cnt;
      before_sum = sh.f_before_sum;
    }
    // Every CTA gets the list of the bin's tokens (in any order).
    uint32_t* cursor = remote(&sh.list_n, 0);
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float zi = z[i];
      if (!matches(mt, zi, first + i)) continue;
      const uint32_t w = Row::fixed(row.w(zi));
      if (w == 0u) continue;
      const uint32_t at = atomicAdd(cursor, 1u);
      const unsigned long long k = rank_key(zi, first + i);
      if (at < kList)
        for (int r = 0; r < cl; ++r) {
          SampleShared* o = remote(&sh, r);
          o->list.key[at] = k;
          o->list.w[at] = w;
        }
    }
    cluster.sync();
    const int cnt = (int)sh.f_cnt;
    for (int i = threadIdx.x; i < cnt; i += kThreads) {
      const unsigned long long k = sh.list.key[i];
      uint32_t c = before_cnt;
      unsigned long long s = before_sum;
      for (int j = 0; j < cnt; ++j)
        if (sh.list.key[j] < k) ++c, s += sh.list.w[j];
      if (tg.holds(c, 1u, s, sh.list.w[i])) {
        sh.f_key = k;
        sh.f_sum = s + sh.list.w[i];
      }
    }
    if (threadIdx.x == 0 && rank == 0) sh.list_n = 0;
    // The list may be filled again (by any CTA) only when all have read it.
    cluster.sync();
    key = sh.f_key;
    sum = sh.f_sum;
    __syncthreads();
  }
};

// Reads a CTA's scores into shared memory, scaled; returns the best
// (order bits, inverted index) seen by this thread.
template <typename T>
struct Loader;
template <>
struct Loader<float> {
  static constexpr int kVec = 4;
  using Vec = float4;
  __device__ static float one(const float* p) { return __ldcs(p); }
  __device__ static void unpack(const float4& v, float (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
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
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleParams p) {
  using L = Loader<T>;
  extern __shared__ __align__(32) uint8_t smp_dyn[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smp_dyn);
  float* zbuf = reinterpret_cast<float*>(smp_dyn + ((sizeof(SampleShared) + 31) & ~(size_t)31));
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cl;
  const int start = rank * p.chunk;
  const int n = start < p.vocab ? (p.vocab - start < p.chunk ? p.vocab - start : p.chunk) : 0;
  const float temp = p.temperature ? __ldg(&p.temperature[r]) : 1.f;
  const bool greedy = temp == 0.f;
  const bool valid = temp >= 0.f;
  const float inv = greedy ? 1.f : 1.f / temp;
  const T* src = (const T*)p.logits + r * p.stride + start;
  // Shared memory takes the scores at the global address's offset within 16
  // bytes, so that both sides of a vector are aligned.
  const int mis = (int)(((uintptr_t)src / sizeof(T)) & (L::kVec - 1));
  float* z = zbuf + mis;
  float best = -CUDART_INF_F;
  uint32_t besti = 0;
  auto put = [&](float x, int i) {
    float v = fmaf(x, inv, 0.f);  // + 0: no negative zeros
    v = v != v ? -CUDART_INF_F : v;
    if (v > best) best = v, besti = start + i;
    return v;
  };
  const int head = n < ((L::kVec - mis) & (L::kVec - 1)) ? n : ((L::kVec - mis) & (L::kVec - 1));
  const int nvec = (n - head) / L::kVec;
  if (tid < head) z[tid] = put(L::one(src + tid), tid);
  {
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
          for (int e = 0; e < L::kVec; ++e) f[e] = put(f[e], head + i * L::kVec + e);
          float4* d = reinterpret_cast<float4*>(z + head + i * L::kVec);
#pragma unroll
          for (int e = 0; e < L::kVec; e += 4) d[e / 4] = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
      }
    }
  }
  {
    const int i = head + nvec * L::kVec + tid;
    if (i < n) z[i] = put(L::one(src + i), i);
  }
  // Best score of the row, lowest index among equals.
  unsigned long long b = ((unsigned long long)order_bits(best) << 32) | (0xFFFFFFFFu - besti);
  b = warp_max(b);
  if (lane == 0) sh.warp_best[warp] = b;
  __syncthreads();
  if (warp == 0) {
    b = warp_max(lane < kWarps ? sh.warp_best[lane] : 0ull);
    if (lane < cl) cluster.map_shared_rank(&sh, lane)->cl_best[rank] = b;
  }
  if (tid == 0) sh.list_n = 0;
  cluster.sync();
  b = 0;
  for (int i = 0; i < cl; ++i) b = sh.cl_best[i] > b ? sh.cl_best[i] : b;
  const uint32_t ob = (uint32_t)(b >> 32);
  const float m = __uint_as_float(ob & 0x80000000u ? ob & 0x7FFFFFFFu : ~ob);
  const uint32_t mi = 0xFFFFFFFFu - (uint32_t)b;
  const bool empty = !valid || m == -CUDART_INF_F;
  float* probs = p.probs ? p.probs + (int64_t)r * p.vocab + start : nullptr;
  if (empty || greedy) {  // uniform over the cluster; no remote access follows
    if (rank == 0 && tid == 0) {
      p.token[r] = empty ? -1 : (int)mi;
      if (p.logprob) p.logprob[r] = empty ? -CUDART_INF_F : 0.f;
      if (p.kept) p.kept[r] = empty ? 0 : 1;
    }
    if (probs)
      for (int i = tid; i < n; i += kThreads) probs[i] = !empty && start + i == (int)mi ? 1.f : 0.f;
    return;
  }
  Sampler s(sh, z, n, (uint32_t)start);
  s.row.m = m;
  s.row.inf = m == CUDART_INF_F;
  const float mp = p.min_p ? __ldg(&p.min_p[r]) : 0.f;
  s.row.min_p = mp > 0.f ? fminf(mp, 1.f) : 0.f;  // the best token passes
  s.row.key_max = kKeyAll;
  const int k = p.top_k ? __ldg(&p.top_k[r]) : 0;
  const float tp = p.top_p ? __ldg(&p.top_p[r]) : 1.f;
  const bool use_k = k > 0 && k < p.vocab, use_p = tp < 1.f;
  if (use_k || use_p) {
    Match all;
    all.b0 = -1;
    all.shift = 50;
    all.prefix = 0;
    s.histogram(all);
    bool fresh = true;
    uint32_t ac = 0;
    unsigned long long key_k = kKeyAll, sum_k = 0, as = 0;
    Target tg;
    tg.by_count = true;
    tg.count = use_k ? (uint32_t)k : 0xFFFFFFFFu;
    tg.bound = 0.0;
    if (s.find_bin(tg, 0u, 0ull, ac, as)) s.resolve(tg, key_k, sum_k, fresh);
    else sum_k = as;
    if (use_p) {
      tg.by_count = false;
      tg.bound = (double)tp * (double)sum_k;
      const unsigned long long key_best = rank_key(m, mi);
      unsigned long long key_p = key_best, sum_p;
      if (tg.bound > 0.0) {
        if (!fresh) s.histogram(all);
        if (s.find_bin(tg, 0u, 0ull, ac, as)) s.resolve(tg, key_p, sum_p, fresh);
      }
      key_k = key_p < key_k ? key_p : key_k;
    }
    s.row.key_max = key_k;
  }
  // Kept weight by warp: warp w owns a contiguous piece of the CTA's tokens.
  const Row row = s.row;
  const int piece = (((n + kWarps - 1) / kWarps) + 31) & ~31;
  const int p0 = warp * piece < n ? warp * piece : n, p1 = p0 + piece < n ? p0 + piece : n;
  unsigned long long sum = 0;
  uint32_t cnt = 0;
  for (int i = p0 + lane; i < p1; i += 32) {
    const uint32_t w = row.kept(z[i], (uint32_t)(start + i));
    sum += w;
    cnt += w != 0u;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    cnt += __shfl_xor_sync(0xFFFFFFFFu, cnt, o);
  }
  __syncthreads();  // warp_sum, warp_cnt are also find_bin's
  if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_cnt[warp] = cnt;
  __syncthreads();
  if (tid < cl) {
    unsigned long long a = 0;
    uint32_t c = 0;
    for (int i = 0; i < kWarps; ++i) a += sh.warp_sum[i], c += sh.warp_cnt[i];
    SampleShared* o = cluster.map_shared_rank(&sh, tid);
    o->cl_sum[rank] = a;
    o->cl_cnt[rank] = c;
  }
  cluster.sync();  // no remote access follows
  unsigned long long total = 0, before = 0;
  uint32_t kept = 0;
  for (int i = 0; i < cl; ++i) {
    if (i < rank) before += sh.cl_sum[i];
    total += sh.cl_sum[i];
    kept += sh.cl_cnt[i];
  }
  const float u = __ldg(&p.u[r]);
  unsigned long long target = u > 0.f ? (unsigned long long)((double)fminf(u, 1.f) * (double)total) : 0ull;
  if (target >= total) target = total - 1;
  for (int i = 0; i < warp; ++i) before += sh.warp_sum[i];
  if (target >= before && target < before + sum) {  // one warp of the cluster
    unsigned long long run = before;
    for (int i0 = p0; i0 < p1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t w = i < p1 ? row.kept(z[i], (uint32_t)(start + i)) : 0u;
      unsigned long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, target < run + inc);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          p.token[r] = start + i;
          if (p.logprob) p.logprob[r] = logf(__uint2float_rn(w) / __ull2float_rn(total));
        }
        break;
      }
      run += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  if (rank == 0 && tid == 0 && p.kept) p.kept[r] = (int)kept;
  if (probs) {
    const float scale = 1.f / __ull2float_rn(total);
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t w = row.kept(z[i], (uint32_t)(start + i));
      __stcs(&probs[i], __uint2float_rn(w) * scale);
    }
  }
}

template <typename T>
cudaError_t launch(SampleParams p, cudaStream_t s) {
  // CTAs of a row: enough that its piece is small against shared memory (two
  // CTAs an SM overlap one's loads with another's passes) and that few rows
  // still spread over the chip; at least 2,048 scores each.
  int cl = 1;
  while (cl < kMaxCl) {
    const int piece = (p.vocab + cl - 1) / cl;
    if (piece <= 12288 && ((long long)p.rows * cl >= kNumSMs || piece <= 2048)) break;
    cl *= 2;
  }
  p.chunk = ((p.vocab + cl - 1) / cl + 7) & ~7;
  const size_t smem = ((sizeof(SampleShared) + 31) & ~(size_t)31) + (size_t)(p.chunk + 8) * 4;
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
