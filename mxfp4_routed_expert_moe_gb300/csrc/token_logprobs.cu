// token_logprobs.cu — log probabilities of given tokens, ranks, entropies and
// the best alternatives of rows of logits.
//
// With m the row's largest logit, S = sum e^(z - m) and U = sum e^(z - m) (z - m):
//   logprob = z_t - m - log S,   entropy = log S - U / S.
// Every thread keeps (m, S, U) of what it has seen and rescales them where m
// grows; threads, warps and the CTAs of a row join theirs in a fixed order.
//
// The best alternatives come out of the same pass: the first tile of a piece
// gives 128 maxima of disjoint groups of logits, and the top-th of those is a
// bound that at least `top` logits reach; whatever is not below it goes to a list,
// a few times `top` of a row in random order.  One comparison per eight logits
// decides that there is nothing to list.  A list that overflows (rows that grow
// with the index) is made again in small steps, thinned by the same bound.
//
// A cluster of 1 to 8 CTAs takes a row; logits are read once.  Bound by HBM and by
// the instructions of a logit (ten) alike for many rows, by latency for one.
#include <cooperative_groups.h>

#include "dense.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;                       // vectors of 8 logits a thread has in flight
constexpr int kTile = kThreads * kUnroll;        // vectors
constexpr int kList = 2048;
constexpr int kGroups = kThreads / 4;
constexpr int kMaxCl = 8;
constexpr int kTop = MOE_LOGPROBS_MAX_TOP;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -200.f;                   // e^-200 is 0 in fp32

typedef unsigned long long Key;  // (order bits of a logit) << 32 | ~index: larger is better; 0: none

struct Stats {
  float m, s, u;
  int count;
};

struct ScoreShared {
  Key list[kList];
  Key group[kGroups];
  Key best[kTop];
  Key cl_best[kMaxCl][kTop];
  Stats warp[kWarps];
  Stats cl[kMaxCl];
  Key bound;
  uint32_t list_n;
};

__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_float(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }
// A logit that may be listed has a key above 0.
__device__ __forceinline__ Key key_of(float z, uint32_t index) {
  return z > -INFINITY ? ((Key)order_bits(z) << 32) | (uint32_t)~index : 0ull;
}
__device__ __forceinline__ Key key_max(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ float exp_of(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * kLog2e));
  return e;
}

// Statistics over a larger maximum M (m <= M; both may be -inf).
__device__ __forceinline__ void raise(float M, float& m, float& s, float& u) {
  const float d = fmaxf(m - M, kFar), f = exp_of(d);  // NaN (both infinite) as far
  u = f * (u + s * d);
  s *= f;
  m = M;
}
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float M = fmaxf(a.m, b.m);
  if (a.m != M) raise(M, a.m, a.s, a.u);
  if (b.m != M) raise(M, b.m, b.s, b.u);
  a.s += b.s;
  a.u += b.u;
  a.count += b.count;
  return a;
}

// The logits of a CTA's piece as vectors of eight from an address aligned to 16
// bytes; entries before and after the piece read as -inf.
template <bool BF16>
struct Piece {
  const uint8_t* base;  // of entry 0, `mis` entries before the piece
  int mis, n;           // entries of the piece
  int vectors;
  uint32_t first;       // index in the row of entry 0 (may wrap; added to)

  static constexpr int kSize = BF16 ? 2 : 4;
  __device__ Piece(const void* row, int start, int count) : n(count) {
    const uint8_t* src = (const uint8_t*)row + (size_t)start * kSize;
    mis = (int)(((uintptr_t)src & 15) / kSize);
    base = src - mis * kSize;
    vectors = n > 0 ? (mis + n + 7) / 8 : 0;
    first = (uint32_t)(start - mis);
  }
  __device__ __forceinline__ bool whole(int v) const { return 8 * v >= mis && 8 * v + 8 <= mis + n; }
  __device__ __forceinline__ float one(int i) const {
    if (i < mis || i >= mis + n) return -INFINITY;
    return BF16 ? bf16_f32(__ldg(reinterpret_cast<const uint16_t*>(base) + i)) : __ldg(reinterpret_cast<const float*>(base) + i);
  }
  __device__ __forceinline__ void edge(int v, float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = one(8 * v + e);
  }
};

__device__ __forceinline__ float max8(const float (&x)[8]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

// The top-th best of the 128 group maxima into sh.bound (0 where fewer groups
// hold something), each thread giving the best key that it knows.  Barriers on
// both sides.
__device__ __forceinline__ void find_bound(ScoreShared& sh, Key mine, int top) {
  mine = key_max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 1));
  mine = key_max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 2));
  if ((threadIdx.x & 3) == 0) sh.group[threadIdx.x >> 2] = mine;
  if (threadIdx.x == 0) sh.bound = 0ull;
  __syncthreads();
  if (threadIdx.x < kGroups) {
    const Key k = sh.group[threadIdx.x];
    int better = 0;
#pragma unroll 8
    for (int i = 0; i < kGroups; ++i) better += sh.group[i] > k;
    if (better == top - 1 && k) sh.bound = k;  // keys differ: one thread at most
  }
  __syncthreads();
}

__device__ __forceinline__ void list_add(ScoreShared& sh, Key k) {
  const uint32_t i = atomicAdd(&sh.list_n, 1u);
  if (i < kList) sh.list[i] = k;
}

// Drops from a list of up to kList keys what is below the bound of its groups;
// at most 16 keys of each of `top` groups stay.  All threads; barriers inside.
__device__ void thin(ScoreShared& sh, int top) {
  const uint32_t n = sh.list_n;
  Key k[kList / kThreads], most = 0ull;
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j) {
    const uint32_t i = threadIdx.x + j * kThreads;
    k[j] = i < n ? sh.list[i] : 0ull;
    most = key_max(most, k[j]);
  }
  find_bound(sh, most, top);
  if (threadIdx.x == 0) sh.list_n = 0;
  __syncthreads();
  const Key bound = sh.bound;
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j)
    if (k[j] && k[j] >= bound) list_add(sh, k[j]);
  __syncthreads();
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) k_token_logprobs(const LogprobParams p) {
  __shared__ ScoreShared sh;
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cl;
  const int start = rank * p.chunk;
  const int n = start < p.vocab ? min(p.chunk, p.vocab - start) : 0;
  const void* row = (const uint8_t*)p.logits + r * p.stride * (BF16 ? 2 : 4);
  const Piece<BF16> in(row, start, n);
  const int top = p.top;
  if (tid == 0) sh.list_n = 0;
  pdl_wait();

  // The given token: its logit, and the bounds above which a logit before or
  // after it in the row is ahead of it.
  int token = p.tokens ? __ldg(&p.tokens[r]) : -1;
  const bool known = token >= 0 && token < p.vocab;
  float zt = -INFINITY, ahead_before = INFINITY, ahead_after = INFINITY;
  if (known) {
    zt = BF16 ? bf16_f32(__ldg((const uint16_t*)row + token)) : __ldg((const float*)row + token);
    zt = fmaxf(zt, -INFINITY);  // NaN as -inf
    ahead_after = zt;
    // Logits before the token are ahead where they are equal, too: above the next
    // lower number.  (All of them, where the token's is -inf: added at the end.)
    if (zt > -INFINITY) ahead_before = zt == 0.f ? __uint_as_float(0x80000001u) : order_float(order_bits(zt) - 1u);
  }

  float m = -INFINITY, s = 0.f, u = 0.f;
  int count = 0;
  float bound_z = INFINITY;  // logits above are listed, after the first tile
  for (int v0 = 0; v0 < in.vectors || v0 == 0; v0 += kTile) {
    float x[kUnroll][8];
    {
      Eight<BF16> raw[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int v = v0 + j * kThreads + tid;
        if (v < in.vectors && in.whole(v)) raw[j].load(in.base, v);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int v = v0 + j * kThreads + tid;
        if (v < in.vectors && in.whole(v))
          raw[j].get(x[j]);
        else
          in.edge(v, x[j]);  // -inf past the end
      }
    }
    float most[kUnroll], all = -INFINITY;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) most[j] = max8(x[j]), all = fmaxf(all, most[j]);
    if (all > m) raise(all, m, s, u);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = fmaxf(x[j][e] - m, kFar);  // NaN, and -inf less -inf, as far
        const float w = exp_of(d);
        s += w;
        u = fmaf(w, d, u);
      }
    }
    if (known) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int i0 = (int)in.first + 8 * (v0 + j * kThreads + tid);
        if (i0 <= token && i0 + 7 >= token) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i0 + e != token) count += x[j][e] > (i0 + e < token ? ahead_before : ahead_after);
        } else {
          const float ahead = i0 < token ? ahead_before : ahead_after;
#pragma unroll
          for (int e = 0; e < 8; ++e) count += x[j][e] > ahead;
        }
      }
    }
    if (top) {
      if (v0 == 0) {
        Key mine = 0ull;
#pragma unroll
        for (int j = kUnroll - 1; j >= 0; --j) {
          const uint32_t i0 = in.first + 8 * (j * kThreads + tid);
          if (most[j] == all)
#pragma unroll
            for (int e = 7; e >= 0; --e)
              if (x[j][e] == all) mine = key_of(all, i0 + e);
        }
        find_bound(sh, mine, top);
        const Key bound = sh.bound;
        bound_z = bound ? order_float((uint32_t)(bound >> 32)) : -INFINITY;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
          if (most[j] >= bound_z)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const Key k = key_of(x[j][e], in.first + 8 * (j * kThreads + tid) + e);
              if (k && k >= bound) list_add(sh, k);
            }
      } else {
        // Indices behind the first tile's: an equal logit is not ahead.
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
          if (most[j] > bound_z)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (x[j][e] > bound_z) list_add(sh, key_of(x[j][e], in.first + 8 * (v0 + j * kThreads + tid) + e));
      }
    }
  }

  // Statistics: lanes, warps, CTAs.
  Stats st = {m, s, u, count};
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    Stats b;
    b.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    b.s = __shfl_xor_sync(0xFFFFFFFFu, st.s, o);
    b.u = __shfl_xor_sync(0xFFFFFFFFu, st.u, o);
    b.count = __shfl_xor_sync(0xFFFFFFFFu, st.count, o);
    st = (lane & o) ? join(b, st) : join(st, b);
  }
  if (lane == 0) sh.warp[warp] = st;
  __syncthreads();
  if (top) {
    if (sh.list_n > kList) {
      // Again in steps that the list has room for.
      __syncthreads();
      if (tid == 0) sh.list_n = 0, sh.bound = 0ull;
      __syncthreads();
      for (int i0 = 0; i0 < in.mis + in.n; i0 += kList / 2) {
        const Key bound = sh.bound;
#pragma unroll
        for (int j = 0; j < kList / 2 / kThreads; ++j) {
          const int i = i0 + j * kThreads + tid;
          const Key k = key_of(in.one(i), in.first + i);
          if (k && k >= bound) list_add(sh, k);
        }
        __syncthreads();
        if (sh.list_n > kList / 2) thin(sh, top);  // uniform: the count changes behind barriers only
        __syncthreads();
      }
    }
    if (sh.list_n > kThreads) thin(sh, top);
    // Ranks by counting: at most a key a thread.
    const uint32_t listed = sh.list_n;
    if (tid < kTop) sh.best[tid] = 0ull;
    __syncthreads();
    if (tid < (int)listed) {
      const Key k = sh.list[tid];
      int better = 0;
#pragma unroll 4
      for (uint32_t i = 0; i < listed; ++i) better += sh.list[i] > k;
      if (better < top) sh.best[better] = k;
    }
    __syncthreads();
  }
  if (warp == 0) {
    st = lane < kWarps ? sh.warp[lane] : Stats{-INFINITY, 0.f, 0.f, 0};
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      Stats b;
      b.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
      b.s = __shfl_xor_sync(0xFFFFFFFFu, st.s, o);
      b.u = __shfl_xor_sync(0xFFFFFFFFu, st.u, o);
      b.count = __shfl_xor_sync(0xFFFFFFFFu, st.count, o);
      st = (lane & o) ? join(b, st) : join(st, b);
    }
  }
  if (cl > 1) {
    cluster.sync();  // every CTA has started
    if (warp == 0) {
      ScoreShared* o = cluster.map_shared_rank(&sh, 0);
      if (lane == 0) o->cl[rank] = st;
      if (top) o->cl_best[rank][lane] = sh.best[lane];
    }
    cluster.sync();  // no remote access follows
    if (rank != 0) return;
    if (warp == 0) {
      st = sh.cl[0];
      for (int i = 1; i < cl; ++i) st = join(st, sh.cl[i]);
    }
    if (top) {
      if (tid < kTop) sh.best[tid] = 0ull;
      __syncthreads();
      if (tid < cl * kTop) {
        const Key* all = &sh.cl_best[0][0];
        const Key k = all[tid];
        int better = 0;
#pragma unroll 8
        for (int i = 0; i < cl * kTop; ++i) better += all[i] > k;
        if (k && better < top) sh.best[better] = k;
      }
    }
  }
  if (tid == 0) sh.cl[0] = st;
  __syncthreads();
  st = sh.cl[0];
  float log_s = logf(st.s);
  const bool infinite = st.m == INFINITY;
  if (infinite) {  // those logits share the probability: their number
    int c = 0;
    for (int i = tid; i < p.vocab; i += kThreads)
      c += (BF16 ? bf16_f32(__ldg((const uint16_t*)row + i)) : __ldg((const float*)row + i)) == INFINITY;
    c = __reduce_add_sync(0xFFFFFFFFu, c);
    if (lane == 0) sh.warp[warp].count = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < kWarps; ++w) c += sh.warp[w].count;
    log_s = logf((float)c);
  }
  if (warp != 0) return;
  auto log_prob = [&](float z) {
    if (infinite) return z == INFINITY ? -log_s : -INFINITY;
    return z == -INFINITY ? -INFINITY : (z - st.m) - log_s;
  };
  if (lane == 0) {
    if (p.logprob) p.logprob[r] = known ? log_prob(zt) : -INFINITY;
    if (p.rank) p.rank[r] = known ? st.count + (zt == -INFINITY ? token : 0) : -1;
    if (p.entropy) p.entropy[r] = infinite ? log_s : st.m == -INFINITY ? 0.f : log_s - st.u / st.s;
  }
  if (lane < top) {
    const Key k = sh.best[lane];
    p.top_ids[(int64_t)r * top + lane] = k ? (int)~(uint32_t)k : -1;
    p.top_logprobs[(int64_t)r * top + lane] = k ? log_prob(order_float((uint32_t)(k >> 32))) : -INFINITY;
  }
}

template <bool BF16>
cudaError_t launch(LogprobParams p, cudaStream_t s) {
  // CTAs of a row: as many as run at once with all rows' others, down to 4,096
  // logits each.
  int cl = 1;
  auto piece = [&](int c) { return (p.vocab + c - 1) / c; };
  while (cl < kMaxCl && 2ll * cl * p.rows <= 2 * kNumSMs && piece(cl) > 4096) cl *= 2;
  p.chunk = (piece(cl) + 7) & ~7;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.rows * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<BF16>, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DT_BF16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace moe
