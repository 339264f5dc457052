// token_logprobs.cu — log probabilities of given tokens, ranks, entropies and
// the best alternatives of rows of logits.
//
// With S = sum e^(z - m) and U = sum e^(z - m) (z - m), whatever the reference m is,
//   logprob = z_t - m - log S,   entropy = log S - U / S.
// Sums are in base 2: with L = log2(e) and c = -m L rounded, a logit weighs
// 2^(z L + c), one FMA with one rounding; the rounding of c is common to all and
// cancels in every result, all of which are taken by the same FMA.  A warp's
// reference is the largest logit of its part of the first tile, and is raised only
// for logits more than 3 above it: were it each thread's own maximum, some lane of a
// warp would have a new one at nearly every step.  (512 rows of 163,840 without
// alternatives: 40.4 us at 3, 41.2 at 2.)  It may not stay far below the maximum,
// where log S and U / S would be large numbers with a small difference (40 below, an
// entropy of 0 erred by 5e-6, to either side).  The reference is a logit of the row, so
// that one token 3 above all others is at the reference, and otherwise the entropy is
// no small number.  Threads, warps and the CTAs of a row join their (m, c, S, U) in a
// fixed order.  What rounding leaves on the wrong side of 0 is 0.
//
// One comparison per 16 logits of a thread decides whether there is more to do with them: a
// far new maximum, logits ahead of the given token (which are counted one by one), or
// candidates for the alternatives.  Those come from a bound that the first tile of a
// piece gives: 128 maxima of disjoint groups of its logits, of which the top-th is
// reached by at least `top` logits; whatever is not below it goes to a list, a few
// times `top` of a row in random order, which gives better bounds on the way.  A list that overflows (rows that grow with
// the index) is made again in small steps, thinned by the same bound.
//
// A cluster of 1 to 8 CTAs takes a row; logits are read once.  512 rows of 163,840 in
// bf16 with given tokens take 63 us with 20 alternatives (2.7 TB/s; 15.5 warp
// instructions per 32 logits, issue slots 58 % busy) and 40 without (4.2 TB/s; 9.6, 55
// %): bound by instructions on the half of an SM's warps that 64 registers a thread
// leave, and by two rounds of CTAs (512 on 304 places) with barriers and latencies at
// each row's end.  What is above the alternatives' bound costs the instructions between
// the two.  Logits of -inf (a masked vocabulary) have the 16 of their thread summed
// twice: with a third of them, 54 and 78 us.  One row is bound by latency: 100,003
// logits, 8.8 us.  More warps an SM, or logits on their way through shared memory, were
// not faster.
#include <cooperative_groups.h>

#include <cuda/std/type_traits>

#include "async.cuh"
#include "dense.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kUnroll = 2;                       // vectors of 8 logits that a thread has in flight (with 4 registers spill)
constexpr int kGroups = 128;                     // of the first bound
constexpr int kMaxCl = 8;
constexpr int kTop = MOE_LOGPROBS_MAX_TOP;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = -300.f;                   // 2^-300 is 0 in fp32
constexpr float kPlain = 1048576.f;              // references beyond, whose c is rounded by 0.1 and more, are summed again at the end
constexpr float kAbove = 3.f;                    // logits this far above the reference raise it: weights below 2^5

typedef unsigned long long Key;  // (order bits of a logit) << 32 | ~index: larger is better; 0: none

struct Stats {
  float m, c, s, u;
  int count;
};

// Of a CTA of T threads.
template <int T>
struct ScoreShared {
  static constexpr int kList = 4 * T;
  Key list[kList];
  Key group[kGroups];
  Key best[kTop];
  Key cl_best[kMaxCl * kTop];  // [CTA][top]
  Stats warp[T / 32];
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
__device__ __forceinline__ float exp2_of(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}

// Two fp32 values in a register pair, for the packed FMA and add.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void apart(Two v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Sums over a larger reference.  Those around a far one (masked logits) may be
// infinite or NaN; they leave nothing here.
__device__ __forceinline__ void raise(float M, float C, Stats& a) {
  const float d = fmaxf(C - a.c, kFar), f = exp2_of(d);
  const bool left = a.s > 0.f && f > 0.f;
  a.u = left ? f * (a.u + a.s * d) : 0.f;
  a.s = left ? f * a.s : 0.f;
  a.m = M;
  a.c = C;
}
__device__ __forceinline__ float shift_of(float m) { return m > -INFINITY ? -m * kLog2e : 0.f; }
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  if (b.m > a.m) raise(b.m, b.c, a);
  if (a.m > b.m) raise(a.m, a.c, b);
  a.s += b.s;
  a.u += b.u;
  a.count += b.count;
  return a;
}
__device__ __forceinline__ Stats other(const Stats& a, int o) {
  Stats b;
  b.m = __shfl_xor_sync(0xFFFFFFFFu, a.m, o);
  b.c = __shfl_xor_sync(0xFFFFFFFFu, a.c, o);
  b.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
  b.u = __shfl_xor_sync(0xFFFFFFFFu, a.u, o);
  b.count = __shfl_xor_sync(0xFFFFFFFFu, a.count, o);
  return b;
}
__device__ __forceinline__ Stats warp_join(Stats st) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const Stats b = other(st, o);
    st = (threadIdx.x & o) ? join(b, st) : join(st, b);
  }
  return st;
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
    return BF16 ? bf16_f32(reinterpret_cast<const uint16_t*>(base)[i]) : reinterpret_cast<const float*>(base)[i];
  }
  __device__ __forceinline__ void edge(int v, float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = one(8 * v + e);
  }
};

__device__ __forceinline__ float max8(const float (&x)[8]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

// Largest of the logits of some vectors as they are held.
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int N>
__device__ __forceinline__ float most_of(const Eight<true> (&raw)[N]) {
  uint32_t m = 0xFF80FF80u;
#pragma unroll
  for (int j = 0; j < N; ++j) m = most2(m, most2(most2(raw[j].v.x, raw[j].v.y), most2(raw[j].v.z, raw[j].v.w)));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
template <int N>
__device__ __forceinline__ float most_of(const Eight<false> (&raw)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float x[8];
    raw[j].get(x);
    m = fmaxf(m, max8(x));
  }
  return m;
}

// f(key, rank) for each of n keys that differ (but for 0, none), a warp a key: rank is
// the number of better ones.  Every lane calls f with the same.
template <int T, typename F>
__device__ __forceinline__ void ranks(const Key* keys, int n, F f) {
  constexpr int kWarps = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (n <= 128) {  // a lane holds its share of them
    Key other[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) other[j] = lane + 32 * j < n ? keys[lane + 32 * j] : 0ull;
    for (int i = warp; i < n; i += kWarps) {
      const Key key = keys[i];
      int better = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) better += __popc(__ballot_sync(0xFFFFFFFFu, other[j] > key));
      f(key, better);
    }
    return;
  }
  for (int i = warp; i < n; i += kWarps) {
    const Key key = keys[i];
    int better = 0;
    for (int c = lane; c - lane < n; c += 32) {
      const Key other = c < n ? keys[c] : 0ull;
      better += __popc(__ballot_sync(0xFFFFFFFFu, other > key));
    }
    f(key, better);
  }
}

// The top-th best of the 128 group maxima into sh.bound (0 where fewer groups
// hold something), each thread giving the best key that it knows.  Barriers on
// both sides.
template <int T>
__device__ __forceinline__ void find_bound(ScoreShared<T>& sh, Key mine, int top) {
  constexpr int kLanes = T / kGroups;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) mine = key_max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
  if (threadIdx.x % kLanes == 0) sh.group[threadIdx.x / kLanes] = mine;
  if (threadIdx.x == 0) sh.bound = 0ull;
  __syncthreads();
  ranks<T>(sh.group, kGroups, [&](Key k, int better) {
    if (k && better == top - 1 && (threadIdx.x & 31) == 0) sh.bound = k;
  });
  __syncthreads();
}

template <int T>
__device__ __forceinline__ void list_add(ScoreShared<T>& sh, Key k) {
  const uint32_t i = atomicAdd(&sh.list_n, 1u);
  if (i < ScoreShared<T>::kList) sh.list[i] = k;
}

// Drops from a list of up to 4 T keys what is below the bound of its groups; the
// keys of `top` groups stay at most, 4 T / 128 each: T at most, a quarter of the list.
// All threads; barriers inside.
template <int T>
__device__ void thin(ScoreShared<T>& sh, int top) {
  const uint32_t n = sh.list_n;
  Key k[4], most = 0ull;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t i = threadIdx.x + j * T;
    k[j] = i < n ? sh.list[i] : 0ull;
    most = key_max(most, k[j]);
  }
  find_bound(sh, most, top);
  if (threadIdx.x == 0) sh.list_n = 0;
  __syncthreads();
  const Key bound = sh.bound;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (k[j] && k[j] >= bound) list_add(sh, k[j]);
  __syncthreads();
}

// The top-th best key of the list so far into sh.bound, if it is short; at least
// that many logits reach it.  All threads, barriers on both sides: named ones, which
// warps may reach by different ways through the code.
template <int T>
__device__ __forceinline__ void tighten(ScoreShared<T>& sh, int top) {
  named_sync(1, T);
  const int n = (int)sh.list_n;
  if (n >= top && n <= T)
    ranks<T>(sh.list, n, [&](Key k, int better) {
      if (better == top - 1 && (threadIdx.x & 31) == 0) sh.bound = k;
    });
  named_sync(1, T);
}

template <bool BF16, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_token_logprobs(const LogprobParams p) {
  constexpr int U = kUnroll, kTile = kThreads * U, kWarps = kThreads / 32, T = kThreads;
  typedef ScoreShared<T> Shared;
  constexpr int kList = Shared::kList;
  __shared__ Shared sh;
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
  const int token = p.tokens ? p.tokens[r] : -1;
  const bool known = token >= 0 && token < p.vocab;
  float zt = -INFINITY, ahead_before = INFINITY, ahead_after = INFINITY;
  if (known) {
    zt = BF16 ? bf16_f32(((const uint16_t*)row)[token]) : ((const float*)row)[token];
    zt = fmaxf(zt, -INFINITY) + 0.f;  // NaN as -inf, -0 as 0: a difference's sign tells what is ahead
    ahead_after = zt;
    // Logits before the token are ahead where they are equal, too: above the next
    // lower number.  (All of them, where the token's is -inf: added at the end.)
    if (zt > -INFINITY) ahead_before = zt == 0.f ? __uint_as_float(0x80000001u) : order_float(order_bits(zt) - 1u);
  }

  Stats st = {-INFINITY, 0.f, 0.f, 0.f, 0};
  Two s2 = 0, u2 = 0;        // the sums, in two lanes
  float bound_z = INFINITY;  // logits above are listed, behind the first tile
  float ahead = fminf(ahead_before, ahead_after);
  float limit = -INFINITY;   // vectors up to here need nothing but their sums
  const Two log2e2 = two(kLog2e, kLog2e);
  auto sums = [&](const float (&x)[U][8]) {
    const Two c2 = two(st.c, st.c);
    Two s = s2, u = u2;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const Two t2 = fma2(two(x[j][e], x[j][e + 1]), log2e2, c2);
        float t0, t1;
        apart(t2, t0, t1);
        const Two w2 = two(exp2_of(t0), exp2_of(t1));
        s = add2(s, w2);
        u = fma2(w2, t2, u);
      }
    float u0, u1;
    apart(u, u0, u1);
    if (!(u0 + u1 <= INFINITY)) {
      // An infinity or a NaN among them (0 times -inf): again with those far away.
      s = s2, u = u2;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float t0 = fmaxf(fmaf(x[j][e], kLog2e, st.c), kFar), t1 = fmaxf(fmaf(x[j][e + 1], kLog2e, st.c), kFar);
          const Two w2 = two(exp2_of(t0), exp2_of(t1));
          s = add2(s, w2);
          u = fma2(w2, two(t0, t1), u);
        }
    }
    s2 = s, u2 = u;
  };
  auto gather = [&] {
    float a, b;
    apart(s2, a, b);
    st.s = a + b;
    apart(u2, a, b);
    st.u = a + b;
  };
  auto counts = [&](const float (&x)[8], int i0) {
    if (i0 <= token && i0 + 7 >= token) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e != token) st.count += x[e] > (i0 + e < token ? ahead_before : ahead_after);
    } else {
      // By the sign of a - x, an addition of a shifted word each (44 against 41 us for
      // 512 rows of 163,840 without alternatives).  NaN, as of equal infinities, comes
      // without a sign.
      const float a = i0 < token ? ahead_before : ahead_after;
      const Two a2 = two(a, a), minus = two(-1.f, -1.f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float d0, d1;
        apart(fma2(two(x[e], x[e + 1]), minus, a2), d0, d1);
        st.count += (int)(__float_as_uint(d0) >> 31);
        st.count += (int)(__float_as_uint(d1) >> 31);
      }
    }
  };
  bool crowded;  // many logits are ahead of the token: counted without asking
  {
    float x[U][8], most[U];
    {
      Eight<BF16> raw[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (in.whole(j * kThreads + tid)) raw[j].load(in.base, j * kThreads + tid);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (in.whole(j * kThreads + tid))
          raw[j].get(x[j]);
        else
          in.edge(j * kThreads + tid, x[j]);  // -inf past the end
        most[j] = max8(x[j]);
        st.m = fmaxf(st.m, most[j]);
      }
    }
    Key bound = 0ull;
    if (top) {
      uint32_t at = 0u;  // of the thread's largest
#pragma unroll
      for (int j = U - 1; j >= 0; --j)
#pragma unroll
        for (int e = 7; e >= 0; --e) at = x[j][e] == st.m ? 8 * j * kThreads + e : at;
      find_bound(sh, key_of(st.m, in.first + 8 * tid + at), top);
      bound = sh.bound;
      bound_z = bound ? order_float((uint32_t)(bound >> 32)) : -INFINITY;
    }
    st.m = order_float(__reduce_max_sync(0xFFFFFFFFu, order_bits(st.m)));
    st.c = shift_of(st.m);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t i0 = in.first + 8 * (j * kThreads + tid);
      if (known && most[j] > ahead) counts(x[j], (int)i0);
      if (top && most[j] >= bound_z) {
        uint32_t which = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) which |= x[j][e] >= bound_z ? 1u << e : 0u;
        for (; which; which &= which - 1) {
          const int e = __ffs(which) - 1;
          const Key k = key_of(in.one(8 * (j * kThreads + tid) + e), i0 + e);
          if (k && k >= bound) list_add(sh, k);
        }
      }
    }
    sums(x);
    // A step of a warp sees as many logits as this: one of them ahead each time costs
    // more than counting all.
    crowded = __any_sync(0xFFFFFFFFu, st.count > 0);
  }
  // The tiles behind the first, the next one's logits in flight.
  auto pass = [&](auto count_all) {
    constexpr bool ALL = decltype(count_all)::value;
    auto set_limit = [&] { limit = fminf(st.m + kAbove, ALL ? bound_z : fminf(ahead, bound_z)); };
    auto step = [&](const float (&x)[U][8], float all, int v0) {
      if (ALL)
#pragma unroll
        for (int j = 0; j < U; ++j) counts(x[j], (int)in.first + 8 * (v0 + j * kThreads));
      if (all > limit) {
        if (all > st.m + kAbove) {
          gather();
          raise(all, shift_of(all), st);
          s2 = two(st.s, 0.f), u2 = two(st.u, 0.f);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const float most = max8(x[j]);
          const int v = v0 + j * kThreads, i0 = (int)in.first + 8 * v;
          if (!ALL && most > ahead) counts(x[j], i0);  // `ahead` is infinite without a token
          if (most > bound_z) {
            // Behind the first tile: an equal logit has a larger index and is not ahead.
            uint32_t which = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) which |= x[j][e] > bound_z ? 1u << e : 0u;
            for (; which; which &= which - 1) {
              const int e = __ffs(which) - 1;
              list_add(sh, key_of(in.one(8 * v + e), (uint32_t)(i0 + e)));
            }
          }
        }
        set_limit();
      }
      sums(x);
    };
    set_limit();
    // Tiles of whole vectors, then what is left of the piece.
    const int tiles = in.vectors > 0 ? (in.vectors - !in.whole(in.vectors - 1)) / kTile : 0;
    Eight<BF16> raw[U];
    if (tiles > 1)
#pragma unroll
      for (int j = 0; j < U; ++j) raw[j].load(in.base, kTile + tid + j * kThreads);
    for (int tile = 1; tile < tiles; ++tile) {
      const int v0 = tile * kTile + tid;
      float x[U][8];
      const float all = most_of(raw);
#pragma unroll
      for (int j = 0; j < U; ++j) raw[j].get(x[j]);
      if (tile + 1 < tiles)
#pragma unroll
        for (int j = 0; j < U; ++j) raw[j].load(in.base, v0 + kTile + j * kThreads);
      step(x, all, v0);
      // What is listed so far gives a better bound, of 2, 4 and 10 times the first
      // tile's logits.
      if (top && (tile == 1 || tile == 3 || tile == 9) && (tile + 1) * kTile < in.vectors) {
        tighten(sh, top);
        const Key bound = sh.bound;
        if (bound) bound_z = fmaxf(bound_z, order_float((uint32_t)(bound >> 32)));
        set_limit();
      }
    }
    if ((tiles > 1 ? tiles : 1) * kTile < in.vectors) {
      const int v0 = (tiles > 1 ? tiles : 1) * kTile + tid;
      float x[U][8], all = -INFINITY;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = v0 + j * kThreads;
        if (in.whole(v)) {
          raw[j].load(in.base, v);
          raw[j].get(x[j]);
        } else {
          in.edge(v, x[j]);  // -inf past the end
        }
        all = fmaxf(all, max8(x[j]));
      }
      step(x, all, v0);
    }
  };
  if (crowded)
    pass(cuda::std::true_type{});
  else
    pass(cuda::std::false_type{});
  gather();

  // Statistics: lanes, of one reference, then warps, CTAs.
  {
    const float m = order_float(__reduce_max_sync(0xFFFFFFFFu, order_bits(st.m)));
    raise(m, shift_of(m), st);
  }
  st = warp_join(st);
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
    // Ranks by counting.
    if (tid < kTop) sh.best[tid] = 0ull;
    __syncthreads();
    ranks<T>(sh.list, (int)sh.list_n, [&](Key k, int better) {
      if (better < top && lane == 0) sh.best[better] = k;
    });
    __syncthreads();
  }
  if (warp == 0) st = warp_join(lane < kWarps ? sh.warp[lane] : Stats{-INFINITY, 0.f, 0.f, 0.f, 0});
  if (cl > 1) {
    cluster.sync();  // every CTA has started
    if (warp == 0) {
      Shared* o = cluster.map_shared_rank(&sh, 0);
      if (lane == 0) o->cl[rank] = st;
      if (lane < top) o->cl_best[rank * top + lane] = sh.best[lane];
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
      ranks<T>(sh.cl_best, cl * top, [&](Key k, int better) {
        if (k && better < top && lane == 0) sh.best[better] = k;
      });
    }
  }
  if (tid == 0) sh.cl[0] = st;
  __syncthreads();
  st = sh.cl[0];
  const bool infinite = st.m == INFINITY, nothing = st.m == -INFINITY;
  bool plain = true;  // base 2 and the common shift
  if (!nothing && fabsf(st.m) > kPlain) {
    // Infinite logits, which share the probability, are counted; those around a far
    // maximum are summed by their differences.
    plain = false;
    float s = 0.f, u = 0.f;
    for (int i = tid; i < p.vocab; i += kThreads) {
      const float z = BF16 ? bf16_f32(((const uint16_t*)row)[i]) : ((const float*)row)[i];
      if (infinite) {
        s += z == INFINITY ? 1.f : 0.f;
      } else {
        const float d = fmaxf((z - st.m) * kLog2e, kFar), w = exp2_of(d);
        s += w;
        u = fmaf(w, d, u);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    }
    if (lane == 0) sh.warp[warp].s = s, sh.warp[warp].u = u;
    __syncthreads();
    st.s = st.u = 0.f;
    for (int w = 0; w < kWarps; ++w) st.s += sh.warp[w].s, st.u += sh.warp[w].u;
  }
  if (warp != 0) return;
  const float log2_s = log2f(st.s);
  auto log_prob = [&](float z) {
    if (infinite) return z == INFINITY ? -log2_s * kLn2 : -INFINITY;
    if (z == -INFINITY) return -INFINITY;
    if (plain && fabsf(z) <= kPlain) return fminf((fmaf(z, kLog2e, st.c) - log2_s) * kLn2, 0.f);
    return (z - st.m) - log2_s * kLn2;
  };
  if (lane == 0) {
    if (p.logprob) p.logprob[r] = known ? log_prob(zt) : -INFINITY;
    if (p.rank) p.rank[r] = known ? st.count + (zt == -INFINITY ? token : 0) : -1;
    if (p.entropy) p.entropy[r] = nothing ? 0.f : fmaxf((log2_s - st.u / st.s) * kLn2, 0.f);  // infinite: u = 0
  }
  if (lane < top) {
    const Key k = sh.best[lane];
    p.top_ids[(int64_t)r * top + lane] = k ? (int)~(uint32_t)k : -1;
    p.top_logprobs[(int64_t)r * top + lane] = k ? log_prob(order_float((uint32_t)(k >> 32))) : -INFINITY;
  }
}

template <bool BF16, int T>
cudaError_t launch(LogprobParams p, cudaStream_t s) {
  // CTAs of a row: as many as run at once with all rows' others, down to 8 logits a
  // thread.
  int cl = 1;
  auto piece = [&](int c) { return (p.vocab + c - 1) / c; };
  while (cl < kMaxCl && 2ll * cl * p.rows <= 2 * kNumSMs && piece(cl) > 8 * T) cl *= 2;
  p.chunk = (piece(cl) + 7) & ~7;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.rows * cl));
  cfg.blockDim = dim3(T);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<BF16, T>, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, int dtype, cudaStream_t s) {
  // Many short rows by small CTAs, whose barriers and latencies overlap.  With 20
  // alternatives, us by CTAs of 128 / 256 / 512 threads: 4,096 rows of 1,000: 42 / 59 /
  // 99, of 4,099: 75 / 74 / 104, of 16,000: 134 / 124 / 132, 1,024 of 64,000: 81 / 72 /
  // 69, 320 of 163,840: 246 / 73 / 52.
  const bool many = p.rows > 2 * kNumSMs;
  if (many && p.vocab <= 2048) return dtype == MOE_DT_BF16 ? launch<true, 128>(p, s) : launch<false, 128>(p, s);
  if (many && p.vocab <= 16384) return dtype == MOE_DT_BF16 ? launch<true, 256>(p, s) : launch<false, 256>(p, s);
  return dtype == MOE_DT_BF16 ? launch<true, 512>(p, s) : launch<false, 512>(p, s);
}

}  // namespace moe
