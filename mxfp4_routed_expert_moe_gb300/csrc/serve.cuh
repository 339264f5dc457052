// serve.cuh — parameter blocks and shared device helpers of the operators
// around the layer (moe_serve.h): paged append, shared-prefix attention,
// sampling.
#pragma once

#include <math_constants.h>

#include "async.cuh"
#include "kernels.h"
#include "moe_serve.h"

namespace moe {

// Record the first problem a kernel finds in the caller's sticky status word.
__device__ __forceinline__ void set_status_word(int32_t* status, int32_t code) {
  if (status) atomicCAS(reinterpret_cast<int*>(status), 0, code);
}

// The last b in [0, B) with start[b] <= n, found by the whole warp 32 probes
// at a time (two rounds up to 1,024 sequences: two dependent loads instead of
// ten).  Always inside [0, B), whatever the array holds.
__device__ __forceinline__ int find_sequence(const int32_t* start, int B, int n) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool below = i < hi && __ldg(&start[i]) <= n;
    const int cnt = __popc(__ballot_sync(0xFFFFFFFFu, below));
    lo += cnt > 0 ? (cnt - 1) * step : 0;
    hi = hi < lo + step ? hi : lo + step;
  }
  return lo;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tensor-map (TMA) load of one 4-D box at element coordinates (x, y, z, w).
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ append --
struct AppendParams {
  moe_kv_cache c;
  moe_kv_batch b;
  const void *q, *k, *v;
  int q_heads;
  int64_t q_stride, k_stride, v_stride;
  uint16_t* q_out;
  int64_t q_out_stride;
  const float* rope;
  int rope_rows, rot;
  int32_t* status;
};
cudaError_t launch_kv_append(const AppendParams& p, int x_dtype, bool interleaved, cudaStream_t s);

// ---------------------------------------------------------------- sampling --
struct SampleParams {
  int rows, vocab;
  const void* logits;
  int64_t stride;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* token;
  float* logprob;
  int32_t* kept;
  float* probs;
  int chunk;  // scores of a row per CTA of its cluster
};
cudaError_t launch_sample(const SampleParams& p, int dtype, cudaStream_t s);

// --------------------------------------------------------------- attention --
// Work of one attention kernel.  A "set" is a group of query rows that read
// the same tokens: sequence b's own part (set b), or the prefix (set `batch`,
// all rows).  Rows of a set for one key head: (token, head of the group), in
// tiles of `rows`; its tokens in units of `unit`.  The units of all sets, in
// (set, key head, row tile, unit) order, are cut into equal contiguous ranges,
// one per worker (a warp of the warp kernel, a CTA of the other); a worker's
// piece of one tile is a segment.  Its partial sums go to slot worker + tile,
// which is unique because every step to the next segment raises the worker or
// the tile by one.  A tile counts tile_cost units more than its tokens have,
// at its start: what loading its queries and storing its sums cost, so that
// ranges of many short tiles take as long as ranges of few long ones.
struct AttnSide {
  int own, prefix;       // which sets this kernel takes
  int rows, unit;        // query rows of a tile, tokens of a unit (powers of two)
  int rows_shift, unit_shift;
  int workers;           // most workers
  int tile_cost;         // units that a tile counts beside its tokens'
  float* slots;          // [workers + tiles][rows * (head_dim + 2)]
  long long* unit_start; // [batch + 1] first unit of each set; [batch + 1]: units per worker, 0: nothing was done
  int32_t* tile_start;   // [batch + 1] first tile of each set
};

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  int q_heads, group;  // query heads, query heads per key head
  float scale_log2;    // scale * log2(e)
  int kv_heads, head_dim, page_size, page_shift, num_pages;
  const uint16_t* v;  // the cache's values, for what the tensor maps do not serve
  int64_t page_stride, token_stride, head_stride;
  moe_kv_batch b;
  AttnSide side[2];    // 0: warps, 1: Tensor Memory
  int tile_rows;       // tile kernel: row tiles of a sequence and key head
  int32_t* status;
  long long wait_limit;
};

// The warp side: seven workers a CTA (32 KB of ring each), tiles of 16 rows,
// units of 16 KB of keys and values.
constexpr int kAttnWarpRows = 16;
__host__ __device__ constexpr int attn_warp_unit(int head_dim) { return head_dim == 128 ? 32 : 64; }
// The Tensor Memory side: one worker a CTA, tiles of 256 rows, units of 128
// tokens.
constexpr int kAttnTcRows = 256;
constexpr int kAttnTcUnit = 128;
// For sharing the CTAs out: time of a unit in us, of a worker among seven and of
// a tile of more than 128 rows; how much longer the Tensor Memory side takes to
// get going; and the units that a tile of the warp side counts beside its
// tile_cost, since few CTAs take many tiles in turn next to a busy other side
// (256 sequences with one token each of their own behind 32,768: 190 us, 221
// without; with up to 509 tokens 235 and 240).
constexpr float kAttnWarpUnitCost = 1.5f, kAttnTcUnitCost = 1.6f, kAttnTcStart = 5.f, kAttnWarpTileMore = 0.7f;

// What a set's entries say, as loaded.
struct AttnRaw {
  int q0, q1, len;
};

__device__ __forceinline__ AttnRaw attn_load(const AttnParams& p, int s) {
  AttnRaw r;
  r.q0 = 0;
  r.q1 = p.b.tokens;
  r.len = p.b.prefix_len;
  if (s < p.b.batch) {
    r.q0 = p.b.q_start ? __ldg(&p.b.q_start[s]) : s;
    r.q1 = p.b.q_start ? __ldg(&p.b.q_start[s + 1]) : s + 1;
    r.len = __ldg(&p.b.kv_len[s]);
  }
  return r;
}

// One set as an attention kernel sees it.
struct AttnSet {
  int rows;      // query rows per key head
  int tok0;      // first query token
  int len;       // tokens of the set
  int first_vis; // tokens the first query token sees (each later one sees one more); len for the prefix
  int tiles;     // row tiles per key head
  int units;     // units per row tile, with the tile's own cost
};

// Whether a sequence's entries fit the batch and its table (reported if not).
__device__ __forceinline__ bool attn_valid(const AttnParams& p, const AttnRaw& r) {
  if (r.q0 >= 0 && r.q1 >= r.q0 && r.q1 <= p.b.tokens && r.q1 - r.q0 <= p.b.max_q && r.len >= 0 &&
      r.len <= MOE_SERVE_MAX_LEN && r.len <= (long long)p.b.table_pages * p.page_size)
    return true;
  set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
  return false;
}

__device__ __forceinline__ AttnSet attn_set(const AttnParams& p, const AttnSide& sd, int s, const AttnRaw& r) {
  AttnSet a;
  a.rows = a.tok0 = a.len = a.first_vis = a.tiles = a.units = 0;
  const bool prefix = s == p.b.batch;
  if (!(prefix ? sd.prefix : sd.own)) return a;
  const int ql = r.q1 - r.q0;
  if (!prefix && !attn_valid(p, r)) return a;
  if (ql == 0 || r.len == 0) return a;
  a.tok0 = r.q0;
  a.len = r.len;
  a.first_vis = prefix ? r.len : r.len - ql + 1;
  a.rows = ql * p.group;
  a.tiles = (a.rows + sd.rows - 1) >> sd.rows_shift;
  a.units = ((a.len + sd.unit - 1) >> sd.unit_shift) + sd.tile_cost;
  return a;
}

// The page table of set s.
__device__ __forceinline__ const int32_t* attn_table(const AttnParams& p, int s) {
  return s == p.b.batch ? p.b.prefix_table : p.b.table + (int64_t)s * p.b.table_stride;
}

// Tokens that query token i (of the set's tokens) sees, in [0, len].
__device__ __forceinline__ int attn_visible(const AttnParams& p, const AttnSet& a, int s, int i) {
  if (s == p.b.batch) return a.len;
  const int v = a.first_vis + i;
  return v < 0 ? 0 : (v > a.len ? a.len : v);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A worker's walk over its range of units.  The entries of the next set are
// loaded one set ahead, so that stepping to it waits for no memory.
struct AttnWalk {
  int set;
  AttnSet a;
  AttnRaw next;
  long long unit0;   // first unit of the set
  int tile0;         // first tile of the set
  int worker;
  long long u, u1;   // next unit, end of the range
};

// The plan as the CTAs of one launch share it.  Blocks [0, ctas[1]) work on
// side 1 (Tensor Memory), the others on side 0 (warps).
constexpr int kAttnWarpWorkers = 7;
struct AttnPlan {
  long long part_u[32];
  int part_t[32];
  long long unit0[kAttnWarpWorkers];
  int set[kAttnWarpWorkers], tile0[kAttnWarpWorkers];
  // Everything below is the same in every CTA.
  long long total[2], per[2];
  int ctas[2];
};

// All threads of the CTA: add up the sets' units, share the CTAs out between
// the two sides by what their units cost, cut each side's units into ranges for
// its workers (worker w of a side's CTA c is number w * ctas + c, so that few
// units spread over the SMs) and find where the ranges of this CTA's workers
// begin.  Only the side of the own parts needs a scan; a prefix alone on its
// side is one set.  CTA 0 writes the plan for the joining kernel.
__device__ __forceinline__ void attn_plan(const AttnParams& p, AttnPlan& sh) {
  const int own = p.side[1].own ? 1 : 0;  // the side that is scanned
  const AttnSide& sd = p.side[own];
  const bool two = p.side[own ^ 1].prefix != 0;
  const int nsets = p.b.batch + 1, nt = blockDim.x, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5, nwarps = nt >> 5;
  const int per_thread = (nsets + nt - 1) / nt;
  const int s0 = tid * per_thread < nsets ? tid * per_thread : nsets;
  const int s1 = s0 + per_thread < nsets ? s0 + per_thread : nsets;
  long long u = 0;
  int t = 0;
  bool falls = false;
  for (int s = s0; s < s1; ++s) {
    const AttnRaw raw = attn_load(p, s);
    falls |= raw.q1 < raw.q0;
    const AttnSet a = attn_set(p, sd, s, raw);
    const int tiles = a.tiles * p.kv_heads;
    u += (long long)tiles * a.units;
    t += tiles;
  }
  long long eu = u;  // inclusive scans
  int et = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ou = __shfl_up_sync(0xFFFFFFFFu, eu, o);
    const int ot = __shfl_up_sync(0xFFFFFFFFu, et, o);
    if (lane >= o) {
      eu += ou;
      et += ot;
    }
  }
  if (lane == 31) {
    sh.part_u[warp] = eu;
    sh.part_t[warp] = et;
  }
  // Where q_start falls, sequences may overlap, and their tiles be more than
  // the workspace has slots for: nothing is done on their side (attn_valid has
  // reported it).
  const bool broken = __syncthreads_or(falls);
  long long total = 0;
  int tiles = 0;
  eu -= u;  // exclusive
  et -= t;
  for (int i = 0; i < nwarps; ++i) {
    const long long x = sh.part_u[i];
    if (i < warp) {
      eu += x;
      et += sh.part_t[i];
    }
    total += x;
    tiles += sh.part_t[i];
  }
  if (broken) total = 0;
  if (tid == 0) {
    long long other = 0;
    if (two) {
      const AttnSet a = attn_set(p, p.side[own ^ 1], p.b.batch, attn_load(p, p.b.batch));
      other = (long long)a.tiles * p.kv_heads * a.units;
    }
    sh.total[own] = total;
    sh.total[own ^ 1] = other;
    // CTAs of side 1, x of n: both sides should end together,
    //   kAttnTcStart + c1 / x = c0 / (n - x),
    // with c the time that their units cost one CTA.  Sides with units get one
    // CTA at least.
    const int n = gridDim.x;
    const float more = own == 0 ? kAttnWarpTileMore * (float)tiles : 0.f;
    const float c1 = (float)sh.total[1] * kAttnTcUnitCost;
    const float c0 = ((float)sh.total[0] + more) * (kAttnWarpUnitCost / kAttnWarpWorkers);
    int n1 = sh.total[1] == 0 ? 0 : n;
    if (n1 > 0 && sh.total[0] > 0) {
      int lo = 1, hi = n - 1;
      while (lo < hi) {
        const int x = (lo + hi) / 2;
        if (kAttnTcStart + __fdividef(c1, (float)x) > __fdividef(c0, (float)(n - x))) lo = x + 1;
        else hi = x;
      }
      n1 = lo;
    }
    if (sh.total[1] > 0 && n1 < 1) n1 = 1;
    if (sh.total[0] > 0 && n1 > n - 1) n1 = n - 1;
    sh.ctas[1] = n1;
    sh.ctas[0] = n - n1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long workers = (long long)sh.ctas[i] * (i == 0 ? kAttnWarpWorkers : 1);
      const long long x = workers > 0 ? (sh.total[i] + workers - 1) / workers : 0;
      sh.per[i] = x < 1 ? 1 : x;
    }
    // A prefix alone on its side: every worker's range begins in it.
    if (two) {
      for (int w = 0; w < kAttnWarpWorkers; ++w) {
        sh.set[w] = p.b.batch;
        sh.unit0[w] = 0;
        sh.tile0[w] = 0;
      }
    }
    if (blockIdx.x == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (p.side[i].unit_start) p.side[i].unit_start[nsets] = broken && i == own ? 0 : sh.per[i];
      if (two) {
        p.side[own ^ 1].unit_start[p.b.batch] = 0;
        p.side[own ^ 1].tile_start[p.b.batch] = 0;
      }
    }
  }
  __syncthreads();
  // Where this CTA's workers of the scanned side begin.
  const int side = (int)blockIdx.x < sh.ctas[1] ? 1 : 0;
  const int workers = side != own ? 0 : own == 0 ? kAttnWarpWorkers : 1;
  const int cta = side == 1 ? (int)blockIdx.x : (int)blockIdx.x - sh.ctas[1], ctas = sh.ctas[side];
  const long long per = sh.per[own];
  bool mine = blockIdx.x == 0;
  for (int w = 0; w < workers; ++w) {
    const long long u0 = ((long long)w * ctas + cta) * per;
    mine |= u0 >= eu && u0 < eu + u;
  }
  if (mine) {
    long long su = eu;
    int st = et;
    for (int s = s0; s < s1; ++s) {
      const AttnSet a = attn_set(p, sd, s, attn_load(p, s));
      const int tiles = a.tiles * p.kv_heads;
      const long long n = (long long)tiles * a.units;
      for (int w = 0; w < workers; ++w) {
        const long long u0 = ((long long)w * ctas + cta) * per;
        if (u0 >= su && u0 < su + n) {
          sh.set[w] = s;
          sh.unit0[w] = su;
          sh.tile0[w] = st;
        }
      }
      if (blockIdx.x == 0 && (s < p.b.batch || !two)) {
        sd.unit_start[s] = su;
        sd.tile_start[s] = st;
      }
      su += n;
      st += tiles;
    }
  }
  __syncthreads();
}

// The walk of this CTA's worker w on its side; false: nothing to do.
__device__ __forceinline__ bool attn_begin(const AttnParams& p, const AttnPlan& sh, int side, int w, AttnWalk& k) {
  const int cta = side == 1 ? (int)blockIdx.x : (int)blockIdx.x - sh.ctas[1];
  k.worker = w * sh.ctas[side] + cta;
  k.u = k.worker * sh.per[side];
  if (k.u >= sh.total[side]) return false;
  k.u1 = k.u + sh.per[side] < sh.total[side] ? k.u + sh.per[side] : sh.total[side];
  k.set = sh.set[w];
  k.unit0 = sh.unit0[w];
  k.tile0 = sh.tile0[w];
  k.a = attn_set(p, p.side[side], k.set, attn_load(p, k.set));
  k.next = attn_load(p, k.set < p.b.batch ? k.set + 1 : k.set);
  return true;
}

// The next segment of the walk.
struct AttnSeg {
  int set, tok0, len;  // the set
  int first_vis;       // of an own part: tokens its first query token sees; of the prefix: where in [kv0, kv1) to begin
  int slot, kvh;
  int row0;      // first row of the tile in its set
  int rows;      // rows of the tile
  int kv0, kv1;  // token range [kv0, kv1) of the set, cut to what the tile's last row sees (may be empty)
  int odd;       // values were taken out of it (clear_odd_values)
};

// Where in [kv0, kv1) a segment begins; the rest follows in order, then what is
// before it, from kv0 on.
__device__ __forceinline__ int attn_first(const AttnParams& p, const AttnSeg& g) {
  return g.set == p.b.batch ? g.first_vis : g.kv0;
}

__device__ __forceinline__ int attn_visible(const AttnParams& p, const AttnSeg& g, int i) {
  if (g.set == p.b.batch) return g.len;
  const int v = g.first_vis + i;
  return v < 0 ? 0 : (v > g.len ? g.len : v);
}

// TURN: the segments of a long prefix begin where the ranges of other tiles are
// at the same time, unit x as near as can be to x modulo the ranges' length
// after the start.  The row tiles of a key head read the same cache; with every
// range in plain order each unit came from HBM for most of them, once the
// prefix was longer than L2 holds (256 sequences of one token behind 32,768, 134
// MB of prefix, 7 tiles a key head: 207 us in plain order, 190 turned; of up to
// 509 tokens 240 and 235).  What L2 holds is left in plain order, in which the
// CTAs ask for different lines (9 prompts of up to 301 tokens behind 4,001: 123.5
// us either way).
constexpr long long kAttnTurnBytes = 96ll << 20;
template <bool TURN>
__device__ __forceinline__ bool attn_next(const AttnParams& p, const AttnPlan& sh, const AttnSide& sd, AttnWalk& w,
                                          AttnSeg& g) {
  if (w.u >= w.u1) return false;
  int tiles = w.a.tiles * p.kv_heads;
  while (w.u >= w.unit0 + (long long)tiles * w.a.units) {
    w.unit0 += (long long)tiles * w.a.units;
    w.tile0 += tiles;
    ++w.set;
    w.a = attn_set(p, sd, w.set, w.next);
    w.next = attn_load(p, w.set < p.b.batch ? w.set + 1 : w.set);
    tiles = w.a.tiles * p.kv_heads;
  }
  const long long lu = w.u - w.unit0;
  int tile, k0;
  if (lu < 0x7FFFFFFFll) {
    tile = (int)((uint32_t)lu / (uint32_t)w.a.units);
    k0 = (int)((uint32_t)lu - (uint32_t)tile * (uint32_t)w.a.units);
  } else {
    tile = (int)(lu / w.a.units);
    k0 = (int)(lu - (long long)tile * w.a.units);
  }
  long long n = w.a.units - k0;
  if (n > w.u1 - w.u) n = w.u1 - w.u;
  w.u += n;
  g.set = w.set;
  g.tok0 = w.a.tok0;
  g.first_vis = w.a.first_vis;
  g.len = w.a.len;
  g.slot = w.worker + w.tile0 + tile;
  g.kvh = tile / w.a.tiles;
  g.row0 = (tile - g.kvh * w.a.tiles) * sd.rows;
  g.rows = w.a.rows - g.row0 < sd.rows ? w.a.rows - g.row0 : sd.rows;
  const int vis = attn_visible(p, g, (g.row0 + g.rows - 1) / p.group);
  const int r0 = k0 > sd.tile_cost ? k0 - sd.tile_cost : 0;
  const long long r1 = k0 + n > sd.tile_cost ? k0 + n - sd.tile_cost : 0;
  g.kv0 = r0 << sd.unit_shift;
  const long long e = r1 << sd.unit_shift;
  g.kv1 = e < vis ? (int)e : vis;
  if (g.kv1 < g.kv0) g.kv1 = g.kv0;
  g.odd = 0;
  if (g.set == p.b.batch) g.first_vis = g.kv0;
  if (TURN && g.set == p.b.batch && 4ll * p.head_dim * p.kv_heads * g.len > kAttnTurnBytes &&
      sh.per[1] <= 0x7FFFFFFF) {
    const int per = (int)sh.per[1], at = r0 % per;
    const int past = (int)(w.u - n - (long long)w.worker * per);
    const int turn = past >= at ? past - at : past - at + per;
    if (turn < ((g.kv1 - g.kv0 + sd.unit - 1) >> sd.unit_shift)) g.first_vis += turn << sd.unit_shift;
  }
  return true;
}

// Values of tokens that some rows of a tile see and others do not: in the product
// with the others' weights of 0 an infinity or NaN would become NaN.  So these
// are taken out of the copy in shared memory (clear_odd_values) and added to the
// sums of the rows that see them (add_odd_values), which a positive weight leaves
// what they are.  With the search for them 9 prompts of up to 301 tokens behind
// 4,001 take 123 us instead of 118 and 8 tokens over 16,001 34.6 instead of 33.3;
// tiles of one new token have none, and pay for code in the way alone (256
// sequences of up to 509 tokens behind 32,768: 235 instead of 229).
__device__ __forceinline__ bool odd_bf16(uint32_t x) { return (x & 0x7F80u) == 0x7F80u; }

// By one warp: tokens [t0, t1) of V in shared memory, 128 bytes a token in each
// half of 64 values.  True, in all lanes, if there were any.
template <int HALVES>
__device__ __forceinline__ bool clear_odd_values(uint8_t* v, int half_bytes, int t0, int t1) {
  const int lane = threadIdx.x & 31;
  uint32_t most = 0;  // largest magnitudes, as integers
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll 4
    for (int i = t0 * 8 + lane; i < t1 * 8; i += 32) {
      const uint4 x = *reinterpret_cast<const uint4*>(v + h * half_bytes + i * 16);
      most = __vmaxu2(__vmaxu2(most, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
      most = __vmaxu2(__vmaxu2(most, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
    }
  if (__builtin_expect(!__any_sync(0xFFFFFFFFu, odd_bf16(most) || odd_bf16(most >> 16)), 1)) return false;
#pragma unroll 1
  for (int h = 0; h < HALVES; ++h)
#pragma unroll 1
    for (int i = t0 * 64 + lane; i < t1 * 64; i += 32) {
      uint16_t* x = reinterpret_cast<uint16_t*>(v + h * half_bytes) + i;
      if (odd_bf16(*x)) *x = 0;
    }
  return true;
}

// By one warp, whose other values are in `dst` already: rows [r0, r1) of the
// segment's tile, D floats each.  The values are read from the cache again.
template <int D>
__device__ __forceinline__ void add_odd_values(const AttnParams& p, const AttnSeg& g, int r0, int r1, float* dst) {
  const int32_t* table = attn_table(p, g.set);
  const int all = attn_visible(p, g, g.row0 / p.group), first = all > g.kv0 ? all : g.kv0;
  __syncwarp();
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const int vis = attn_visible(p, g, (g.row0 + r) / p.group), end = vis < g.kv1 ? vis : g.kv1;
#pragma unroll 1
    for (int d = threadIdx.x & 31; d < D; d += 32) {
#pragma unroll 1
      for (int tok = first; tok < end; ++tok) {
        const int page = __ldg(&table[tok >> p.page_shift]);
        if (page < 0 || page >= p.num_pages) continue;  // reported where it was loaded
        const uint32_t x = __ldg(p.v + page * p.page_stride + (tok & (p.page_size - 1)) * p.token_stride +
                                 g.kvh * p.head_stride + d);
        if (odd_bf16(x)) dst[r * D + d] += __uint_as_float(x << 16);
      }
    }
  }
  __syncwarp();
}

// Token rows of one tensor-map box: pages shorter than a unit give several.
__host__ __device__ __forceinline__ int attn_box(int page_size, int unit) { return page_size < unit ? page_size : unit; }

cudaError_t launch_attn_split(const AttnParams& p, const CUtensorMap (&maps)[4], cudaStream_t s);
cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_tile(const AttnParams& p, int cl, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s);
// One CTA per SM of the chip that the library is built for: the workspace goes by
// it, so it is not asked of the device as the layer's launches do.
constexpr int kAttnCtas = kNumSMs;

}  // namespace moe
