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
// one per CTA; a CTA's piece of one tile is a segment.  Its partial sums go to
// slot CTA + tile, which is unique because every step to the next segment
// raises the CTA or the tile by one.
struct AttnSide {
  int own, prefix;       // which sets this kernel takes
  int rows, unit;        // query rows of a tile, tokens of a unit
  int ctas;              // CTAs launched
  int min_units;         // least units of a CTA's range
  float* slots;          // [ctas + tiles][rows * (head_dim + 2)]
  long long* unit_start; // [batch + 2] first unit of each set, then the total; [batch + 2]: units per CTA
  int32_t* tile_start;   // [batch + 2] first tile of each set
};

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  int q_heads, group;  // query heads, query heads per key head
  float scale_log2;    // scale * log2(e)
  int kv_heads, head_dim, page_size, page_shift, num_pages;
  moe_kv_batch b;
  AttnSide side[2];    // 0: warp kernel, 1: Tensor Memory kernel
  int32_t* status;
  long long wait_limit;
};

// One set as an attention kernel sees it.
struct AttnSet {
  int rows;      // query rows per key head
  int tok0;      // first query token
  int len;       // tokens of the set
  int first_vis; // tokens the first query token sees (each later one sees one more); len for the prefix
  int tiles;     // row tiles per key head
  int units;     // units per row tile
  const int32_t* table;
};

__device__ __forceinline__ AttnSet attn_set(const AttnParams& p, const AttnSide& sd, int s) {
  AttnSet a;
  a.rows = a.tok0 = a.len = a.first_vis = a.tiles = a.units = 0;
  a.table = nullptr;
  int ql;
  if (s == p.b.batch) {
    if (!sd.prefix) return a;
    ql = p.b.tokens;
    a.len = a.first_vis = p.b.prefix_len;
    a.table = p.b.prefix_table;
  } else {
    if (!sd.own) return a;
    int q0 = s, q1 = s + 1;
    if (p.b.q_start) {
      q0 = __ldg(&p.b.q_start[s]);
      q1 = __ldg(&p.b.q_start[s + 1]);
    }
    const int len = __ldg(&p.b.kv_len[s]);
    if (q0 < 0 || q1 < q0 || q1 > p.b.tokens || q1 - q0 > p.b.max_q || len < 0 ||
        len > (long long)p.b.table_pages * p.page_size) {
      set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
      return a;
    }
    ql = q1 - q0;
    a.tok0 = q0;
    a.len = len;
    a.first_vis = len - ql + 1;
    a.table = p.b.table + (int64_t)s * p.b.table_stride;
  }
  if (ql == 0 || a.len == 0) return a;
  a.rows = ql * p.group;
  a.tiles = (a.rows + sd.rows - 1) / sd.rows;
  a.units = (a.len + sd.unit - 1) / sd.unit;
  return a;
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

// A CTA's walk over its range of units.
struct AttnWalk {
  int set;
  AttnSet a;
  long long unit0;  // first unit of the set
  int tile0;        // first tile of the set
  long long u, u1;  // next unit, end of the range
};

struct AttnPlanShared {
  long long part_u[32];
  int part_t[32];
  long long total;
  int set, tile0;
  long long unit0;
};

// All threads of the CTA: add up the sets' units, cut them into gridDim.x
// ranges and find where this CTA's begins.  CTA 0 writes the plan for the
// joining kernel.  False (CTA-uniform): nothing to do.
__device__ __forceinline__ bool attn_plan(const AttnParams& p, const AttnSide& sd, AttnPlanShared& sh, AttnWalk& w) {
  const int nsets = p.b.batch + 1, nt = blockDim.x, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5, nwarps = nt >> 5;
  const int per_thread = (nsets + nt - 1) / nt;
  const int s0 = tid * per_thread < nsets ? tid * per_thread : nsets;
  const int s1 = s0 + per_thread < nsets ? s0 + per_thread : nsets;
  long long u = 0;
  int t = 0;
  for (int s = s0; s < s1; ++s) {
    const AttnSet a = attn_set(p, sd, s);
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
  __syncthreads();
  long long total = 0, bu = 0;
  int bt = 0;
  for (int i = 0; i < nwarps; ++i) {
    if (i == warp) {
      bu = total;
    }
    total += sh.part_u[i];
  }
  for (int i = 0; i < warp; ++i) bt += sh.part_t[i];
  eu += bu - u;  // exclusive
  et += bt - t;
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < sd.min_units) per = sd.min_units;
  const long long u0 = (long long)blockIdx.x * per;
  long long su = eu;
  int stl = et;
  const bool mine = u0 >= eu && u0 < eu + u;
  if (mine || blockIdx.x == 0) {
    for (int s = s0; s < s1; ++s) {
      const AttnSet a = attn_set(p, sd, s);
      const int tiles = a.tiles * p.kv_heads;
      const long long n = (long long)tiles * a.units;
      if (u0 >= su && u0 < su + n) {
        sh.set = s;
        sh.unit0 = su;
        sh.tile0 = stl;
      }
      if (blockIdx.x == 0) {
        sd.unit_start[s] = su;
        sd.tile_start[s] = stl;
      }
      su += n;
      stl += tiles;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    sd.unit_start[nsets] = total;
    sd.unit_start[nsets + 1] = per;
  }
  __syncthreads();
  if (u0 >= total) return false;
  w.set = sh.set;
  w.unit0 = sh.unit0;
  w.tile0 = sh.tile0;
  w.a = attn_set(p, sd, w.set);
  w.u = u0;
  w.u1 = u0 + per < total ? u0 + per : total;
  return true;
}

// The next segment of the walk.
struct AttnSeg {
  int slot, kvh;
  int row0;      // first row of the tile in its set
  int rows;      // rows of the tile
  int kv0, kv1;  // token range [kv0, kv1) of the set, cut to what the tile's last row sees (may be empty)
};

__device__ __forceinline__ bool attn_next(const AttnParams& p, const AttnSide& sd, AttnWalk& w, AttnSeg& g) {
  if (w.u >= w.u1) return false;
  long long set_units = (long long)w.a.tiles * p.kv_heads * w.a.units;
  while (w.u >= w.unit0 + set_units) {
    w.unit0 += set_units;
    w.tile0 += w.a.tiles * p.kv_heads;
    w.a = attn_set(p, sd, ++w.set);
    set_units = (long long)w.a.tiles * p.kv_heads * w.a.units;
  }
  const long long lu = w.u - w.unit0;
  const int tile = (int)(lu / w.a.units);
  const int k0 = (int)(lu - (long long)tile * w.a.units);
  long long n = w.a.units - k0;
  if (n > w.u1 - w.u) n = w.u1 - w.u;
  w.u += n;
  g.slot = (int)blockIdx.x + w.tile0 + tile;
  g.kvh = tile / w.a.tiles;
  g.row0 = (tile % w.a.tiles) * sd.rows;
  g.rows = w.a.rows - g.row0 < sd.rows ? w.a.rows - g.row0 : sd.rows;
  const int vis = attn_visible(p, w.a, w.set, (g.row0 + g.rows - 1) / p.group);
  g.kv0 = k0 * sd.unit;
  const long long e = (long long)(k0 + n) * sd.unit;
  g.kv1 = e < vis ? (int)e : vis;
  if (g.kv1 < g.kv0) g.kv1 = g.kv0;
  return true;
}

// Token rows of one tensor-map box: pages shorter than a unit give several.
__host__ __device__ __forceinline__ int attn_box(int page_size, int unit) { return page_size < unit ? page_size : unit; }

cudaError_t launch_attn_tc(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s);
cudaError_t launch_attn_warp(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s);
cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s);
// CTAs of the warp kernel (two per SM).
constexpr int kAttnWarpCtas = 2 * kNumSMs;
constexpr int kAttnWarpUnit = 64;
// The Tensor Memory kernel: one CTA per SM, tiles of 256 rows, units of 128 tokens.
constexpr int kAttnTcCtas = kNumSMs;
constexpr int kAttnTcRows = 256;
constexpr int kAttnTcUnit = 128;

}  // namespace moe
