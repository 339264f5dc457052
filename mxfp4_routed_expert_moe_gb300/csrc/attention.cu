// attention.cu — attention over the paged cache: the tile kernel (small
// problems, in one launch) and the kernel that joins the split kernel's sums.
//
// For a query row q and its tokens j, with t_j = scale log2(e) q.k_j:
//   m = max t_j,  l = sum 2^(t_j - m),  o = sum 2^(t_j - m) v_j
// over any part of the tokens; parts join by
//   M = max m_i,  out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,
//   lse = (M + log2 l) ln 2.
// A part without visible tokens has m = -inf, l = 0, o = 0 and drops out.
#include <cooperative_groups.h>

#include "attention_warp.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------- tile kernel --
// Small problems, where launches and latencies are the time: one launch, no
// plan, no joining kernel.  A cluster takes 16 rows of one (sequence, key head)
// over everything they see, the prefix and then the own part; its warps take
// the units in turn and join through (distributed) shared memory.
// A prefix is read once per sequence here, from L2.
struct TileShared {
  uint64_t full[kWorkers][2];
  float ml[kWorkers][2 * kAttnWarpRows];  // m, l of each warp's rows
};

template <int D>
__global__ void __launch_bounds__(kWorkers * 32, 1)
    k_attn_tile(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = WarpCfg<D>;
  constexpr int kUnit = C::kUnit;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ TileShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = dyn + warp * (C::kStages * C::kStage);
  uint64_t* full = sh.full[warp];
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_trigger();
  pdl_wait();
  const int tile = blockIdx.x / cl;
  const int rt = tile % p.tile_rows, kvh = tile / p.tile_rows % p.kv_heads, b = tile / p.tile_rows / p.kv_heads;
  const AttnRaw raw = attn_load(p, b);
  const int ql = raw.q1 - raw.q0, row0 = rt * kAttnWarpRows;
  if ((b == 0 && raw.q0 != 0) || (b == p.b.batch - 1 && raw.q1 != p.b.tokens)) set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
  if (!attn_valid(p, raw)) return;  // uniform over the cluster, like all of the above
  const int rows = ql * p.group - row0 < kAttnWarpRows ? ql * p.group - row0 : kAttnWarpRows;
  if (rows <= 0) return;
  // Own tokens that row r sees: len - ql + 1 + its token, within [0, len].
  auto visible = [&](int r) {
    const int v = raw.len - ql + 1 + (row0 + r) / p.group;
    return v < 0 ? 0 : (v > raw.len ? raw.len : v);
  };
  const int own_end = visible(rows - 1), own_all = visible(0);
  const int units_p = (p.b.prefix_len + kUnit - 1) / kUnit, units = units_p + (own_end + kUnit - 1) / kUnit;
  const int box = attn_box(p.page_size, kUnit);
  const int my_box = lane >> 2, my_half = (lane >> 1) & 1, my_v = lane & 1;
  const bool my_lane = my_half < D / 64 && my_box * box < kUnit;
  const int step = cl * kWorkers;
  auto unit_at = [&](int u, int& kv, int& end) {  // its first token and the end of its part
    const bool pre = u < units_p;
    kv = (pre ? u : u - units_p) * kUnit;
    end = pre ? p.b.prefix_len : own_end;
    return pre ? p.b.batch : b;
  };
  auto fetch = [&](int u) {  // this lane's page of unit u
    if (u >= units) return 0;
    int kv, end;
    const int set = unit_at(u, kv, end);
    const int tok = kv + my_box * box;
    return my_lane && tok < end ? __ldg(&attn_table(p, set)[tok >> p.page_shift]) : 0;
  };
  auto load = [&](int u, int st, int page) {
    int kv, end;
    unit_at(u, kv, end);
    const int left = end - kv < kUnit ? end - kv : kUnit;
    const int nb = (left + box - 1) / box;
    if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nb * box * D * 4));
    __syncwarp();
    if (my_lane && my_box < nb) {
      if (page < 0 || page >= p.num_pages) {
        set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
        page = p.num_pages;  // past the map: the box is filled with zeros
      }
      tma_load_4d(ring + st * C::kStage + my_v * C::kMat + my_half * C::kHalf + my_box * box * 128, my_v ? &vmap : &kmap,
                  my_half * 64, (kv + my_box * box) & (p.page_size - 1), kvh, page, &full[st]);
    }
    __syncwarp();
  };
  const int u0 = warp * cl + rank;  // few units spread over the CTAs first
  int page[C::kStages], n_in = 0;
#pragma unroll
  for (int s = 0; s < C::kStages; ++s) page[s] = fetch(u0 + s * step);
#pragma unroll
  for (int s = 0; s < C::kStages; ++s)
    if (u0 + s * step < units) {
      load(u0 + s * step, s, page[s]);
      ++n_in;
    }
  int next = fetch(u0 + C::kStages * step);
  WarpRows<D> acc;
  acc.load(p, raw.q0, kvh, row0, rows);
  int vis[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) vis[h] = (lane >> 2) + 8 * h < rows ? visible((lane >> 2) + 8 * h) : 0;
  int n = 0;
  bool alive = true, odd = false;
  for (int u = u0; u < units; u += step, ++n) {
    const int st = n % C::kStages;
    alive = __all_sync(0xFFFFFFFFu, mbar_wait_for(&full[st], (n / C::kStages) & 1, p.wait_limit));
    if (!alive) {
      set_status_word(p.status, MOE_ERR_TIMEOUT);
      break;
    }
    int kv, end;
    const bool pre = unit_at(u, kv, end) == p.b.batch;
    const int see[2] = {(pre ? end : vis[0]) - kv, (pre ? end : vis[1]) - kv};
    odd |= acc.unit(ring + st * C::kStage, p.scale_log2, (pre ? end : own_all) - kv, see, end - kv);
    __syncwarp();  // every lane has read the stage
    if (u + C::kStages * step < units) {
      load(u + C::kStages * step, st, next);
      ++n_in;
      next = fetch(u + (C::kStages + 1) * step);
    }
  }
  // Copies still in flight after a wait gave up must land before the ring is
  // used again or left.
  for (int i = n; i < n_in; ++i)
    if (!mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1)) set_status_word(p.status, MOE_ERR_TIMEOUT);
  acc.close();
  acc.store(reinterpret_cast<float*>(ring), sh.ml[warp], rows);
  if (odd) {
    AttnSeg own;
    own.set = b;
    own.len = own.kv1 = raw.len;
    own.first_vis = raw.len - ql + 1;
    own.kvh = kvh;
    own.row0 = row0;
    own.kv0 = 0;
    add_odd_values<D>(p, own, 0, rows, reinterpret_cast<float*>(ring));
  }
  cluster.sync();
  // CTA `rank` joins rows rank, rank + cl, ...: D / 4 threads a row, the warps
  // in order.
  constexpr int L = D / 4;
  static_assert(C::kStages * C::kStage >= kAttnWarpRows * D * 4, "a warp's ring holds its sums");
  for (int i = threadIdx.x; i < (rows - rank + cl - 1) / cl * L; i += kWorkers * 32) {
    const int r = rank + i / L * cl, col = i % L * 4;
    float mx = -CUDART_INF_F;
    for (int w = 0; w < step; ++w) mx = fmaxf(mx, cluster.map_shared_rank(&sh, w % cl)->ml[w / cl][r]);
    float acc4[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
    for (int w = 0; w < step; ++w) {
      const TileShared* o = cluster.map_shared_rank(&sh, w % cl);
      const float m = o->ml[w / cl][r];
      const float f = m == -CUDART_INF_F ? 0.f : ex2(m - mx);
      l += o->ml[w / cl][kAttnWarpRows + r] * f;  // a NaN sum stays one
      const float4 v = *reinterpret_cast<const float4*>(
          cluster.map_shared_rank(dyn, w % cl) + (w / cl) * (C::kStages * C::kStage) + (r * D + col) * 4);
      if (f > 0.f) {
        acc4[0] = fmaf(f, v.x, acc4[0]);
        acc4[1] = fmaf(f, v.y, acc4[1]);
        acc4[2] = fmaf(f, v.z, acc4[2]);
        acc4[3] = fmaf(f, v.w, acc4[3]);
      }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int rr = row0 + r, tok = rr / p.group, head = kvh * p.group + rr - tok * p.group;
    *reinterpret_cast<uint2*>(p.out + (int64_t)(raw.q0 + tok) * p.out_stride + head * D + col) =
        make_uint2(pack_bf16(acc4[0] * inv, acc4[1] * inv), pack_bf16(acc4[2] * inv, acc4[3] * inv));
    if (p.lse && col == 0)
      p.lse[(int64_t)(raw.q0 + tok) * p.q_heads + head] = l == 0.f ? -CUDART_INF_F : (mx + log2f(l)) * 0.69314718055994531f;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int D>
cudaError_t launch_tile(const AttnParams& p, int cl, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  cudaError_t err = ensure_smem_attr((const void*)k_attn_tile<D>, WarpCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.b.batch * p.kv_heads * p.tile_rows * cl));
  cfg.blockDim = dim3(kWorkers * 32);
  cfg.dynamicSmemBytes = WarpCfg<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_attn_tile<D>, p, km, vm);
}

// --------------------------------------------------------------- join kernel --
// A row's segments are the workers whose ranges meet its tile's units, in
// order, first the prefix's and then the own part's.  A CTA takes some heads
// of one token: two warps look up the token's sets, one thread per head and
// part finds the segments, then each warp joins four heads at a time.  Bound by
// instructions: about 100 per row and segment.
constexpr int kJoinWarps = 4;
constexpr int kJoinHeads = 64;  // heads of a CTA at a time

struct JoinPart {
  const float* slots;
  long long unit0, per;
  int units, tiles, tile0;  // of the set (units 0: no part)
  int i;                    // the token in its set
  int rows_shift;
};

// A head's segments in one part.
struct JoinRow {
  const float* first;  // slot of the first segment, at the row's sums
  const float* m;      // the same slot, at the row's maximum (its sum: `rows` further)
  int n;
};

__device__ __forceinline__ JoinRow join_row(const AttnParams& p, const JoinPart& t, int head, int64_t slot_floats) {
  JoinRow j;
  j.n = 0;
  j.first = j.m = nullptr;
  if (t.units == 0) return j;
  const int kvh = head / p.group;
  const int r = t.i * p.group + head - kvh * p.group;
  const int tile = kvh * t.tiles + (r >> t.rows_shift), row = r & ((1 << t.rows_shift) - 1);
  const long long u0 = t.unit0 + (long long)tile * t.units, u1 = u0 + t.units - 1;
  int c0, c1;
  if (u1 < 0x7FFFFFFFll) {
    c0 = (int)((uint32_t)u0 / (uint32_t)t.per);
    c1 = (int)((uint32_t)u1 / (uint32_t)t.per);
  } else {
    c0 = (int)(u0 / t.per);
    c1 = (int)(u1 / t.per);
  }
  j.n = c1 - c0 + 1;
  const float* slot = t.slots + (int64_t)(c0 + t.tile0 + tile) * slot_floats;
  j.first = slot + (int64_t)row * p.head_dim;
  j.m = slot + ((int64_t)p.head_dim << t.rows_shift) + row;
  return j;
}

// The joined row, divided and rounded once, and its logarithm of the sum.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, int n, int head, int lane, const float (&acc)[D / 32],
                                          float l, float mx) {
  constexpr int E = D / 32;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint16_t* dst = p.out + (int64_t)n * p.out_stride + head * D + lane * E;
  if (E == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[E - 2] * inv, acc[E - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (p.lse && lane == 0)
    p.lse[(int64_t)n * p.q_heads + head] = l == 0.f ? -CUDART_INF_F : (mx + log2f(l)) * 0.69314718055994531f;
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const AttnParams p) {
  __shared__ JoinPart sh_part[2];
  __shared__ JoinRow sh_row[2][kJoinHeads];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x;
  if (warp < 2) {  // 0: the prefix, 1: the own part
    JoinPart t;
    t.units = 0;
    int b = p.b.batch, i = n;
    bool any = p.b.prefix_len > 0;
    if (warp == 1) {
      b = n;
      i = 0;
      if (p.b.q_start) {
        b = find_sequence(p.b.q_start, p.b.batch, n);
        i = n - __ldg(&p.b.q_start[b]);
      }
      any = i >= 0 && i < p.b.max_q;  // attn_set refuses what else does not fit
    }
    const AttnRaw raw = attn_load(p, b);
    if (i < 0 || i >= raw.q1 - raw.q0) {  // of no sequence
      any = false;
      if (lane == 0) set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
    }
    const AttnSide& sd = p.side[warp ? (p.side[1].own ? 1 : 0) : (p.side[1].prefix ? 1 : 0)];
    if (any) {
      // The batch's own entries are as the split kernel saw them: it lets this
      // kernel start only after everything before it is complete.
      const AttnSet a = attn_set(p, sd, b, raw);
      t.units = a.units;
      t.tiles = a.tiles;
      t.i = i;
      t.slots = sd.slots;
      t.rows_shift = sd.rows_shift;
    }
    pdl_wait();
    if (t.units) {
      t.unit0 = sd.unit_start[b];
      t.per = sd.unit_start[p.b.batch + 1];
      t.tile0 = sd.tile_start[b];
      if (t.per == 0) t.units = 0;
    }
    if (lane == 0) sh_part[warp] = t;
  } else {
    pdl_wait();
  }
  __syncthreads();
  constexpr int E = D / 32;
  int64_t sf[2];
  int rows[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    rows[k] = 1 << sh_part[k].rows_shift;
    sf[k] = (int64_t)(D + 2) << sh_part[k].rows_shift;
  }
  // This CTA's heads, kJoinHeads at a time.
  const int per_cta = (p.q_heads + gridDim.y - 1) / gridDim.y;
  const int h_end = (int)(blockIdx.y + 1) * per_cta < p.q_heads ? (int)(blockIdx.y + 1) * per_cta : p.q_heads;
  for (int h0 = blockIdx.y * per_cta; h0 < h_end; h0 += kJoinHeads) {
    const int heads = h_end - h0 < kJoinHeads ? h_end - h0 : kJoinHeads;
    __syncthreads();
    static_assert(2 * kJoinHeads == kJoinWarps * 32, "a thread per head and part");
    {
      const int k = threadIdx.x / kJoinHeads, h = threadIdx.x % kJoinHeads;
      if (h < heads) sh_row[k][h] = join_row(p, sh_part[k], h0 + h, sf[k]);
    }
    __syncthreads();
    // A head a warp where there are no more heads than warps, or segments for
    // more than 8 lanes: eight of a row's loads in flight, one latency for most.
    // Else four heads at a time: lane 8 h + s looks after segment s of head h,
    // and the loads of the four overlap.
    const bool wide = (int)threadIdx.x < heads && sh_row[0][threadIdx.x].n + sh_row[1][threadIdx.x].n > 8;
    const bool many = __syncthreads_or(heads <= kJoinWarps || wide);
    for (int done = warp * 4; done < heads && !many; done += 4 * kJoinWarps) {
      const int hl = done + (lane >> 3), s = lane & 7;
      JoinRow a, b;
      a.n = b.n = 0;
      int rw = 0;
      const float *src = nullptr, *ms = nullptr;
      if (hl < heads) {
        a = sh_row[0][hl];
        b = sh_row[1][hl];
        if (s < a.n) {
          src = a.first + s * sf[0];
          ms = a.m + s * sf[0];
          rw = rows[0];
        } else if (s < a.n + b.n) {
          src = b.first + (s - a.n) * sf[1];
          ms = b.m + (s - a.n) * sf[1];
          rw = rows[1];
        }
      }
      float m = -CUDART_INF_F, l = 0.f;
      if (ms) {
        m = *ms;
        l = ms[rw];
      }
      float mx = m;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      const float f = m == -CUDART_INF_F ? 0.f : ex2(m - mx);
      l *= f;  // a NaN sum stays one
      // In segment order: the same order whichever way a row is joined.
      float lt = 0.f;
      float acc[4][E] = {};
      const int most = __reduce_max_sync(0xFFFFFFFFu, a.n + b.n);
#pragma unroll 2
      for (int k = 0; k < most; ++k) {
        lt += __shfl_sync(0xFFFFFFFFu, l, (lane & 24) + k);
        float v[4][E], fs[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          fs[h] = __shfl_sync(0xFFFFFFFFu, f, 8 * h + k);
          const float* row = (const float*)__shfl_sync(0xFFFFFFFFu, (unsigned long long)src, 8 * h + k);
#pragma unroll
          for (int e = 0; e < E; ++e) v[h][e] = 0.f;
          if (fs[h] > 0.f) {  // a segment without weight may hold an unwritten sum
            if (E == 4) {
              const float4 x = *reinterpret_cast<const float4*>(row + lane * E);
              v[h][0] = x.x, v[h][1] = x.y, v[h][E - 2] = x.z, v[h][E - 1] = x.w;
            } else {
              const float2 x = *reinterpret_cast<const float2*>(row + lane * E);
              v[h][0] = x.x, v[h][1] = x.y;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[h][e] = fmaf(fs[h], v[h][e], acc[h][e]);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (done + h >= heads) break;
        store_row<D>(p, n, h0 + done + h, lane, acc[h], __shfl_sync(0xFFFFFFFFu, lt, 8 * h), __shfl_sync(0xFFFFFFFFu, mx, 8 * h));
      }
    }
    // Else a head at a time.
    for (int hl = warp; hl < heads && many; hl += kJoinWarps) {
      const int head = h0 + hl;
      JoinRow part[2];
      part[0] = sh_row[0][hl];
      part[1] = sh_row[1][hl];
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        for (int s = lane; s < part[k].n; s += 32) mx = fmaxf(mx, part[k].m[s * sf[k]]);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      float acc[E] = {}, l = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        for (int s0 = 0; s0 < part[k].n; s0 += 32) {
          // Lane s holds segment s0 + s's weight and sum.
          float f = 0.f, ls = 0.f;
          if (s0 + lane < part[k].n) {
            const float* b = part[k].m + (s0 + lane) * sf[k];
            const float ms = *b;
            f = ms == -CUDART_INF_F ? 0.f : ex2(ms - mx);
            ls = b[rows[k]] * f;  // a NaN sum stays one
          }
          const int cnt = part[k].n - s0 < 32 ? part[k].n - s0 : 32;
#pragma unroll 8
          for (int s = 0; s < cnt; ++s) {
            const float fs = __shfl_sync(0xFFFFFFFFu, f, s);
            l += __shfl_sync(0xFFFFFFFFu, ls, s);
            const float* src = part[k].first + (s0 + s) * sf[k] + lane * E;
            float v[E];
            if (E == 4) {
              const float4 x = *reinterpret_cast<const float4*>(src);
              v[0] = x.x, v[1] = x.y, v[E - 2] = x.z, v[E - 1] = x.w;
            } else {
              const float2 x = *reinterpret_cast<const float2*>(src);
              v[0] = x.x, v[1] = x.y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fs > 0.f ? fmaf(fs, v[e], acc[e]) : acc[e];
          }
        }
      }
      store_row<D>(p, n, head, lane, acc, l, mx);
    }
  }
}

}  // namespace

cudaError_t launch_attn_tile(const AttnParams& p, int cl, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  return p.head_dim == 128 ? launch_tile<128>(p, cl, km, vm, s) : launch_tile<64>(p, cl, km, vm, s);
}

cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s) {
  // All heads of a token in one CTA for long batches, down to a head a warp
  // while the CTAs are few.
  const int most = (p.q_heads + kJoinWarps - 1) / kJoinWarps;
  int ny = (8 * kNumSMs + p.b.tokens - 1) / p.b.tokens;
  ny = ny < 1 ? 1 : (ny > most ? most : ny);
  const dim3 grid((unsigned)p.b.tokens, (unsigned)ny);
  return p.head_dim == 128 ? launch_pdl(k_attn_join<128>, grid, dim3(kJoinWarps * 32), 0, s, p)
                           : launch_pdl(k_attn_join<64>, grid, dim3(kJoinWarps * 32), 0, s, p);
}

}  // namespace moe
