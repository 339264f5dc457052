// attention.cu — attention over the paged cache: the warp kernel (few query
// rows per key head) and the kernel that joins partial sums.
//
// For a query row q and its tokens j, with t_j = scale log2(e) q.k_j:
//   m = max t_j,  l = sum 2^(t_j - m),  o = sum 2^(t_j - m) v_j
// over any part of the tokens; parts join by
//   M = max m_i,  out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,
//   lse = (M + log2 l) ln 2.
// A part without visible tokens has m = -inf, l = 0, o = 0 and drops out.
#include "serve.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------- warp kernel --
// For at most 64 query rows per (set, key head): decode, speculative steps.
// Bound by HBM: 2 * 2 * head_dim bytes per token and key head against 4 *
// head_dim * rows operations, so warp MMAs (m16n8k16) keep up, and 16 rows
// waste less than a Tensor Memory tile of 128.  A producer warp copies 64
// tokens of K and V per ring stage with tensor-map boxes (one per page);
// four consumer warps share a stage: with MT row tiles of 16, warp w takes row
// tile w % MT and 16 * MT of its tokens.  The warps that split tokens join
// through shared memory at the end of a segment.
constexpr int kUnit = kAttnWarpUnit;
constexpr int kConsumers = 4;
constexpr int kWarpThreads = (kConsumers + 1) * 32;

template <int D>
struct WarpCfg {
  static constexpr int kHalf = kUnit * 128;            // bytes of 64 tokens x 64 dims
  static constexpr int kMat = kHalf * (D / 64);        // K or V of a stage
  static constexpr int kStage = 2 * kMat;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRed = 2 * 36 * 32 * 4;         // two writers' 32 sums + m, l per thread
  static constexpr int kSmem = kStages * kStage + kRed + 256;
};

struct WarpShared {
  uint64_t full[8], empty[8];
  AttnPlanShared plan;
  int abort_flag;
};

__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, int* abort_flag, int32_t* status,
                                          long long limit) {
  const bool diag = limit < kWaitCycles;
  if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (diag ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)abort_flag) return false;
    if (clock64() - t0 > limit) {
      set_status_word(status, MOE_ERR_TIMEOUT);
      *(volatile int*)abort_flag = 1;
      return false;
    }
  }
}

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

// Keep the 16-bit halves of v whose token (t, t + 1) is below n.
__device__ __forceinline__ uint32_t keep_tokens(uint32_t v, int t, int n) {
  return t + 1 < n ? v : (t < n ? v & 0xFFFFu : 0u);
}

template <int D, int MT>
__global__ void __launch_bounds__(kWarpThreads, 2)
    k_attn_warp(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = WarpCfg<D>;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ WarpShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnSide& sd = p.side[0];
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kConsumers);
    }
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  // After the Tensor Memory kernel (side 1), which starts it only when all
  // earlier work is complete, this kernel overlaps that one's tail: they take
  // different parts.  It then waits for it at its end, so that the joining
  // kernel finds both complete.
  const bool overlap = p.side[1].own || p.side[1].prefix;
  if (!overlap) pdl_wait();
  pdl_trigger();
  AttnWalk w;
  if (!attn_plan(p, sd, sh.plan, w)) {  // its barriers also publish the mbarriers
    if (overlap) pdl_wait();
    return;
  }
  AttnSeg g;
  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer --
    const int box = attn_box(p.page_size, kUnit);
    int st = 0, use = 0;
    bool ok = true;
    while (ok && attn_next(p, sd, w, g)) {
      for (int kv = g.kv0; kv < g.kv1; kv += kUnit) {
        bool got = true;
        if (use > 0 && lane == 0) got = attn_wait(&sh.empty[st], (use - 1) & 1, &sh.abort_flag, p.status, p.wait_limit);
        if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
          ok = false;
          break;
        }
        const int left = g.kv1 - kv < kUnit ? g.kv1 - kv : kUnit;
        const int nb = (left + box - 1) / box;
        uint8_t* base = dyn + st * C::kStage;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], (uint32_t)(nb * box * D * 4));
        __syncwarp();
        if (lane < nb) {
          const int tok = kv + lane * box;
          int page = __ldg(&w.a.table[tok >> p.page_shift]);
          if (page < 0 || page >= p.num_pages) {
            set_status_word(p.status, MOE_ERR_DEVICE_CHECK);
            page = p.num_pages;  // past the map: the box is filled with zeros
          }
          const int y = tok & (p.page_size - 1);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            tma_load_4d(base + h * C::kHalf + lane * box * 128, &kmap, h * 64, y, g.kvh, page, &sh.full[st]);
            tma_load_4d(base + C::kMat + h * C::kHalf + lane * box * 128, &vmap, h * 64, y, g.kvh, page, &sh.full[st]);
          }
        }
        __syncwarp();
        if (++st == C::kStages) st = 0, ++use;
      }
    }
    // No copy may be in flight when the CTA exits: wait for the last use of
    // each stage (stage s was filled `use` times, once more if s < st).
    if (lane == 0)
      for (int s = 0; s < C::kStages; ++s) {
        const int n = use + (s < st ? 1 : 0);
        if (n > 0 && !mbar_wait(&sh.full[s], (n - 1) & 1)) set_status_word(p.status, MOE_ERR_TIMEOUT);
      }
    if (overlap) pdl_wait();
    return;
  }
  // ------------------------------------------------------------- consumers --
  constexpr int NG = kConsumers / MT;  // token groups
  constexpr int TG = 16 * MT;          // tokens of a group
  constexpr int NT = D / 8;
  const int wr = warp % MT, wg = warp / MT;
  float* red = reinterpret_cast<float*>(dyn + C::kStages * C::kStage);
  int st = 0, use = 0;
  bool alive = true;
  while (attn_next(p, sd, w, g)) {
    // This thread's two rows and their queries, as MMA fragments.
    const int r0 = wr * 16 + (lane >> 2);
    uint32_t qf[D / 16][4];
    int vis[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 8 * h;
      const bool in = r < g.rows;
      const int i = (g.row0 + (in ? r : 0)) / p.group;
      vis[h] = in ? attn_visible(p, w.a, w.set, i) : 0;
      const uint16_t* src = p.q + (int64_t)(w.a.tok0 + i) * p.q_stride +
                            (int64_t)(g.kvh * p.group + (g.row0 + (in ? r : 0)) - i * p.group) * D + 2 * (lane & 3);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][h] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk)) : 0u;
        qf[kk][h + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8)) : 0u;
      }
    }
    // Units that end above the first row's tokens need the mask.
    const int vis_min = attn_visible(p, w.a, w.set, g.row0 / p.group);
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    for (int kv = g.kv0; kv < g.kv1; kv += kUnit) {
      if (alive) alive = attn_wait(&sh.full[st], use & 1, &sh.abort_flag, p.status, p.wait_limit);
      alive = __all_sync(0xFFFFFFFFu, alive);
      if (!alive) break;
      const uint32_t kb = smem_u32(dyn + st * C::kStage), vb = kb + C::kMat;
      const int t0 = wg * TG;  // the warp's first token of the stage
      const bool edge = kv + kUnit > vis_min;
      if (kv + t0 < g.kv1) {
        // Scores of 16 rows x TG tokens.
        float sc[TG / 8][4];
#pragma unroll
        for (int i = 0; i < TG / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
          for (int j = 0; j < TG / 16; ++j) {
            const int tok = t0 + 16 * j + (lane & 7) + ((lane >> 4) << 3);
            const int c = (kk & 3) * 2 + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm4(kb + (kk >> 2) * C::kHalf + tok * 128 + ((c ^ (tok & 7)) << 4), b);
            mma_bf16(sc[2 * j], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b[0], b[1]);
            mma_bf16(sc[2 * j + 1], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b[2], b[3]);
          }
        }
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int i = 0; i < TG / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float t = sc[i][e] * p.scale_log2;
            if (edge && kv + t0 + 8 * i + 2 * (lane & 3) + (e & 1) >= vis[e >> 1]) t = -CUDART_INF_F;
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
        for (int j = 0; j < TG / 16; ++j) {
          uint32_t a[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* s4 = sc[2 * j + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s4[e] = ex2(s4[e] - ms[e >> 1]);
              l[e >> 1] += s4[e];
            }
            // bf16 weights: half an ulp of 2^-9 each, averaged over the sum,
            // below the rounding of the bf16 output.
            a[2 * i] = pack_bf16(s4[0], s4[1]);
            a[2 * i + 1] = pack_bf16(s4[2], s4[3]);
          }
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            const int tok = t0 + 16 * j + (lane & 15);
            const int c = (n & 7) + (lane >> 4);
            uint32_t b[4];
            ldsm4t(vb + (n >> 3) * C::kHalf + tok * 128 + ((c ^ (tok & 7)) << 4), b);
            if (edge) {
              // Rows of V past the length may hold anything: 0 * NaN is NaN.
              const int tk = kv + t0 + 16 * j + 2 * (lane & 3);
              b[0] = keep_tokens(b[0], tk, g.kv1);
              b[1] = keep_tokens(b[1], tk + 8, g.kv1);
              b[2] = keep_tokens(b[2], tk, g.kv1);
              b[3] = keep_tokens(b[3], tk + 8, g.kv1);
            }
            mma_bf16(o[n], a[0], a[1], a[2], a[3], b[0], b[1]);
            mma_bf16(o[n + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (++st == C::kStages) st = 0, ++use;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
    }
    // Join the token groups pairwise: (g, g + off) in fixed order.
#pragma unroll
    for (int off = NG / 2; off >= 1; off /= 2) {
      const bool writer = wg >= off && wg < 2 * off, reader = wg < off;
      float* buf = red + ((wg % off) * MT + wr) * (36 * 32) + lane;
      float fa[2] = {1.f, 1.f}, fb[2] = {0.f, 0.f};
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        if (writer) {
#pragma unroll
          for (int i = 0; i < 32; ++i) buf[i * 32] = o[half * 8 + i / 4][i & 3];
#pragma unroll
          for (int h = 0; h < 2; ++h) buf[(32 + h) * 32] = m[h], buf[(34 + h) * 32] = l[h];
        }
        named_sync(1, kConsumers * 32);
        if (reader) {
          if (half == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float mb = buf[(32 + h) * 32], lb = buf[(34 + h) * 32];
              const float mm = fmaxf(m[h], mb);
              fa[h] = m[h] == mm ? 1.f : ex2(m[h] - mm);
              fb[h] = mb == mm ? 1.f : ex2(mb - mm);
              m[h] = mm;
              l[h] = l[h] * fa[h] + lb * fb[h];
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float& v = o[half * 8 + i / 4][i & 3];
            v = v * fa[(i >> 1) & 1] + buf[i * 32] * fb[(i >> 1) & 1];
          }
        }
        named_sync(1, kConsumers * 32);
      }
    }
    if (wg == 0) {
      float* slot = sd.slots + (int64_t)g.slot * sd.rows * (D + 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 8 * h;
        if (r >= g.rows) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2*>(slot + r * D + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
        if ((lane & 3) == 0) {
          slot[sd.rows * D + r] = m[h];
          slot[sd.rows * (D + 1) + r] = l[h];
        }
      }
    }
  }
  if (overlap) pdl_wait();
}

template <int D, int MT>
cudaError_t launch_warp(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  auto kern = k_attn_warp<D, MT>;
  cudaError_t err = ensure_smem_attr((const void*)kern, WarpCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(p.side[0].ctas), dim3(kWarpThreads), WarpCfg<D>::kSmem, s, p, km, vm);
}

// --------------------------------------------------------------- join kernel --
// One warp per (token, head): the row's segments are the CTAs whose ranges
// meet its tile's units, in order, first the prefix's and then the own part's.
constexpr int kJoinWarps = 4;

struct JoinRow {
  const float* slots;  // slot of the first segment
  int64_t slot_floats;
  int n, row, rows;
};

// The segments of a row of set s: units [u0, u0 + units) of ranges of `per`.
__device__ __forceinline__ JoinRow join_row(const AttnParams& p, const AttnSide& sd, int s, int i, int head) {
  JoinRow j;
  const AttnSet a = attn_set(p, sd, s);
  j.n = 0;
  j.rows = sd.rows;
  j.slot_floats = (int64_t)sd.rows * (p.head_dim + 2);
  j.slots = nullptr;
  j.row = 0;
  if (a.units == 0) return j;
  const long long per = sd.unit_start[p.b.batch + 2];
  const int kvh = head / p.group;
  const int r = i * p.group + head - kvh * p.group;
  const int tile = kvh * a.tiles + r / sd.rows;
  j.row = r % sd.rows;
  const long long u0 = sd.unit_start[s] + (long long)tile * a.units;
  const int c0 = (int)(u0 / per), c1 = (int)((u0 + a.units - 1) / per);
  j.n = c1 - c0 + 1;
  j.slots = sd.slots + (int64_t)(c0 + sd.tile_start[s] + tile) * j.slot_floats;
  return j;
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const AttnParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= (long long)p.b.tokens * p.q_heads) return;
  const int n = (int)(row / p.q_heads), head = (int)(row - (long long)n * p.q_heads);
  JoinRow part[2];
  part[0].n = part[1].n = 0;
  if (p.b.prefix_len > 0) part[0] = join_row(p, p.side[p.side[1].prefix ? 1 : 0], p.b.batch, n, head);
  {
    int b = n, i = 0;
    if (p.b.q_start) {
      b = find_sequence(p.b.q_start, p.b.batch, n);
      i = n - __ldg(&p.b.q_start[b]);
    }
    // attn_set refuses a sequence whose entries do not fit; then there is no part.
    if (i >= 0 && i < p.b.max_q) part[1] = join_row(p, p.side[p.side[1].own ? 1 : 0], b, i, head);
  }
  float mx = -CUDART_INF_F;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    for (int s = lane; s < part[k].n; s += 32)
      mx = fmaxf(mx, part[k].slots[s * part[k].slot_floats + (int64_t)part[k].rows * D + part[k].row]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  constexpr int E = D / 32;
  float acc[E] = {}, l = 0.f;
  {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* base = part[k].slots;
      for (int s0 = 0; s0 < part[k].n; s0 += 32) {
        // Lane s holds segment s0 + s's weight and sum.
        float f = 0.f, ls = 0.f;
        if (s0 + lane < part[k].n) {
          const float* b = base + (s0 + lane) * part[k].slot_floats + (int64_t)part[k].rows * D;
          const float ms = b[part[k].row];
          f = ms == -CUDART_INF_F ? 0.f : ex2(ms - mx);
          ls = b[part[k].rows + part[k].row] * f;  // a NaN sum stays one
        }
        const int cnt = part[k].n - s0 < 32 ? part[k].n - s0 : 32;
#pragma unroll 4
        for (int s = 0; s < cnt; ++s) {
          const float fs = __shfl_sync(0xFFFFFFFFu, f, s);
          l += __shfl_sync(0xFFFFFFFFu, ls, s);
          const float* src = base + (s0 + s) * part[k].slot_floats + (int64_t)part[k].row * D + lane * E;
          float v[E];
          if (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[0] = x.x, v[1] = x.y, v[E - 2] = x.z, v[E - 1] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[0] = x.x, v[1] = x.y;
          }
          if (fs > 0.f)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += fs * v[e];
        }
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint16_t* dst = p.out + (int64_t)n * p.out_stride + head * D + lane * E;
  if (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[E - 2] * inv, acc[E - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (mx + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_attn_warp(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  const int mt = p.side[0].rows / 16;
  if (p.head_dim == 128)
    return mt == 1 ? launch_warp<128, 1>(p, km, vm, s) : mt == 2 ? launch_warp<128, 2>(p, km, vm, s)
                                                                  : launch_warp<128, 4>(p, km, vm, s);
  return mt == 1 ? launch_warp<64, 1>(p, km, vm, s) : mt == 2 ? launch_warp<64, 2>(p, km, vm, s)
                                                               : launch_warp<64, 4>(p, km, vm, s);
}

cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s) {
  const long long rows = (long long)p.b.tokens * p.q_heads;
  const dim3 grid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
  return p.head_dim == 128 ? launch_pdl(k_attn_join<128>, grid, dim3(kJoinWarps * 32), 0, s, p)
                           : launch_pdl(k_attn_join<64>, grid, dim3(kJoinWarps * 32), 0, s, p);
}

}  // namespace moe
