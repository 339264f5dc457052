// serve.cu — exported entry points of the operators around the layer
// (moe_serve.h): argument checks, workspace layout, tensor maps and launch
// sequences.  Nothing here allocates or synchronises.
#include <math.h>
#include <string.h>

#include "serve.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int check_cache(const moe_kv_cache* c) {
  if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return MOE_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->head_dim < 1) return MOE_ERR_INVALID_ARG;
  if (c->page_stride < 1 || c->token_stride < 1 || c->head_stride < 1) return MOE_ERR_INVALID_ARG;
  if (c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8) return MOE_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return MOE_ERR_UNSUPPORTED;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->kv_heads > 256) return MOE_ERR_UNSUPPORTED;
  // Tensor-map strides: below 2^40 bytes.
  const int64_t lim = (int64_t)1 << 39;
  if (c->page_stride >= lim || c->token_stride >= lim || c->head_stride >= lim) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_batch(const moe_kv_batch* b) {
  if (!b || b->batch < 1 || b->tokens < 1 || b->max_q < 1 || b->prefix_len < 0 || b->table_pages < 0) return MOE_ERR_INVALID_ARG;
  if (!b->kv_len || !aligned(b->kv_len, 4) || !b->table || !aligned(b->table, 4)) return MOE_ERR_INVALID_ARG;
  if (b->table_stride < b->table_pages || (b->q_start && !aligned(b->q_start, 4))) return MOE_ERR_INVALID_ARG;
  if (!b->q_start && b->tokens != b->batch) return MOE_ERR_INVALID_ARG;
  if (b->prefix_len > 0 && (!b->prefix_table || !aligned(b->prefix_table, 4))) return MOE_ERR_INVALID_ARG;
  if (b->prefix_len > MOE_SERVE_MAX_LEN || b->batch > MOE_SERVE_MAX_BATCH || b->tokens > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ------------------------------------------------------ attention: the plan --
// Most new tokens a sequence can have: max_q is the caller's bound and may be
// any number above that.
int most_new(const moe_kv_batch& b) {
  const int most = b.q_start ? b.tokens : 1;
  return b.max_q < most ? b.max_q : most;
}

// Row tiles per key head that the kernel may have: the sum over sets of
// ceil(rows / tile), bounded by what the host knows.
int64_t max_tiles(const moe_kv_batch& b, int group, const AttnSide& s) {
  const int64_t rows = (int64_t)b.tokens * group;
  int64_t t = 0;
  if (s.prefix) t += (rows + s.rows - 1) / s.rows;
  if (s.own) t += b.q_start ? rows / s.rows + b.batch : (int64_t)b.batch * ((group + s.rows - 1) / s.rows);
  return t;
}

// Which side of the split kernel takes which part: the warps take parts of at
// most 16 rows per key head (one tile), the Tensor Memory side the others.  A
// sequence has no more rows than the batch, so own parts on the Tensor Memory
// side have their prefix there too: attn_plan scans one side and takes the other
// for a prefix alone.
void plan_sides(const moe_kv_batch& b, int group, int head_dim, AttnSide (&side)[2]) {
  memset(side, 0, sizeof side);
  const bool own_tc = (int64_t)most_new(b) * group > kAttnWarpRows, prefix = b.prefix_len > 0;
  const bool prefix_tc = (int64_t)b.tokens * group > kAttnWarpRows;
  AttnSide &w = side[0], &t = side[1];
  w.own = !own_tc;
  w.prefix = prefix && !prefix_tc;
  w.rows = kAttnWarpRows;
  w.unit = attn_warp_unit(head_dim);
  w.workers = kAttnCtas * kAttnWarpWorkers;
  w.tile_cost = 1;
  t.own = own_tc;
  t.prefix = prefix && prefix_tc;
  t.rows = kAttnTcRows;
  t.unit = kAttnTcUnit;
  t.workers = kAttnCtas;
  t.tile_cost = 4;
  for (AttnSide& s : side) {
    while ((1 << s.rows_shift) < s.rows) ++s.rows_shift;
    while ((1 << s.unit_shift) < s.unit) ++s.unit_shift;
  }
}

// Whether the tile kernel takes the call, and on clusters of how many CTAs
// (0: no): as many CTAs a tile as keep all tiles on the chip at once.  A wave of
// it costs about 6 us and each unit that a warp takes in turn 1.2 us; the split
// kernel and its join cost 10 us and more before their first byte, or 20 us
// where prefix and own parts go to different sides.  Measured at 56 / 8 heads of
// 128, tile against split: 1 sequence of 200 tokens 6.7 / 11.2 us, of 16,000 (11
// units in turn) 23.3 / 50.8; 16 of 1,000 11.2 / 16.1, of 4,000 (21 units) 31.8
// / 34.9; 32 of 100 behind 1,000 (two waves, 6 units each) 23.0 / 25.6; 64 of
// 200 (four waves) 22.5 / 15.1.  The call does not know lengths, so the rule
// goes by the most tokens a sequence may have, its table's width: with a table
// for 40,000 tokens the sequence of 200 takes the 11.2 us.
int tile_cluster(const moe_kv_batch& b, const moe_kv_cache& c, int group) {
  const int64_t row_tiles = ((int64_t)most_new(b) * group + kAttnWarpRows - 1) / kAttnWarpRows;
  const int64_t tiles = b.batch * c.kv_heads * row_tiles;
  const int unit = attn_warp_unit(c.head_dim);
  const int64_t units = ((int64_t)b.prefix_len + unit - 1) / unit + ((int64_t)b.table_pages * c.page_size + unit - 1) / unit;
  int cl = 1;
  while (cl < 8 && tiles * cl * 2 <= kNumSMs && (int64_t)cl * kAttnWarpWorkers < units) cl *= 2;
  const int64_t each = (units + cl * kAttnWarpWorkers - 1) / (cl * kAttnWarpWorkers);
  if (tiles * cl <= kNumSMs) return each <= 16 ? cl : 0;
  const bool two_sides = b.prefix_len > 0 && (int64_t)b.tokens * group > kAttnWarpRows &&
                         (int64_t)most_new(b) * group <= kAttnWarpRows;
  return tiles <= 2 * kNumSMs && two_sides && each <= 6 ? cl : 0;
}

size_t side_layout(const moe_kv_batch& b, int group, int kv_heads, int head_dim, AttnSide (&side)[2], void* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return (char*)base + o;
  };
  for (int i = 0; i < 2; ++i) {
    AttnSide& s = side[i];
    if (!s.own && !s.prefix) continue;
    const size_t slots = (size_t)s.workers + (size_t)max_tiles(b, group, s) * kv_heads;
    s.unit_start = (long long*)take((size_t)(b.batch + 2) * 8);
    s.tile_start = (int32_t*)take((size_t)(b.batch + 1) * 4);
    s.slots = (float*)take(slots * s.rows * (head_dim + 2) * 4);
  }
  return off;
}

// [page][head][token][64-element half]: boxes of `rows` tokens x 64 values,
// 128-byte swizzle.
int cache_map(CUtensorMap* m, const moe_kv_cache* c, void* base, int rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return MOE_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)c->kv_heads,
                              (cuuint64_t)c->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c->token_stride * 2, (cuuint64_t)c->head_stride * 2,
                                 (cuuint64_t)c->page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  // L2 fetches what one token of a head holds: with more, short heads bring in
  // their neighbours, which other CTAs read at other times (24 sequences of up
  // to 32,771 tokens, 4 key heads of 64: 79 us, 89 with 256 bytes; no difference
  // for heads of 128).
  const CUtensorMapL2promotion fetch =
      c->head_dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, fetch,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int check_heads(const moe_kv_cache* c, int q_heads) {
  if (q_heads < 1 || q_heads % c->kv_heads) return MOE_ERR_INVALID_ARG;
  if (q_heads > 1024) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether the rows of an output lie apart.
bool rows_apart(const moe_kv_batch* b, int64_t stride, int64_t width) {
  return b->tokens == 1 || stride >= width || stride <= -width;
}

}  // namespace

extern "C" {

int moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, int x_dtype, const void* q, const void* k,
                  const void* v, int q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out,
                  int64_t q_out_stride, const float* rope, int rope_rows, int rot_dim, int interleaved,
                  int32_t* status, void* stream) {
  int st;
  if ((st = check_cache(cache)) != MOE_OK || (st = check_batch(batch)) != MOE_OK) return st;
  if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  const int vec = x_dtype == MOE_DT_F32 ? 4 : 8;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || k_stride % vec || v_stride % vec) return MOE_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return MOE_ERR_INVALID_ARG;
  if (q) {
    if ((st = check_heads(cache, q_heads)) != MOE_OK) return st;
    if (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % vec || q_out_stride % 8) return MOE_ERR_INVALID_ARG;
    if (!rows_apart(batch, q_out_stride, (int64_t)q_heads * cache->head_dim)) return MOE_ERR_INVALID_ARG;
    // In place: every row over itself.
    if (q_out == q && (x_dtype != MOE_DT_BF16 || (q_out_stride != q_stride && batch->tokens > 1))) return MOE_ERR_INVALID_ARG;
  }
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 || (interleaved != 0 && interleaved != 1)) return MOE_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!rope || !aligned(rope, 16) || rope_rows < 1)) return MOE_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MOE_ERR_INVALID_ARG;
  AppendParams p;
  p.c = *cache;
  p.b = *batch;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_heads = q_heads;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = (uint16_t*)q_out;
  p.q_out_stride = q_out_stride;
  p.rope = rope;
  p.rope_rows = rope_rows;
  p.rot = rot_dim;
  p.status = status;
  return cuda_status(launch_kv_append(p, x_dtype, interleaved != 0, (cudaStream_t)stream));
}

size_t moe_attention_workspace_bytes(const moe_kv_cache* cache, const moe_kv_batch* batch, int q_heads) {
  if (check_cache(cache) != MOE_OK || check_batch(batch) != MOE_OK || check_heads(cache, q_heads) != MOE_OK) return 0;
  AttnSide side[2];
  const int group = q_heads / cache->kv_heads;
  plan_sides(*batch, group, cache->head_dim, side);
  return side_layout(*batch, group, cache->kv_heads, cache->head_dim, side, nullptr);
}

int moe_prefix_attention(const moe_kv_cache* cache, const moe_kv_batch* batch, const void* q, int q_heads,
                         int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse, void* ws,
                         size_t ws_bytes, int32_t* status, void* stream) {
  int st;
  if ((st = check_cache(cache)) != MOE_OK || (st = check_batch(batch)) != MOE_OK) return st;
  if ((st = check_heads(cache, q_heads)) != MOE_OK) return st;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8) return MOE_ERR_INVALID_ARG;
  if (!rows_apart(batch, out_stride, (int64_t)q_heads * cache->head_dim)) return MOE_ERR_INVALID_ARG;
  if ((lse && !aligned(lse, 4)) || (status && !aligned(status, 4))) return MOE_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !isfinite(scale_log2)) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  AttnParams p;
  memset(&p, 0, sizeof p);
  p.group = q_heads / cache->kv_heads;
  plan_sides(*batch, p.group, cache->head_dim, p.side);
  if (ws_bytes < side_layout(*batch, p.group, cache->kv_heads, cache->head_dim, p.side, ws)) return MOE_ERR_WORKSPACE;
  p.q = (const uint16_t*)q;
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.q_heads = q_heads;
  p.scale_log2 = scale_log2;
  p.kv_heads = cache->kv_heads;
  p.head_dim = cache->head_dim;
  p.page_size = cache->page_size;
  for (p.page_shift = 0; (1 << p.page_shift) < cache->page_size; ++p.page_shift) {
  }
  p.num_pages = cache->num_pages;
  p.v = (const uint16_t*)cache->v;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.b = *batch;
  p.status = status;
  p.wait_limit = wait_limit();
  cudaStream_t s = (cudaStream_t)stream;
  if (const int cl = tile_cluster(*batch, *cache, p.group)) {
    CUtensorMap km, vm;
    const int box = attn_box(cache->page_size, attn_warp_unit(cache->head_dim));
    if ((st = cache_map(&km, cache, cache->k, box)) != MOE_OK || (st = cache_map(&vm, cache, cache->v, box)) != MOE_OK)
      return st;
    p.tile_rows = (int)(((int64_t)most_new(*batch) * p.group + kAttnWarpRows - 1) / kAttnWarpRows);
    return cuda_status(launch_attn_tile(p, cl, km, vm, s));
  }
  CUtensorMap maps[4];  // K and V in the boxes of either side
  for (int i = 0; i < 2; ++i) {
    const int box = attn_box(cache->page_size, p.side[i].unit);
    if ((st = cache_map(&maps[2 * i], cache, cache->k, box)) != MOE_OK ||
        (st = cache_map(&maps[2 * i + 1], cache, cache->v, box)) != MOE_OK)
      return st;
  }
  if ((st = cuda_status(launch_attn_split(p, maps, s))) != MOE_OK) return st;
  return cuda_status(launch_attn_join(p, s));
}

int moe_sample(int rows, int vocab, const void* logits, int dtype, int64_t stride, const float* u,
               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
               int32_t* token, float* logprob, int32_t* kept, float* probs, void* stream) {
  if (rows < 1 || vocab < 1 || !logits || !u || !token || stride < vocab) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, dtype == MOE_DT_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
  const void* words[] = {u, temperature, top_k, top_p, min_p, token, logprob, kept, probs};
  for (const void* w : words)
    if (!aligned(w, 4)) return MOE_ERR_INVALID_ARG;
  if (vocab > MOE_SAMPLE_MAX_VOCAB || rows > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  SampleParams p;
  p.rows = rows;
  p.vocab = vocab;
  p.logits = logits;
  p.stride = stride;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.token = token;
  p.logprob = logprob;
  p.kept = kept;
  p.probs = probs;
  p.chunk = 0;
  return cuda_status(launch_sample(p, dtype, (cudaStream_t)stream));
}

}  // extern "C"
