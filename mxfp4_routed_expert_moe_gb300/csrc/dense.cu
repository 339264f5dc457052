// dense.cu — exported entry points of the dense half of a serving step
// (moe_dense.h): argument checks and launches.  Nothing here allocates or
// synchronises.
#include "dense.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool is_dtype(int d) { return d == MOE_DT_F32 || d == MOE_DT_BF16; }
int64_t size_of(int dtype) { return dtype == MOE_DT_F32 ? 4 : 2; }
uint64_t magnitude(int64_t stride) { return stride < 0 ? -(uint64_t)stride : (uint64_t)stride; }

constexpr uint64_t kMaxStride = 4 * MOE_DENSE_MAX_STRIDE;  // bytes: tensor maps, and products with a row that stay in range

int check_mx(const moe_mx* a) {
  if (!a || !a->q || !a->s || !aligned(a->q, 16)) return MOE_ERR_INVALID_ARG;
  if (a->type != MOE_MX_E2M1 && a->type != MOE_MX_E4M3) return MOE_ERR_INVALID_ARG;
  if (a->rows < 1 || a->cols < 32 || a->cols % 32) return MOE_ERR_INVALID_ARG;
  const int64_t row = a->type == MOE_MX_E4M3 ? a->cols : a->cols / 2;
  if (a->q_stride % 16 || a->q_stride < row || a->s_stride < a->cols / 32) return MOE_ERR_INVALID_ARG;
  if (a->cols > MOE_DENSE_MAX_COLS || magnitude(a->q_stride) >= kMaxStride || magnitude(a->s_stride) >= kMaxStride) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows of `cols` elements at 16-byte vectors; apart: an output's.
int check_rows(const void* x, int dtype, int64_t stride, int rows, int cols, bool apart) {
  if (!x || !is_dtype(dtype) || !aligned(x, 16) || (uint64_t)stride * size_of(dtype) % 16) return MOE_ERR_INVALID_ARG;
  if (magnitude(stride) >= kMaxStride / 4) return MOE_ERR_UNSUPPORTED;
  if (apart && rows > 1 && magnitude(stride) < (uint64_t)cols) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

MxRows rows_of(const moe_mx& a) { return {a.q, a.s, a.q_stride, a.s_stride}; }

// Values that one launch of the conversions covers: counts of eights, its last CTA's behind the end too, stay in 32 bits.
bool too_many(const moe_mx* a) { return (int64_t)a->rows * a->cols > MOE_MX_MAX_VALUES; }
static_assert(MOE_MX_MAX_VALUES / 8 < (1LL << 32) - 1024 && MOE_MX_MAX_VALUES / 8 + 4 >= (1LL << 32) - 1024, "blocks of 32");

}  // namespace

extern "C" {

int moe_mx_quantize(const void* x, int x_dtype, int64_t x_stride, const moe_mx* out, void* stream) {
  int st;
  if ((st = check_mx(out)) != MOE_OK) return st;
  if ((st = check_rows(x, x_dtype, x_stride, out->rows, out->cols, false)) != MOE_OK) return st;
  if (out->q == x) return MOE_ERR_INVALID_ARG;
  if (too_many(out)) return MOE_ERR_UNSUPPORTED;
  QuantizeParams p = {(uint32_t)out->rows, (uint32_t)out->cols, x, nullptr, x_stride * size_of(x_dtype), rows_of(*out)};
  return cuda_status(launch_mx_quantize(p, x_dtype, out->type, (cudaStream_t)stream));
}

int moe_mx_dequantize(const moe_mx* x, void* out, int out_dtype, int64_t out_stride, void* stream) {
  int st;
  if ((st = check_mx(x)) != MOE_OK) return st;
  if ((st = check_rows(out, out_dtype, out_stride, x->rows, x->cols, true)) != MOE_OK) return st;
  if (x->q == out) return MOE_ERR_INVALID_ARG;
  if (too_many(x)) return MOE_ERR_UNSUPPORTED;
  QuantizeParams p = {(uint32_t)x->rows, (uint32_t)x->cols, nullptr, out, out_stride * size_of(out_dtype), rows_of(*x)};
  return cuda_status(launch_mx_dequantize(p, out_dtype, x->type, (cudaStream_t)stream));
}

int moe_rms_norm(int rows, int cols, const void* x, int x_dtype, int64_t x_stride, const void* residual,
                 void* residual_out, int res_dtype, int64_t res_stride, const float* weight, float eps, void* out,
                 int out_dtype, int64_t out_stride, const moe_mx* mx, void* stream) {
  int st;
  if (rows < 1 || cols < 8 || cols % 8) return MOE_ERR_INVALID_ARG;
  if (cols > MOE_DENSE_MAX_COLS) return MOE_ERR_UNSUPPORTED;
  if (!(eps > 0.f) || !(eps < 3.4e38f) || !aligned(weight, 16)) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(x, x_dtype, x_stride, rows, cols, false)) != MOE_OK) return st;
  if ((residual == nullptr) != (residual_out == nullptr)) return MOE_ERR_INVALID_ARG;
  if (residual) {
    if ((st = check_rows(residual, res_dtype, res_stride, rows, cols, false)) != MOE_OK) return st;
    if ((st = check_rows(residual_out, res_dtype, res_stride, rows, cols, true)) != MOE_OK) return st;
  }
  if ((out == nullptr) == (mx == nullptr)) return MOE_ERR_INVALID_ARG;
  NormParams p = {};
  if (mx) {
    if ((st = check_mx(mx)) != MOE_OK) return st;
    if (mx->rows != rows || mx->cols != cols) return MOE_ERR_INVALID_ARG;
    p.mx = rows_of(*mx);
  } else if ((st = check_rows(out, out_dtype, out_stride, rows, cols, true)) != MOE_OK) {
    return st;
  }
  // In place: every row over itself.
  const int64_t xb = x_stride * size_of(x_dtype), rb = residual ? res_stride * size_of(res_dtype) : 0;
  const int64_t ob = out ? out_stride * size_of(out_dtype) : 0;
  auto over = [&](const void* o, int ot, int64_t os, const void* i, int it, int64_t is) {
    return o && o == i && (ot != it || (rows > 1 && os != is));
  };
  if (over(out, out_dtype, ob, x, x_dtype, xb) || over(out, out_dtype, ob, residual, res_dtype, rb) ||
      over(residual_out, res_dtype, rb, x, x_dtype, xb) || (out && out == residual_out) ||
      (mx && (mx->q == x || mx->q == residual || mx->q == residual_out)))
    return MOE_ERR_INVALID_ARG;
  p.rows = rows;
  p.cols = cols;
  p.x = x;
  p.res = residual;
  p.res_out = residual_out;
  p.out = out;
  p.x_stride = xb;
  p.res_stride = rb;
  p.out_stride = ob;
  p.weight = weight;
  p.eps = eps;
  // Also where eps beside the sum's mean leaves fp32's range.
  const double room = (3.4028234e38 - eps) * cols * (1 - 0x1p-20);
  p.most = room < 3.0e38 ? (float)room : 3.0e38f;
  return cuda_status(launch_rms_norm(p, x_dtype, res_dtype, mx ? 2 + mx->type : out_dtype, (cudaStream_t)stream));
}

int moe_mx_linear(const moe_mx* x, const moe_mx* w, const void* add, int64_t add_stride, void* out, int out_dtype,
                  int64_t out_stride, int32_t* status, void* stream) {
  int st;
  if ((st = check_mx(x)) != MOE_OK || (st = check_mx(w)) != MOE_OK) return st;
  if (x->cols != w->cols || !out || !is_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  const int64_t size = size_of(out_dtype);
  if (!aligned(out, size) || !aligned(add, size) || (status && !aligned(status, 4))) return MOE_ERR_INVALID_ARG;
  for (const moe_mx* a : {x, w})
    if (!aligned(a->q, 32) || a->q_stride % 32 || !aligned(a->s, 4) || a->s_stride % 4) return MOE_ERR_INVALID_ARG;
  if (x->rows > 1 && magnitude(out_stride) < (uint64_t)w->rows) return MOE_ERR_INVALID_ARG;
  // In place: every row over itself.
  if (add == out && x->rows > 1 && add_stride != out_stride) return MOE_ERR_INVALID_ARG;
  if (w->type != MOE_MX_E2M1 || x->cols % 128 || x->rows > MOE_LINEAR_MAX_ROWS || w->rows > MOE_LINEAR_MAX_OUTS)
    return MOE_ERR_UNSUPPORTED;
  if (magnitude(out_stride) >= kMaxStride / 4 || magnitude(add_stride) >= kMaxStride / 4) return MOE_ERR_UNSUPPORTED;
  LinearParams p = {};
  p.T = x->rows;
  p.N = w->rows;
  p.K = x->cols;
  p.xs = x->s;
  p.ws = w->s;
  p.xs_stride = x->s_stride;
  p.ws_stride = w->s_stride;
  p.add = add;
  p.out = out;
  p.add_stride = add_stride;
  p.out_stride = out_stride;
  p.status = status;
  p.wait_limit = wait_limit();
  return cuda_status(launch_mx_linear(p, *x, *w, out_dtype, (cudaStream_t)stream));
}

int moe_token_logprobs(int rows, int vocab, const void* logits, int dtype, int64_t stride, const int32_t* tokens,
                       float* logprob, int32_t* rank, float* entropy, int top, int32_t* top_ids, float* top_logprobs,
                       void* stream) {
  if (rows < 1 || vocab < 1 || !logits || !is_dtype(dtype) || !aligned(logits, size_of(dtype))) return MOE_ERR_INVALID_ARG;
  if (rows > 1 && magnitude(stride) < (uint64_t)vocab) return MOE_ERR_INVALID_ARG;
  if (!tokens && (logprob || rank)) return MOE_ERR_INVALID_ARG;
  if (top < 0 || (top > 0) != (top_ids != nullptr) || (top > 0) != (top_logprobs != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!logprob && !rank && !entropy && !top) return MOE_ERR_INVALID_ARG;
  const void* words[] = {tokens, logprob, rank, entropy, top_ids, top_logprobs};
  for (const void* w : words)
    if (!aligned(w, 4)) return MOE_ERR_INVALID_ARG;
  if (vocab > MOE_LOGPROBS_MAX_VOCAB || rows > MOE_LOGPROBS_MAX_ROWS || top > MOE_LOGPROBS_MAX_TOP || magnitude(stride) >= kMaxStride / 4)
    return MOE_ERR_UNSUPPORTED;
  LogprobParams p = {};
  p.rows = rows;
  p.vocab = vocab;
  p.top = top;
  p.logits = logits;
  p.stride = stride;
  p.tokens = tokens;
  p.logprob = logprob;
  p.rank = rank;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  return cuda_status(launch_token_logprobs(p, dtype, (cudaStream_t)stream));
}

}  // extern "C"
