// api_block.cu - C entry points of the operators around a block's sparse layers:
// argument checks, tensor maps and launches (the checks, errors and device
// set-up are those of api.cu).
#include <cmath>

#include "abi_internal.cuh"
#include "fp4.cuh"
#include "kernels.cuh"

namespace {

using cm::record_errorf;

#define CM_CHECK(expr)                         \
  do {                                         \
    chipmunk_status _st = (expr);              \
    if (_st != CHIPMUNK_OK) return _st;        \
  } while (0)

#define CM_CUDA(expr, what)                                                              \
  do {                                                                                   \
    cudaError_t _e = (expr);                                                             \
    if (_e != cudaSuccess)                                                               \
      return record_errorf(CHIPMUNK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(_e));   \
  } while (0)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A pointer argument: required or optional, 16-byte aligned where given.
struct Ptr {
  const void *p;
  const char *name;
  bool required;
};

chipmunk_status check_ptrs(const Ptr *ptrs, int n) {
  for (int i = 0; i < n; ++i) {
    if (ptrs[i].p == nullptr && ptrs[i].required)
      return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "%s is NULL", ptrs[i].name);
    if (!aligned16(ptrs[i].p)) return record_errorf(CHIPMUNK_ERR_ALIGNMENT, "%s is not 16-byte aligned", ptrs[i].name);
  }
  return CHIPMUNK_OK;
}

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxN = int64_t(1) << 20;

bool fp4_sizes_ok(int64_t rows, int64_t cols, int32_t format) {
  return rows >= 0 && rows <= kMaxRows && cols >= 32 && cols <= 65536 && cols % 32 == 0 &&
         (format == CHIPMUNK_NVFP4 || format == CHIPMUNK_MXFP4);
}

// The product's tiles are counted in 31 bits.
bool linear_tiles_ok(int64_t T, int64_t N) { return ((T + 127) / 128) * ((N + 127) / 128) < (int64_t(1) << 31); }

chipmunk_status check_fp4(const chipmunk_fp4_rows *q, const char *what) {
  if (q == nullptr) return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "%s is NULL", what);
  if (q->format != CHIPMUNK_NVFP4 && q->format != CHIPMUNK_MXFP4)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "%s: format %d unknown", what, q->format);
  if (!fp4_sizes_ok(q->rows, q->cols, q->format))
    return record_errorf(CHIPMUNK_ERR_SHAPE, "%s: %lld rows x %lld columns (columns a multiple of 32 up to 65536)", what,
                         (long long)q->rows, (long long)q->cols);
  if (q->rows == 0) return CHIPMUNK_OK;
  const Ptr ptrs[] = {{q->codes, "codes", true},
                      {q->scales, "scales", true},
                      {q->row_scales, "row_scales", q->format == CHIPMUNK_NVFP4}};
  return check_ptrs(ptrs, 3);
}

cm::Fp4QuantParams quant_params(const void *x, const chipmunk_fp4_rows *q, int *status) {
  return {q->rows,
          q->cols,
          q->format == CHIPMUNK_NVFP4 ? cm::kNvfp4 : cm::kMxfp4,
          static_cast<const uint16_t *>(x),
          static_cast<uint8_t *>(q->codes),
          static_cast<uint8_t *>(q->scales),
          q->row_scales,
          status};
}

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// The quantised x of a linear call inside its workspace: codes, block scales, row scales.
chipmunk_fp4_rows ws_rows(const chipmunk_linear_fp4_args *a, void *ws) {
  uint8_t *p = static_cast<uint8_t *>(ws);
  const size_t codes = round_up(size_t(a->T) * size_t(a->w.cols / 2), 256);
  const size_t scales = cm::fp4_scale_bytes(a->T, a->w.cols, a->w.format);
  return {a->T, a->w.cols, a->w.format, p, p + codes, reinterpret_cast<float *>(p + codes + scales)};
}

// Tensor maps of a linear call. Codes: rows of bytes, boxes of 128 bytes (256 columns) x 128
// rows. Block scales: 512-byte tiles as 128 words, boxes of the tiles of 256 columns of
// one row tile of x and of as many of w as the product's tile has. out: boxes of 128 bytes x 32 rows.
chipmunk_status linear_maps(cm::LinearFp4Maps *m, const chipmunk_linear_fp4_args *a, const chipmunk_fp4_rows &xq) {
  const uint64_t T = a->T, N = a->N, bytes = uint64_t(a->w.cols) / 2;
  const uint64_t tiles = cm::fp4_scale_tiles(a->w.cols, a->w.format);
  const uint32_t per_stage = a->w.format == CHIPMUNK_NVFP4 ? 4 : 2;
  const bool f32 = a->out_type == CHIPMUNK_FP32;
  const uint64_t out_es = f32 ? 4 : 2;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, i32 = CU_TENSOR_MAP_DATA_TYPE_INT32;
  const uint64_t dx[] = {bytes, T}, dw[] = {bytes, N}, dsx[] = {128, tiles, (T + 127) / 128},
                 dsw[] = {128, tiles, (N + 127) / 128}, dout[] = {N, T};
  const uint64_t sb[] = {bytes}, ss[] = {512, tiles * 512}, so[] = {N * out_es};
  const uint32_t box[] = {128, 128}, boxw[] = {128, 256}, bsx[] = {128, per_stage, 1}, bsw1[] = {128, per_stage, 1},
                 bsw2[] = {128, per_stage, 2}, bout[] = {uint32_t(128 / out_es), 32};
  const bool wide = m->form == cm::kLinearPair || m->form == cm::kLinearWide;  // 256 columns per tile
  CM_CHECK(cm::encode_map(&m->w, u8, a->w.codes, 2, dw, sb, m->form == cm::kLinearWide ? boxw : box, true, "w codes"));
  CM_CHECK(cm::encode_map(&m->sw, i32, a->w.scales, 3, dsw, ss, wide ? bsw2 : bsw1, false, "w scales"));
  if (m->form == cm::kLinearRows) return CHIPMUNK_OK;
  CM_CHECK(cm::encode_map(&m->x, u8, xq.codes, 2, dx, sb, box, true, "x codes"));
  CM_CHECK(cm::encode_map(&m->sx, i32, xq.scales, 3, dsx, ss, bsx, false, "x scales"));
  return cm::encode_map(&m->out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->out, 2,
                        dout, so, bout, true, "out");
}

}  // namespace

namespace cm {

size_t linear_fp4_ws(const chipmunk_linear_fp4_args *a) {
  if (a->x == nullptr || a->T < 1 || !fp4_sizes_ok(a->T, a->w.cols, a->w.format)) return 0;
  if (linear_fp4_form(a->T, a->N, a->w.cols, false) == kLinearRows) return 0;
  size_t n = round_up(size_t(a->T) * size_t(a->w.cols / 2), 256) + fp4_scale_bytes(a->T, a->w.cols, a->w.format);
  if (a->w.format == CHIPMUNK_NVFP4) n += round_up(size_t(a->T) * 4, 256);
  return n;
}

}  // namespace cm

extern "C" {

size_t chipmunk_fp4_scale_bytes(int64_t rows, int64_t cols, int32_t format) {
  return fp4_sizes_ok(rows, cols, format) ? cm::fp4_scale_bytes(rows, cols, format) : 0;
}

chipmunk_status chipmunk_quantize_fp4_rows(const void *x, const chipmunk_fp4_rows *q, chipmunk_stream stream) {
  CM_CHECK(check_fp4(q, "q"));
  if (q->rows == 0) return CHIPMUNK_OK;
  const Ptr ptrs[] = {{x, "x", true}};
  CM_CHECK(check_ptrs(ptrs, 1));
  int *status = nullptr;
  CM_CHECK(cm::device_ready(&status));
  CM_CUDA(cm::launch_quantize_fp4_rows(quant_params(x, q, status), static_cast<cudaStream_t>(stream)),
          "4-bit quantise launch");
  return CHIPMUNK_OK;
}

chipmunk_status chipmunk_dequantize_fp4_rows(const chipmunk_fp4_rows *q, int32_t out_type, void *out,
                                             chipmunk_stream stream) {
  CM_CHECK(check_fp4(q, "q"));
  if (out_type != CHIPMUNK_BF16 && out_type != CHIPMUNK_FP32)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "out_type %d unknown", out_type);
  if (q->rows == 0) return CHIPMUNK_OK;
  const Ptr ptrs[] = {{out, "out", true}};
  CM_CHECK(check_ptrs(ptrs, 1));
  int *status = nullptr;
  CM_CHECK(cm::device_ready(&status));
  CM_CUDA(cm::launch_dequantize_fp4_rows(quant_params(nullptr, q, status), out_type == CHIPMUNK_FP32, out,
                                         static_cast<cudaStream_t>(stream)),
          "4-bit dequantise launch");
  return CHIPMUNK_OK;
}

chipmunk_status chipmunk_linear_fp4(const chipmunk_linear_fp4_args *a, void *ws, size_t ws_bytes,
                                    chipmunk_stream stream) {
  if (a == nullptr) return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "args is NULL");
  if (a->T < 1 || a->T > kMaxRows) return record_errorf(CHIPMUNK_ERR_SHAPE, "T=%lld out of range", (long long)a->T);
  if (a->N < 8 || a->N > kMaxN || a->N % 8 != 0)
    return record_errorf(CHIPMUNK_ERR_SHAPE, "N=%lld must be a multiple of 8 in [8, 2^20]", (long long)a->N);
  if (!linear_tiles_ok(a->T, a->N))
    return record_errorf(CHIPMUNK_ERR_SHAPE, "T=%lld x N=%lld is too large", (long long)a->T, (long long)a->N);
  if (a->act != CHIPMUNK_ACT_NONE && a->act != CHIPMUNK_ACT_GELU)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "act %d unknown", a->act);
  if (a->out_type != CHIPMUNK_BF16 && a->out_type != CHIPMUNK_FP32)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "out_type %d unknown", a->out_type);
  CM_CHECK(check_fp4(&a->w, "w"));
  if (a->w.rows != a->N)
    return record_errorf(CHIPMUNK_ERR_SHAPE, "w has %lld rows, N is %lld", (long long)a->w.rows, (long long)a->N);
  const Ptr ptrs[] = {{a->x, "x", false}, {a->bias, "bias", false}, {a->out, "out", true}};
  CM_CHECK(check_ptrs(ptrs, 3));
  chipmunk_fp4_rows xq = a->xq;
  cm::LinearFp4Maps m;
  m.form = cm::linear_fp4_form(a->T, a->N, a->w.cols, a->x == nullptr);
  if (m.form == cm::kLinearRows) {
    // quantised inside the product's kernel: no workspace
  } else if (a->x != nullptr) {
    const size_t need = cm::linear_fp4_ws(a);
    if (ws == nullptr || ws_bytes < need)
      return record_errorf(CHIPMUNK_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                           ws == nullptr ? size_t(0) : ws_bytes);
    if (!aligned16(ws)) return record_errorf(CHIPMUNK_ERR_ALIGNMENT, "ws is not 16-byte aligned");
    xq = ws_rows(a, ws);
  } else {
    CM_CHECK(check_fp4(&a->xq, "xq"));
    if (xq.rows != a->T || xq.cols != a->w.cols || xq.format != a->w.format)
      return record_errorf(CHIPMUNK_ERR_SHAPE, "xq (%lld x %lld, format %d) does not fit T=%lld and w's %lld columns, format %d",
                           (long long)xq.rows, (long long)xq.cols, xq.format, (long long)a->T, (long long)a->w.cols,
                           a->w.format);
  }
  int *status = nullptr;
  CM_CHECK(cm::device_ready(&status));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = a->out_type == CHIPMUNK_FP32;
  CM_CHECK(linear_maps(&m, a, xq));
  if (a->x != nullptr && m.form != cm::kLinearRows)
    CM_CUDA(cm::launch_quantize_fp4_rows(quant_params(a->x, &xq, status), s), "4-bit quantise launch");
  cm::LinearFp4Params p{int(a->T),
                        int(a->N),
                        int(a->w.cols),
                        a->w.format == CHIPMUNK_NVFP4 ? cm::kNvfp4 : cm::kMxfp4,
                        a->act == CHIPMUNK_ACT_GELU,
                        f32,
                        xq.row_scales,
                        a->w.row_scales,
                        static_cast<const uint16_t *>(a->bias),
                        static_cast<const uint16_t *>(a->x),
                        a->out,
                        status};
  CM_CUDA(cm::launch_linear_fp4(p, m, s), "4-bit linear launch");
  return CHIPMUNK_OK;
}

int32_t chipmunk_selftest_linear_fp4_form(int64_t T, int64_t N, int64_t K, int32_t quantised) {
  if (T < 1 || N < 8 || N > kMaxN || N % 8 != 0 || !fp4_sizes_ok(T, K, CHIPMUNK_NVFP4) || !linear_tiles_ok(T, N)) return -1;
  return cm::linear_fp4_form(T, N, K, quantised != 0);
}

chipmunk_status chipmunk_norm_residual(const chipmunk_norm_args *a, chipmunk_stream stream) {
  if (a == nullptr) return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "args is NULL");
  if (a->T < 1 || a->T > kMaxRows) return record_errorf(CHIPMUNK_ERR_SHAPE, "T=%lld out of range", (long long)a->T);
  if (a->D < 8 || a->D > 16384 || a->D % 8 != 0)
    return record_errorf(CHIPMUNK_ERR_SHAPE, "D=%lld must be a multiple of 8 in [8, 16384]", (long long)a->D);
  if (a->B < 1 || a->B > kMaxRows) return record_errorf(CHIPMUNK_ERR_SHAPE, "B=%lld out of range", (long long)a->B);
  const int32_t types[] = {a->res_type, a->y_type, a->mod_type};
  for (int32_t t : types)
    if (t != CHIPMUNK_BF16 && t != CHIPMUNK_FP32) return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "type %d unknown", t);
  if (a->post_norm < CHIPMUNK_NORM_NONE || a->post_norm > CHIPMUNK_NORM_RMS)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "post_norm %d unknown", a->post_norm);
  if (a->out != nullptr && a->norm != CHIPMUNK_NORM_LAYER && a->norm != CHIPMUNK_NORM_RMS)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "norm %d unknown", a->norm);
  if (a->out_format < CHIPMUNK_OUT_BF16 || a->out_format > CHIPMUNK_OUT_MXFP4)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "out_format %d unknown", a->out_format);
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps) || !std::isfinite(a->res_scale))
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "eps must be >= 0 and finite, res_scale finite");
  if (a->y == nullptr && (a->gate != nullptr || a->post_weight != nullptr || a->post_norm != CHIPMUNK_NORM_NONE))
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "gate, post_norm and post_weight need y");
  if (a->post_weight != nullptr && a->post_norm == CHIPMUNK_NORM_NONE)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "post_weight needs a post_norm");
  if (a->out == nullptr && a->res_out == nullptr)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "out and res_out are both NULL");
  if ((a->gate != nullptr || a->scale != nullptr || a->shift != nullptr) && (a->ld_mod < a->D || a->ld_mod % 8 != 0))
    return record_errorf(CHIPMUNK_ERR_SHAPE, "ld_mod=%lld must be a multiple of 8, at least D", (long long)a->ld_mod);
  if (a->offsets == nullptr && a->B != 1)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "B=%lld samples need offsets", (long long)a->B);
  const bool fp4 = a->out_format == CHIPMUNK_OUT_NVFP4 || a->out_format == CHIPMUNK_OUT_MXFP4;
  const bool quant = a->out != nullptr && a->out_format != CHIPMUNK_OUT_BF16;
  if (quant && a->D % (fp4 ? 32 : 16) != 0)
    return record_errorf(CHIPMUNK_ERR_SHAPE, "D=%lld must be a multiple of %d for quantised rows", (long long)a->D,
                         fp4 ? 32 : 16);
  const Ptr ptrs[] = {{a->res, "res", true},
                      {a->y, "y", false},
                      {a->post_weight, "post_weight", false},
                      {a->gate, "gate", false},
                      {a->res_out, "res_out", false},
                      {a->weight, "weight", false},
                      {a->bias, "bias", false},
                      {a->scale, "scale", false},
                      {a->shift, "shift", false},
                      {a->out, "out", false},
                      {a->out_scales, "out_scales", quant && fp4},
                      {a->out_row_scales, "out_row_scales", quant && a->out_format != CHIPMUNK_OUT_MXFP4}};
  CM_CHECK(check_ptrs(ptrs, 12));
  if ((reinterpret_cast<uintptr_t>(a->offsets) & 3u) != 0)
    return record_errorf(CHIPMUNK_ERR_ALIGNMENT, "offsets is not 4-byte aligned");
  int *status = nullptr;
  CM_CHECK(cm::device_ready(&status));
  cm::NormParams p{a->T,
                   int(a->D),
                   int(a->B),
                   a->res_type == CHIPMUNK_FP32,
                   a->y_type == CHIPMUNK_FP32,
                   a->mod_type == CHIPMUNK_FP32,
                   a->norm,
                   a->post_norm,
                   a->out_format,
                   a->eps,
                   a->res_scale,
                   a->res,
                   a->y,
                   a->post_weight,
                   a->gate,
                   a->res_out,
                   a->weight,
                   a->bias,
                   a->scale,
                   a->shift,
                   a->ld_mod,
                   a->offsets,
                   a->out,
                   static_cast<uint8_t *>(a->out_scales),
                   a->out_row_scales,
                   status};
  CM_CUDA(cm::launch_norm_residual(p, static_cast<cudaStream_t>(stream)), "norm launch");
  return CHIPMUNK_OK;
}

chipmunk_status chipmunk_qk_norm_rope(const chipmunk_heads_args *a, chipmunk_stream stream) {
  if (a == nullptr) return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "args is NULL");
  if (a->h < 1 || a->h > 1024) return record_errorf(CHIPMUNK_ERR_SHAPE, "h=%d out of range", a->h);
  if (a->T < 1 || a->T > kMaxRows || a->T * a->h >= (int64_t(1) << 31))
    return record_errorf(CHIPMUNK_ERR_SHAPE, "T=%lld out of range (T * h below 2^31)", (long long)a->T);
  if (a->ld < int64_t(3) * a->h * 128 || a->ld % 8 != 0 || a->ld > (int64_t(1) << 32))
    return record_errorf(CHIPMUNK_ERR_SHAPE, "ld=%lld must be a multiple of 8, at least 3*h*128", (long long)a->ld);
  if (a->pairs != CHIPMUNK_PAIRS_INTERLEAVED && a->pairs != CHIPMUNK_PAIRS_HALVES)
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "pairs %d unknown", a->pairs);
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps))
    return record_errorf(CHIPMUNK_ERR_INVALID_ARG, "eps must be >= 0 and finite");
  const Ptr ptrs[] = {{a->qkv, "qkv", true}, {a->q_weight, "q_weight", true}, {a->k_weight, "k_weight", true},
                      {a->cos, "cos", true}, {a->sin, "sin", true},           {a->q, "q", true},
                      {a->k, "k", true},     {a->v, "v", true}};
  CM_CHECK(check_ptrs(ptrs, 8));
  int *status = nullptr;
  CM_CHECK(cm::device_ready(&status));
  cm::HeadsParams p{a->T,
                    a->h,
                    a->pairs == CHIPMUNK_PAIRS_HALVES,
                    a->ld,
                    a->eps,
                    static_cast<const uint16_t *>(a->qkv),
                    static_cast<const uint16_t *>(a->q_weight),
                    static_cast<const uint16_t *>(a->k_weight),
                    a->cos,
                    a->sin,
                    static_cast<uint16_t *>(a->q),
                    static_cast<uint16_t *>(a->k),
                    static_cast<uint16_t *>(a->v),
                    status};
  CM_CUDA(cm::launch_qk_norm_rope(p, static_cast<cudaStream_t>(stream)), "heads launch");
  return CHIPMUNK_OK;
}

}  // extern "C"
