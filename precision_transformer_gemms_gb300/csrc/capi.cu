// C ABI of liblpq: argument validation, status codes and the host-only
// helpers (copy sizes, the 12 GEMM shapes of a layer).  No entry point
// allocates device memory or falls back to another format ("How to optimize
// Transformer-based models for low-precision training", interpreting
// real-model results: a silent fallback to FP8/BF16 is what to avoid).
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <map>
#include <set>
#include <utility>

#include "lpq_internal.h"

namespace lpq {

namespace {
thread_local char g_last_error[512] = "";

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool is_fp8_pertensor(int32_t f) { return f == LPQ_FP8_E4M3 || f == LPQ_FP8_E5M2; }
bool is_nvfp4(int32_t f) { return f == LPQ_NVFP4 || f == LPQ_NVFP4_2D; }
bool is_block(int32_t f) { return f == LPQ_FP8_BLOCK_1x128 || f == LPQ_FP8_BLOCK_128x128; }
bool is_mx8(int32_t f) { return f == LPQ_MXFP8 || f == LPQ_MXFP8_E5M2; }
// Formats with u8 block scales in the tensor-core scale layout.
bool is_u8_scaled(int32_t f) { return is_mx8(f) || f == LPQ_MXFP4 || is_nvfp4(f); }
bool valid_fmt(int32_t f) { return f >= LPQ_BF16 && f <= LPQ_MXFP4; }

// Column-block length of a format's row-wise scales (0 = none).
int64_t row_block(int32_t f) {
  switch (f) {
    case LPQ_MXFP8: case LPQ_MXFP8_E5M2: case LPQ_MXFP4: return 32;
    case LPQ_NVFP4: case LPQ_NVFP4_2D: return 16;
    case LPQ_FP8_BLOCK_1x128: case LPQ_FP8_BLOCK_128x128: return 128;
  }
  return 0;
}

// Rows of the input that a column-wise copy needs as a multiple.
int64_t col_rows_multiple(int32_t f) {
  switch (f) {
    case LPQ_MXFP8: case LPQ_MXFP8_E5M2: case LPQ_MXFP4: return 32;
    case LPQ_FP8_BLOCK_1x128: case LPQ_FP8_BLOCK_128x128: return 128;
  }
  return 16;
}

lpq_status check_arch() {
  static int ok = -1;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_check(e, "cudaGetDevice");
  static int checked_dev = -1;
  if (ok < 0 || checked_dev != dev) {
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    ok = (major == 10 && minor == 3) ? 1 : 0;
    checked_dev = dev;
    if (!ok)
      return set_error(LPQ_ERR_ARCH, "device %d is sm_%d%d; liblpq is built for sm_103a only", dev, major, minor);
  }
  return ok ? LPQ_OK : set_error(LPQ_ERR_ARCH, "device is not sm_103");
}

lpq_status check_view(const lpq_qview* v, const char* name, int32_t fmt, int64_t rows, int64_t cols, int colwise,
                      bool need_ts, bool need_amax) {
  if (v->fmt != fmt) return set_error(LPQ_ERR_INVALID_ARG, "%s.fmt is %d, expected %d", name, v->fmt, fmt);
  if (v->rows != rows || v->cols != cols)
    return set_error(LPQ_ERR_SHAPE, "%s is %lld x %lld, expected %lld x %lld", name, (long long)v->rows,
                     (long long)v->cols, (long long)rows, (long long)cols);
  if (v->colwise != colwise) return set_error(LPQ_ERR_INVALID_ARG, "%s.colwise must be %d", name, colwise);
  if (v->sf_layout != LPQ_SF_PLAIN && v->sf_layout != LPQ_SF_GEMM)
    return set_error(LPQ_ERR_INVALID_ARG, "%s.sf_layout %d", name, v->sf_layout);
  if (rows * cols > 0 && !v->codes) return set_error(LPQ_ERR_INVALID_ARG, "%s.codes is NULL", name);
  if (!aligned16(v->codes)) return set_error(LPQ_ERR_ALIGN, "%s.codes not 16-byte aligned", name);
  if (row_block(fmt) && rows * cols > 0 && !v->scales) return set_error(LPQ_ERR_INVALID_ARG, "%s.scales is NULL", name);
  if (row_block(fmt) && v->sf_layout == LPQ_SF_GEMM && !aligned16(v->scales))
    return set_error(LPQ_ERR_ALIGN, "%s.scales not 16-byte aligned", name);
  if (is_block(fmt) && (reinterpret_cast<uintptr_t>(v->scales) & 3u))
    return set_error(LPQ_ERR_ALIGN, "%s.scales not 4-byte aligned", name);
  if (need_ts && !v->tensor_scale) return set_error(LPQ_ERR_INVALID_ARG, "%s.tensor_scale is NULL", name);
  if (need_amax && !v->amax) return set_error(LPQ_ERR_INVALID_ARG, "%s.amax is NULL", name);
  return LPQ_OK;
}
}  // namespace

lpq_status set_error(lpq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

lpq_status cuda_check(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return LPQ_OK;
  return set_error(LPQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

namespace {
std::mutex g_dev_mu;
std::set<int>* g_sms_known = nullptr;  // devices whose SM count is cached
int g_sms_of[256];
std::set<std::pair<int, const void*>>* g_smem_set = nullptr;  // (device, kernel) pairs already raised
std::map<std::pair<int, const void*>, int>* g_resident = nullptr;  // (device, kernel) -> CTAs per SM
}  // namespace

int device_sms() {
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!g_sms_known) g_sms_known = new std::set<int>();
  if (dev >= 0 && dev < 256 && g_sms_known->count(dev)) return g_sms_of[dev];
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (n <= 0) n = 148;
  if (dev >= 0 && dev < 256) {
    g_sms_of[dev] = n;
    g_sms_known->insert(dev);
  }
  return n;
}

int resident_ctas(const void* kernel, int threads, int smem) {
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!g_resident) g_resident = new std::map<std::pair<int, const void*>, int>();
  auto it = g_resident->find({dev, kernel});
  if (it != g_resident->end()) return it->second;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
  (*g_resident)[{dev, kernel}] = n;
  return n;
}

lpq_status set_smem_attr(const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_check(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!g_smem_set) g_smem_set = new std::set<std::pair<int, const void*>>();
  if (g_smem_set->count({dev, kernel})) return LPQ_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_check(e, "cudaFuncSetAttribute(max dynamic shared memory)");
  g_smem_set->insert({dev, kernel});
  return LPQ_OK;
}

}  // namespace lpq

using namespace lpq;

extern "C" {

int32_t lpq_version(void) { return 100; }

const char* lpq_last_error(void) { return g_last_error; }

lpq_status lpq_copy_bytes(int32_t fmt, int64_t rows, int64_t cols, int32_t sf_layout, size_t* codes_bytes,
                          size_t* scale_bytes) {
  if (!codes_bytes || !scale_bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  if (!valid_fmt(fmt)) return set_error(LPQ_ERR_INVALID_ARG, "unknown format %d", fmt);
  if (rows < 0 || cols < 0) return set_error(LPQ_ERR_SHAPE, "negative dimension");
  if (sf_layout != LPQ_SF_PLAIN && sf_layout != LPQ_SF_GEMM) return set_error(LPQ_ERR_INVALID_ARG, "sf_layout");
  const int64_t blk = row_block(fmt);
  if (blk && cols % blk) return set_error(LPQ_ERR_SHAPE, "cols %lld not a multiple of %lld", (long long)cols, (long long)blk);
  const size_t n = (size_t)rows * (size_t)cols;
  size_t cb = 0, sb = 0;
  switch (fmt) {
    case LPQ_BF16: cb = 2 * n; break;
    case LPQ_FP8_E4M3: case LPQ_FP8_E5M2: cb = n; break;
    case LPQ_MXFP8: case LPQ_MXFP8_E5M2: case LPQ_MXFP4: case LPQ_NVFP4: case LPQ_NVFP4_2D:
      cb = is_mx8(fmt) ? n : n / 2;
      sb = sf_layout == LPQ_SF_GEMM ? (size_t)sf_row_groups(rows) * (size_t)sf_kt_atoms(fmt, cols) * 512
                                    : (size_t)rows * (size_t)(cols / blk);
      break;
    case LPQ_FP8_BLOCK_1x128: cb = n; sb = 4 * (size_t)rows * (size_t)(cols / 128); break;
    case LPQ_FP8_BLOCK_128x128: cb = n; sb = 4 * (size_t)((rows + 127) / 128) * (size_t)(cols / 128); break;
  }
  *codes_bytes = cb;
  *scale_bytes = sb;
  return LPQ_OK;
}

lpq_status lpq_quantize(const void* x, int64_t rows, int64_t cols, int32_t fmt, int32_t scaling, uint32_t flags,
                        uint64_t seed, uint64_t counter_offset, uint32_t rht_seed, const lpq_delayed_state* state,
                        lpq_qtensor* out, lpq_stream_t stream) {
  if (!valid_fmt(fmt)) return set_error(LPQ_ERR_INVALID_ARG, "unknown format %d", fmt);
  if (!out) return set_error(LPQ_ERR_INVALID_ARG, "out is NULL");
  if (rows < 0 || cols < 0) return set_error(LPQ_ERR_SHAPE, "negative dimension");
  if (flags & ~uint32_t(LPQ_ROWWISE | LPQ_COLWISE | LPQ_RHT_COLWISE | LPQ_STOCHASTIC | LPQ_GIVEN_AMAX))
    return set_error(LPQ_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  const bool do_row = flags & LPQ_ROWWISE, do_col = flags & LPQ_COLWISE;
  if (!do_row && !do_col) return set_error(LPQ_ERR_INVALID_ARG, "neither LPQ_ROWWISE nor LPQ_COLWISE requested");
  if ((flags & (LPQ_RHT_COLWISE | LPQ_STOCHASTIC)) && fmt != LPQ_NVFP4)
    return set_error(LPQ_ERR_UNSUPPORTED, "Hadamard transform and stochastic rounding apply to 1D NVFP4 only");
  if ((flags & LPQ_RHT_COLWISE) && !do_col)
    return set_error(LPQ_ERR_INVALID_ARG, "LPQ_RHT_COLWISE needs LPQ_COLWISE");
  if (counter_offset % 4) return set_error(LPQ_ERR_INVALID_ARG, "counter_offset must be a multiple of 4");
  const bool pt = is_fp8_pertensor(fmt);
  if (pt && scaling != LPQ_SCALING_CURRENT && scaling != LPQ_SCALING_DELAYED)
    return set_error(LPQ_ERR_INVALID_ARG, "scaling %d", scaling);
  if (!pt && scaling != LPQ_SCALING_CURRENT)
    return set_error(LPQ_ERR_UNSUPPORTED, "delayed scaling applies to per-tensor FP8 only");
  if ((flags & LPQ_GIVEN_AMAX) && !((pt && scaling == LPQ_SCALING_CURRENT) || is_nvfp4(fmt)))
    return set_error(LPQ_ERR_UNSUPPORTED, "LPQ_GIVEN_AMAX applies to current-scaled FP8 and NVFP4 only");
  if (pt && scaling == LPQ_SCALING_DELAYED) {
    if (!state || !state->scale || !state->scale_inv || !state->amax_history || !state->pos || state->len < 1 ||
        state->len > 1024)
      return set_error(LPQ_ERR_INVALID_ARG, "delayed scaling needs a complete state");
  }
  if (rows * cols > 0 && !x) return set_error(LPQ_ERR_INVALID_ARG, "x is NULL");
  if (!aligned16(x)) return set_error(LPQ_ERR_ALIGN, "x not 16-byte aligned");
  // shape rules
  if (cols % 16) return set_error(LPQ_ERR_SHAPE, "cols %lld not a multiple of 16", (long long)cols);
  const int64_t blk = row_block(fmt);
  if (blk && cols % blk) return set_error(LPQ_ERR_SHAPE, "cols %lld not a multiple of %lld", (long long)cols, (long long)blk);
  if (fmt == LPQ_NVFP4_2D && rows % 16) return set_error(LPQ_ERR_SHAPE, "NVFP4_2D needs rows % 16 == 0");
  if (do_col && rows % col_rows_multiple(fmt))
    return set_error(LPQ_ERR_SHAPE, "column-wise copy needs rows %% %lld == 0 (rows = %lld)",
                     (long long)col_rows_multiple(fmt), (long long)rows);
  const bool need_ts = pt || is_nvfp4(fmt);
  const bool need_amax = pt || is_nvfp4(fmt);
  lpq_status st;
  if (do_row && (st = check_view(&out->row, "out.row", fmt, rows, cols, 0, need_ts, need_amax)) != LPQ_OK) return st;
  if (do_col && (st = check_view(&out->col, "out.col", fmt, cols, rows, 1, need_ts, need_amax)) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  return launch_quantize(x, rows, cols, fmt, scaling, flags, seed, counter_offset, rht_seed, state, out,
                         reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_amax(const void* x, int64_t rows, int64_t cols, uint32_t flags, uint32_t rht_seed, float* amax,
                    float* rht_amax, lpq_stream_t stream) {
  if (flags & ~uint32_t(LPQ_RHT_COLWISE)) return set_error(LPQ_ERR_INVALID_ARG, "lpq_amax flags 0x%x", flags);
  const bool rht = flags & LPQ_RHT_COLWISE;
  if (!amax && !(rht && rht_amax)) return set_error(LPQ_ERR_INVALID_ARG, "no amax output");
  if (rht && !rht_amax) return set_error(LPQ_ERR_INVALID_ARG, "LPQ_RHT_COLWISE needs rht_amax");
  if (rows < 0 || cols < 0) return set_error(LPQ_ERR_SHAPE, "negative dimension");
  if (cols % 16) return set_error(LPQ_ERR_SHAPE, "cols %lld not a multiple of 16", (long long)cols);
  if (rht && rows % 16) return set_error(LPQ_ERR_SHAPE, "the RHT amax needs rows %% 16 == 0 (rows = %lld)", (long long)rows);
  if (rows * cols > 0 && !x) return set_error(LPQ_ERR_INVALID_ARG, "x is NULL");
  if (!aligned16(x)) return set_error(LPQ_ERR_ALIGN, "x not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(amax) & 3u) || (reinterpret_cast<uintptr_t>(rht_amax) & 3u))
    return set_error(LPQ_ERR_ALIGN, "amax outputs not 4-byte aligned");
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_amax(x, rows, cols, rht, rht_seed, amax, rht_amax, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_scale_update(const lpq_delayed_state* state, const float* amax, float fmax, lpq_stream_t stream) {
  if (!state || !amax || !state->scale || !state->scale_inv || !state->amax_history || !state->pos)
    return set_error(LPQ_ERR_INVALID_ARG, "NULL state or amax");
  if (state->len < 1 || state->len > 1024) return set_error(LPQ_ERR_INVALID_ARG, "history length %d", state->len);
  if (!(fmax > 0.f)) return set_error(LPQ_ERR_INVALID_ARG, "fmax must be positive");
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_scale_update(state, amax, fmax, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_gemm(int32_t layout, const lpq_qview* a, const lpq_qview* b, void* c, int32_t c_is_fp32, int64_t m,
                    int64_t n, int64_t k, lpq_stream_t stream) {
  return lpq_gemm_ex(layout, a, b, c, c_is_fp32, m, n, k, nullptr, stream);
}

lpq_status lpq_gemm_ex(int32_t layout, const lpq_qview* a, const lpq_qview* b, void* c, int32_t c_is_fp32, int64_t m,
                       int64_t n, int64_t k, const lpq_gemm_opts* opts, lpq_stream_t stream) {
  if (!a || !b) return set_error(LPQ_ERR_INVALID_ARG, "NULL operand");
  if (opts) {
    if (opts->single_cta < 0 || opts->single_cta > 1 || opts->scale_copies < 0 || opts->scale_copies > 1 ||
        opts->direct_store < 0 || opts->direct_store > 1 || opts->whole_tiles < 0 || opts->whole_tiles > 1 ||
        !(opts->tile_n == 0 || opts->tile_n == 128 || opts->tile_n == 256))
      return set_error(LPQ_ERR_INVALID_ARG,
                       "lpq_gemm_opts: single_cta, scale_copies, direct_store, whole_tiles 0/1; tile_n 0, 128 or 256");
    for (int i = 0; i < 3; ++i)
      if (opts->reserved[i]) return set_error(LPQ_ERR_INVALID_ARG, "lpq_gemm_opts.reserved must be 0");
  }
  if (layout < LPQ_FPROP || layout > LPQ_WGRAD) return set_error(LPQ_ERR_INVALID_ARG, "layout %d", layout);
  if (m < 0 || n < 0 || k < 0) return set_error(LPQ_ERR_SHAPE, "negative dimension");
  if (a->rows != m || a->cols != k) return set_error(LPQ_ERR_SHAPE, "a is %lld x %lld, expected m x k = %lld x %lld",
                                                     (long long)a->rows, (long long)a->cols, (long long)m, (long long)k);
  if (b->rows != n || b->cols != k) return set_error(LPQ_ERR_SHAPE, "b is %lld x %lld, expected n x k = %lld x %lld",
                                                     (long long)b->rows, (long long)b->cols, (long long)n, (long long)k);
  const int want_a = layout == LPQ_WGRAD ? 1 : 0, want_b = layout == LPQ_FPROP ? 0 : 1;
  if (a->colwise != want_a || b->colwise != want_b)
    return set_error(LPQ_ERR_INVALID_ARG, "layout %d reads a %s a and a %s b", layout, want_a ? "column-wise" : "row-wise",
                     want_b ? "column-wise" : "row-wise");
  const int32_t fa = a->fmt, fb = b->fmt;
  const bool pair_ok = (fa == LPQ_BF16 && fb == LPQ_BF16) || (is_fp8_pertensor(fa) && is_fp8_pertensor(fb)) ||
                       (is_mx8(fa) && is_mx8(fb)) || (fa == LPQ_MXFP4 && fb == LPQ_MXFP4) ||
                       (is_nvfp4(fa) && is_nvfp4(fb)) ||
                       (is_block(fa) && is_block(fb));
  if (!pair_ok) return set_error(LPQ_ERR_UNSUPPORTED, "no GEMM for the pairing %d x %d (no fallback)", fa, fb);
  const int64_t kmul = is_block(fa) ? 128 : 32;
  if (k % kmul) return set_error(LPQ_ERR_SHAPE, "k %lld not a multiple of %lld", (long long)k, (long long)kmul);
  if (m > 0 && n > 0) {
    if (!c) return set_error(LPQ_ERR_INVALID_ARG, "c is NULL");
    if (!aligned16(c)) return set_error(LPQ_ERR_ALIGN, "c not 16-byte aligned");
    if (k > 0) {
      for (const lpq_qview* v : {a, b}) {
        if (!v->codes) return set_error(LPQ_ERR_INVALID_ARG, "operand codes NULL");
        if (!aligned16(v->codes)) return set_error(LPQ_ERR_ALIGN, "operand codes not 16-byte aligned");
        if (is_u8_scaled(v->fmt)) {
          if (v->sf_layout != LPQ_SF_GEMM)
            return set_error(LPQ_ERR_INVALID_ARG, "block-scaled operands need LPQ_SF_GEMM scales");
          if (!v->scales || !aligned16(v->scales)) return set_error(LPQ_ERR_ALIGN, "operand scales NULL/unaligned");
        }
        if (is_block(v->fmt)) {
          if (v->sf_layout != LPQ_SF_GEMM)
            return set_error(LPQ_ERR_INVALID_ARG, "sub-channel operands need LPQ_SF_GEMM factors");
          if (!v->scales || (reinterpret_cast<uintptr_t>(v->scales) & 3u))
            return set_error(LPQ_ERR_ALIGN, "operand factors NULL/unaligned");
        }
        if ((is_fp8_pertensor(v->fmt) || is_nvfp4(v->fmt)) && !v->tensor_scale)
          return set_error(LPQ_ERR_INVALID_ARG, "operand tensor_scale NULL");
      }
    }
  }
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_gemm(a, b, c, c_is_fp32, m, n, k, opts, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool valid_type(int32_t t) { return t == LPQ_TYPE_BF16 || t == LPQ_TYPE_FP32; }
bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t type_bytes(int32_t t) { return t == LPQ_TYPE_FP32 ? 4 : 2; }

// What both directions of the norm check.
lpq_status check_norm(int32_t x_type, int32_t w_type, int64_t rows, int64_t cols) {
  if (!valid_type(x_type)) return set_error(LPQ_ERR_INVALID_ARG, "x_type %d", x_type);
  if (!valid_type(w_type)) return set_error(LPQ_ERR_INVALID_ARG, "w_type %d", w_type);
  if (rows < 0 || cols < 1) return set_error(LPQ_ERR_SHAPE, "layer norm of %lld x %lld", (long long)rows, (long long)cols);
  if (cols > (int64_t)1 << 30 || rows > (int64_t)1 << 40) return set_error(LPQ_ERR_SHAPE, "layer norm: too large");
  return LPQ_OK;
}
lpq_status check_matrix(const void* p, const char* name, int64_t ld, int64_t rows, int64_t cols, uintptr_t elem) {
  if (ld < cols) return set_error(LPQ_ERR_SHAPE, "%s: leading dimension %lld below %lld", name, (long long)ld, (long long)cols);
  if (rows > 0 && !p) return set_error(LPQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned_to(p, elem)) return set_error(LPQ_ERR_ALIGN, "%s not aligned to its elements", name);
  return LPQ_OK;
}

// What both directions of the vocabulary loss check.
lpq_status check_ce_shape(int64_t t, int64_t v, int64_t d) {
  if (t < 0 || v < 1) return set_error(LPQ_ERR_SHAPE, "t %lld, v %lld", (long long)t, (long long)v);
  if (d < 8 || d % 8) return set_error(LPQ_ERR_SHAPE, "d %lld not a positive multiple of 8", (long long)d);
  const int64_t most = (int64_t)1 << 30;
  if (t > most || v > most || d > most) return set_error(LPQ_ERR_SHAPE, "dimension beyond 2^30");
  return LPQ_OK;
}
lpq_status check_ce(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* labels, int64_t t,
                    int64_t v, int64_t d) {
  lpq_status st = check_ce_shape(t, v, d);
  if (st != LPQ_OK) return st;
  if (ldh < d || ldw < d || ldh % 8 || ldw % 8)
    return set_error(LPQ_ERR_SHAPE, "ldh %lld and ldw %lld must be multiples of 8, at least d = %lld", (long long)ldh,
                     (long long)ldw, (long long)d);
  if (ldh > (int64_t)1 << 38 || ldw > (int64_t)1 << 38) return set_error(LPQ_ERR_SHAPE, "leading dimension beyond 2^38");
  if ((t > 0 && (!h || !labels)) || !w) return set_error(LPQ_ERR_INVALID_ARG, "h, w or labels is NULL");
  if (!aligned16(h) || !aligned16(w)) return set_error(LPQ_ERR_ALIGN, "h or w not 16-byte aligned");
  if (!aligned_to(labels, 8)) return set_error(LPQ_ERR_ALIGN, "labels not 8-byte aligned");
  return LPQ_OK;
}
lpq_status check_piece(int64_t piece) {
  if (piece < 0 || piece % 64) return set_error(LPQ_ERR_SHAPE, "vocab_piece %lld not a multiple of 64", (long long)piece);
  return LPQ_OK;
}
lpq_status check_workspace(const void* ws, size_t have, size_t need) {
  if (have < need) return set_error(LPQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
  if (need > 0 && !ws) return set_error(LPQ_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned16(ws)) return set_error(LPQ_ERR_ALIGN, "workspace not 16-byte aligned");
  return LPQ_OK;
}
}  // namespace

lpq_status lpq_layer_norm(const void* x, int64_t ldx, int32_t x_type, const void* weight, const void* bias,
                          int32_t w_type, int64_t rows, int64_t cols, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, float* amax, lpq_stream_t stream) {
  lpq_status st = check_norm(x_type, w_type, rows, cols);
  if (st != LPQ_OK) return st;
  if (!(eps >= 0.f)) return set_error(LPQ_ERR_INVALID_ARG, "eps must be at least 0");
  if ((st = check_matrix(x, "x", ldx, rows, cols, type_bytes(x_type))) != LPQ_OK) return st;
  if ((st = check_matrix(y, "y", ldy, rows, cols, type_bytes(x_type))) != LPQ_OK) return st;
  if (!aligned_to(weight, type_bytes(w_type)) || !aligned_to(bias, type_bytes(w_type)))
    return set_error(LPQ_ERR_ALIGN, "weight or bias not aligned to its elements");
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(amax, 4))
    return set_error(LPQ_ERR_ALIGN, "mean, rstd or amax not 4-byte aligned");
  if ((st = check_arch()) != LPQ_OK) return st;
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.weight = weight; a.bias = bias; a.rows = rows; a.cols = cols; a.eps = eps;
  a.out = y; a.ldo = ldy; a.mean = mean; a.rstd = rstd; a.amax = amax;
  return launch_norm(a, x_type, w_type, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_layer_norm_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  lpq_status st = check_norm(LPQ_TYPE_BF16, LPQ_TYPE_BF16, rows, cols);
  if (st != LPQ_OK) return st;
  *bytes = (size_t)norm_parts(rows, cols) * 2 * (size_t)cols * sizeof(float);
  return LPQ_OK;
}

lpq_status lpq_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t x_type,
                                   const float* mean, const float* rstd, const void* weight, int32_t w_type,
                                   int64_t rows, int64_t cols, void* dx, int64_t lddx, float* dweight, float* dbias,
                                   void* workspace, size_t workspace_bytes, lpq_stream_t stream) {
  size_t need = 0;
  lpq_status st = check_norm(x_type, w_type, rows, cols);
  if (st != LPQ_OK) return st;
  if ((st = check_matrix(dy, "dy", lddy, rows, cols, type_bytes(x_type))) != LPQ_OK) return st;
  if ((st = check_matrix(x, "x", ldx, rows, cols, type_bytes(x_type))) != LPQ_OK) return st;
  if ((st = check_matrix(dx, "dx", lddx, rows, cols, type_bytes(x_type))) != LPQ_OK) return st;
  if (rows > 0 && (!mean || !rstd)) return set_error(LPQ_ERR_INVALID_ARG, "mean or rstd is NULL");
  if (!aligned_to(weight, type_bytes(w_type))) return set_error(LPQ_ERR_ALIGN, "weight not aligned to its elements");
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return set_error(LPQ_ERR_ALIGN, "mean, rstd, dweight or dbias not 4-byte aligned");
  if ((st = lpq_layer_norm_workspace(rows, cols, &need)) != LPQ_OK) return st;
  if (dweight || dbias)
    if ((st = check_workspace(workspace, workspace_bytes, need)) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  NormArgs a{};
  a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx; a.weight = weight; a.rows = rows; a.cols = cols;
  a.mean_in = mean; a.rstd_in = rstd; a.out = dx; a.ldo = lddx; a.dweight = dweight; a.dbias = dbias;
  a.parts = static_cast<float*>(workspace);
  return launch_norm_backward(a, x_type, w_type, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_linear_ce_workspace(int64_t t, int64_t v, int64_t d, int32_t backward, int64_t vocab_piece,
                                   size_t* bytes) {
  if (!bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  lpq_status st = check_ce_shape(t, v, d);
  if (st != LPQ_OK) return st;
  if ((st = check_piece(vocab_piece)) != LPQ_OK) return st;
  *bytes = ce_workspace(t, v, d, backward != 0, vocab_piece, backward == 2);
  return LPQ_OK;
}

lpq_status lpq_linear_ce(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* labels, int64_t t,
                         int64_t v, int64_t d, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                         lpq_stream_t stream) {
  lpq_status st = check_ce(h, ldh, w, ldw, labels, t, v, d);
  if (st != LPQ_OK) return st;
  if (t > 0 && (!loss || !lse)) return set_error(LPQ_ERR_INVALID_ARG, "loss or lse is NULL");
  if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return set_error(LPQ_ERR_ALIGN, "loss or lse not 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, ce_workspace(t, v, d, false, 0, false))) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  CeArgs a{};
  a.h = h; a.w = w; a.labels = labels; a.ldh = ldh; a.ldw = ldw; a.t = t; a.v = v; a.d = d;
  a.loss = loss; a.lse_out = lse; a.workspace = static_cast<uint8_t*>(workspace);
  return launch_ce(a, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_linear_ce_backward(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* labels,
                                  const float* lse, const float* dloss, int64_t t, int64_t v, int64_t d, void* dh,
                                  void* dw, int32_t grads_fp32, int64_t vocab_piece, void* workspace,
                                  size_t workspace_bytes, lpq_stream_t stream) {
  return lpq_linear_ce_backward_ex(h, ldh, w, ldw, labels, lse, dloss, t, v, d, dh, dw, grads_fp32, vocab_piece, workspace,
                                   workspace_bytes, nullptr, stream);
}

lpq_status lpq_linear_ce_backward_ex(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* labels,
                                     const float* lse, const float* dloss, int64_t t, int64_t v, int64_t d, void* dh,
                                     void* dw, int32_t grads_fp32, int64_t vocab_piece, void* workspace,
                                     size_t workspace_bytes, const lpq_ce_opts* opts, lpq_stream_t stream) {
  const lpq_ce_opts none{};
  if (!opts) opts = &none;
  lpq_status st = check_ce(h, ldh, w, ldw, labels, t, v, d);
  if (st != LPQ_OK) return st;
  if (opts->two_terms < 0 || opts->two_terms > 1) return set_error(LPQ_ERR_INVALID_ARG, "two_terms %d", opts->two_terms);
  for (int32_t r : opts->reserved)
    if (r) return set_error(LPQ_ERR_INVALID_ARG, "reserved option %d", r);
  if ((st = check_piece(vocab_piece)) != LPQ_OK) return st;
  if (grads_fp32 < 0 || grads_fp32 > 1) return set_error(LPQ_ERR_INVALID_ARG, "grads_fp32 %d", grads_fp32);
  if ((t > 0 && (!lse || !dloss || !dh)) || !dw) return set_error(LPQ_ERR_INVALID_ARG, "lse, dloss, dh or dw is NULL");
  if (!aligned_to(lse, 4) || !aligned_to(dloss, 4)) return set_error(LPQ_ERR_ALIGN, "lse or dloss not 4-byte aligned");
  if (!aligned16(dh) || !aligned16(dw)) return set_error(LPQ_ERR_ALIGN, "dh or dw not 16-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, ce_workspace(t, v, d, true, vocab_piece, opts->two_terms))) != LPQ_OK)
    return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  CeArgs a{};
  a.h = h; a.w = w; a.labels = labels; a.ldh = ldh; a.ldw = ldw; a.t = t; a.v = v; a.d = d;
  a.lse = lse; a.dloss = dloss; a.dh = dh; a.dw = dw; a.grads_fp32 = grads_fp32; a.piece = vocab_piece;
  a.two_terms = opts->two_terms;
  a.workspace = static_cast<uint8_t*>(workspace);
  return launch_ce_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
lpq_status check_matvec(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, const void* y, int32_t y_is_fp32) {
  if (!w) return set_error(LPQ_ERR_INVALID_ARG, "w is NULL");
  if (!(is_nvfp4(w->fmt) || w->fmt == LPQ_MXFP4))
    return set_error(LPQ_ERR_UNSUPPORTED, "lpq_matvec reads NVFP4, NVFP4_2D and MXFP4 weights, not format %d", w->fmt);
  if (w->colwise) return set_error(LPQ_ERR_INVALID_ARG, "lpq_matvec reads a row-wise copy");
  if (w->sf_layout != LPQ_SF_PLAIN && w->sf_layout != LPQ_SF_GEMM)
    return set_error(LPQ_ERR_INVALID_ARG, "w.sf_layout %d", w->sf_layout);
  if (y_is_fp32 < 0 || y_is_fp32 > 1) return set_error(LPQ_ERR_INVALID_ARG, "y_is_fp32 %d", y_is_fp32);
  if (m < 0 || w->rows < 0 || w->cols < 0) return set_error(LPQ_ERR_SHAPE, "negative dimension");
  if (w->cols % 32) return set_error(LPQ_ERR_SHAPE, "k %lld not a multiple of 32", (long long)w->cols);
  if (w->rows > (int64_t)1 << 30 || m > (int64_t)1 << 30) return set_error(LPQ_ERR_SHAPE, "dimension beyond 2^30");
  const int64_t most_k = (int64_t)1 << (w->sf_layout == LPQ_SF_PLAIN ? 16 : 19);
  if (w->cols > most_k) return set_error(LPQ_ERR_SHAPE, "k %lld beyond %lld", (long long)w->cols, (long long)most_k);
  if (m > 0 && w->cols > 0 && (ldx < w->cols || ldx % 8))
    return set_error(LPQ_ERR_SHAPE, "ldx %lld must be a multiple of 8, at least k = %lld", (long long)ldx, (long long)w->cols);
  if (m > 0 && w->rows > 0) {
    if (!y) return set_error(LPQ_ERR_INVALID_ARG, "y is NULL");
    if (!aligned16(y)) return set_error(LPQ_ERR_ALIGN, "y not 16-byte aligned");
    if (w->cols > 0) {
      if (!x || !w->codes || !w->scales) return set_error(LPQ_ERR_INVALID_ARG, "x, w.codes or w.scales is NULL");
      if (is_nvfp4(w->fmt) && !w->tensor_scale) return set_error(LPQ_ERR_INVALID_ARG, "w.tensor_scale is NULL");
      if (!aligned16(x) || !aligned16(w->codes)) return set_error(LPQ_ERR_ALIGN, "x or w.codes not 16-byte aligned");
      if (!aligned_to(w->scales, 4) || !aligned_to(w->tensor_scale, 4))
        return set_error(LPQ_ERR_ALIGN, "w.scales or w.tensor_scale not 4-byte aligned");
    }
  }
  return LPQ_OK;
}
}  // namespace

lpq_status lpq_matvec(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, void* y, int32_t y_is_fp32,
                      lpq_stream_t stream) {
  lpq_status st = check_matvec(w, x, ldx, m, y, y_is_fp32);
  if (st != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  return launch_matvec(w, x, ldx, m, y, y_is_fp32, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_matvec_adapted_workspace(int64_t m, int64_t rank, size_t* bytes) {
  if (!bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  if (m < 0 || m > (int64_t)1 << 30 || rank < 8 || rank > 256 || rank % 8)
    return set_error(LPQ_ERR_SHAPE, "m %lld, rank %lld (a multiple of 8, 8 to 256)", (long long)m, (long long)rank);
  *bytes = (size_t)m * (size_t)rank * sizeof(float);
  return LPQ_OK;
}

lpq_status lpq_matvec_adapted(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, void* y, int32_t y_is_fp32,
                              const lpq_adapters* adapters, const int64_t* index, void* workspace, size_t workspace_bytes,
                              lpq_stream_t stream) {
  lpq_status st = check_matvec(w, x, ldx, m, y, y_is_fp32);
  if (st != LPQ_OK) return st;
  if (!adapters) return set_error(LPQ_ERR_INVALID_ARG, "adapters is NULL");
  if (adapters->count < 0 || adapters->count > (int64_t)1 << 30) return set_error(LPQ_ERR_SHAPE, "adapters.count %lld", (long long)adapters->count);
  size_t need = 0;
  if ((st = lpq_matvec_adapted_workspace(m, adapters->rank, &need)) != LPQ_OK) return st;
  const bool any = m > 0 && w->rows > 0 && w->cols > 0 && adapters->count > 0;
  if (any && (!adapters->a || !adapters->b || !index)) return set_error(LPQ_ERR_INVALID_ARG, "adapters.a, adapters.b or index is NULL");
  if (!aligned16(adapters->a) || !aligned16(adapters->b)) return set_error(LPQ_ERR_ALIGN, "adapters.a or adapters.b not 16-byte aligned");
  if (!aligned_to(adapters->scale, 4)) return set_error(LPQ_ERR_ALIGN, "adapters.scale not 4-byte aligned");
  if (!aligned_to(index, 8)) return set_error(LPQ_ERR_ALIGN, "index not 8-byte aligned");
  if (any && (st = check_workspace(workspace, workspace_bytes, need)) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  AdapterArgs a{};
  a.a = adapters->a; a.b = adapters->b; a.scale = adapters->scale; a.index = index; a.count = adapters->count; a.rank = adapters->rank;
  a.inner = static_cast<float*>(workspace);
  return launch_matvec(w, x, ldx, m, y, y_is_fp32, any ? &a : nullptr, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_moe_route(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t m, int64_t d, int64_t experts, int64_t k,
                         int32_t renormalize, int64_t* ids, float* probs, lpq_stream_t stream) {
  if (renormalize < 0 || renormalize > 1) return set_error(LPQ_ERR_INVALID_ARG, "renormalize %d", renormalize);
  if (m < 0 || m > kRouteMostTokens) return set_error(LPQ_ERR_SHAPE, "m %lld", (long long)m);
  if (d < 8 || d % 8 || d > 65536) return set_error(LPQ_ERR_SHAPE, "d %lld not a multiple of 8, 8 to 65536", (long long)d);
  if (experts < 1 || experts > kMoeMostExperts) return set_error(LPQ_ERR_SHAPE, "experts %lld, at most %d", (long long)experts, kMoeMostExperts);
  if (k < 1 || k > kMoeMostChoices || k > experts)
    return set_error(LPQ_ERR_SHAPE, "k %lld of %lld experts, at most %d", (long long)k, (long long)experts, kMoeMostChoices);
  if (ldx < d || ldx % 8 || ldw < d || ldw % 8)
    return set_error(LPQ_ERR_SHAPE, "ldx %lld and ldw %lld must be multiples of 8, at least d = %lld", (long long)ldx, (long long)ldw, (long long)d);
  if (!w || (m > 0 && (!x || !ids || !probs))) return set_error(LPQ_ERR_INVALID_ARG, "x, w, ids or probs is NULL");
  if (!aligned16(x) || !aligned16(w)) return set_error(LPQ_ERR_ALIGN, "x or w not 16-byte aligned");
  if (!aligned_to(ids, 8) || !aligned_to(probs, 4)) return set_error(LPQ_ERR_ALIGN, "ids or probs not aligned to its elements");
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  RouteArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x); a.w = static_cast<const __nv_bfloat16*>(w); a.ldx = ldx; a.ldw = ldw; a.m = m;
  a.d = (int)d; a.experts = (int)experts; a.k = (int)k; a.renormalize = renormalize != 0; a.ids = ids; a.probs = probs;
  return launch_moe_route(a, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
lpq_status check_moe_shape(int64_t m, int64_t k, int64_t d, int64_t f) {
  const int64_t most = 65536;
  if (m < 0 || m > (int64_t)1 << 30) return set_error(LPQ_ERR_SHAPE, "m %lld", (long long)m);
  if (k < 0 || k > kMoeMostChoices) return set_error(LPQ_ERR_SHAPE, "k %lld, at most %d", (long long)k, kMoeMostChoices);
  if (d < 32 || d % 32 || d > most || f < 32 || f % 32 || f > most)
    return set_error(LPQ_ERR_SHAPE, "d %lld and f %lld must be multiples of 32, 32 to %lld", (long long)d, (long long)f, (long long)most);
  return LPQ_OK;
}
lpq_status check_experts(const lpq_qview* w, const char* name, int64_t rows) {
  if (!w) return set_error(LPQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!(is_nvfp4(w->fmt) || w->fmt == LPQ_MXFP4))
    return set_error(LPQ_ERR_UNSUPPORTED, "lpq_moe reads NVFP4, NVFP4_2D and MXFP4 weights, not format %d (%s)", w->fmt, name);
  if (w->sf_layout != LPQ_SF_GEMM) return set_error(LPQ_ERR_UNSUPPORTED, "lpq_moe reads LPQ_SF_GEMM scales (%s)", name);
  if (rows >= 0 && w->rows != rows)
    return set_error(LPQ_ERR_SHAPE, "%s has %lld rows, %lld expected", name, (long long)w->rows, (long long)rows);
  return check_view(w, name, w->fmt, w->rows, w->cols, 0, is_nvfp4(w->fmt), false);
}
}  // namespace

lpq_status lpq_moe_workspace(int64_t m, int64_t k, int64_t d, int64_t f, size_t* bytes) {
  if (!bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  lpq_status st = check_moe_shape(m, k, d, f);
  if (st != LPQ_OK) return st;
  *bytes = moe_workspace(m, k, d, f);
  return LPQ_OK;
}

lpq_status lpq_moe(const lpq_qview* up, const lpq_qview* down, int64_t experts, const void* x, int64_t ldx, int64_t m,
                   const int64_t* ids, const float* probs, int64_t k, void* y, void* workspace, size_t workspace_bytes,
                   lpq_stream_t stream) {
  if (!up || !down) return set_error(LPQ_ERR_INVALID_ARG, "up or down is NULL");
  const int64_t d = up->cols, f = down->cols;
  lpq_status st = check_moe_shape(m, k, d, f);
  if (st != LPQ_OK) return st;
  if (experts < 1 || experts > kMoeMostExperts) return set_error(LPQ_ERR_SHAPE, "experts %lld, at most %d", (long long)experts, kMoeMostExperts);
  if ((st = check_experts(up, "up", experts * 2 * f)) != LPQ_OK) return st;
  if ((st = check_experts(down, "down", experts * d)) != LPQ_OK) return st;
  if (ldx < d || ldx % 8) return set_error(LPQ_ERR_SHAPE, "ldx %lld must be a multiple of 8, at least d = %lld", (long long)ldx, (long long)d);
  if (m > 0 && (!x || !y || (k > 0 && (!ids || !probs)))) return set_error(LPQ_ERR_INVALID_ARG, "x, y, ids or probs is NULL");
  if (!aligned16(x)) return set_error(LPQ_ERR_ALIGN, "x not 16-byte aligned");
  if (!aligned_to(y, 2) || !aligned_to(ids, 8) || !aligned_to(probs, 4) || !aligned_to(up->tensor_scale, 4) || !aligned_to(down->tensor_scale, 4))
    return set_error(LPQ_ERR_ALIGN, "y, ids, probs or a tensor_scale not aligned to its elements");
  if (m > 0 && (st = check_workspace(workspace, workspace_bytes, moe_workspace(m, k, d, f))) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  MoeArgs a{};
  a.up = up; a.down = down; a.x = x; a.ldx = ldx; a.m = m; a.experts = experts; a.top = k; a.ids = ids; a.probs = probs; a.y = y;
  a.workspace = static_cast<uint8_t*>(workspace);
  return launch_moe(a, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
// What both directions of the head norm check; fills the shared arguments.
lpq_status check_qk(QkArgs& a, const void* x, int64_t ldx, int32_t type, int64_t rows, int64_t q_heads, int64_t k_heads,
                    int64_t head_dim, const void* q_weight, const void* k_weight, int32_t w_type, const int64_t* positions,
                    const double* freqs, int64_t rotary_dim, int32_t interleaved, float eps) {
  if (!valid_type(type)) return set_error(LPQ_ERR_INVALID_ARG, "type %d", type);
  if (!valid_type(w_type)) return set_error(LPQ_ERR_INVALID_ARG, "w_type %d", w_type);
  if (interleaved < 0 || interleaved > 1) return set_error(LPQ_ERR_INVALID_ARG, "interleaved %d", interleaved);
  if (!(eps >= 0.f)) return set_error(LPQ_ERR_INVALID_ARG, "eps must be at least 0");
  if (head_dim < 2 || head_dim > kQkMaxDim || head_dim % 2)
    return set_error(LPQ_ERR_SHAPE, "head_dim %lld must be even, 2 to %d", (long long)head_dim, kQkMaxDim);
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2)
    return set_error(LPQ_ERR_SHAPE, "rotary_dim %lld must be even, 0 to head_dim", (long long)rotary_dim);
  const int64_t most = (int64_t)1 << 20;
  if (rows < 0 || q_heads < 0 || k_heads < 0 || rows > (int64_t)1 << 30 || q_heads > most || k_heads > most)
    return set_error(LPQ_ERR_SHAPE, "rows %lld, heads %lld and %lld", (long long)rows, (long long)q_heads, (long long)k_heads);
  const int64_t cols = (q_heads + k_heads) * head_dim;
  lpq_status st = check_matrix(cols ? x : &a, "x", ldx, rows, cols, type_bytes(type));
  if (st != LPQ_OK) return st;
  if (!aligned_to(q_weight, type_bytes(w_type)) || !aligned_to(k_weight, type_bytes(w_type)))
    return set_error(LPQ_ERR_ALIGN, "q_weight or k_weight not aligned to its elements");
  if (rows > 0 && cols > 0 && !positions) return set_error(LPQ_ERR_INVALID_ARG, "positions is NULL");
  if (!aligned_to(positions, 8)) return set_error(LPQ_ERR_ALIGN, "positions not 8-byte aligned");
  if (rotary_dim > 0 && !freqs) return set_error(LPQ_ERR_INVALID_ARG, "freqs is NULL");
  for (int64_t i = 0; i < rotary_dim / 2; ++i)
    if (!(freqs[i] - freqs[i] == 0)) return set_error(LPQ_ERR_INVALID_ARG, "freqs[%lld] is not finite", (long long)i);
  a.x = x; a.ldx = ldx; a.rows = rows; a.q_heads = (int)q_heads; a.k_heads = (int)k_heads; a.dim = (int)head_dim;
  a.q_weight = q_weight; a.k_weight = k_weight; a.w_type = w_type; a.positions = positions; a.freqs = freqs;
  a.rotary = (int)rotary_dim; a.neighbours = interleaved != 0; a.eps = eps;
  return LPQ_OK;
}
}  // namespace

lpq_status lpq_qk_norm_rope(const void* x, int64_t ldx, int32_t type, int64_t rows, int64_t q_heads, int64_t k_heads,
                            int64_t head_dim, const void* q_weight, const void* k_weight, int32_t w_type,
                            const int64_t* positions, const double* freqs, int64_t rotary_dim, int32_t interleaved, float eps,
                            void* y, int64_t ldy, lpq_stream_t stream) {
  QkArgs a{};
  lpq_status st = check_qk(a, x, ldx, type, rows, q_heads, k_heads, head_dim, q_weight, k_weight, w_type, positions, freqs,
                           rotary_dim, interleaved, eps);
  if (st != LPQ_OK) return st;
  const int64_t cols = (q_heads + k_heads) * head_dim;
  if ((st = check_matrix(cols ? y : &a, "y", ldy, rows, cols, type_bytes(type))) != LPQ_OK) return st;
  if (y == x && ldy != ldx && rows > 1 && cols > 0) return set_error(LPQ_ERR_SHAPE, "y in x's place needs x's leading dimension");
  if ((st = check_arch()) != LPQ_OK) return st;
  a.out = y; a.ldo = ldy;
  return launch_qk_norm(a, type, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_qk_norm_rope_workspace(int64_t rows, int64_t head_dim, size_t* bytes) {
  if (!bytes) return set_error(LPQ_ERR_INVALID_ARG, "NULL output pointer");
  if (rows < 0 || head_dim < 2 || head_dim > kQkMaxDim)
    return set_error(LPQ_ERR_SHAPE, "rows %lld, head_dim %lld", (long long)rows, (long long)head_dim);
  *bytes = qk_norm_workspace(rows, head_dim);
  return LPQ_OK;
}

lpq_status lpq_qk_norm_rope_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t type, int64_t rows,
                                     int64_t q_heads, int64_t k_heads, int64_t head_dim, const void* q_weight,
                                     const void* k_weight, int32_t w_type, const int64_t* positions, const double* freqs,
                                     int64_t rotary_dim, int32_t interleaved, float eps, void* dx, int64_t lddx,
                                     float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                     lpq_stream_t stream) {
  QkArgs a{};
  lpq_status st = check_qk(a, x, ldx, type, rows, q_heads, k_heads, head_dim, q_weight, k_weight, w_type, positions, freqs,
                           rotary_dim, interleaved, eps);
  if (st != LPQ_OK) return st;
  const int64_t cols = (q_heads + k_heads) * head_dim;
  if ((st = check_matrix(cols ? dy : &a, "dy", lddy, rows, cols, type_bytes(type))) != LPQ_OK) return st;
  if ((st = check_matrix(cols ? dx : &a, "dx", lddx, rows, cols, type_bytes(type))) != LPQ_OK) return st;
  if (rows > 1 && cols > 0 && ((dx == x && lddx != ldx) || (dx == dy && lddx != lddy)))
    return set_error(LPQ_ERR_SHAPE, "dx in another's place needs its leading dimension");
  if (!aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4))
    return set_error(LPQ_ERR_ALIGN, "dq_weight or dk_weight not 4-byte aligned");
  if (dq_weight || dk_weight)
    if ((st = check_workspace(workspace, workspace_bytes, qk_norm_workspace(rows, head_dim))) != LPQ_OK) return st;
  if ((st = check_arch()) != LPQ_OK) return st;
  a.dy = dy; a.lddy = lddy; a.out = dx; a.ldo = lddx; a.dq_weight = dq_weight; a.dk_weight = dk_weight;
  a.parts = static_cast<float*>(workspace);
  return launch_qk_norm_backward(a, type, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_adjust_logits(const void* logits, int64_t ld, int32_t type, int64_t rows, int64_t v,
                             const lpq_logit_controls* controls, void* out, int64_t ldo, lpq_stream_t stream) {
  if (!controls) return set_error(LPQ_ERR_INVALID_ARG, "controls is NULL");
  const lpq_logit_controls& c = *controls;
  if (!valid_type(type)) return set_error(LPQ_ERR_INVALID_ARG, "type %d", type);
  if (rows < 0 || v < 0 || rows > (int64_t)1 << 30 || v > (int64_t)1 << 30)
    return set_error(LPQ_ERR_SHAPE, "rows %lld, v %lld", (long long)rows, (long long)v);
  const bool any = rows > 0 && v > 0;
  lpq_status st = check_matrix(any ? logits : &c, "logits", ld, rows, v, type_bytes(type));
  if (st != LPQ_OK) return st;
  if ((st = check_matrix(any ? out : &c, "out", ldo, rows, v, type_bytes(type))) != LPQ_OK) return st;
  if (out == logits && rows > 1 && v > 0 && ld != ldo) return set_error(LPQ_ERR_SHAPE, "out in the logits' place needs their leading dimension");
  if (c.history) {
    if (c.max_len < 0 || c.max_len > (int64_t)1 << 30 || c.ld_history < c.max_len)
      return set_error(LPQ_ERR_SHAPE, "history of %lld in rows of %lld", (long long)c.max_len, (long long)c.ld_history);
    if (!c.lengths) return set_error(LPQ_ERR_INVALID_ARG, "lengths is NULL");
  } else if (c.repetition || c.frequency || c.presence) {
    return set_error(LPQ_ERR_INVALID_ARG, "penalties without a history");
  }
  if (c.bias_words) {
    if (!c.bias_offsets || !c.bias_values) return set_error(LPQ_ERR_INVALID_ARG, "bias_offsets or bias_values is NULL");
    if (c.bias_count < 0) return set_error(LPQ_ERR_SHAPE, "bias_count %lld", (long long)c.bias_count);
  }
  if (c.allowed && c.ld_allowed < (v + 31) / 32)
    return set_error(LPQ_ERR_SHAPE, "ld_allowed %lld below %lld", (long long)c.ld_allowed, (long long)((v + 31) / 32));
  for (const void* p : {(const void*)c.history, (const void*)c.lengths, (const void*)c.prompt, (const void*)c.bias_offsets,
                        (const void*)c.bias_words})
    if (!aligned_to(p, 8)) return set_error(LPQ_ERR_ALIGN, "an int64 array is not 8-byte aligned");
  for (const void* p : {(const void*)c.repetition, (const void*)c.frequency, (const void*)c.presence, (const void*)c.bias_values,
                        (const void*)c.allowed})
    if (!aligned_to(p, 4)) return set_error(LPQ_ERR_ALIGN, "a 4-byte array is not 4-byte aligned");
  if ((st = check_arch()) != LPQ_OK) return st;
  LogitsArgs a{};
  a.logits = logits; a.out = out; a.ld = ld; a.ldo = ldo; a.rows = rows; a.v = v; a.c = c;
  if (!c.repetition && !c.frequency && !c.presence) a.c.history = nullptr;
  return launch_adjust_logits(a, type, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_layer_shapes(const lpq_transformer_cfg* cfg, lpq_gemm_shape out[12], int32_t* count) {
  if (!cfg || !out || !count) return set_error(LPQ_ERR_INVALID_ARG, "NULL argument");
  if (cfg->hidden <= 0 || cfg->intermediate <= 0 || cfg->micro_batch <= 0 || cfg->seq <= 0)
    return set_error(LPQ_ERR_SHAPE, "config dimensions must be positive");
  const int64_t M = cfg->micro_batch * cfg->seq;
  const int64_t h = cfg->hidden, f = cfg->intermediate;
  const struct {
    const char* name;
    int64_t k, n;
  } lin[4] = {{"qkv", h, 3 * h}, {"attn_out", h, h}, {"mlp_up", h, f}, {"mlp_down", f, h}};
  const char* pass[3] = {"fprop", "dgrad", "wgrad"};
  int i = 0;
  for (const auto& l : lin)
    for (int p = 0; p < 3; ++p, ++i) {
      lpq_gemm_shape& s = out[i];
      memset(&s, 0, sizeof(s));
      snprintf(s.name, sizeof(s.name), "%s_%s", l.name, pass[p]);
      s.layout = p;
      if (p == 0) { s.m = M; s.k = l.k; s.n = l.n; }
      else if (p == 1) { s.m = M; s.k = l.n; s.n = l.k; }
      else { s.m = l.n; s.k = M; s.n = l.k; }
    }
  *count = 12;
  return LPQ_OK;
}

lpq_status lpq_device_status(lpq_stream_t stream, int32_t* code) {
  if (!code) return set_error(LPQ_ERR_INVALID_ARG, "code is NULL");
  return read_and_clear_device_error(reinterpret_cast<cudaStream_t>(stream), code);
}

lpq_status lpq_selftest_wait(uint64_t limit_ns, lpq_stream_t stream) {
  if (limit_ns == 0 || limit_ns > kWaitLimitNs) return set_error(LPQ_ERR_INVALID_ARG, "limit_ns must be in (0, 1 s]");
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_selftest_wait(limit_ns, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_selftest_arith(int32_t which, uint64_t begin, uint64_t count, uint32_t param, int64_t* result,
                              lpq_stream_t stream) {
  if (which < 0 || which > 2) return set_error(LPQ_ERR_INVALID_ARG, "which %d", which);
  if (!result || (reinterpret_cast<uintptr_t>(result) & 7u)) return set_error(LPQ_ERR_INVALID_ARG, "result");
  const uint64_t limit = which == 0 ? 0x7F800001ull : which == 1 ? 8ull * 0x100000000ull : 1ull << 24;
  if (begin > limit || count > limit - begin) return set_error(LPQ_ERR_INVALID_ARG, "index range beyond %llu",
                                                               (unsigned long long)limit);
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_selftest_arith(which, begin, count, param, result, reinterpret_cast<cudaStream_t>(stream));
}

lpq_status lpq_mma_peak(int32_t kind, int32_t iters, int32_t with_scale_copies, lpq_stream_t stream) {
  if (kind < 0 || kind > 3) return set_error(LPQ_ERR_INVALID_ARG, "kind %d", kind);
  if (iters < 1 || iters > (1 << 24)) return set_error(LPQ_ERR_INVALID_ARG, "iters %d", iters);
  const bool ok_mode = (with_scale_copies >= 0 && with_scale_copies <= 1) ||
                       (with_scale_copies >= 2 && with_scale_copies <= 5 && kind == 3) || with_scale_copies == 6 ||
                       with_scale_copies == 8 ||
                       (with_scale_copies == 7 && (kind == 2 || kind == 3));
  if (!ok_mode) return set_error(LPQ_ERR_INVALID_ARG, "with_scale_copies %d for kind %d", with_scale_copies, kind);
  lpq_status st = check_arch();
  if (st != LPQ_OK) return st;
  return launch_mma_peak(kind, iters, with_scale_copies, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
