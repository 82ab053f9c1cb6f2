// Products of a few bf16 token rows with 4-bit weights and group scales.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kTokens = 8;  // tokens per pass over the weights

struct MatvecArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;
  const __nv_bfloat16* x;
  void* y;
  int64_t ldx;
  int64_t n, k, m;
  int64_t kt;  // scale atoms per 128-row group
  int gemm_layout, mx, y_fp32;
};

// FP32 value of a 4-bit code times its group scale (exact).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23) * (1.0f + 0.5f * (float)(m & 1u));
  return (code & 8u) ? -v : v;
}

// One warp per weight row.
__global__ void __launch_bounds__(256) matvec_row_kernel(const MatvecArgs g) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= g.n) return;
  const int blk = g.mx ? 32 : 16;
  for (int64_t m0 = 0; m0 < g.m; m0 += kTokens) {
    float acc[kTokens] = {};
    const int mm = (int)min((int64_t)kTokens, g.m - m0);
    for (int64_t b = lane; b < g.k / blk; b += 32) {
      const uint32_t sc = g.scales[g.gemm_layout ? sf_gemm_offset(row, b, g.kt) : row * (g.k / blk) + b];
      const float scale = g.mx ? (sc == 255u ? __int_as_float(0x7FC00000) : pow2_exact((int)sc - 127)) : e4m3_value(sc);
      const uint8_t* c = g.codes + row * (g.k / 2) + b * (blk / 2);
      for (int i = 0; i < blk; ++i) {
        const float wv = e2m1_value((c[i >> 1] >> (4 * (i & 1))) & 15u) * scale;
        for (int j = 0; j < mm; ++j) acc[j] += wv * __bfloat162float(g.x[(m0 + j) * g.ldx + b * blk + i]);
      }
    }
    for (int j = 0; j < mm; ++j) {
      float v = acc[j];
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (g.tensor_scale) v *= *g.tensor_scale;
      if (lane == 0) {
        const int64_t at = (m0 + j) * g.n + row;
        if (g.y_fp32) static_cast<float*>(g.y)[at] = v;
        else static_cast<__nv_bfloat16*>(g.y)[at] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace

lpq_status launch_matvec(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, void* y, int32_t y_is_fp32,
                         cudaStream_t s) {
  if (m == 0 || w->rows == 0) return LPQ_OK;
  if (w->cols == 0)  // empty reduction: y = 0
    return cuda_check(cudaMemsetAsync(y, 0, (size_t)m * (size_t)w->rows * (y_is_fp32 ? 4 : 2), s), "cudaMemsetAsync(y)");
  MatvecArgs g{};
  g.codes = static_cast<const uint8_t*>(w->codes);
  g.scales = static_cast<const uint8_t*>(w->scales);
  g.mx = w->fmt == LPQ_MXFP4;
  g.tensor_scale = g.mx ? nullptr : w->tensor_scale;
  g.x = static_cast<const __nv_bfloat16*>(x);
  g.y = y;
  g.ldx = ldx;
  g.n = w->rows;
  g.k = w->cols;
  g.m = m;
  g.kt = sf_kt_atoms(w->fmt, w->cols);
  g.gemm_layout = w->sf_layout == LPQ_SF_GEMM;
  g.y_fp32 = y_is_fp32;
  matvec_row_kernel<<<(unsigned)((g.n + 7) / 8), 256, 0, s>>>(g);
  return cuda_check(cudaGetLastError(), "matvec launch");
}

}  // namespace lpq
