// Layer norm and its backward pass on sm_103a.
//
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps)
//   dx = rstd (g - sum(g) / n - xhat sum(g xhat) / n),  g = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// All sums are FP32; the variance is taken from the centred values (a second
// pass over the row), so a row's offset does not cancel its digits.
#include <cuda_bf16.h>

#include <algorithm>

#include "lpq_device.cuh"

namespace lpq {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v; else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4) return v; else return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

constexpr int kRowThreads = 256;

// Sum over the CTA, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = warp_sum(v);
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[warp] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) s += sh[i];
  return s;
}

// One CTA per row, element by element: any size, stride and alignment.
template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_row_kernel(const NormArgs a) {
  __shared__ float sh[kRowThreads / 32];
  const int n = (int)a.cols;
  const W* w = static_cast<const W*>(a.weight);
  const W* b = static_cast<const W*>(a.bias);
  float top = 0.f;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.out) + r * a.ldo;
    float s = 0.f;
    for (int i = threadIdx.x; i < n; i += kRowThreads) s += to_f32(x[i]);
    const float mean = block_sum(s, sh) / (float)n;
    s = 0.f;
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const float c = to_f32(x[i]) - mean;
      s += c * c;
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, sh) / (float)n + a.eps);
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const float c = (to_f32(x[i]) - mean) * rstd;
      const T o = from_f32<T>(c * (w ? to_f32(w[i]) : 1.0f) + (b ? to_f32(b[i]) : 0.0f));
      y[i] = o;
      top = absmax_acc(top, to_f32(o));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
  if (a.amax) {
    top = warp_max_xor(top, 32);
    if ((threadIdx.x & 31) == 0) atomic_max_nonneg(a.amax, top);
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_dx_row_kernel(const NormArgs a) {
  __shared__ float sh[kRowThreads / 32];
  const int n = (int)a.cols;
  const W* w = static_cast<const W*>(a.weight);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dx = static_cast<T*>(a.out) + r * a.ldo;
    const float mean = a.mean_in[r], rstd = a.rstd_in[r];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const float g = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.0f);
      s1 += g;
      s2 += g * ((to_f32(x[i]) - mean) * rstd);
    }
    const float m1 = block_sum(s1, sh) / (float)n;
    const float m2 = block_sum(s2, sh) / (float)n;
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const float g = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.0f);
      const float xh = (to_f32(x[i]) - mean) * rstd;
      dx[i] = from_f32<T>(rstd * (g - m1 - xh * m2));
    }
  }
}

// Part p of the parameter gradients: the rows p, p + parts, ...; one thread per column.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_parts_kernel(const NormArgs a, int parts) {
  const int64_t c = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (c >= a.cols) return;
  for (int p = blockIdx.y; p < parts; p += gridDim.y) {
    float dw = 0.f, db = 0.f;
    for (int64_t r = p; r < a.rows; r += parts) {
      const float dy = to_f32(static_cast<const T*>(a.dy)[r * a.lddy + c]);
      const float xh = (to_f32(static_cast<const T*>(a.x)[r * a.ldx + c]) - a.mean_in[r]) * a.rstd_in[r];
      dw += dy * xh;
      db += dy;
    }
    a.parts[(int64_t)p * 2 * a.cols + c] = dw;
    a.parts[((int64_t)p * 2 + 1) * a.cols + c] = db;
  }
}

// Joins the parts: 32 columns per CTA, its 8 warps each summing every eighth
// part, then the 8 sums in order.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* parts, int nparts, int64_t cols, float* dweight,
                                                        float* dbias) {
  __shared__ float sh[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int which = blockIdx.y;  // 0: dweight, 1: dbias
  float* out = which ? dbias : dweight;
  if (!out) return;
  float s = 0.f;
  if (c < cols)
    for (int p = warp; p < nparts; p += 8) s += parts[((int64_t)p * 2 + which) * cols + c];
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int i = 1; i < 8; ++i) s += sh[i][lane];
    out[c] = s;
  }
}

template <typename T, typename W>
lpq_status forward_t(const NormArgs& a, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(a.rows, (int64_t)device_sms() * 8);
  norm_row_kernel<T, W><<<grid, kRowThreads, 0, s>>>(a);
  return cuda_check(cudaGetLastError(), "layer norm launch");
}

template <typename T, typename W>
lpq_status backward_t(const NormArgs& a, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(a.rows, (int64_t)device_sms() * 8);
  norm_dx_row_kernel<T, W><<<grid, kRowThreads, 0, s>>>(a);
  lpq_status st = cuda_check(cudaGetLastError(), "layer norm backward launch");
  if (st != LPQ_OK || (!a.dweight && !a.dbias)) return st;
  const int parts = (int)norm_parts(a.rows, a.cols);
  norm_parts_kernel<T><<<dim3((unsigned)((a.cols + kRowThreads - 1) / kRowThreads), parts), kRowThreads, 0, s>>>(a, parts);
  if ((st = cuda_check(cudaGetLastError(), "layer norm parts launch")) != LPQ_OK) return st;
  norm_join_kernel<<<dim3((unsigned)((a.cols + 31) / 32), 2), 256, 0, s>>>(a.parts, parts, a.cols, a.dweight, a.dbias);
  return cuda_check(cudaGetLastError(), "layer norm join launch");
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
  return std::min<int64_t>({rows, 304, std::max<int64_t>(1, ((int64_t)1 << 24) / cols)});
}

lpq_status launch_norm(const NormArgs& a, int32_t x_type, int32_t w_type, cudaStream_t s) {
  if (a.amax) {
    lpq_status st = cuda_check(cudaMemsetAsync(a.amax, 0, sizeof(float), s), "cudaMemsetAsync(amax)");
    if (st != LPQ_OK) return st;
  }
  if (a.rows == 0) return LPQ_OK;
  if (x_type == LPQ_TYPE_BF16)
    return w_type == LPQ_TYPE_BF16 ? forward_t<__nv_bfloat16, __nv_bfloat16>(a, s) : forward_t<__nv_bfloat16, float>(a, s);
  return w_type == LPQ_TYPE_BF16 ? forward_t<float, __nv_bfloat16>(a, s) : forward_t<float, float>(a, s);
}

lpq_status launch_norm_backward(const NormArgs& a, int32_t x_type, int32_t w_type, cudaStream_t s) {
  if (a.rows == 0) {
    lpq_status st = LPQ_OK;
    for (float* p : {a.dweight, a.dbias})
      if (p && (st = cuda_check(cudaMemsetAsync(p, 0, (size_t)a.cols * sizeof(float), s), "cudaMemsetAsync")) != LPQ_OK)
        return st;
    return LPQ_OK;
  }
  if (x_type == LPQ_TYPE_BF16)
    return w_type == LPQ_TYPE_BF16 ? backward_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                   : backward_t<__nv_bfloat16, float>(a, s);
  return w_type == LPQ_TYPE_BF16 ? backward_t<float, __nv_bfloat16>(a, s) : backward_t<float, float>(a, s);
}

}  // namespace lpq
