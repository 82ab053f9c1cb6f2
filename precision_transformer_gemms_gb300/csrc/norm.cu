// Layer norm and its backward pass on sm_103a.
//
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps)
//   dx = rstd (g - sum(g) / n - xhat sum(g xhat) / n),  g = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// All sums are FP32; the variance is taken from the centred values (a second
// pass over the row), so a row's offset does not cancel its digits.
//
// HBM bounds both: one read and one write of the rows forward, two reads and one
// write backward.  Measured against the copy bandwidth of 6787 GB/s, bf16:
//   forward   15872 x 4096 42.4 us (90%), 65536 x 1024 46.6 us (85%), 8192 x 16384 82.4 us (96%)
//   backward  15872 x 4096 66.5 us (86%), 63488 x 4096 231 us (99%), 65536 x 1024 70 us (85%),
//             8192 x 16384 196 us (60%: two passes over the ring, one CTA per SM)
// What is left at 15872 x 4096 is the start and the end of a 40 us kernel, and
// backward the join of its 152 parts (5 us).  FP32 rows of 8193 to 16384 columns
// leave the backward ring room for one row, so that loads and work take turns:
// 4000 x 16384 90 us forward (86%), 164 us backward (71%).
//
// Unaligned rows go element by element, forward and up to 4096 columns backward
// with the next row loaded to registers while this one is worked on: 15872 x 4095
// bf16 79 us forward (49%), 115 us backward (50%), bound by the count of 2-byte
// loads; 15872 x 2047 FP32 45 us (85%) and 78 us (74%).  Wider ones are loaded
// backward when their turn comes, and beyond 8192 columns spill: 4000 x 8191 bf16
// 80 and 124 us (24%, 23%), FP32 51 and 214 (75%, 27%); 4000 x 16383 bf16 157 and
// 355 us (25%, 16%), FP32 236 and 498 (33%, 23%).
//
// Rows beyond 16384 columns are read again from the L2: 4096 x 32768 137 us
// forward (58%), 277 us backward (43%: the parameter gradients are a launch of
// their own).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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

__device__ __forceinline__ float load_param(const void* p, int w_fp32, int c) {
  return w_fp32 ? static_cast<const float*>(p)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The launch's max |y|: a single CTA stores it, several raise the value that
// was set to 0 before the launch.
__device__ __forceinline__ void store_amax(float* amax, float top) {
  __shared__ float sh[32];
  top = warp_max_xor(top, 32);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x < 32) {
    top = warp_max_xor(threadIdx.x < blockDim.x / 32 ? sh[threadIdx.x] : 0.f, 32);
    if (threadIdx.x == 0) {
      if (gridDim.x == 1) *amax = top; else atomic_max_nonneg(amax, top);
    }
  }
}

constexpr int kRowThreads = 512;

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

// Joins the parts: 32 columns per CTA, its 16 warps each summing every 16th
// part, then the 16 sums in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const float* parts, int nparts, int64_t cols,
                                                                    float* dweight, float* dbias) {
  __shared__ float sh[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int which = blockIdx.y;  // 0: dweight, 1: dbias
  float* out = which ? dbias : dweight;
  let_dependents_start();
  wait_for_stream();
  if (!out) return;
  float s = 0.f;
  if (c < cols) {
    const float* p = parts + which * cols + c;
#pragma unroll 10
    for (int i = warp; i < nparts; i += kJoinWarps) s += p[(int64_t)i * 2 * cols];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i) s += sh[i][lane];
    out[c] = s;
  }
}

// ------------------------------------------------------------------ rows in registers
// A row belongs to TPR threads, each holding NE of its elements in FP32; a CTA
// works on kBlock / TPR rows at a time and loops over the rest.  Vector form
// (16-byte aligned rows of whole 16-byte vectors): every thread streams its own
// vectors of the next rows through a ring in shared memory with cp.async, so
// that the loads in flight take no registers and need no barrier (a thread
// reads back only what it copied itself, and refills a slot after its values
// have entered a sum).  Scalar form: any alignment and length.

// The backward pass holds 120 registers a thread: one CTA of 512 threads per
// SM, whose row groups join their parameter gradients (152 parts to add up
// afterwards; with two CTAs of 256 threads, 304 parts, 68.2 us instead of
// 66.7 at 15872 x 4096 bf16).
template <int TPR, bool BACKWARD>
struct RowGroup {
  static constexpr int kBlock = BACKWARD ? 512 : TPR > 256 ? TPR : 256;
  static constexpr int kGroups = kBlock / TPR;
};

// Rows in flight for a ring stage of this many bytes.  Forward, with several
// CTAs per SM: two or three (four are slower: 182 us instead of 174 at 63488 x
// 4096 bf16).  Backward, one CTA per SM: four while they fit, down to one of FP32
// rows beyond 8192 columns.
template <bool BACKWARD>
constexpr int rows_ahead(int stage) {
  constexpr int most = BACKWARD ? 196608 : 24576;
  return BACKWARD && 4 * stage <= most ? 4 : 3 * stage <= most ? 3 : 2 * stage <= 200000 ? 2 : 1;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sums of the N values of v over the TPR threads of a row group.  `sh`
// alternates between two places from call to call, so one barrier is enough.
template <int TPR, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*sh)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (TPR > 32) {
    constexpr int kW = TPR / 32;
    const int w0 = (int)threadIdx.x / TPR * kW;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sh[i][threadIdx.x / 32] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
      if constexpr (kW >= 4) {
#pragma unroll
        for (int j = 0; j < kW; j += 4) {
          const float4 q = *reinterpret_cast<const float4*>(&sh[i][w0 + j]);
          s += (q.x + q.y) + (q.z + q.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kW; ++j) s += sh[i][w0 + j];
      }
      v[i] = s;
    }
  }
}

// s / n from the rounded 1 / n: the product and what it leaves out, s - q n, which
// one FMA gives exactly.  Without it a row of one value c would not have the mean
// c, and what is left of the row would not be 0 (a division: 42.5 -> 44.7 us at
// 15872 x 4096 bf16 and 23.9 -> 26.1 at 15872 x 1023).  An infinite sum stays one.
__device__ __forceinline__ float mean_of(float s, float n, float inv_n) {
  const float q = s * inv_n, mean = __fmaf_rn(__fmaf_rn(-q, n, s), inv_n, q);
  return fabsf(q) == __builtin_huge_valf() ? q : mean;
}

// Column of element i of thread `tid` of a row: vectors are dealt out in turn.
template <typename T, bool VEC, int TPR>
__device__ __forceinline__ int column_of(int tid, int i) {
  if constexpr (VEC) {
    constexpr int V = 16 / (int)sizeof(T);
    return ((i / V) * TPR + tid) * V + i % V;
  } else {
    return i * TPR + tid;
  }
}

__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

// 16 bytes <-> FP32 pairs (8 bf16 values or 4 floats).
template <typename T>
__device__ __forceinline__ void unpack_vector(const uint4& v, float2* f) {
  if constexpr (sizeof(T) == 2) {
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
  } else {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack_vector(const float2* f) {
  if constexpr (sizeof(T) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __float22bfloat162_rn(f[j]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  }
}

// 2 NP consecutive parameters from column c on (weight or bias, bf16 or FP32).
template <int NP>
__device__ __forceinline__ void load_params(const void* p, int w_fp32, int c, float2* f) {
  if (w_fp32) {
#pragma unroll
    for (int j = 0; j < NP; j += 2)
      unpack_vector<float>(__ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c + 2 * j)), f + j);
  } else if constexpr (NP == 4) {
    unpack_vector<__nv_bfloat16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c)), f);
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + c));
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
  }
}

// ------------------------------------------------------------------ rows beyond 16384 columns
// One CTA per row, in passes over it: the first from memory, the others mostly
// from the L2 (two CTAs an SM: 304 rows).  VEC: 16 bytes at a time.
template <typename T, bool VEC>
struct RowSpan {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, NP = VEC ? V / 2 : 1;  // elements, pairs (scalar: y = 0)
  static __device__ __forceinline__ void load(const T* p, int c, float2 (&f)[NP]) {
    if constexpr (VEC) unpack_vector<T>(*reinterpret_cast<const uint4*>(p + c), f);
    else f[0] = make_float2(to_f32(p[c]), 0.f);
  }
  static __device__ __forceinline__ void param(const void* p, int w_fp32, int c, float2 (&f)[NP], float none) {
    if (!p) {
#pragma unroll
      for (int j = 0; j < NP; ++j) f[j] = pair_of(none);
    } else if constexpr (VEC) {
      load_params<NP>(p, w_fp32, c, f);
    } else {
      f[0] = make_float2(load_param(p, w_fp32, c), 0.f);
    }
  }
  static __device__ __forceinline__ void store(T* p, int c, const float2 (&f)[NP]) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(p + c) = pack_vector<T>(f);
    else p[c] = from_f32<T>(f[0].x);
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) norm_row_kernel(const NormArgs a, int w_fp32) {
  using R = RowSpan<T, VEC>;
  __shared__ float sh[kRowThreads / 32];
  const int n = (int)a.cols;
  float top = 0.f;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.out) + r * a.ldo;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * R::V; c < n; c += kRowThreads * R::V) {
      float2 f[R::NP];
      R::load(x, c, f);
#pragma unroll
      for (int j = 0; j < R::NP; ++j) s += f[j].x + f[j].y;
    }
    const float mean = block_sum(s, sh) / (float)n;
    s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * R::V; c < n; c += kRowThreads * R::V) {
      float2 f[R::NP];
      R::load(x, c, f);
#pragma unroll
      for (int j = 0; j < R::NP; ++j) {
        const float dx = f[j].x - mean, dy = VEC ? f[j].y - mean : 0.f;
        s += dx * dx + dy * dy;
      }
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, sh) / (float)n + a.eps);
#pragma unroll 2
    for (int c = threadIdx.x * R::V; c < n; c += kRowThreads * R::V) {
      float2 f[R::NP], w[R::NP], b[R::NP];
      R::load(x, c, f);
      R::param(a.weight, w_fp32, c, w, 1.0f);
      R::param(a.bias, w_fp32, c, b, 0.0f);
#pragma unroll
      for (int j = 0; j < R::NP; ++j) {
        f[j] = make_float2((f[j].x - mean) * rstd * w[j].x + b[j].x, VEC ? (f[j].y - mean) * rstd * w[j].y + b[j].y : 0.f);
        top = absmax_acc(absmax_acc(top, to_f32(from_f32<T>(f[j].x))), to_f32(from_f32<T>(f[j].y)));
      }
      R::store(y, c, f);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
  if (a.amax) store_amax(a.amax, top);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) norm_dx_row_kernel(const NormArgs a, int w_fp32) {
  using R = RowSpan<T, VEC>;
  __shared__ float sh[kRowThreads / 32];
  const int n = (int)a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dx = static_cast<T*>(a.out) + r * a.ldo;
    const float mean = a.mean_in[r], rstd = a.rstd_in[r];
    float s1 = 0.f, s2 = 0.f;
    // xhat and g = dy w
    auto take = [&](int c, float2 (&xh)[R::NP], float2 (&g)[R::NP]) {
      float2 w[R::NP];
      R::load(x, c, xh);
      R::load(dy, c, g);
      R::param(a.weight, w_fp32, c, w, 1.0f);
#pragma unroll
      for (int j = 0; j < R::NP; ++j) {
        xh[j] = make_float2((xh[j].x - mean) * rstd, VEC ? (xh[j].y - mean) * rstd : 0.f);
        g[j] = make_float2(g[j].x * w[j].x, VEC ? g[j].y * w[j].y : 0.f);
      }
    };
#pragma unroll 2
    for (int c = threadIdx.x * R::V; c < n; c += kRowThreads * R::V) {
      float2 xh[R::NP], g[R::NP];
      take(c, xh, g);
#pragma unroll
      for (int j = 0; j < R::NP; ++j) {
        s1 += g[j].x + g[j].y;
        s2 += g[j].x * xh[j].x + g[j].y * xh[j].y;
      }
    }
    const float m1 = block_sum(s1, sh) / (float)n;
    const float m2 = block_sum(s2, sh) / (float)n;
#pragma unroll 2
    for (int c = threadIdx.x * R::V; c < n; c += kRowThreads * R::V) {
      float2 xh[R::NP], g[R::NP];
      take(c, xh, g);
#pragma unroll
      for (int j = 0; j < R::NP; ++j)
        g[j] = make_float2(rstd * (g[j].x - m1 - xh[j].x * m2), rstd * (g[j].y - m1 - xh[j].y * m2));
      R::store(dx, c, g);
    }
  }
}

// Part p of the parameter gradients: the rows p, p + parts, ...; a thread per
// column or 16 bytes of columns.
constexpr int kPartThreads = 128;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPartThreads) norm_parts_kernel(const NormArgs a, int parts) {
  using R = RowSpan<T, VEC>;
  const int64_t c = ((int64_t)blockIdx.x * kPartThreads + threadIdx.x) * R::V;
  if (c >= a.cols) return;
  const int p = blockIdx.y;
  float2 dw[R::NP] = {}, db[R::NP] = {};
#pragma unroll 4
  for (int64_t r = p; r < a.rows; r += parts) {
    float2 x[R::NP], dy[R::NP];
    R::load(static_cast<const T*>(a.x) + r * a.ldx, (int)c, x);
    R::load(static_cast<const T*>(a.dy) + r * a.lddy, (int)c, dy);
    const float mean = a.mean_in[r], rstd = a.rstd_in[r];
#pragma unroll
    for (int j = 0; j < R::NP; ++j) {
      dw[j].x += dy[j].x * ((x[j].x - mean) * rstd);
      dw[j].y += dy[j].y * ((x[j].y - mean) * rstd);
      db[j].x += dy[j].x;
      db[j].y += dy[j].y;
    }
  }
  float* to = a.parts + (int64_t)p * 2 * a.cols + c;
  auto put = [&](float* q, const float2 (&f)[R::NP]) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < R::NP; ++j) *reinterpret_cast<float2*>(q + 2 * j) = f[j];
    } else {
      q[0] = f[0].x;
    }
  };
  put(to, dw);
  put(to + a.cols, db);
}

// The parameters of a thread's vectors.  HELD (parameters of the rows' own
// type): kept as they are in registers over all rows; else read for each row
// (both would be 2 registers per element and cost resident warps).
template <typename T, int TPR, int NE, bool HELD>
struct Params {
  static constexpr int V = 16 / (int)sizeof(T), NV = NE / V;
  uint4 held[HELD ? NV : 1];
  const void* p;
  int w_fp32;
  __device__ __forceinline__ Params(const void* param, int fp32, int tid, int n, uint32_t fill) : p(param), w_fp32(fp32) {
    if constexpr (HELD) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        held[v] = make_uint4(fill, fill, fill, fill);
        if (p && c < n) held[v] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + c));
      }
    }
  }
  __device__ __forceinline__ void get(int v, int c, float2 (&f)[V / 2], float none) const {
    if constexpr (HELD) {
      unpack_vector<T>(held[v], f);
    } else if (p) {
      load_params<V / 2>(p, w_fp32, c, f);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) f[j] = pair_of(none);
    }
  }
};
// The same for the scalar form, in FP32.
template <int TPR, int NE, bool HELD>
struct ScalarParams {
  float held[HELD ? NE : 1];
  const void* p;
  int w_fp32;
  float none;
  __device__ __forceinline__ ScalarParams(const void* param, int fp32, int tid, int n, float fill) : p(param), w_fp32(fp32), none(fill) {
    if constexpr (HELD)
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = i * TPR + tid;
        held[i] = p && c < n ? load_param(p, w_fp32, c) : none;
      }
  }
  __device__ __forceinline__ float get(int i, int c) const {
    if constexpr (HELD) return held[i];
    return p ? load_param(p, w_fp32, c) : none;
  }
};
// 1.0 in every element of a register of T.
template <typename T>
constexpr uint32_t ones() { return sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u; }

// max of |values| of a stored vector, two bf16 values at a time (NaN ignored).
template <typename T>
__device__ __forceinline__ void absmax_vector(uint32_t& top, const uint4& q) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 2)
      asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %1;\n\tmax.bf16x2 %0, %0, t;\n\t}" : "+r"(top) : "r"(u[j]));
    else
      top = __float_as_uint(absmax_acc(__uint_as_float(top), __uint_as_float(u[j])));
  }
}
template <typename T>
__device__ __forceinline__ float absmax_value(uint32_t top) {
  if constexpr (sizeof(T) == 2) return fmaxf(bf16_lo(top), bf16_hi(top)); else return __uint_as_float(top);
}

// The elements of one row tensor of a thread as pairs, from its ring slot; 0
// past the row's end.
template <typename T, int TPR, int NE>
__device__ __forceinline__ void take_row(const uint4* slot, int stride, int tid, int n, float2 (&f)[NE / 2]) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int v = 0; v < NE / V; ++v) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (column_of<T, true, TPR>(tid, v * V) < n) q = slot[v * stride];
    unpack_vector<T>(q, f + v * V / 2);
  }
}
// Scalar form: the next row's elements, loaded while the row before is worked on.
template <typename T, bool VEC, int TPR, int NE>
struct NextRow {
  T raw[VEC ? 1 : NE];
  __device__ __forceinline__ void load(const T* row, bool there, int tid, int n) {
    if constexpr (!VEC)
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = i * TPR + tid;
        raw[i] = there && c < n ? row[c] : from_f32<T>(0.f);
      }
  }
  __device__ __forceinline__ void take(float2 (&f)[NE / 2]) const {
#pragma unroll
    for (int i = 0; i < NE; i += 2) f[i / 2] = make_float2(to_f32(raw[i]), to_f32(raw[i + 1]));
  }
};

// f(i, in): for the pairs of a thread, whether their elements lie in the row
// (a vector's all do or none; a scalar form's pair may be cut).
template <typename T, bool VEC, int TPR, int NE, typename F>
__device__ __forceinline__ void each_pair(int tid, int n, F f) {
  if constexpr (VEC) {
    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
    for (int v = 0; v < NE / V; ++v)
      if (column_of<T, true, TPR>(tid, v * V) < n)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) f(v * V / 2 + j, true, true);
  } else {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i)
      f(i, column_of<T, false, TPR>(tid, 2 * i) < n, column_of<T, false, TPR>(tid, 2 * i + 1) < n);
  }
}

template <typename T, bool VEC, bool HELD, int TPR, int NE>
__global__ void __launch_bounds__(RowGroup<TPR, false>::kBlock) norm_kernel(const NormArgs a, int w_fp32) {
  constexpr int kBlock = RowGroup<TPR, false>::kBlock, kGroups = RowGroup<TPR, false>::kGroups;
  constexpr int V = 16 / (int)sizeof(T), NV = NE / V;
  constexpr int kAhead = rows_ahead<false>(NV * 16 * kBlock);
  extern __shared__ uint4 ring[];  // [kAhead][NV][kBlock]
  __shared__ alignas(16) float sh[2][1][32];
  const int tid = threadIdx.x % TPR, n = (int)a.cols;
  const int64_t first = (int64_t)blockIdx.x * kGroups + threadIdx.x / TPR, step = (int64_t)gridDim.x * kGroups;
  const float inv_n = 1.0f / (float)n;
  let_dependents_start();
  wait_for_stream();
  // the row whose copy is next: its number and this thread's first vector
  int64_t ahead = first;
  const T* ahead_x = static_cast<const T*>(a.x) + first * a.ldx + tid * V;
  const int64_t x_step = step * a.ldx;
  auto copy = [&](int slot) {
    if constexpr (VEC) {
      if (ahead < a.rows) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (column_of<T, true, TPR>(tid, v * V) < n)
            cp_async16(&ring[(slot * NV + v) * kBlock + threadIdx.x], ahead_x + v * TPR * V);
      }
      ahead += step;
      ahead_x += x_step;
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) copy(s);
  constexpr bool kHeld = VEC && HELD;
  const Params<T, TPR, VEC ? NE : V, kHeld> weight(a.weight, w_fp32, tid, n, ones<T>()), bias(a.bias, w_fp32, tid, n, 0u);
  using Scalars = ScalarParams<TPR, VEC ? 1 : NE, (NE <= 16)>;
  const Scalars weight1(a.weight, w_fp32, tid, n, 1.0f), bias1(a.bias, w_fp32, tid, n, 0.0f);
  uint32_t top = 0;
  float top_scalar = 0.f;
  int slot = 0;
  NextRow<T, VEC, TPR, NE> next_x;
  next_x.load(static_cast<const T*>(a.x) + first * a.ldx, first < a.rows, tid, n);
  T* y = static_cast<T*>(a.out) + first * a.ldo;
  const int64_t y_step = step * a.ldo;
  for (int64_t r = first; r < a.rows; r += step, y += y_step) {
    float2 x[NE / 2];
    if constexpr (VEC) cp_async_wait<kAhead - 1>();
    if constexpr (VEC) {
      take_row<T, TPR, NE>(&ring[slot * NV * kBlock + threadIdx.x], kBlock, tid, n, x);
    } else {
      next_x.take(x);
      next_x.load(static_cast<const T*>(a.x) + (r + step) * a.ldx, r + step < a.rows, tid, n);
    }
    float2 s2 = pair_of(0.f);
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) s2 = __fadd2_rn(s2, x[i]);
    float s[1] = {s2.x + s2.y};
    group_sum<TPR, 1>(s, sh[0]);
    copy(slot);
    slot = (slot + 1) % kAhead;
    const float mean = mean_of(s[0], (float)n, inv_n);
    s2 = pair_of(0.f);
    each_pair<T, VEC, TPR, NE>(tid, n, [&](int i, bool in0, bool in1) {
      x[i] = __fadd2_rn(x[i], pair_of(-mean));
      if constexpr (!VEC) x[i] = make_float2(in0 ? x[i].x : 0.f, in1 ? x[i].y : 0.f);
      s2 = __ffma2_rn(x[i], x[i], s2);
    });
    s[0] = s2.x + s2.y;
    group_sum<TPR, 1>(s, sh[1]);
    const float rstd = 1.0f / sqrtf(s[0] * inv_n + a.eps);
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        if (c < n) {
          float2 w[V / 2], b[V / 2], o[V / 2];
          weight.get(v, c, w, 1.0f);
          bias.get(v, c, b, 0.0f);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) o[j] = __ffma2_rn(__fmul2_rn(x[v * V / 2 + j], pair_of(rstd)), w[j], b[j]);
          const uint4 q = pack_vector<T>(o);
          *reinterpret_cast<uint4*>(y + c) = q;
          if (a.amax) absmax_vector<T>(top, q);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = column_of<T, false, TPR>(tid, i);
        if (c < n) {
          const T q = from_f32<T>(__fmaf_rn((i & 1 ? x[i / 2].y : x[i / 2].x) * rstd, weight1.get(i, c), bias1.get(i, c)));
          y[c] = q;
          top_scalar = absmax_acc(top_scalar, to_f32(q));
        }
      }
    }
    if (tid == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
  if constexpr (VEC) cp_async_wait<0>();
  if (a.amax) store_amax(a.amax, VEC ? absmax_value<T>(top) : top_scalar);
}

// dx of each row; the parameter gradients' sums over this CTA's rows go to its
// part (a.parts [CTA][dweight, dbias][cols]), which norm_join_kernel adds up.
template <typename T, bool VEC, bool HELD, int TPR, int NE>
__global__ void __launch_bounds__(RowGroup<TPR, true>::kBlock, 1) norm_backward_kernel(const NormArgs a, int w_fp32) {
  constexpr int kBlock = RowGroup<TPR, true>::kBlock, kGroups = RowGroup<TPR, true>::kGroups;
  constexpr int V = 16 / (int)sizeof(T), NV = NE / V;
  constexpr int kAhead = rows_ahead<true>(2 * NV * 16 * kBlock);
  constexpr bool kAgain = VEC && NE > 16;
  extern __shared__ uint4 ring[];  // [kAhead][x, dy][NV][kBlock]
  __shared__ alignas(16) float sh[2][2][32];
  const int tid = threadIdx.x % TPR, n = (int)a.cols;
  const int64_t first = (int64_t)blockIdx.x * kGroups + threadIdx.x / TPR, step = (int64_t)gridDim.x * kGroups;
  const float inv_n = 1.0f / (float)n;
  let_dependents_start();
  wait_for_stream();
  // the row whose copy is next: its number and this thread's first vectors
  int64_t ahead = first;
  const T* ahead_x = static_cast<const T*>(a.x) + first * a.ldx + tid * V;
  const T* ahead_dy = static_cast<const T*>(a.dy) + first * a.lddy + tid * V;
  const int64_t x_step = step * a.ldx, dy_step = step * a.lddy;
  auto copy = [&](int slot) {
    if constexpr (VEC) {
      if (ahead < a.rows) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (column_of<T, true, TPR>(tid, v * V) < n) {
            cp_async16(&ring[(slot * 2 * NV + v) * kBlock + threadIdx.x], ahead_x + v * TPR * V);
            cp_async16(&ring[((slot * 2 + 1) * NV + v) * kBlock + threadIdx.x], ahead_dy + v * TPR * V);
          }
      }
      ahead += step;
      ahead_x += x_step;
      ahead_dy += dy_step;
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) copy(s);
  float2 dw[NE / 2], db[NE / 2];
#pragma unroll
  for (int i = 0; i < NE / 2; ++i) dw[i] = db[i] = pair_of(0.f);
  constexpr bool kHeld = VEC && HELD && !kAgain;
  const Params<T, TPR, VEC ? NE : V, kHeld> weight(a.weight, w_fp32, tid, n, ones<T>());
  int slot = 0, turn = 0;
  float mean = first < a.rows ? a.mean_in[first] : 0.f, rstd = first < a.rows ? a.rstd_in[first] : 0.f;
  const ScalarParams<TPR, VEC ? 1 : NE, (NE <= 8)> weight1(a.weight, w_fp32, tid, n, 1.0f);
  constexpr bool kNext = !VEC && NE <= 8;  // (wider threads have no registers for the next row)
  NextRow<T, !kNext, TPR, NE> next_x, next_dy;
  next_x.load(static_cast<const T*>(a.x) + first * a.ldx, first < a.rows, tid, n);
  next_dy.load(static_cast<const T*>(a.dy) + first * a.lddy, first < a.rows, tid, n);
  T* dx = static_cast<T*>(a.out) + first * a.ldo;
  const int64_t dx_step = step * a.ldo;
  for (int64_t r = first; r < a.rows; r += step, dx += dx_step) {
    // the next row's statistics are on their way while this row is worked on
    const int64_t rn = r + step < a.rows ? r + step : r;
    const float next_mean = a.mean_in[rn], next_rstd = a.rstd_in[rn];
    float2 x[NE / 2], g[NE / 2];
    if constexpr (VEC) cp_async_wait<kAhead - 1>();
    if constexpr (kAgain) {
      // 32 elements of x, dy and both gradients are more than a thread can
      // hold: the row's sums first, then its vectors once more from the ring
      float2 s0 = pair_of(0.f), s1 = pair_of(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        if (c < n) {
          float2 xv[V / 2], gv[V / 2], w[V / 2];
          unpack_vector<T>(ring[(slot * 2 * NV + v) * kBlock + threadIdx.x], xv);
          unpack_vector<T>(ring[((slot * 2 + 1) * NV + v) * kBlock + threadIdx.x], gv);
          weight.get(v, c, w, 1.0f);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            xv[j] = __fmul2_rn(__fadd2_rn(xv[j], pair_of(-mean)), pair_of(rstd));
            dw[v * V / 2 + j] = __ffma2_rn(gv[j], xv[j], dw[v * V / 2 + j]);
            db[v * V / 2 + j] = __fadd2_rn(db[v * V / 2 + j], gv[j]);
            gv[j] = __fmul2_rn(gv[j], w[j]);
            s0 = __fadd2_rn(s0, gv[j]);
            s1 = __ffma2_rn(gv[j], xv[j], s1);
          }
        }
      }
      float s[2] = {s0.x + s0.y, s1.x + s1.y};
      group_sum<TPR, 2>(s, sh[turn]);
      turn ^= 1;
      const float2 m1 = pair_of(-s[0] * inv_n), m2 = pair_of(-s[1] * inv_n);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        if (c < n) {
          float2 xv[V / 2], gv[V / 2], w[V / 2];
          unpack_vector<T>(ring[(slot * 2 * NV + v) * kBlock + threadIdx.x], xv);
          unpack_vector<T>(ring[((slot * 2 + 1) * NV + v) * kBlock + threadIdx.x], gv);
          weight.get(v, c, w, 1.0f);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            xv[j] = __fmul2_rn(__fadd2_rn(xv[j], pair_of(-mean)), pair_of(rstd));
            gv[j] = __fmul2_rn(__ffma2_rn(xv[j], m2, __ffma2_rn(gv[j], w[j], m1)), pair_of(rstd));
          }
          *reinterpret_cast<uint4*>(dx + c) = pack_vector<T>(gv);
        }
      }
      copy(slot);
      slot = (slot + 1) % kAhead;
      mean = next_mean;
      rstd = next_rstd;
      continue;
    }
    if constexpr (VEC) {
      take_row<T, TPR, NE>(&ring[slot * 2 * NV * kBlock + threadIdx.x], kBlock, tid, n, x);
      take_row<T, TPR, NE>(&ring[(slot * 2 + 1) * NV * kBlock + threadIdx.x], kBlock, tid, n, g);
    } else if constexpr (kNext) {
      next_x.take(x);
      next_dy.take(g);
      next_x.load(static_cast<const T*>(a.x) + rn * a.ldx, rn > r, tid, n);
      next_dy.load(static_cast<const T*>(a.dy) + rn * a.lddy, rn > r, tid, n);
    } else {
      NextRow<T, false, TPR, NE> row;
      row.load(static_cast<const T*>(a.x) + r * a.ldx, true, tid, n);
      row.take(x);
      row.load(static_cast<const T*>(a.dy) + r * a.lddy, true, tid, n);
      row.take(g);
    }
    // (past the row's end g is 0, and with it everything that x enters)
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
      x[i] = __fmul2_rn(__fadd2_rn(x[i], pair_of(-mean)), pair_of(rstd));
      if constexpr (!VEC)
        x[i] = make_float2(column_of<T, false, TPR>(tid, 2 * i) < n ? x[i].x : 0.f,
                           column_of<T, false, TPR>(tid, 2 * i + 1) < n ? x[i].y : 0.f);
      dw[i] = __ffma2_rn(g[i], x[i], dw[i]);
      db[i] = __fadd2_rn(db[i], g[i]);
    }
    float2 s0 = pair_of(0.f), s1 = pair_of(0.f);
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        if (c < n) {
          float2 w[V / 2];
          weight.get(v, c, w, 1.0f);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) g[v * V / 2 + j] = __fmul2_rn(g[v * V / 2 + j], w[j]);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            s0 = __fadd2_rn(s0, g[v * V / 2 + j]);
            s1 = __ffma2_rn(g[v * V / 2 + j], x[v * V / 2 + j], s1);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE / 2; ++i) {
        const int c = column_of<T, false, TPR>(tid, 2 * i), d = column_of<T, false, TPR>(tid, 2 * i + 1);
        if (c < n) g[i].x *= weight1.get(2 * i, c);
        if (d < n) g[i].y *= weight1.get(2 * i + 1, d);
        s0 = __fadd2_rn(s0, g[i]);
        s1 = __ffma2_rn(g[i], x[i], s1);
      }
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    group_sum<TPR, 2>(s, sh[turn]);
    turn ^= 1;
    copy(slot);
    slot = (slot + 1) % kAhead;
    const float2 m1 = pair_of(-s[0] * inv_n), m2 = pair_of(-s[1] * inv_n);
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = column_of<T, true, TPR>(tid, v * V);
        if (c < n) {
          float2 o[V / 2];
#pragma unroll
          for (int j = 0; j < V / 2; ++j)
            o[j] = __fmul2_rn(__ffma2_rn(x[v * V / 2 + j], m2, __fadd2_rn(g[v * V / 2 + j], m1)), pair_of(rstd));
          *reinterpret_cast<uint4*>(dx + c) = pack_vector<T>(o);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = column_of<T, false, TPR>(tid, i);
        const float gi = i & 1 ? g[i / 2].y : g[i / 2].x, xi = i & 1 ? x[i / 2].y : x[i / 2].x;
        if (c < n) dx[c] = from_f32<T>(rstd * __fmaf_rn(xi, m2.x, gi + m1.x));
      }
    }
    mean = next_mean;
    rstd = next_rstd;
  }
  if constexpr (VEC) cp_async_wait<0>();
  if (!a.parts) return;
  float* part = a.parts + (int64_t)blockIdx.x * 2 * n;
  // the CTA's row groups in order, through the ring's memory
  float* all = reinterpret_cast<float*>(ring);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float2 v = which ? db[i / 2] : dw[i / 2];
      all[(threadIdx.x / TPR) * TPR * NE + column_of<T, VEC, TPR>(tid, i)] = i & 1 ? v.y : v.x;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += kBlock) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kGroups; ++q) s += all[q * TPR * NE + c];
      part[(int64_t)which * n + c] = s;
    }
  }
}

// Whether rows can be read and written 16 bytes at a time.
bool vector_rows(const NormArgs& a, size_t elem, bool backward) {
  auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int64_t per = (int64_t)(16 / elem);
  if (a.cols % per || a.ldx % per || a.ldo % per || !ok(a.x) || !ok(a.out) || !ok(a.weight) || !ok(a.bias)) return false;
  return !backward || (ok(a.dy) && a.lddy % per == 0);
}

// amax = 0 before the CTAs of a launch raise it.  A kernel, and not a memset: the
// norm's kernel starts under it.
__global__ void clear_amax_kernel(float* amax) {
  let_dependents_start();
  wait_for_stream();
  *amax = 0.f;
}
lpq_status clear_amax(const NormArgs& a, int grid, cudaStream_t s) {
  if (!a.amax || grid == 1) return LPQ_OK;
  return cuda_check(launch_dependent(clear_amax_kernel, 1, 1, 0, s, a.amax), "layer norm amax launch");
}

template <typename T, bool VEC, bool HELD, int TPR, int NE>
lpq_status run_forward(const NormArgs& a, int w_fp32, cudaStream_t s) {
  constexpr int kBlock = RowGroup<TPR, false>::kBlock, kGroups = RowGroup<TPR, false>::kGroups;
  constexpr int kStage = NE * (int)sizeof(T) * kBlock, kSmem = VEC ? rows_ahead<false>(kStage) * kStage : 0;
  const void* kernel = reinterpret_cast<const void*>(norm_kernel<T, VEC, HELD, TPR, NE>);
  lpq_status st = set_smem_attr(kernel, kSmem);
  if (st != LPQ_OK) return st;
  const int64_t most = (int64_t)device_sms() * resident_ctas(kernel, kBlock, kSmem);
  const int grid = (int)std::min<int64_t>((a.rows + kGroups - 1) / kGroups, most);
  if ((st = clear_amax(a, grid, s)) != LPQ_OK) return st;
  return cuda_check(launch_dependent(norm_kernel<T, VEC, HELD, TPR, NE>, grid, kBlock, kSmem, s, a, w_fp32), "layer norm launch");
}

template <typename T, bool VEC, bool HELD, int TPR, int NE>
lpq_status run_backward(const NormArgs& a, int w_fp32, int& parts, cudaStream_t s) {
  constexpr int kBlock = RowGroup<TPR, true>::kBlock, kGroups = RowGroup<TPR, true>::kGroups;
  constexpr int kStage = 2 * NE * (int)sizeof(T) * kBlock, kRing = VEC ? rows_ahead<true>(kStage) * kStage : 0;
  constexpr int kJoin = kBlock * NE * 4;
  constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  lpq_status st = set_smem_attr(reinterpret_cast<const void*>(norm_backward_kernel<T, VEC, HELD, TPR, NE>), kSmem);
  if (st != LPQ_OK) return st;
  parts = (int)std::min<int64_t>((a.rows + kGroups - 1) / kGroups, norm_parts(a.rows, a.cols));
  return cuda_check(launch_dependent(norm_backward_kernel<T, VEC, HELD, TPR, NE>, parts, kBlock, kSmem, s, a, w_fp32),
                    "layer norm backward launch");
}

// Threads per row and elements per thread by width; beyond 16384 columns the
// rows are read from memory again.
// kFewer: half the threads, with 32 elements each, for 4097 to 8192 columns (bf16
// forward, where two CTAs then fit an SM: 15872 x 8192 104 -> 86 us).  kNarrow:
// 8 elements a thread up to 4096 columns (scalar backward, which then has
// registers for the next row: 15872 x 4095 248 -> 116 us).
enum { kUsual, kFewer, kNarrow };
template <int HOW, typename F>
lpq_status by_width(int64_t cols, F f) {
  using std::integral_constant;
  constexpr int K = HOW == kNarrow ? 2 : 1;
  if (cols <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (cols <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  if (cols <= 1024) return f(integral_constant<int, 64 * K>{}, integral_constant<int, 16 / K>{});
  if (cols <= 2048) return f(integral_constant<int, 128 * K>{}, integral_constant<int, 16 / K>{});
  if (cols <= 4096) return f(integral_constant<int, 256 * K>{}, integral_constant<int, 16 / K>{});
  if (cols <= 8192) return f(integral_constant<int, HOW == kFewer ? 256 : 512>{}, integral_constant<int, HOW == kFewer ? 32 : 16>{});
  return f(integral_constant<int, 512>{}, integral_constant<int, 32>{});
}

template <typename T>
lpq_status forward_t(const NormArgs& a, int w_fp32, cudaStream_t s) {
  if (a.cols <= 16384) {
    const bool vec = vector_rows(a, sizeof(T), false), held = (sizeof(T) == 4) == (w_fp32 != 0);
    return by_width<sizeof(T) == 2 ? kFewer : kUsual>(a.cols, [&](auto tpr, auto ne) {
      return !vec ? run_forward<T, false, false, tpr, ne>(a, w_fp32, s)
             : held ? run_forward<T, true, true, tpr, ne>(a, w_fp32, s) : run_forward<T, true, false, tpr, ne>(a, w_fp32, s);
    });
  }
  const int grid = (int)std::min<int64_t>(a.rows, (int64_t)device_sms() * 2);
  lpq_status st = clear_amax(a, grid, s);
  if (st != LPQ_OK) return st;
  (vector_rows(a, sizeof(T), false) ? norm_row_kernel<T, true> : norm_row_kernel<T, false>)<<<grid, kRowThreads, 0, s>>>(a, w_fp32);
  return cuda_check(cudaGetLastError(), "layer norm launch");
}

template <typename T>
lpq_status backward_t(NormArgs a, int w_fp32, cudaStream_t s) {
  int parts = 0;
  lpq_status st;
  if (!a.dweight && !a.dbias) a.parts = nullptr;
  if (a.cols <= 16384) {
    const bool vec = vector_rows(a, sizeof(T), true), held = (sizeof(T) == 4) == (w_fp32 != 0);
    if (vec)
      st = by_width<kUsual>(a.cols, [&](auto tpr, auto ne) {
        return held ? run_backward<T, true, true, tpr, ne>(a, w_fp32, parts, s)
                    : run_backward<T, true, false, tpr, ne>(a, w_fp32, parts, s);
      });
    else
      st = by_width<kNarrow>(a.cols, [&](auto tpr, auto ne) { return run_backward<T, false, false, tpr, ne>(a, w_fp32, parts, s); });
    if (st != LPQ_OK || !a.parts) return st;
  } else {
    const bool vec = vector_rows(a, sizeof(T), true);
    const int grid = (int)std::min<int64_t>(a.rows, (int64_t)device_sms() * 2);
    (vec ? norm_dx_row_kernel<T, true> : norm_dx_row_kernel<T, false>)<<<grid, kRowThreads, 0, s>>>(a, w_fp32);
    st = cuda_check(cudaGetLastError(), "layer norm backward launch");
    if (st != LPQ_OK || !a.parts) return st;
    parts = (int)norm_parts(a.rows, a.cols);
    const int64_t threads = a.cols / (vec ? 16 / (int)sizeof(T) : 1);
    const dim3 blocks((unsigned)((threads + kPartThreads - 1) / kPartThreads), (unsigned)parts);
    (vec ? norm_parts_kernel<T, true> : norm_parts_kernel<T, false>)<<<blocks, kPartThreads, 0, s>>>(a, parts);
    if ((st = cuda_check(cudaGetLastError(), "layer norm parts launch")) != LPQ_OK) return st;
  }
  return cuda_check(launch_dependent(norm_join_kernel, dim3((unsigned)((a.cols + 31) / 32), 2), 32 * kJoinWarps, 0, s,
                                     a.parts, parts, a.cols, a.dweight, a.dbias),
                    "layer norm join launch");
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
  return std::min<int64_t>({rows, 152, std::max<int64_t>(1, ((int64_t)1 << 24) / cols)});
}

lpq_status launch_norm(const NormArgs& a, int32_t x_type, int32_t w_type, cudaStream_t s) {
  if (a.rows == 0) return clear_amax(a, 0, s);
  const int w_fp32 = w_type == LPQ_TYPE_FP32;
  return x_type == LPQ_TYPE_BF16 ? forward_t<__nv_bfloat16>(a, w_fp32, s) : forward_t<float>(a, w_fp32, s);
}

lpq_status launch_norm_backward(const NormArgs& a, int32_t x_type, int32_t w_type, cudaStream_t s) {
  if (a.rows == 0) {
    lpq_status st = LPQ_OK;
    for (float* p : {a.dweight, a.dbias})
      if (p && (st = cuda_check(cudaMemsetAsync(p, 0, (size_t)a.cols * sizeof(float), s), "cudaMemsetAsync")) != LPQ_OK)
        return st;
    return LPQ_OK;
  }
  const int w_fp32 = w_type == LPQ_TYPE_FP32;
  return x_type == LPQ_TYPE_BF16 ? backward_t<__nv_bfloat16>(a, w_fp32, s) : backward_t<float>(a, w_fp32, s);
}

}  // namespace lpq
