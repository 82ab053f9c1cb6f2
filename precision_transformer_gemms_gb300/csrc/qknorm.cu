// RMS norm of every query and key head with the position rotation in the same
// pass, and its backward pass, on sm_103a.
//
//   n = x rstd w,  rstd = 1 / sqrt(sum(x^2) / D + eps)          per head of D values
//   y1 = n1 cos a - n2 sin a,  y2 = n2 cos a + n1 sin a          per pair, a = position * frequency
//   backward: g = dy turned by -a;  dw = sum over tokens and heads of g x rstd;
//   dx = rstd (g w - x rstd^2 sum(g w x) / D)
//
// HBM bounds both: one read and one write forward, two reads and one write
// backward.  A pair's two values lie in one thread, so the rotation needs no
// exchange: a thread holds V values of the first half and V of the second (or
// 2 V neighbours, where neighbours are turned together), and D / (2 V) lanes
// hold a head, whose sums take log2 of that many shuffles.  The statistics are
// taken again backward rather than kept: x is read anyway.
//
// The angle in turns is position * (frequency / 2 pi), of which only the
// fraction matters: as a 64-bit integer product modulo 2^64 that is exact but
// for the frequency's own rounding (2^-53 of it), so an angle at position 2^20
// is as near as one at 0.  cos and sin are taken once per token, thread and
// pair, and serve all heads that a warp takes of the token.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kWarps = 8;                    // per CTA
constexpr int kMaxPairs = kQkMaxDim / 2;

// Head groups on their way per warp in the vector form (1 or 2 KB each way, FP32
// twice that), and CTAs per SM.
template <typename T, bool BACKWARD>
struct Ring {
  static constexpr int kDepth = sizeof(T) == 4 ? 3 : 4;
  static constexpr int kPieces = 2 * 8 * sizeof(T) / 16 * (BACKWARD ? 2 : 1);  // 16-byte pieces of a lane
  static constexpr int kStage = kPieces * 512;
  static constexpr int kBytes = kWarps * kDepth * kStage;
  static constexpr int kCtas = BACKWARD ? 2 : 3;
};

struct QkKernelArgs {
  const void* x;
  const void* dy;
  void* out;
  int64_t ldx, lddy, ldo;
  const void* weight[2];  // of the query heads, of the key heads; NULL: 1
  const int64_t* positions;
  float* parts;  // backward: [CTA][2][D], or NULL
  int64_t rows;
  int64_t groups;  // of heads: tokens * (those of the queries and of the keys)
  int heads[2];    // query heads, key heads
  int runs[2];     // groups of 32 / lanes heads
  int dim, rotary;
  int lanes;       // that hold a head
  int w_fp32;
  float eps;
  uint64_t turns[kMaxPairs];  // frequency / 2 pi in units of 2^-64
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v; else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4) return v; else return __float2bfloat16_rn(v);
}

// V values as they lie in memory.
template <typename T, int V>
struct Raw {
  uint4 v[V * sizeof(T) / 16];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  // Through a lane's places in shared memory, 512 bytes apart.
  static __device__ __forceinline__ void copy(uint32_t to, const T* p, bool there) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 512), "l"(reinterpret_cast<const uint4*>(p) + i),
                   "r"(there ? 16 : 0) : "memory");
  }
  __device__ __forceinline__ void take(uint32_t from) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                   : "r"(from + i * 512) : "memory");
  }
  __device__ __forceinline__ float get(int i) const {  // i is a constant after unrolling
    if constexpr (sizeof(T) == 4) {
      const uint4& u = v[i >> 2];
      return __uint_as_float((i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w);
    } else {
      const uint4& u = v[i >> 3];
      const uint32_t p = ((i >> 1) & 3) == 0 ? u.x : ((i >> 1) & 3) == 1 ? u.y : ((i >> 1) & 3) == 2 ? u.z : u.w;
      return i & 1 ? bf16_hi(p) : bf16_lo(p);
    }
  }
  __device__ __forceinline__ void set2(int i, float a, float b) {  // values i and i + 1, i even
    uint4& u = v[sizeof(T) == 4 ? i >> 2 : i >> 3];
    if constexpr (sizeof(T) == 4) {
      if ((i & 3) == 0) { u.x = __float_as_uint(a); u.y = __float_as_uint(b); }
      else { u.z = __float_as_uint(a); u.w = __float_as_uint(b); }
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      const uint32_t p = *reinterpret_cast<const uint32_t*>(&h);
      if (((i >> 1) & 3) == 0) u.x = p; else if (((i >> 1) & 3) == 1) u.y = p; else if (((i >> 1) & 3) == 2) u.z = p; else u.w = p;
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
};

// A thread's part of a head: P pairs, as NU units of V pairs.  Vectors: V = 8,
// one unit.  Any alignment and sizes: V = 1, units 32 apart.
template <typename T, int V, int NU, bool NEIGHBOURS>
struct Slice {
  static constexpr int P = V * NU;
  Raw<T, V> a[NU], b[NU];

  // Offsets in a head of a unit's two halves; false: the thread holds no such unit.
  static __device__ __forceinline__ bool place(const QkKernelArgs& g, int lane, int j, int& at, int& bt) {
    const int u = lane + j * g.lanes;
    const int turned = g.rotary / (2 * V);
    if (NEIGHBOURS || u >= turned) {  // (values that are not turned lie side by side)
      at = u * 2 * V;
      bt = at + V;
    } else {
      at = u * V;
      bt = g.rotary / 2 + at;
    }
    return u * 2 * V < g.dim;
  }
  __device__ __forceinline__ void load(const QkKernelArgs& g, const T* head, int lane, bool there) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      int at, bt;
      if (place(g, lane, j, at, bt) && there) {
        a[j].load(head + at);
        b[j].load(head + bt);
      } else {
        a[j] = Raw<T, V>{};
        b[j] = Raw<T, V>{};
      }
    }
  }
  // The same through the ring (V > 1); `head` is any address of the tensor where nothing is there.
  static __device__ __forceinline__ void copy(const QkKernelArgs& g, uint32_t to, const T* head, int lane, bool there) {
    int at, bt;
    there = place(g, lane, 0, at, bt) && there;
    Raw<T, V>::copy(to, there ? head + at : head, there);
    Raw<T, V>::copy(to + V * sizeof(T) / 16 * 512, there ? head + bt : head, there);
  }
  __device__ __forceinline__ void take(uint32_t from) {
    a[0].take(from);
    b[0].take(from + V * sizeof(T) / 16 * 512);
  }
  // Pair i of the thread as its two values.
  __device__ __forceinline__ void pair(int i, float& p, float& q) const {
    const int j = i / V, k = i % V;
    if constexpr (V == 1) {
      p = to_f32(a[j].v);
      q = to_f32(b[j].v);
    } else if constexpr (NEIGHBOURS) {
      const Raw<T, V>& r = k < V / 2 ? a[j] : b[j];
      p = r.get(2 * k % V);
      q = r.get(2 * k % V + 1);
    } else {
      p = a[j].get(k);
      q = b[j].get(k);
    }
  }
  __device__ __forceinline__ void store(const QkKernelArgs& g, T* head, int lane, const float (&p)[P], const float (&q)[P]) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      int at, bt;
      if (!place(g, lane, j, at, bt)) continue;
      if constexpr (V == 1) {
        a[j].v = from_f32<T>(p[j]);
        b[j].v = from_f32<T>(q[j]);
      } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          if constexpr (NEIGHBOURS) {
            a[j].set2(k, p[k / 2], q[k / 2]);
            b[j].set2(k, p[V / 2 + k / 2], q[V / 2 + k / 2]);
          } else {
            a[j].set2(k, p[k], p[k + 1]);
            b[j].set2(k, q[k], q[k + 1]);
          }
        }
      }
      a[j].store(head + at);
      b[j].store(head + bt);
    }
  }
  // Places in the head of pair i's two values.
  static __device__ __forceinline__ bool where(const QkKernelArgs& g, int lane, int i, int& p, int& q) {
    int at, bt;
    const bool in = place(g, lane, i / V, at, bt);
    if (NEIGHBOURS && V > 1) {
      p = at + 2 * (i % V);
      q = p + 1;
    } else {
      p = at + i % V;
      q = bt + i % V;
    }
    return in;
  }
};

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A warp takes a run of the head groups (32 / lanes heads each), in token order.
template <typename T, int V, int NU, bool NEIGHBOURS, bool BACKWARD>
__global__ void __launch_bounds__(32 * kWarps, BACKWARD ? 2 : 3) qk_norm_kernel(const __grid_constant__ QkKernelArgs g) {
  using S = Slice<T, V, NU, NEIGHBOURS>;
  using R = Ring<T, BACKWARD>;
  constexpr int P = S::P;
  constexpr bool kRing = V > 1;
  extern __shared__ __align__(16) uint8_t smem[];
  float* sh = reinterpret_cast<float*>(smem + (kRing ? R::kBytes : 0));  // weights [2][dim]; backward, at the end: sums [warp][2][dim]
  __shared__ uint64_t turns[kMaxPairs];
  let_dependents_start();
  wait_for_stream();
  const int warp = threadIdx.x >> 5;
  const int lane = (threadIdx.x & 31) & (g.lanes - 1), sub = (threadIdx.x & 31) / g.lanes;
  for (int i = threadIdx.x; i < g.rotary / 2; i += 32 * kWarps) turns[i] = g.turns[i];
  for (int i = threadIdx.x; i < 2 * g.dim; i += 32 * kWarps) {
    const void* w = g.weight[i >= g.dim];
    const int c = i >= g.dim ? i - g.dim : i;
    sh[i] = !w ? 1.0f : g.w_fp32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  }
  __syncthreads();

  const int64_t workers = (int64_t)gridDim.x * kWarps, me = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t each = g.groups / workers, more = g.groups % workers;
  const int64_t begin = me * each + min(me, more), end = begin + each + (me < more);
  const int per_token = g.runs[0] + g.runs[1];
  const float inv_dim = 1.0f / (float)g.dim;
  const T* x = static_cast<const T*>(g.x);
  const T* dy = static_cast<const T*>(g.dy);
  T* out = static_cast<T*>(g.out);

  float cs[P], sn[P], wp[P], wq[P];
  float dwp[BACKWARD ? 2 : 1][P], dwq[BACKWARD ? 2 : 1][P];
  if constexpr (BACKWARD) {
#pragma unroll
    for (int i = 0; i < P; ++i) dwp[0][i] = dwp[1][i] = dwq[0][i] = dwq[1][i] = 0.f;
  }
  int64_t token = begin / per_token;
  int run = (int)(begin - token * per_token);
  // The head of a group that this thread's lanes take; false: the group has no such head.
  auto head_of = [&](int r, int& kind, int& head) {
    kind = r >= g.runs[0];
    head = (r - (kind ? g.runs[0] : 0)) * (32 / g.lanes) + sub;
    const bool there = head < g.heads[kind];
    head += kind ? g.heads[0] : 0;
    return there;
  };
  // The groups to come: in registers, or in the warp's ring (a lane reads back what it copied itself).
  S nx, ny;
  int64_t f_left = end - begin, f_token = token;
  int f_run = run;
  uint32_t f_at = 0, at = 0;
  const uint32_t ring = smem_u32(smem) + warp * (R::kDepth * R::kStage) + (threadIdx.x & 31) * 16;
  auto fetch = [&]() {
    if (f_left > 0) {
      --f_left;
      int kind, head;
      const bool there = head_of(f_run, kind, head);
      const T* px = x + f_token * g.ldx + (there ? (int64_t)head * g.dim : 0);
      const T* py = BACKWARD ? dy + f_token * g.lddy + (there ? (int64_t)head * g.dim : 0) : nullptr;
      if constexpr (kRing) {
        S::copy(g, ring + f_at, px, lane, there);
        if constexpr (BACKWARD) S::copy(g, ring + f_at + R::kStage / 2, py, lane, there);
      } else {
        nx.load(g, px, lane, there);
        if constexpr (BACKWARD) ny.load(g, py, lane, there);
      }
      if (++f_run == per_token) {
        f_run = 0;
        ++f_token;
      }
    }
    if constexpr (kRing) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      f_at = f_at == (R::kDepth - 1) * R::kStage ? 0 : f_at + R::kStage;
    }
  };
#pragma unroll
  for (int i = 0; i < (kRing ? R::kDepth : 1); ++i) fetch();
  int held = -1;  // the kind whose weights are in registers
  bool new_token = true;
  int64_t next_position = begin < end ? g.positions[token] : 0;
  for (int64_t i = begin; i < end; ++i) {
    if (new_token) {
      const int64_t position = next_position;
      if (token + 1 < g.rows) next_position = g.positions[token + 1];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int u = lane + (k / V) * g.lanes, f = u * V + k % V;
        cs[k] = 1.0f;
        sn[k] = 0.0f;
        if (f < g.rotary / 2) {
          const int32_t half_turns = (int32_t)((turns[f] * (uint64_t)position) >> 32);  // of 2^-31
          sincospif((float)half_turns * 4.65661287e-10f, &sn[k], &cs[k]);
        }
      }
    }
    int kind, head;
    const bool there = head_of(run, kind, head);
    if (kind != held) {
      held = kind;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        int p, q;
        const bool in = S::where(g, lane, k, p, q);
        wp[k] = in ? sh[kind * g.dim + p] : 0.f;
        wq[k] = in ? sh[kind * g.dim + q] : 0.f;
      }
    }
    S cx, cy;
    if constexpr (kRing) {
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
      cx.take(ring + at);
      if constexpr (BACKWARD) cy.take(ring + at + R::kStage / 2);
      at = at == (R::kDepth - 1) * R::kStage ? 0 : at + R::kStage;
    } else {
      cx = nx;
      if constexpr (BACKWARD) cy = ny;
      fetch();
    }
    const int64_t this_token = token;
    new_token = ++run == per_token;
    if (new_token) {
      run = 0;
      ++token;
    }

    float p[P], q[P];
    float square = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      cx.pair(k, p[k], q[k]);
      square = fmaf(p[k], p[k], square);
      square = fmaf(q[k], q[k], square);
    }
    T* to = out + this_token * g.ldo + (int64_t)head * g.dim;
    if constexpr (!BACKWARD) {
      const float rstd = __frsqrt_rn(fmaf(lanes_sum(square, g.lanes), inv_dim, g.eps));
      if constexpr (kRing) fetch();  // into the place whose values have entered the sum
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const float a = p[k] * rstd * wp[k], b = q[k] * rstd * wq[k];
        p[k] = fmaf(a, cs[k], -(b * sn[k]));
        q[k] = fmaf(b, cs[k], a * sn[k]);
      }
      if (there) cx.store(g, to, lane, p, q);
    } else {
      float gp[P], gq[P], dot = 0.f;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float u, v;
        cy.pair(k, u, v);
        gp[k] = fmaf(u, cs[k], v * sn[k]);
        gq[k] = fmaf(v, cs[k], -(u * sn[k]));
        dot = fmaf(gp[k] * wp[k], p[k], dot);
        dot = fmaf(gq[k] * wq[k], q[k], dot);
      }
      for (int o = g.lanes >> 1; o > 0; o >>= 1) {
        square += __shfl_xor_sync(0xFFFFFFFFu, square, o);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      }
      if constexpr (kRing) fetch();  // into the place whose values have entered the sums
      const float rstd = __frsqrt_rn(fmaf(square, inv_dim, g.eps));
      const float back = dot * inv_dim * rstd * rstd;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const float a = gp[k] * (p[k] * rstd), b = gq[k] * (q[k] * rstd);
        if (there) {
          if (kind == 0) {
            dwp[0][k] += a;
            dwq[0][k] += b;
          } else {
            dwp[1][k] += a;
            dwq[1][k] += b;
          }
        }
        p[k] = rstd * fmaf(gp[k], wp[k], -(p[k] * back));
        q[k] = rstd * fmaf(gq[k], wq[k], -(q[k] * back));
      }
      if (there) cx.store(g, to, lane, p, q);
    }
  }
  if constexpr (BACKWARD) {
    if (!g.parts) return;
    // the warp's groups of lanes, then the warps, in a fixed order
    if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float a = dwp[kind][k], b = dwq[kind][k];
        for (int o = 16; o >= g.lanes; o >>= 1) {
          a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
          b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        int pa, pb;
        if (S::where(g, lane, k, pa, pb) && sub == 0) {
          sh[(warp * 2 + kind) * g.dim + pa] = a;
          sh[(warp * 2 + kind) * g.dim + pb] = b;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.dim; i += 32 * kWarps) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sh[w * 2 * g.dim + i];
      g.parts[(int64_t)blockIdx.x * 2 * g.dim + i] = s;
    }
  }
}

// The weights' gradients: 32 values per CTA, its 16 warps each summing every
// 16th part, then the 16 sums in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps) qk_join_kernel(const float* parts, int nparts, int dim, float* dq, float* dk) {
  __shared__ float sh[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  let_dependents_start();
  wait_for_stream();
  float s = 0.f;
  if (c < 2 * dim) {
#pragma unroll 8
    for (int i = warp; i < nparts; i += kJoinWarps) s += parts[(int64_t)i * 2 * dim + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * dim) {
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i) s += sh[i][lane];
    float* out = c < dim ? dq : dk;
    if (out) out[c < dim ? c : c - dim] = s;
  }
}

// Most CTAs of the backward pass, each of which leaves a part of the weights' gradients.
int64_t most_parts() { return 2 * 160; }

template <typename T, int V, int NU, bool NEIGHBOURS, bool BACKWARD>
lpq_status run(QkKernelArgs& g, int64_t rows, float* dq, float* dk, cudaStream_t s) {
  const void* kernel = reinterpret_cast<const void*>(qk_norm_kernel<T, V, NU, NEIGHBOURS, BACKWARD>);
  const int units = (g.dim / 2 + V - 1) / V;
  g.lanes = 1;
  while (g.lanes < 32 && g.lanes < units) g.lanes *= 2;
  for (int i = 0; i < 2; ++i) g.runs[i] = (g.heads[i] * g.lanes + 31) / 32;
  g.groups = rows * (g.runs[0] + g.runs[1]);
  g.rows = rows;
  const int ring = V > 1 ? Ring<T, BACKWARD>::kBytes : 0;
  const int smem = ring + (BACKWARD ? kWarps : 1) * 2 * g.dim * (int)sizeof(float);
  lpq_status st = set_smem_attr(kernel, ring + (BACKWARD ? kWarps : 1) * 2 * kQkMaxDim * (int)sizeof(float));
  if (st != LPQ_OK) return st;
  int64_t most = (int64_t)device_sms() * std::max(1, std::min(Ring<T, BACKWARD>::kCtas, 226 * 1024 / (smem + 4 * 1024)));
  if (BACKWARD) most = std::min(most, most_parts());
  const int64_t grid = std::max<int64_t>(1, std::min(most, (g.groups + kWarps - 1) / kWarps));
  st = cuda_check(launch_dependent(qk_norm_kernel<T, V, NU, NEIGHBOURS, BACKWARD>, dim3((unsigned)grid), dim3(32 * kWarps), smem, s, g),
                  BACKWARD ? "qk norm backward launch" : "qk norm launch");
  if (st != LPQ_OK || !BACKWARD || !g.parts) return st;
  return cuda_check(launch_dependent(qk_join_kernel, dim3((2 * g.dim + 31) / 32), dim3(32 * kJoinWarps), 0, s, g.parts, (int)grid, g.dim,
                                     dq, dk),
                    "qk norm join launch");
}

template <typename T, bool BACKWARD>
lpq_status dispatch(QkKernelArgs& g, int64_t rows, bool neighbours, float* dq, float* dk, cudaStream_t s) {
  auto whole = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * sizeof(T) % 16 == 0; };
  if (g.dim % 16 == 0 && g.rotary % 16 == 0 && whole(g.x, g.ldx) && whole(g.out, g.ldo) && (!BACKWARD || whole(g.dy, g.lddy)))
    return neighbours ? run<T, 8, 1, true, BACKWARD>(g, rows, dq, dk, s) : run<T, 8, 1, false, BACKWARD>(g, rows, dq, dk, s);
  // value by value
  if (g.dim <= 64) return neighbours ? run<T, 1, 1, true, BACKWARD>(g, rows, dq, dk, s) : run<T, 1, 1, false, BACKWARD>(g, rows, dq, dk, s);
  if (g.dim <= 128) return neighbours ? run<T, 1, 2, true, BACKWARD>(g, rows, dq, dk, s) : run<T, 1, 2, false, BACKWARD>(g, rows, dq, dk, s);
  if (g.dim <= 256) return neighbours ? run<T, 1, 4, true, BACKWARD>(g, rows, dq, dk, s) : run<T, 1, 4, false, BACKWARD>(g, rows, dq, dk, s);
  return neighbours ? run<T, 1, 8, true, BACKWARD>(g, rows, dq, dk, s) : run<T, 1, 8, false, BACKWARD>(g, rows, dq, dk, s);
}

QkKernelArgs kernel_args(const QkArgs& a) {
  QkKernelArgs g{};
  g.x = a.x; g.dy = a.dy; g.out = a.out;
  g.ldx = a.ldx; g.lddy = a.lddy; g.ldo = a.ldo;
  g.weight[0] = a.q_weight; g.weight[1] = a.k_weight;
  g.positions = a.positions;
  g.heads[0] = a.q_heads; g.heads[1] = a.k_heads;
  g.dim = a.dim; g.rotary = a.rotary;
  g.w_fp32 = a.w_type == LPQ_TYPE_FP32;
  g.eps = a.eps;
  g.parts = a.parts;
  for (int i = 0; i < a.rotary / 2; ++i) {
    double whole;  // (modf leaves the fraction with the value's sign)
    double turn = std::modf(a.freqs[i] * 0.15915494309189535, &whole);  // 1 / (2 pi)
    if (turn < 0) turn += 1.0;
    g.turns[i] = turn < 1.0 ? (uint64_t)std::ldexp(turn, 64) : 0;
  }
  return g;
}

}  // namespace

size_t qk_norm_workspace(int64_t rows, int64_t dim) { return rows > 0 ? (size_t)most_parts() * 2 * (size_t)dim * sizeof(float) : 0; }

lpq_status launch_qk_norm(const QkArgs& a, int32_t type, cudaStream_t s) {
  if (a.rows == 0 || a.q_heads + a.k_heads == 0) return LPQ_OK;
  QkKernelArgs g = kernel_args(a);
  return type == LPQ_TYPE_FP32 ? dispatch<float, false>(g, a.rows, a.neighbours, nullptr, nullptr, s)
                               : dispatch<__nv_bfloat16, false>(g, a.rows, a.neighbours, nullptr, nullptr, s);
}

lpq_status launch_qk_norm_backward(const QkArgs& a, int32_t type, cudaStream_t s) {
  if (a.rows == 0 || a.q_heads + a.k_heads == 0) {  // empty sums
    for (float* p : {a.dq_weight, a.dk_weight})
      if (p) {
        lpq_status st = cuda_check(cudaMemsetAsync(p, 0, (size_t)a.dim * sizeof(float), s), "cudaMemsetAsync(weight gradient)");
        if (st != LPQ_OK) return st;
      }
    return LPQ_OK;
  }
  QkKernelArgs g = kernel_args(a);
  if (!a.dq_weight && !a.dk_weight) g.parts = nullptr;
  return type == LPQ_TYPE_FP32 ? dispatch<float, true>(g, a.rows, a.neighbours, a.dq_weight, a.dk_weight, s)
                               : dispatch<__nv_bfloat16, true>(g, a.rows, a.neighbours, a.dq_weight, a.dk_weight, s);
}

}  // namespace lpq
