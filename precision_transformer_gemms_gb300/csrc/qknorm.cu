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
// exchange: a thread holds 16-byte vectors from both halves of a head (or whole pairs,
// where neighbours are turned together), 8 pairs in all; D / 16 lanes hold a head,
// whose sums take log2 of that many shuffles.  Rows stream through per-lane rings of
// asynchronous copies; arithmetic is two-wide.  The statistics are taken again backward
// rather than kept: x is read anyway.
//
// The angle in turns is position * (frequency / 2 pi), of which only the fraction
// matters: an integer product modulo 2^96 takes the frequency's 53 bits whole, so that
// an angle at position 2^20 is as near as one at 0 but for the frequency's own rounding
// in turns (2^-52 of the angle) and 2^-33 turns.  cos and sin are taken once per token, shared by a warp's
// lanes, and serve all heads that the warp takes of the token.
//
// Measured against the copy bandwidth of 6677 GB/s, 15872 tokens, bf16 unless said:
//   forward   64 heads of 128 78.5 us (99%), of 64 78.2, 32 of 256 with 64 turned 79.5,
//             neighbours turned 78.6, 8192 tokens FP32 81.7 (98%), 32 + 8 heads of 128
//             54.6 (89%), 16 of 512 110 (71%)
//   backward  64 heads of 128 129 us (90%; 4 of it the join of the parts), of 64 132,
//             32 of 256 135, 8192 tokens FP32 154 (78%: a ring of two), 32 + 8 106 (69%)
// Heads that are no power of two times 16 leave lanes idle (96 of 80: 120 us, 61%).
// bf16 that goes in 8-byte vectors: 112 heads of 72 145 us (53%, backward 273), 96 of 80
// with halves of 20 turned 126 (value by value 348, 499 and 302).  What goes value by
// value (64 of 130: 260 us, 30%; backward 370, 32%) is bound by the count of accesses;
// beyond 256 values a head it spills, too (16 of 510 FP32 or bf16: 160 bytes a thread
// forward, 240 to 280 backward, 205 and 301 us at 8192 tokens).  The vector forms spill 16
// to 40 bytes a thread backward, those of 8 bytes 8 to 24 forward.
// Grouped heads lose more backward (40 + 0 heads 87 us, 84%; 24 + 16 92; 32 + 8 106; 36 +
// 4 123, 59%): warps have equal counts of head groups, and those with the keys set up a
// token's angles and weights for two groups, or one, where queries have eight.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "lpq_device.cuh"
#include "turns.h"

namespace lpq {
namespace {

constexpr int kWarps = 8;                    // per CTA
constexpr int kMaxPairs = kQkMaxDim / 2;

// Head groups on their way per warp in the vector form (1 or 2 KB each way, FP32
// twice that), and CTAs per SM.
template <typename T, bool BACKWARD>
struct Ring {
  static constexpr int kDepth = sizeof(T) == 4 ? (BACKWARD ? 2 : 3) : 4;
  static constexpr int kStage = 32 * 2 * 8 * sizeof(T) * (BACKWARD ? 2 : 1);  // 8 pairs a lane
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
  int rows;
  int64_t groups;  // of heads: tokens * (those of the queries and of the keys)
  int heads[2];    // query heads, key heads
  int runs[2];     // groups of 32 / lanes heads
  int dim, rotary;
  int lanes;       // that hold a head
  int neighbours;  // the pairs are neighbours
  int w_fp32;
  float eps;
  uint64_t turns[kMaxPairs];  // frequency / 2 pi: the words of Turns
  uint32_t low_turns[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v; else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4) return v; else return __float2bfloat16_rn(v);
}

// V values as they lie in memory: 16 bytes (8 of 4 bf16 values), or one value.
template <typename T, int V>
struct Raw {
  static constexpr int kBytes = V * sizeof(T);
  static_assert(kBytes == 16 || kBytes == 8, "a vector is 8 or 16 bytes");
  using Word = std::conditional_t<kBytes == 16, uint4, uint2>;
  Word v;
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Word*>(p) = v; }
  // Through a lane's place in shared memory.
  static __device__ __forceinline__ void copy(uint32_t to, const T* p, bool there) {
    if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(there ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(there ? 8 : 0) : "memory");
  }
  __device__ __forceinline__ void take(uint32_t from) {
    if constexpr (kBytes == 16)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
    else
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(from) : "memory");
  }
  // 32-bit word i (a constant after unrolling).
  __device__ __forceinline__ uint32_t& word(int i) {
    if constexpr (kBytes == 16) return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    else return i == 0 ? v.x : v.y;
  }
  __device__ __forceinline__ uint32_t word(int i) const { return const_cast<Raw*>(this)->word(i); }
  // Values 2 i and 2 i + 1.
  __device__ __forceinline__ float2 get2(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    else return make_float2(bf16_lo(word(i)), bf16_hi(word(i)));
  }
  __device__ __forceinline__ void set2(int i, float a, float b) {
    if constexpr (sizeof(T) == 4) {
      word(2 * i) = __float_as_uint(a);
      word(2 * i + 1) = __float_as_uint(b);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      word(i) = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
};

// A thread's part of a head: P pairs (even), as NU units of two vectors of V values.
// Neighbouring lanes' vectors are neighbours, so that a warp's accesses take whole
// sectors: the two vectors lie half a head apart, or half of the turned values, where
// the pairs are made of their halves.  Vectors hold 8 pairs a thread; any alignment and
// sizes: V = 1, units 32 apart.  Pairs 2 j and 2 j + 1 lie in one float2
// of firsts and one of seconds, for the two-wide operations.
template <typename T, int V, int NU, bool NEIGHBOURS>
struct Slice {
  static constexpr int P = V * NU;
  Raw<T, V> a[NU], b[NU];

  // Offsets in a head of unit j's two vectors; false: the thread holds no such unit.
  static __device__ __forceinline__ bool place(const QkKernelArgs& g, int lanes, int lane, int j, int& at, int& bt) {
    const int u = lane + j * lanes, turned = g.rotary / (2 * V);
    if (V == 1 && g.neighbours) {
      at = 2 * u;
      bt = at + 1;
    } else if (V > 1 && NEIGHBOURS) {
      at = u * V;
      bt = g.dim / 2 + at;
    } else if (u < turned) {
      at = u * V;
      bt = g.rotary / 2 + at;
    } else {
      at = g.rotary + (u - turned) * V;
      bt = at + (g.dim - g.rotary) / 2;
    }
    return u * 2 * V < g.dim;
  }
  // Places in the head of pair i's two values.
  static __device__ __forceinline__ bool where(const QkKernelArgs& g, int lanes, int lane, int i, int& p, int& q) {
    int at, bt;
    const bool in = place(g, lanes, lane, i / V, at, bt);
    const int k = i % V;
    if (NEIGHBOURS && V > 1) {
      p = k < V / 2 ? at + 2 * k : bt + 2 * k - V;
      q = p + 1;
    } else {
      p = at + k;
      q = bt + k;
    }
    return in;
  }
  // Which pair of the head that is, among those that are turned (beyond half of `rotary`: it is not).
  static __device__ __forceinline__ int turn_of(const QkKernelArgs& g, int lanes, int lane, int i) {
    if (NEIGHBOURS && V > 1) {
      int p, q;
      where(g, lanes, lane, i, p, q);
      return p / 2;
    }
    return (lane + i / V * lanes) * V + i % V;
  }
  __device__ __forceinline__ void values(float2 (&p)[P / 2], float2 (&q)[P / 2]) const {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (V == 1) {
        p[i] = make_float2(to_f32(a[2 * i].v), to_f32(a[2 * i + 1].v));
        q[i] = make_float2(to_f32(b[2 * i].v), to_f32(b[2 * i + 1].v));
      } else {
        const int j = i / (V / 2), k = i % (V / 2);
        if constexpr (NEIGHBOURS) {
          const Raw<T, V>& r = k < V / 4 ? a[j] : b[j];
          const float2 u = r.get2(2 * k % (V / 2)), v = r.get2(2 * k % (V / 2) + 1);
          p[i] = make_float2(u.x, v.x);
          q[i] = make_float2(u.y, v.y);
        } else {
          p[i] = a[j].get2(k);
          q[i] = b[j].get2(k);
        }
      }
    }
  }
  __device__ __forceinline__ void set(const float2 (&p)[P / 2], const float2 (&q)[P / 2]) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (V == 1) {
        a[2 * i].v = from_f32<T>(p[i].x);
        a[2 * i + 1].v = from_f32<T>(p[i].y);
        b[2 * i].v = from_f32<T>(q[i].x);
        b[2 * i + 1].v = from_f32<T>(q[i].y);
      } else {
        const int j = i / (V / 2), k = i % (V / 2);
        if constexpr (NEIGHBOURS) {
          Raw<T, V>& r = k < V / 4 ? a[j] : b[j];
          r.set2(2 * k % (V / 2), p[i].x, q[i].x);
          r.set2(2 * k % (V / 2) + 1, p[i].y, q[i].y);
        } else {
          a[j].set2(k, p[i].x, p[i].y);
          b[j].set2(k, q[i].x, q[i].y);
        }
      }
    }
  }
};

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

// A warp takes a run of the head groups (32 / lanes heads each).  Forward they come
// token by token, queries then keys, so that a token's angles serve both; backward the
// queries of all tokens, then the keys, so that the sums of the weight's gradient
// change hands once at most.  LANES > 0: heads of 16 LANES values in whole groups,
// every lane with all its units of every group.
template <typename T, int V, int NU, bool NEIGHBOURS, bool BACKWARD, int LANES>
__global__ void __launch_bounds__(32 * kWarps, Ring<T, BACKWARD>::kCtas) qk_norm_kernel(const __grid_constant__ QkKernelArgs g) {
  using S = Slice<T, V, NU, NEIGHBOURS>;
  using R = Ring<T, BACKWARD>;
  constexpr int P = S::P, H = P / 2;
  constexpr bool kRing = V > 1;
  extern __shared__ __align__(16) uint8_t smem[];
  // behind the ring: weights [2][dim], cos and sin [warp][rotary / 2]; backward, sums [warp][2][dim]
  float* sh = reinterpret_cast<float*>(smem + (kRing ? R::kBytes : 0));
  __shared__ uint64_t turns[kMaxPairs];
  let_dependents_start();
  wait_for_stream();
  const int warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : g.lanes;
  const int lane = (threadIdx.x & 31) & (lanes - 1), sub = (threadIdx.x & 31) / lanes;
  const int half = g.rotary / 2;
  float2* trig = reinterpret_cast<float2*>(sh + 2 * g.dim) + warp * half;
  float* sums = sh + 2 * g.dim + kWarps * g.rotary;
  for (int i = threadIdx.x; i < half; i += 32 * kWarps) turns[i] = g.turns[i];
  for (int i = threadIdx.x; i < 2 * g.dim; i += 32 * kWarps) {
    const void* w = g.weight[i >= g.dim];
    const int c = i >= g.dim ? i - g.dim : i;
    sh[i] = !w ? 1.0f : g.w_fp32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  }
  if constexpr (BACKWARD)
    for (int i = threadIdx.x; i < kWarps * 2 * g.dim; i += 32 * kWarps) sums[i] = 0.f;
  __syncthreads();

  const int64_t workers = (int64_t)gridDim.x * kWarps, me = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t each = g.groups / workers, more = g.groups % workers;
  const int64_t begin = me * each + min(me, more);
  const int count = (int)(each + (me < more));
  const float inv_dim = 1.0f / (float)g.dim;
  const int per_group = 32 / lanes, step = per_group * g.dim;  // heads, and values from a group to the next
  int unit_a[NU], unit_b[NU];  // the lane's vectors in a head
  bool unit[NU];
#pragma unroll
  for (int j = 0; j < NU; ++j) unit[j] = S::place(g, lanes, lane, j, unit_a[j], unit_b[j]) || LANES > 0;

  // A place in the run: a group of a token's query or key heads.
  struct Place {
    int token, kind, run;
  };
  Place here;
  if constexpr (BACKWARD) {
    here.kind = begin >= (int64_t)g.rows * g.runs[0];
    const int64_t first = begin - (here.kind ? (int64_t)g.rows * g.runs[0] : 0);
    here.token = g.runs[here.kind] ? (int)(first / g.runs[here.kind]) : 0;
    here.run = (int)(first - (int64_t)here.token * g.runs[here.kind]);
  } else {
    const int per_token = g.runs[0] + g.runs[1];
    here.token = (int)(begin / per_token);
    here.run = (int)(begin - (int64_t)here.token * per_token);
    here.kind = here.run >= g.runs[0];
    here.run -= here.kind ? g.runs[0] : 0;
  }
  auto next = [&](Place& p) {  // true: the next group of the same heads' kind and token
    if (++p.run < g.runs[p.kind]) return true;
    p.run = 0;
    if (BACKWARD) {
      if (++p.token == g.rows) {
        p.token = 0;
        p.kind = 1;
      }
    } else if (p.kind == 0 && g.runs[1] > 0) {
      p.kind = 1;
    } else {
      ++p.token;
      p.kind = g.runs[0] == 0;
    }
    return false;
  };
  auto start = [&](const Place& p, int64_t ld) {  // of its group in a tensor, at this lane's head
    return (int64_t)p.token * ld + (int64_t)(p.kind ? g.heads[0] : 0) * g.dim + (int64_t)p.run * step + sub * g.dim;
  };
  auto has_head = [&](const Place& p) { return LANES > 0 || p.run * per_group + sub < g.heads[p.kind]; };

  // The groups to come: in registers, or in the warp's ring (a lane reads back what it copied itself).
  S nx, ny;
  int f_left = count;
  Place f = here;
  const T* const x = static_cast<const T*>(g.x);
  const T* const dy = static_cast<const T*>(g.dy);
  const T* fx = x + start(f, g.ldx);
  const T* fy = BACKWARD ? dy + start(f, g.lddy) : nullptr;
  uint32_t f_at = 0, at = 0;
  constexpr int kVector = V * sizeof(T);
  const uint32_t ring = smem_u32(smem) + warp * (R::kDepth * R::kStage) + (threadIdx.x & 31) * kVector;
  auto fetch = [&]() {
    if (f_left > 0) {
      --f_left;
      const bool there = has_head(f);
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        const bool in = LANES > 0 || (there && unit[j]);
        if constexpr (kRing) {
          const uint32_t to = ring + f_at + j * 64 * kVector;
          Raw<T, V>::copy(to, in ? fx + unit_a[j] : x, in);
          Raw<T, V>::copy(to + 32 * kVector, in ? fx + unit_b[j] : x, in);
          if constexpr (BACKWARD) {
            Raw<T, V>::copy(to + R::kStage / 2, in ? fy + unit_a[j] : dy, in);
            Raw<T, V>::copy(to + R::kStage / 2 + 32 * kVector, in ? fy + unit_b[j] : dy, in);
          }
        } else {
          nx.a[j] = nx.b[j] = ny.a[j] = ny.b[j] = Raw<T, V>{};
          if (in) {
            nx.a[j].load(fx + unit_a[j]);
            nx.b[j].load(fx + unit_b[j]);
            if constexpr (BACKWARD) {
              ny.a[j].load(fy + unit_a[j]);
              ny.b[j].load(fy + unit_b[j]);
            }
          }
        }
      }
      if (next(f)) {
        fx += step;
        if constexpr (BACKWARD) fy += step;
      } else {
        fx = x + start(f, g.ldx);
        if constexpr (BACKWARD) fy = dy + start(f, g.lddy);
      }
    }
    if constexpr (kRing) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      f_at = f_at == (R::kDepth - 1) * R::kStage ? 0 : f_at + R::kStage;
    }
  };
#pragma unroll
  for (int i = 0; i < (kRing ? R::kDepth : 1); ++i) fetch();

  // Forward: w1 cos, -w2 sin, w2 cos, w1 sin of the thread's pairs.  Backward: w1, w2, cos, sin.
  float2 wa[H], wb[H], wc[H], wd[H];
  float2 dwp[BACKWARD ? H : 1], dwq[BACKWARD ? H : 1];
  if constexpr (BACKWARD) {
#pragma unroll
    for (int i = 0; i < H; ++i) dwp[i] = dwq[i] = twice(0.f);
  }
  auto leave_sums = [&](int kind) {  // the warp's groups of lanes, in a fixed order
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float a = k & 1 ? dwp[k / 2].y : dwp[k / 2].x, b = k & 1 ? dwq[k / 2].y : dwq[k / 2].x;
      for (int o = 16; o >= lanes; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
      }
      int pa, pb;
      if (S::where(g, lanes, lane, k, pa, pb) && sub == 0) {
        sums[(warp * 2 + kind) * g.dim + pa] += a;
        sums[(warp * 2 + kind) * g.dim + pb] += b;
      }
    }
#pragma unroll
    for (int i = 0; i < H; ++i) dwp[i] = dwq[i] = twice(0.f);
  };
  bool new_token = true, new_kind = true;
  int64_t next_position = count > 0 ? g.positions[here.token] : 0;
  T* to = static_cast<T*>(g.out) + start(here, g.ldo);
  for (int i = 0; i < count; ++i) {
    if (new_token) {  // the warp's lanes share the angles
      const int64_t position = next_position;
      next_position = g.positions[here.token + 1 < g.rows ? here.token + 1 : 0];
      __syncwarp();
      for (int j = threadIdx.x & 31; j < half; j += 32) {
        uint64_t angle = turns[j] * (uint64_t)position;
        if (is_far(position)) angle += low_part(g.low_turns[j], position);  // (in shared memory too, heads of 512: 110 -> 115 us)
        const int32_t half_turns = (int32_t)(angle >> 32);  // of 2^-31
        float s, c;
        sincospif((float)half_turns * 4.65661287e-10f, &s, &c);
        trig[j] = make_float2(c, s);
      }
      __syncwarp();
    }
    if (new_token || new_kind) {
      float2 turn[P];  // (cos, sin)
      float w[2 * P];  // of the firsts, of the seconds
      const float* ws = sh + here.kind * g.dim;
      if constexpr (V > 1) {
#pragma unroll
        for (int k = 0; k < P; k += 2) {
          const int t = S::turn_of(g, lanes, lane, k);  // (even, and so is half)
          const float4 r = t < half ? *reinterpret_cast<const float4*>(trig + t) : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
          turn[k] = make_float2(r.x, r.y);
          turn[k + 1] = make_float2(r.z, r.w);
        }
#pragma unroll
        for (int k = 0; k < P; k += 4) {
          const int j = k / V, i0 = k % V;
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 u = unit[j] ? *reinterpret_cast<const float4*>(ws + unit_a[j] + i0) : zero;
          const float4 v = unit[j] ? *reinterpret_cast<const float4*>(ws + unit_b[j] + i0) : zero;
          const float a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {  // (neighbours: value 2 i and 2 i + 1 of a vector are pair i's)
            w[NEIGHBOURS ? j * V + (i0 + h) / 2 + (h & 1 ? P : 0) : k + h] = a[h];
            w[NEIGHBOURS ? j * V + (V + i0 + h) / 2 + (h & 1 ? P : 0) : P + k + h] = b[h];
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int t = S::turn_of(g, lanes, lane, k);
          turn[k] = t < half ? trig[t] : make_float2(1.0f, 0.0f);
          w[k] = unit[k] ? ws[unit_a[k]] : 0.f;
          w[P + k] = unit[k] ? ws[unit_b[k]] : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const float2 c = make_float2(turn[2 * k].x, turn[2 * k + 1].x), n = make_float2(turn[2 * k].y, turn[2 * k + 1].y);
        const float2 w1 = make_float2(w[2 * k], w[2 * k + 1]), w2 = make_float2(w[P + 2 * k], w[P + 2 * k + 1]);
        if constexpr (BACKWARD) {
          wa[k] = w1;
          wb[k] = w2;
          wc[k] = c;
          wd[k] = n;
        } else {
          wa[k] = __fmul2_rn(w1, c);
          wb[k] = __fmul2_rn(make_float2(-w2.x, -w2.y), n);
          wc[k] = __fmul2_rn(w2, c);
          wd[k] = __fmul2_rn(w1, n);
        }
      }
    }
    S cx, cy;
    if constexpr (kRing) {
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        const uint32_t from = ring + at + j * 64 * kVector;
        cx.a[j].take(from);
        cx.b[j].take(from + 32 * kVector);
        if constexpr (BACKWARD) {
          cy.a[j].take(from + R::kStage / 2);
          cy.b[j].take(from + R::kStage / 2 + 32 * kVector);
        }
      }
      at = at == (R::kDepth - 1) * R::kStage ? 0 : at + R::kStage;
    } else {
      cx = nx;
      if constexpr (BACKWARD) cy = ny;
      fetch();
    }

    float2 p[H], q[H];
    cx.values(p, q);
    float2 squares = twice(0.f);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      squares = __ffma2_rn(p[k], p[k], squares);
      squares = __ffma2_rn(q[k], q[k], squares);
    }
    float square = squares.x + squares.y;
    const bool there = has_head(here);
    if constexpr (!BACKWARD) {
#pragma unroll
      for (int o = lanes >> 1; o > 0; o >>= 1) square += __shfl_xor_sync(0xFFFFFFFFu, square, o);
      if constexpr (kRing) fetch();  // into the place whose values have entered the sum
      const float2 rstd = twice(rsqrtf(fmaf(square, inv_dim, g.eps)));
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const float2 a = __fmul2_rn(p[k], rstd), b = __fmul2_rn(q[k], rstd);
        p[k] = __ffma2_rn(b, wb[k], __fmul2_rn(a, wa[k]));
        q[k] = __ffma2_rn(a, wd[k], __fmul2_rn(b, wc[k]));
      }
    } else {
      float2 gp[H], gq[H], dots = twice(0.f);
      cy.values(gp, gq);
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const float2 u = gp[k], v = gq[k];
        gp[k] = __ffma2_rn(v, wd[k], __fmul2_rn(u, wc[k]));
        gq[k] = __ffma2_rn(make_float2(-u.x, -u.y), wd[k], __fmul2_rn(v, wc[k]));
        dots = __ffma2_rn(__fmul2_rn(gp[k], wa[k]), p[k], dots);
        dots = __ffma2_rn(__fmul2_rn(gq[k], wb[k]), q[k], dots);
      }
      float dot = dots.x + dots.y;
#pragma unroll
      for (int o = lanes >> 1; o > 0; o >>= 1) {
        square += __shfl_xor_sync(0xFFFFFFFFu, square, o);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      }
      if constexpr (kRing) fetch();  // into the place whose values have entered the sums
      const float r = rsqrtf(fmaf(square, inv_dim, g.eps));
      const float2 rstd = twice(r), back = twice(-(dot * inv_dim * r * r));
#pragma unroll
      for (int k = 0; k < H; ++k) {
        if (there) {
          dwp[k] = __ffma2_rn(gp[k], __fmul2_rn(p[k], rstd), dwp[k]);
          dwq[k] = __ffma2_rn(gq[k], __fmul2_rn(q[k], rstd), dwq[k]);
        }
        p[k] = __fmul2_rn(rstd, __ffma2_rn(p[k], back, __fmul2_rn(gp[k], wa[k])));
        q[k] = __fmul2_rn(rstd, __ffma2_rn(q[k], back, __fmul2_rn(gq[k], wb[k])));
      }
    }
    if (there) {
      cx.set(p, q);
#pragma unroll
      for (int j = 0; j < NU; ++j)
        if (LANES > 0 || unit[j]) {
          cx.a[j].store(to + unit_a[j]);
          cx.b[j].store(to + unit_b[j]);
        }
    }
    const int token = here.token, kind = here.kind;
    if (next(here)) {
      new_token = new_kind = false;
      to += step;
    } else {
      new_kind = here.kind != kind;
      new_token = here.token != token || (BACKWARD && new_kind);
      to = static_cast<T*>(g.out) + start(here, g.ldo);
      if constexpr (BACKWARD)
        if (new_kind || here.token == 0) leave_sums(kind);
    }
  }
  if constexpr (BACKWARD) {
    if (!g.parts) return;
    leave_sums(here.kind);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.dim; i += 32 * kWarps) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * 2 * g.dim + i];
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

// CTAs per place for one: SMs are not equally fast at memory, and an even split over
// the CTAs that fit at once waits for the slowest (15872 x 64 x 128 bf16: 95.4 us with
// one round, 82.7 with four, 80.1 with eight).  Backward each CTA leaves a part to join,
// which costs more than rounds gain (130 us with one, 133 with two).
constexpr int kWaves = 8;
// Most CTAs of the backward pass, each of which leaves a part of the weights' gradients.
int64_t most_parts() { return 2 * 160; }

template <typename T, int V, int NU, bool NEIGHBOURS, bool BACKWARD, int LANES>
lpq_status run(QkKernelArgs& g, int64_t rows, float* dq, float* dk, cudaStream_t s) {
  const void* kernel = reinterpret_cast<const void*>(qk_norm_kernel<T, V, NU, NEIGHBOURS, BACKWARD, LANES>);
  const int units = g.dim / 2 / V;  // of a head; value by value a warp has a head
  g.lanes = 1;
  while (g.lanes < 32 && g.lanes * (V > 1 ? NU : 1) < units) g.lanes *= 2;
  for (int i = 0; i < 2; ++i) g.runs[i] = (g.heads[i] * g.lanes + 31) / 32;
  g.groups = rows * (g.runs[0] + g.runs[1]);
  g.rows = (int)rows;
  const int ring = V > 1 ? Ring<T, BACKWARD>::kBytes : 0;
  auto rest = [](int dim, int rotary) { return 2 * dim * 4 + kWarps * rotary / 2 * 8 + (BACKWARD ? kWarps * 2 * dim * 4 : 0); };
  const int smem = ring + rest(g.dim, g.rotary);
  lpq_status st = set_smem_attr(kernel, ring + rest(kQkMaxDim, kQkMaxDim));
  if (st != LPQ_OK) return st;
  int64_t most = (int64_t)device_sms() * std::max(1, std::min(Ring<T, BACKWARD>::kCtas, 226 * 1024 / (smem + 4 * 1024)));
  // Forward more rounds of CTAs while every warp keeps a few groups (2000 tokens of 32 +
  // 8 heads of 128: 20.0 us with one group a warp, 9.9 with five).
  if (BACKWARD) most = std::min(most, most_parts());
  else most = std::max(most, std::min(most * kWaves, g.groups / (kWarps * 8)));
  const int64_t grid = std::max<int64_t>(1, std::min(most, (g.groups + kWarps - 1) / kWarps));
  if (g.groups / (grid * kWarps) >= 0x7FFFFFFF) return set_error(LPQ_ERR_SHAPE, "qk norm: too large");
  st = cuda_check(launch_dependent(qk_norm_kernel<T, V, NU, NEIGHBOURS, BACKWARD, LANES>, dim3((unsigned)grid), dim3(32 * kWarps), smem, s, g),
                  BACKWARD ? "qk norm backward launch" : "qk norm launch");
  if (st != LPQ_OK || !BACKWARD || !g.parts) return st;
  return cuda_check(launch_dependent(qk_join_kernel, dim3((2 * g.dim + 31) / 32), dim3(32 * kJoinWarps), 0, s, g.parts, (int)grid, g.dim,
                                     dq, dk),
                    "qk norm join launch");
}

template <typename T, bool NEIGHBOURS, bool BACKWARD>
lpq_status vectors(QkKernelArgs& g, int64_t rows, bool usual, float* dq, float* dk, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T), NU = 8 / V;
  if (usual && g.dim == 64) return run<T, V, NU, NEIGHBOURS, BACKWARD, 4>(g, rows, dq, dk, s);
  if (usual && g.dim == 128) return run<T, V, NU, NEIGHBOURS, BACKWARD, 8>(g, rows, dq, dk, s);
  if (usual && g.dim == 256) return run<T, V, NU, NEIGHBOURS, BACKWARD, 16>(g, rows, dq, dk, s);
  return run<T, V, NU, NEIGHBOURS, BACKWARD, 0>(g, rows, dq, dk, s);
}

template <typename T, bool BACKWARD>
lpq_status dispatch(QkKernelArgs& g, int64_t rows, bool neighbours, float* dq, float* dk, cudaStream_t s) {
  g.neighbours = neighbours;
  // Vectors of v values: both halves of what is turned begin with one, or every vector
  // holds whole pairs, and two lie in a float4 of angles.
  auto fits = [&](int v) {
    auto whole = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % (v * sizeof(T)) == 0 && ld % v == 0; };
    return g.dim % (2 * v) == 0 && g.rotary % (neighbours ? 4 : 2 * v) == 0 && whole(g.x, g.ldx) && whole(g.out, g.ldo) &&
           (!BACKWARD || whole(g.dy, g.lddy));
  };
  if (fits(16 / sizeof(T))) {
    const int per_group = 512 / g.dim;  // whole groups of the usual head sizes
    const bool usual = per_group > 0 && g.heads[0] % per_group == 0 && g.heads[1] % per_group == 0;
    return neighbours ? vectors<T, true, BACKWARD>(g, rows, usual, dq, dk, s) : vectors<T, false, BACKWARD>(g, rows, usual, dq, dk, s);
  }
  if constexpr (sizeof(T) == 2)
    if (fits(4)) return neighbours ? run<T, 4, 2, true, BACKWARD, 0>(g, rows, dq, dk, s) : run<T, 4, 2, false, BACKWARD, 0>(g, rows, dq, dk, s);
  // value by value
  if (g.dim <= 128) return run<T, 1, 2, false, BACKWARD, 0>(g, rows, dq, dk, s);
  if (g.dim <= 256) return run<T, 1, 4, false, BACKWARD, 0>(g, rows, dq, dk, s);
  return run<T, 1, 8, false, BACKWARD, 0>(g, rows, dq, dk, s);
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
    const Turns t = turns_of(a.freqs[i]);
    g.turns[i] = t.high;
    g.low_turns[i] = t.low;
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
