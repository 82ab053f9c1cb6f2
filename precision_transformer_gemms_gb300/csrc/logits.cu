// Penalties for repeated words, biases and a grammar's mask on the logits of
// the next words, one pass over them, on sm_103a.
//
//   c = times word j stands in the row's answer, seen = it stands in its context
//   l = seen ? (l > 0 ? l / r : l r) : l;  l -= f c + p [c > 0];  l += b;  not allowed: -infinity
//
// The logits, read and written once, are the traffic there is.  A CTA takes a
// run of words of a row: it loads them to registers, counts the context's words
// that lie in its run in shared memory (integers: the order of the atomics does
// not matter), adds the biases there in the list's order, and then works on its
// registers.  Contexts of more than a few words are read by a cluster of CTAs
// together, each a part, whose words it counts where they belong, in its own or
// another CTA's shared memory.
#include <cuda_bf16.h>

#include <algorithm>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kClusterContext = 512;  // words of a context that a CTA reads alone
constexpr uint32_t kSeen = 0x80000000u;  // stands in the prompt; the other bits count the answer

// Integer sums in the shared memory of a CTA of the cluster.
__device__ __forceinline__ void count_at(uint32_t addr, bool prompt) {
  if (prompt) asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(kSeen) : "memory");
  else asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(1u) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// `segments` CTAs a row, a multiple of C, the CTAs of a cluster.
template <typename T, int VEC, int NV, int C>
__global__ void __launch_bounds__(kThreads) adjust_logits_kernel(const LogitsArgs g, int64_t segments) {
  constexpr int S = kThreads * VEC * NV;  // words of a CTA
  __shared__ __align__(16) uint32_t counts[S];
  __shared__ __align__(16) float biases[S];
  let_dependents_start();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / segments;
  const T* in = static_cast<const T*>(g.logits) + row * g.ld;
  T* out = static_cast<T*>(g.out) + row * g.ldo;
  // Word w of the row stands at w + lead, counted from a 16-byte boundary.
  const int lead = VEC == 1 ? 0 : (int)((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(T));
  const int64_t first = (blockIdx.x - row * segments) * S - lead;  // word of the run's first place
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  for (int i = tid; i < S / 4; i += kThreads) {
    reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(biases)[i] = make_uint4(0, 0, 0, 0);
  }
  if constexpr (C > 1) cluster_arrive();  // this CTA's counts are ready
  wait_for_stream();

  T val[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t w = first + (j * kThreads + tid) * VEC;
    if (VEC > 1 && w >= 0 && w + VEC <= g.v) {
      *reinterpret_cast<uint4*>(val[j]) = *reinterpret_cast<const uint4*>(in + w);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) val[j][k] = w + k >= 0 && w + k < g.v ? in[w + k] : T(0.f);
    }
  }
  // The word's place among `count` from `from` on, or -1.
  auto place = [&](int64_t word, int64_t from, int count) {
    if ((uint64_t)word >= (uint64_t)g.v) return -1;
    const int64_t at = word - from;
    return at >= 0 && at < count ? (int)at : -1;
  };
  if constexpr (C == 1) __syncthreads();
  if (g.c.history) {
    const int64_t n = max((int64_t)0, min(g.c.lengths[row], g.c.max_len));
    const int64_t prompt = g.c.prompt ? g.c.prompt[row] : 0;
    const int64_t* h = g.c.history + row * g.c.ld_history;
    const uint32_t table = smem_u32(counts);
    constexpr int kAhead = 4;  // words of a thread on their way
    int64_t word[kAhead];
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) word[j] = i0 + j * C * kThreads < n ? h[i0 + j * C * kThreads] : -1;
    };
    int64_t i0 = (int64_t)rank * kThreads + tid;
    load(i0);
    if constexpr (C > 1) {
      __syncwarp();
      cluster_wait();  // the others' counts are ready, too
    }
    for (; i0 < n; load(i0)) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int at = place(word[j], first - (int64_t)rank * S, C * S);
        if (at < 0) continue;
        const bool asked = i0 + j * C * kThreads < prompt;
        if constexpr (C > 1) {
          count_at(mapa_shared(table + (at % S) * 4, (uint32_t)(at / S)), asked);
        } else {
          if (asked) atomicOr(&counts[at], kSeen); else atomicAdd(&counts[at], 1u);
        }
      }
      i0 += kAhead * C * kThreads;
    }
  } else if constexpr (C > 1) {
    cluster_wait();
  }
  if constexpr (C > 1) {
    __syncwarp();
    cluster_arrive();  // its words are counted
  }
  if (g.c.bias_words && tid < 32) {
    const int64_t from = max((int64_t)0, g.c.bias_offsets[row]), to = min(g.c.bias_offsets[row + 1], g.c.bias_count);
    for (int64_t i = from; i < to; i += 32) {
      const int at = i + tid < to ? place(g.c.bias_words[i + tid], first, S) : -1;
      const float b = at >= 0 ? g.c.bias_values[i + tid] : 0.f;
      for (uint32_t left = __ballot_sync(0xFFFFFFFFu, at >= 0); left; left &= left - 1) {  // one after another
        if (tid == __ffs(left) - 1) biases[at] += b;
        __syncwarp();
      }
    }
  }
  __syncthreads();
  if constexpr (C > 1) cluster_wait();
  const float rep = g.c.repetition ? g.c.repetition[row] : 1.f;
  const float freq = g.c.frequency ? g.c.frequency[row] : 0.f, pres = g.c.presence ? g.c.presence[row] : 0.f;
  const uint32_t* allowed = g.c.allowed ? reinterpret_cast<const uint32_t*>(g.c.allowed) + row * g.c.ld_allowed : nullptr;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int p = (j * kThreads + tid) * VEC;
    const int64_t w = first + p;
    if (w >= g.v || w + VEC <= 0) continue;
    uint32_t bits = 0xFFFFFFFFu;
    if (allowed) {
      const int64_t a = max(w, (int64_t)0), z = min(w + VEC, g.v) - 1;
      bits = __funnelshift_r(allowed[a >> 5], allowed[z >> 5], (uint32_t)a & 31u) << (a - w);
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float x;
      if constexpr (sizeof(T) == 4) x = val[j][k]; else x = __bfloat162float(val[j][k]);
      const uint32_t c = counts[p + k];
      if (c) {
        x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
        const uint32_t times = c & ~kSeen;
        if (times) x = x - freq * (float)times - pres;
      }
      if (g.c.bias_words) x += biases[p + k];
      if (!((bits >> k) & 1u)) x = -__int_as_float(0x7F800000);
      if constexpr (sizeof(T) == 4) val[j][k] = x; else val[j][k] = __float2bfloat16_rn(x);
    }
    if (VEC > 1 && w >= 0 && w + VEC <= g.v) {
      *reinterpret_cast<uint4*>(out + w) = *reinterpret_cast<const uint4*>(val[j]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (w + k >= 0 && w + k < g.v) out[w + k] = val[j][k];
    }
  }
}

template <typename T, int VEC, int NV, int C>
lpq_status run(const LogitsArgs& g, cudaStream_t s) {
  constexpr int S = kThreads * VEC * NV;
  const int64_t segments = ((g.v + VEC - 1 + S - 1) / S + C - 1) / C * C;  // (a row may begin VEC - 1 places in)
  const int64_t grid = g.rows * segments;
  if (grid > 0x7FFFFFFF) return set_error(LPQ_ERR_SHAPE, "logits: too large");
  if constexpr (C == 1)
    return cuda_check(launch_dependent(adjust_logits_kernel<T, VEC, NV, 1>, dim3((unsigned)grid), dim3(kThreads), 0, s, g, segments),
                      "logits launch");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_check(cudaLaunchKernelEx(&cfg, adjust_logits_kernel<T, VEC, NV, C>, g, segments), "logits launch");
}

template <typename T, int VEC, int NV>
lpq_status run_context(const LogitsArgs& g, cudaStream_t s) {
  return g.c.history && g.c.max_len > kClusterContext ? run<T, VEC, NV, 8>(g, s) : run<T, VEC, NV, 1>(g, s);
}

template <typename T>
lpq_status dispatch(const LogitsArgs& g, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  // every row must begin equally far from a 16-byte boundary on both sides
  const uintptr_t in = reinterpret_cast<uintptr_t>(g.logits), out = reinterpret_cast<uintptr_t>(g.out);
  const bool vectors = (in - out) % 16 == 0 && (g.rows == 1 || (g.ld - g.ldo) * (int64_t)sizeof(T) % 16 == 0);
  const bool small = g.rows * g.v < (int64_t)device_sms() * 2 * 4096;
  if (vectors) return small ? run_context<T, VEC, 1>(g, s) : run_context<T, VEC, 16 / VEC>(g, s);
  return small ? run_context<T, 1, 4>(g, s) : run_context<T, 1, 16>(g, s);
}

}  // namespace

lpq_status launch_adjust_logits(const LogitsArgs& g, int32_t type, cudaStream_t s) {
  if (g.rows == 0 || g.v == 0) return LPQ_OK;
  return type == LPQ_TYPE_FP32 ? dispatch<float>(g, s) : dispatch<__nv_bfloat16>(g, s);
}

}  // namespace lpq
