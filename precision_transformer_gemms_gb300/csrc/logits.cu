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
// registers.  Every CTA of a row reads the row's whole context, from the L2.
//
// Measured, 64 rows of 131073 FP32 (floor 10.5 us at the copy bandwidth of 6677 GB/s):
// contexts of up to 1000 words 18.6 us, 8192 25, 16384 29, 32768 36; bf16, 4000 words
// 18; 8 rows 4.9; one row of 32000 words 2.1.  What bounds it is the chain of a CTA's
// loads (lengths, context, counts, then words) and the scan of the context, whose 8192
// words take a CTA's 512 threads 16 loads each, in four rounds of four, for the 8192
// words that it writes; clusters that share the scan through distributed shared memory gained for one row
// with a long context alone.
#include <cuda_bf16.h>

#include <algorithm>

#include "logit_runs.h"
#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr uint32_t kSeen = 0x80000000u;  // stands in the prompt; the other bits count the answer

// `segments` CTAs a row.  What a CTA reads at addresses that it knows, it asks for at
// once: the time of a CTA is that of a few loads after one another, not of its bytes.
template <typename T, int VEC, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads, VEC == 1 ? 3 : kThreads == 256 ? 5 : 3) adjust_logits_kernel(const LogitsArgs g, uint32_t segments) {
  constexpr int S = kThreads * VEC * NV;  // words of a CTA
  extern __shared__ __align__(16) uint32_t counts[];  // [S], and with biases their sums [S]
  float* biases = reinterpret_cast<float*>(counts + S);
  let_dependents_start();
  const int tid = threadIdx.x;
  const uint32_t row32 = blockIdx.x / segments;
  const int64_t row = row32;
  const T* in = static_cast<const T*>(g.logits) + row * g.ld;
  T* out = static_cast<T*>(g.out) + row * g.ldo;
  // Word w of the row stands at w + lead, counted from a 16-byte boundary.
  const int lead = VEC == 1 ? 0 : (int)((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(T));
  const int v = (int)g.v;
  const int first = run_first((int)(blockIdx.x - row32 * segments), S, lead);
#pragma unroll
  for (int i = 0; i < S / 4; i += kThreads) {
    reinterpret_cast<uint4*>(counts)[i + tid] = make_uint4(0, 0, 0, 0);
    if (g.c.bias_words) reinterpret_cast<uint4*>(biases)[i + tid] = make_uint4(0, 0, 0, 0);
  }
  wait_for_stream();

  int64_t n = 0, prompt = 0, from = 0, to = 0;
  if (g.c.history) {
    n = g.c.lengths[row];
    if (g.c.prompt) prompt = g.c.prompt[row];
  }
  if (g.c.bias_words) {
    from = g.c.bias_offsets[row];
    to = g.c.bias_offsets[row + 1];
  }
  const float rep = g.c.repetition ? g.c.repetition[row] : 1.f;
  const float freq = g.c.frequency ? g.c.frequency[row] : 0.f, pres = g.c.presence ? g.c.presence[row] : 0.f;
  T val[NV][VEC];
  uint32_t bits[NV];
  const uint32_t* allowed = g.c.allowed ? reinterpret_cast<const uint32_t*>(g.c.allowed) + row * g.c.ld_allowed : nullptr;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int w = first + (j * kThreads + tid) * VEC;
    if (VEC > 1 && w >= 0 && w + VEC <= v) {
      *reinterpret_cast<uint4*>(val[j]) = *reinterpret_cast<const uint4*>(in + w);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) val[j][k] = w + k >= 0 && w + k < v ? in[w + k] : T(0.f);
    }
    bits[j] = 0xFFFFFFFFu;
    if (allowed && w < v && w + VEC > 0) {
      const int a = max(w, 0), z = min(w + VEC, v) - 1;
      bits[j] = __funnelshift_r(allowed[a >> 5], allowed[z >> 5], (uint32_t)a & 31u) << (a - w);
    }
  }
  const int words = run_words(first, S, v);

  // The context's words, and the biases by the last warp.
  const int len = (int)max((int64_t)0, min(n, g.c.max_len));
  const int asked = (int)max((int64_t)0, min(prompt, (int64_t)len));  // words of the prompt
  // Both ends: the last warp's lanes read from + lane at once, which beyond 2^63 would be
  // in front of the list.
  from = within(from, g.c.bias_count);
  to = within(to, g.c.bias_count);
  constexpr int kAhead = 4;  // words of a thread on their way
  constexpr int stride = kThreads;
  int i0 = tid;
  const int64_t* h = g.c.history + row * g.c.ld_history + i0;
  int64_t word[kAhead];
  auto load = [&]() {
    if (i0 + (kAhead - 1) * stride < len) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) word[j] = h[j * stride];
    } else {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) word[j] = i0 + j * stride < len ? h[j * stride] : INT64_MIN;
    }
    h += kAhead * stride;
  };
  const int lane = tid & 31;
  const bool biasing = g.c.bias_words && tid >= kThreads - 32;
  int64_t bias_word = -1;
  float bias = 0.f;
  auto load_bias = [&]() {
    bias_word = from + lane < to ? g.c.bias_words[from + lane] : -1;
    bias = from + lane < to ? g.c.bias_values[from + lane] : 0.f;
  };
  load();
  if (biasing) load_bias();
  __syncthreads();  // (the tables are clear)
  while (i0 < len) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int at = run_place(word[j], first, words);
      if (at < 0) continue;
      if (i0 + j * stride < asked) atomicOr(&counts[at], kSeen); else atomicAdd(&counts[at], 1u);
    }
    i0 += kAhead * stride;
    load();
  }
  if (biasing) {
    for (; from < to; load_bias()) {
      const int at = run_place(bias_word, first, words);
      for (uint32_t left = __ballot_sync(0xFFFFFFFFu, at >= 0); left; left &= left - 1) {  // one after another, in the list's order
        if (lane == __ffs(left) - 1) biases[at] += bias;
        __syncwarp();
      }
      from += 32;
    }
  }
  __syncthreads();
  // rep scaled to where its reciprocal is a normal number (infinity: to 0, whose reciprocal is taken to be 0)
  const float size = fabsf(rep), scale = size < 0x1p-100f ? 0x1p64f : size > 0x1p100f ? 0x1p-64f : 1.f;
  const bool endless = size > 3.402823466e38f;
  const float divisor = endless ? 0.f : rep * scale, inverse = endless ? 0.f : __fdiv_rn(1.f, divisor);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int p = (j * kThreads + tid) * VEC, w = first + p;
    if (w >= v || w + VEC <= 0) continue;
    float x[VEC];
    uint32_t c[VEC], any = 0;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if constexpr (sizeof(T) == 4) x[k] = val[j][k]; else x[k] = __bfloat162float(val[j][k]);
      c[k] = counts[p + k];
      any |= c[k];
    }
    if (any) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        // x / rep by the reciprocal and one correction with the exact remainder (where that is a number)
        float q = x[k] * inverse;
        if (fabsf(q) <= 3.402823466e38f) q = fmaf(fmaf(-q, divisor, x[k]), inverse, q);
        q *= scale;
        const float seen = x[k] > 0.f ? q : x[k] * rep;
        if (c[k]) x[k] = seen;
        const uint32_t times = c[k] & ~kSeen;
        if (times) x[k] = x[k] - freq * (float)times - pres;
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if (g.c.bias_words) x[k] += biases[p + k];
      if (!((bits[j] >> k) & 1u)) x[k] = -__int_as_float(0x7F800000);
      if constexpr (sizeof(T) == 4) val[j][k] = x[k]; else val[j][k] = __float2bfloat16_rn(x[k]);
    }
    if (VEC > 1 && w >= 0 && w + VEC <= v) {
      *reinterpret_cast<uint4*>(out + w) = *reinterpret_cast<const uint4*>(val[j]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (w + k >= 0 && w + k < v) out[w + k] = val[j][k];
    }
  }
}

template <typename T, int VEC, int NV, int kThreads>
lpq_status run(const LogitsArgs& g, cudaStream_t s) {
  constexpr int S = kThreads * VEC * NV;
  const int64_t segments = run_count(g.v, VEC, S);
  const int64_t grid = g.rows * segments;
  if (grid > 0x7FFFFFFF) return set_error(LPQ_ERR_SHAPE, "logits: too large");
  const void* kernel = reinterpret_cast<const void*>(adjust_logits_kernel<T, VEC, NV, kThreads>);
  lpq_status st = set_smem_attr(kernel, 8 * S);
  if (st != LPQ_OK) return st;
  return cuda_check(launch_dependent(adjust_logits_kernel<T, VEC, NV, kThreads>, dim3((unsigned)grid), dim3(kThreads),
                                     (g.c.bias_words ? 8 : 4) * S, s, g, (uint32_t)segments),
                    "logits launch");
}

template <typename T>
lpq_status dispatch(const LogitsArgs& g, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  // every row must begin equally far from a 16-byte boundary on both sides
  const uintptr_t in = reinterpret_cast<uintptr_t>(g.logits), out = reinterpret_cast<uintptr_t>(g.out);
  const bool vectors = (in - out) % 16 == 0 && (g.rows == 1 || (g.ld - g.ldo) * (int64_t)sizeof(T) % 16 == 0);
  // Small runs of words while they give every SM a few CTAs; large ones else, and of
  // twice the words where the context, which every CTA reads, may be long (64 x 131073
  // FP32, contexts of up to 8192: 26.6 -> 24.6 us, of 32768 50.9 -> 34.8, of 1000 18.5 -> 20.0).
  const bool small = g.rows * g.v < (int64_t)device_sms() * 2 * 4096;
  const bool long_context = g.c.history && g.c.max_len >= 2048;
  if (vectors) return small ? run<T, VEC, 1, 256>(g, s) : long_context ? run<T, VEC, 16 / VEC, 512>(g, s) : run<T, VEC, 16 / VEC, 256>(g, s);
  return small ? run<T, 1, 4, 256>(g, s) : run<T, 1, 16, 256>(g, s);
}

}  // namespace

lpq_status launch_adjust_logits(const LogitsArgs& g, int32_t type, cudaStream_t s) {
  if (g.rows == 0 || g.v == 0) return LPQ_OK;
  return type == LPQ_TYPE_FP32 ? dispatch<float>(g, s) : dispatch<__nv_bfloat16>(g, s);
}

}  // namespace lpq
