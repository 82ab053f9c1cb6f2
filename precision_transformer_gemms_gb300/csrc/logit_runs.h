// How a row of v logits is cut into runs of words and which place of a run a word has:
// plain integer arithmetic, shared by the kernel, its launch and a test on the host.
#pragma once
#include <stdint.h>

#ifndef LPQ_HOST_DEVICE
#ifdef __CUDACC__
#define LPQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define LPQ_HOST_DEVICE inline
#endif
#endif

namespace lpq {

// Runs of s words for a row of v, which may begin vec - 1 places into its first one.
LPQ_HOST_DEVICE int64_t run_count(int64_t v, int vec, int s) { return (v + vec - 1 + s - 1) / s; }

// Word of a run's first place, in a row that begins `lead` places into its first run.
LPQ_HOST_DEVICE int run_first(int run, int s, int lead) { return run * s - lead; }

// Places of a run up to the row's end: 0 in a last run that begins behind it (the runs
// are counted for a row that begins as far into its first one as it may).
LPQ_HOST_DEVICE int run_words(int first, int s, int v) {
  const int left = v - first;
  return left < 0 ? 0 : left < s ? left : s;
}

// The word's place in a run of that many, or -1.  (A word just below 0 may be given a
// place in front of the row's first, which nothing reads.)
LPQ_HOST_DEVICE int run_place(int64_t word, int first, int words) {
  const uint64_t p = (uint64_t)word - (uint64_t)(int64_t)first;
  return p < (uint64_t)words ? (int)p : -1;
}

// A control's number of entries or place among `count` of them, whatever it holds.
LPQ_HOST_DEVICE int64_t within(int64_t n, int64_t count) { return n < 0 ? 0 : n < count ? n : count; }

}  // namespace lpq
