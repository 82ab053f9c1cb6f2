// Products of a few bf16 token rows with 4-bit weights and group scales:
// y[i, n] = sum_k x[i, k] w[n, k], w = code * scale (* tensor scale).
//
// The weights are read once and are all the traffic there is, so the kernel is
// built around their stream: a lane keeps three 16-byte loads (32 codes each)
// of two weight rows in flight while it works on a fourth.  What bounds the
// work is instruction issue: at HBM's rate an SM has to take in 40 weights per
// cycle.  A byte of two E2M1 codes becomes an f16 pair in one conversion and
// is multiplied with its group scale (exact: 2 significant bits times 4); the
// products with x run on mma.m16n8k16 (weights as the 16 rows, tokens as the 8
// columns) with FP32 sums, 1.4 instructions per weight and lane in all.
// tcgen05 would need the decoded weights written to shared memory first, for a
// product whose tensor work is small.
//
// x enters as f16 too: a token's values times a power of two that brings its
// largest one to [2^14, 2^15).  A bf16 value has 8 significant bits, so this
// is exact down to 2^-31 of the largest.  Where a nonzero x is smaller than
// that, the CTA takes bf16 operands instead (twice the instructions: bf16 has
// no conversion from E2M1).  Either way codes, scales and x are exact and only
// the FP32 sums round.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 128;         // rows of a group of the tensor-core scale layout: 8 tiles
constexpr int kChunk = 128;         // codes of a row per warp load: 4 lanes x 32
constexpr int kBufs = 4;            // loads per row in registers
constexpr int kStep = kBufs * kChunk;
constexpr int kSegments = 8;        // most parts of K (and CTAs of a cluster)
constexpr int kXBytes = 160 * 1024; // most shared memory for x

struct MatvecArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;
  const __nv_bfloat16* x;
  void* y;
  int64_t ldx;
  int64_t n;
  int k;
  int m;               // tokens
  int64_t kt;          // scale atoms per 128-row group
  int64_t row_scales;  // scales per row (plain layout)
  int y_fp32;
  int steps, segments;  // K in steps, and in parts that are summed by themselves
  int cluster;          // 1, or a CTA per segment
  int items;            // work items of 8 tiles (cluster > 1) or 8 / segments tiles
  int x_words;          // 16-byte words of x that a CTA has room for, per token
};

template <bool F16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 codes -> four pairs.  f16: the codes 2 i and 2 i + 1, their values.
// bf16: the codes i and i + 4, their values * 2^-126 (the code's exponent and
// mantissa bits are the low bits of a bf16 with the same meaning, subnormals
// included, 126 exponent steps down).
template <bool F16>
__device__ __forceinline__ void decode8(uint32_t u, uint32_t (&p)[4]) {
  if constexpr (F16) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3]) : "r"(u));
  } else {
    p[0] = ((u << 12) & 0x80008000u) | ((u << 6) & 0x01C001C0u);
    p[1] = ((u << 8) & 0x80008000u) | ((u << 2) & 0x01C001C0u);
    p[2] = ((u << 4) & 0x80008000u) | ((u >> 2) & 0x01C001C0u);
    p[3] = (u & 0x80008000u) | ((u >> 6) & 0x01C001C0u);
  }
}

// A lane's part of a chunk: 32 codes of two rows and their scales (NVFP4 two
// E4M3 bytes, MXFP4 one E8M0 byte per row).
struct Load {
  uint4 lo, hi;
  uint32_t slo, shi;
};

// The two group scales of a lane's 32 codes as operand pairs.  NVFP4: f16 the
// scale, bf16 the scale * 2^118 (the decoded values lie 2^-126 down, the sums
// come out 2^-8 down).  MXFP4, scale 2^e: f16 2^e (callers see to the range);
// bf16 2^(min(e, 1) + 126) and, where e > 1, the rest by mx_rest.
template <bool MX, bool F16>
__device__ __forceinline__ void scale_pairs(uint32_t s, uint32_t (&o)[2]) {
  if constexpr (MX) {
    if constexpr (F16) {
      const float f = __uint_as_float(s << 23);
      const __half2 h = __floats2half2_rn(f, f);
      o[0] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      o[0] = (min(s, 128u) + 126u) * 0x00800080u;
    }
    o[1] = o[0];
  } else {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)s));
    if constexpr (F16) {
      o[0] = __byte_perm(h2, h2, 0x1010);
      o[1] = __byte_perm(h2, h2, 0x3232);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      const uint32_t a = __float_as_uint(f.x * 3.3230700e35f), b = __float_as_uint(f.y * 3.3230700e35f);  // 2^118
      o[0] = __byte_perm(a, a, 0x3232);
      o[1] = __byte_perm(b, b, 0x3232);
    }
  }
}
__device__ __forceinline__ uint32_t mx_rest(uint32_t s) {  // 2^(e - 1) where e > 1, else 1; NaN for 255
  return s == 255u ? 0x7FC07FC0u : (max(s, 128u) - 1u) * 0x00800080u;
}
// Whether 2^e times some code of c leaves f16: e outside [-23, 13] with a code
// that is not zero, or the scale that is no number.
__device__ __forceinline__ bool mx_outside(uint32_t s, const uint4& c) {
  return (s - 104u > 36u && ((c.x | c.y | c.z | c.w) & 0x77777777u)) || s == 255u;
}
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  uint32_t h2;
  asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h2) : "h"((uint16_t)(code & 15u)));
  return __low2float(*reinterpret_cast<const __half2*>(&h2));
}

// The chunk's products.  e: the lane's x entries per column block (16 bytes per
// word, words 4 * mm entries apart).
template <bool MX, bool F16, int NT>
__device__ __forceinline__ void chunk_products(const Load& l, const uint4* const (&e)[NT], int mm, float (&acc)[NT][4]) {
  uint32_t sl[2], sh[2], xl = 0, xh = 0;
  scale_pairs<MX, F16>(l.slo, sl);
  scale_pairs<MX, F16>(l.shi, sh);
  bool rest = false;
  if constexpr (MX && !F16) {
    rest = __any_sync(0xFFFFFFFFu, l.slo > 128u || l.shi > 128u);
    xl = mx_rest(l.slo);
    xh = mx_rest(l.shi);
  }
  const uint32_t wl[4] = {l.lo.x, l.lo.y, l.lo.z, l.lo.w};
  const uint32_t wh[4] = {l.hi.x, l.hi.y, l.hi.z, l.hi.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t pl[4], ph[4];
    decode8<F16>(wl[w], pl);
    decode8<F16>(wh[w], ph);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pl[i] = mul2<F16>(pl[i], sl[w >> 1]);
      ph[i] = mul2<F16>(ph[i], sh[w >> 1]);
    }
    if constexpr (MX && !F16) {
      if (rest) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pl[i] = mul2<F16>(pl[i], xl);
          ph[i] = mul2<F16>(ph[i], xh);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 b = e[n][w * 4 * mm];
      mma<F16>(acc[n], pl[0], ph[0], pl[1], ph[1], b.x, b.y);
      mma<F16>(acc[n], pl[2], ph[2], pl[3], ph[3], b.z, b.w);
    }
  }
}

// A chunk with MXFP4 groups that f16 cannot hold: plain FP32 dot products of
// the lane's 32 codes with each token, joined over the 4 lanes of a row and
// added to the warp's sums in shared memory ([token][row], x's own scale).
// back: per token 2^-shift of the entries at e.
__device__ __noinline__ void far_chunk(uint4 lo, uint4 hi, uint32_t slo, uint32_t shi, const uint4* e, int mm,
                                       const float* back, float* sums) {
  const int lane = threadIdx.x & 31, t = lane & 3, gid = lane >> 2;
  const float fl = slo == 255u ? __int_as_float(0x7FC00000) : pow2_exact((int)slo - 127);
  const float fh = shi == 255u ? __int_as_float(0x7FC00000) : pow2_exact((int)shi - 127);
#pragma unroll 1
  for (int token = 0; token < mm; ++token) {
    const float f = back[token];
    float dl = 0.f, dh = 0.f;
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
      const uint4 b = e[w * 4 * mm + token];
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
      const uint32_t cl = w == 0 ? lo.x : w == 1 ? lo.y : w == 2 ? lo.z : lo.w;
      const uint32_t ch = w == 0 ? hi.x : w == 1 ? hi.y : w == 2 ? hi.z : hi.w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[i >> 1]));
        const float xv = (i & 1 ? p.y : p.x) * f;
        dl += e2m1_value(cl >> (4 * i)) * xv;
        dh += e2m1_value(ch >> (4 * i)) * xv;
      }
    }
    dl *= fl;
    dh *= fh;
    dl += __shfl_xor_sync(0xFFFFFFFFu, dl, 1);
    dh += __shfl_xor_sync(0xFFFFFFFFu, dh, 1);
    dl += __shfl_xor_sync(0xFFFFFFFFu, dl, 2);
    dh += __shfl_xor_sync(0xFFFFFFFFu, dh, 2);
    if (((token & 7) >> 1) == t) {  // the lane that holds this token's column
      sums[token * 16 + gid] += dl;
      sums[token * 16 + gid + 8] += dh;
    }
  }
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A warp's tile is 16 weight rows: 4 runs of 4 neighbours, 32 apart (rows 32 j
// + i of a 128-row group, i in a run of 4), whose scales of 4 neighbouring
// blocks are 64 consecutive bytes of the tensor-core layout.  K is cut into
// segments by its length alone and a warp sums one segment.  With many tiles a
// CTA's warps take all segments of a few tiles, with x of all of K in shared
// memory; with few a cluster of CTAs takes 8 tiles, one segment (and x of it)
// per CTA, and joins the sums through distributed shared memory.  The segments'
// sums are added in the same order either way: a row's result does not depend
// on the number of rows.
template <bool MX, bool SFG, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 && !MX ? 2 : 2) matvec_kernel(const MatvecArgs g) {
  extern __shared__ uint4 sx[];
  constexpr int kCols = 8 * NT;
  __shared__ uint32_t top_sh[kSegments * kCols], least_sh[kSegments * kCols];
  __shared__ float back_sh[kSegments * kCols];  // 2^-shift
  __shared__ int f16_sh[kSegments];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, t = lane & 3;
  const bool shared_k = g.cluster > 1;  // the cluster's CTAs share K
  const int rank = shared_k ? (int)cluster_ctarank() : 0;
  const int first_item = blockIdx.x / g.cluster, item_step = gridDim.x / g.cluster;
  const int seg = shared_k ? rank : warp % g.segments;                     // this warp's segment,
  const int slot = shared_k ? warp : warp / g.segments;                    // its tile among the item's,
  const int slots = shared_k ? kWarps : kWarps / g.segments;               // and how many those are
  const int64_t m0 = (int64_t)blockIdx.y * g.m;
  const int mm = g.m;
  // segments [seg0, seg1) of this CTA; segment i is steps [i * steps / segments, (i + 1) * steps / segments)
  const int seg0 = shared_k ? rank : 0, seg1 = shared_k ? rank + 1 : g.segments;
  auto seg_begin = [&](int i) { return i * g.steps / g.segments; };
  const int step0 = seg_begin(seg0);
  const int lo = seg_begin(seg), hi = seg_begin(seg + 1);  // this warp's steps
  constexpr int kSums = kCols * 16 * (MX ? 2 : 1);  // a warp's sums: [token][row], then those of far_chunk
  float* sums = reinterpret_cast<float*>(sx + (size_t)g.x_words * mm);  // two buffers of all warps'

  // ---- the weight stream
  constexpr int kChunkS = SFG ? (MX ? 512 : 1024) : (MX ? 4 : 8);  // scale bytes per chunk
  const int lane_s = MX ? t : SFG ? (t >> 1) * 512 + (t & 1) * 2 : t * 2;
  const uint8_t* pc = nullptr;  // the lane's first row: codes and scales
  const uint8_t* ps = nullptr;
  int64_t hi_c = 0, hi_s = 0;  // its second row lies 2 rows on
  auto row_of = [&](int item, int sl, int r) {  // row r of 16 of an item's tile
    const int64_t tile = (int64_t)item * slots + sl;
    return (tile >> 3) * kGroup + 32 * (r & 3) + 4 * (tile & 7) + (r >> 2);
  };
  auto set_item = [&](int item) {
    int64_t row = row_of(item, slot, gid);
    // rows beyond the matrix read its last row; their results are not stored
    const bool two = row + 2 < g.n;
    row = min(row, g.n - 1);
    pc = g.codes + row * (g.k >> 1);
    ps = g.scales + (SFG ? sf_gemm_offset(row, 0, g.kt) : row * g.row_scales);
    hi_c = two ? g.k : 0;
    hi_s = two ? (SFG ? 32 : 2 * g.row_scales) : 0;
  };
  auto fetch = [&](const uint8_t* c, const uint8_t* s, Load& l) {
    l.lo = __ldcs(reinterpret_cast<const uint4*>(c));
    l.hi = __ldcs(reinterpret_cast<const uint4*>(c + hi_c));
    if constexpr (MX) {
      l.slo = *s;
      l.shi = s[hi_s];
    } else {
      l.slo = *reinterpret_cast<const uint16_t*>(s);
      l.shi = *reinterpret_cast<const uint16_t*>(s + hi_s);
    }
  };
  // Chunk h of a step whose first chunk's codes and scales are at c and s.
  auto load = [&](const uint8_t* c, const uint8_t* s, int step, int h, Load& l) {
    if ((step + 1) * kStep <= g.k || step * kStep + h * kChunk + t * 32 < g.k) {
      fetch(c + h * (kChunk / 2), s + h * kChunkS, l);
    } else {  // past the end of K: the row's first block again, with scale 0 (and x 0)
      fetch(pc, ps, l);
      l.slo = l.shi = 0;
    }
  };
  auto codes_at = [&](int step) { return pc + (int64_t)step * (kStep / 2) + t * 16; };
  auto scales_at = [&](int step) { return ps + (int64_t)step * (kBufs * kChunkS) + lane_s; };
  Load buf[kBufs];
  set_item(first_item);
#pragma unroll
  for (int h = 0; h < kBufs; ++h) load(codes_at(lo), scales_at(lo), lo, h, buf[h]);

  // ---- x as operand entries of 16 bytes, ordered by chunk, word, lane, token
  // (a warp's reads are contiguous): first as it is with its range, then converted
  for (int i = threadIdx.x; i < kSegments * kCols; i += kThreads) {
    top_sh[i] = 0;
    least_sh[i] = 0xFFFFu;
  }
  const int words = (seg_begin(seg1) - step0) * (kStep / 8);  // 16-byte words per token, a multiple of 64
  auto segment_of = [&](int i) {  // of word i; a warp's 32 words lie in one token and one segment
    return shared_k ? rank : ((i / (kStep / 8) + 1) * g.segments - 1) / g.steps;
  };
  auto place = [&](int token, int i) { return (((i >> 4) * 4 + (i & 3)) * 4 + ((i >> 2) & 3)) * mm + token; };
  auto advance = [&](int& token, int& i) {
    i += kThreads;
    while (i >= words) {
      i -= words;
      ++token;
    }
  };
  __syncthreads();
  constexpr int kAhead = 8;  // loads in flight per thread
  for (int token = threadIdx.x / words, i = threadIdx.x % words; token < mm;) {
    uint4 v[kAhead];
    int tk = token, at = i;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      v[a] = make_uint4(0, 0, 0, 0);
      const int k = step0 * kStep + at * 8;
      if (tk < mm && k < g.k) v[a] = *reinterpret_cast<const uint4*>(g.x + (m0 + tk) * g.ldx + k);
      advance(tk, at);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (token < mm) {
        const uint32_t u[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
        uint32_t top = 0, least = 0xFFFFFFFFu;  // pairs of 16-bit maxima of |x| and minima of |x| - 1 (0 wraps to the top)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t m = u[j] & 0x7FFF7FFFu;
          top = __vmaxu2(top, m);
          least = __vminu2(least, __vsub2(m, 0x00010001u));
        }
        top = __reduce_max_sync(0xFFFFFFFFu, max(top >> 16, top & 0xFFFFu));
        least = __reduce_min_sync(0xFFFFFFFFu, min(least >> 16, least & 0xFFFFu));
        if (lane == 0) {
          const int to = segment_of(i) * kCols + token;
          atomicMax(&top_sh[to], top);
          atomicMin(&least_sh[to], least);
        }
        sx[place(token, i)] = v[a];
      }
      advance(token, i);
    }
  }
  __syncthreads();
  // x * 2^shift: the largest value's exponent field becomes 14 + 127 (at most
  // 126 steps up).  f16 holds a bf16 value exactly down to the field 110 (a
  // subnormal's leading bit lies up to 7 below field 1).
  if (threadIdx.x < kSegments) f16_sh[threadIdx.x] = 1;
  __syncthreads();
  if (threadIdx.x < kSegments * kCols) {
    const uint32_t top = top_sh[threadIdx.x], least = least_sh[threadIdx.x] + 1u;
    const int shift = top ? min(141 - (int)max(top >> 7, 1u), 126) : 0;
    if (top >= 0x7F80u || (least <= 0xFFFFu && (least >> 7 ? (int)(least >> 7) : -6) + shift < 110))
      f16_sh[threadIdx.x / kCols] = 0;
    back_sh[threadIdx.x] = __uint_as_float((uint32_t)(127 - shift) << 23);
  }
  __syncthreads();
  if (threadIdx.x < kSegments * kCols && !f16_sh[threadIdx.x / kCols]) back_sh[threadIdx.x] = 1.0f;
  __syncthreads();
  for (int token = threadIdx.x / words, i = threadIdx.x % words; token < mm; advance(token, i)) {
    const int sg = segment_of(i);
    uint4& e = sx[place(token, i)];
    const uint32_t u[4] = {e.x, e.y, e.z, e.w};
    if (f16_sh[sg]) {
      const float f = __uint_as_float(0x7F000000u - __float_as_uint(back_sh[sg * kCols + token]));  // 2^shift
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h2 = __floats2half2_rn(bf16_lo(u[j]) * f, bf16_hi(u[j]) * f);
        r[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      e = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      e = make_uint4(__byte_perm(u[0], u[2], 0x5410), __byte_perm(u[0], u[2], 0x7632),
                     __byte_perm(u[1], u[3], 0x5410), __byte_perm(u[1], u[3], 0x7632));
    }
  }
  __syncthreads();

  const float tensor = MX ? 1.0f : *g.tensor_scale;
  auto put = [&](int64_t row, int token, float v) {
    if (row >= g.n || token >= mm) return;
    const int64_t at = (m0 + token) * g.n + row;
    if (g.y_fp32) static_cast<float*>(g.y)[at] = v * tensor;
    else static_cast<__nv_bfloat16*>(g.y)[at] = __float2bfloat16_rn(v * tensor);
  };
  // columns beyond the tokens repeat the last one: their sums are not stored
  int col[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) col[n] = t * mm + min(gid + 8 * n, mm - 1);

  const bool f16 = f16_sh[seg];
  int jbuf = 0;
  for (int item = first_item; item < g.items; item += item_step, jbuf ^= 1) {
    float* mine = sums + (jbuf * kWarps + warp) * kSums;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[n][i] = 0.f;
        if constexpr (MX) mine[kCols * 16 + (8 * n + 2 * t + (i & 1)) * 16 + gid + (i >> 1) * 8] = 0.f;
      }
    auto steps = [&](auto f16_path) {
      constexpr bool F16 = decltype(f16_path)::value;
      for (int s = lo; s < hi; ++s) {
        // the step whose loads go out now (at the very end the last item's first again)
        int ns = s + 1;
        if (ns == hi) {
          ns = lo;
          if (item + item_step < g.items) set_item(item + item_step);
        }
        const uint8_t* c = codes_at(ns);
        const uint8_t* sc = scales_at(ns);
        const uint4* e = sx + (size_t)((s - step0) * (kStep / 8)) * mm;
#pragma unroll
        for (int h = 0; h < kBufs; ++h) {
          const uint4* cols[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) cols[n] = e + h * 16 * mm + col[n];
          if (MX && F16 &&
              __any_sync(0xFFFFFFFFu, mx_outside(buf[h].slo, buf[h].lo) || mx_outside(buf[h].shi, buf[h].hi)))
            far_chunk(buf[h].lo, buf[h].hi, buf[h].slo, buf[h].shi, e + h * 16 * mm + t * mm, mm,
                      back_sh + seg * kCols, mine + kCols * 16);
          else
            chunk_products<MX, F16, NT>(buf[h], cols, mm, acc);
          load(c, sc, ns, h, buf[h]);
        }
      }
    };
    if (f16) steps(std::true_type{}); else steps(std::false_type{});
    // back to x's own scale (bf16 NVFP4 sums lie 2^-8 down)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = 8 * n + 2 * t + (i & 1);
        acc[n][i] *= back_sh[seg * kCols + min(token, mm - 1)] * (f16 || MX ? 1.0f : 256.0f);
      }
    if (g.segments == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = 8 * n + 2 * t + (i & 1), r = gid + (i >> 1) * 8;
          put(row_of(item, slot, r), token, acc[n][i] + (MX ? mine[kCols * 16 + token * 16 + r] : 0.f));
        }
      continue;
    }
    // The segments' sums meet in shared memory (two buffers: one barrier per
    // item) and are added in order; in a cluster each CTA adds its share.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(8 * n + 2 * t + (i & 1)) * 16 + gid + (i >> 1) * 8] = acc[n][i];
    __syncwarp();
    if (shared_k) cluster_sync_all(); else __syncthreads();
    const int per = shared_k ? kGroup / g.cluster : 16 * slots;  // (tile, row) places of this CTA, per token
    for (int e = threadIdx.x; e < per * mm; e += kThreads) {
      const int token = e / per, r = rank * per + e % per;
      const int sl = r >> 4, at = token * 16 + (r & 15);
      float v = 0.f, f = 0.f;
      if (shared_k) {
        const uint32_t here = smem_u32(sums + (jbuf * kWarps + sl) * kSums + at);
        for (int c = 0; c < g.segments; ++c) {
          const uint32_t from = mapa_shared(here, (uint32_t)c);
          v += ld_shared_cluster(from);
          if constexpr (MX) f += ld_shared_cluster(from + kCols * 16 * 4);
        }
      } else {
        const float* from = sums + (jbuf * kWarps + sl * g.segments) * kSums + at;
        for (int c = 0; c < g.segments; ++c) {
          v += from[c * kSums];
          if constexpr (MX) f += from[c * kSums + kCols * 16];
        }
      }
      put(row_of(item, sl, r & 15), token, v + f);
    }
  }
  if (shared_k) cluster_sync_all();  // no CTA leaves while another may still read its sums
}

template <bool MX, bool SFG, int NT>
lpq_status run_matvec(MatvecArgs g, int passes, cudaStream_t s) {
  constexpr int kSumBytes = 2 * kWarps * NT * 128 * 4 * (MX ? 2 : 1);
  const int seg_steps = (g.steps + g.segments - 1) / g.segments;
  g.x_words = (g.cluster > 1 ? seg_steps : g.steps) * (kStep / 8);
  const int smem = g.x_words * 16 * g.m + (MX || g.segments > 1 ? kSumBytes : 0);
  lpq_status st = set_smem_attr(reinterpret_cast<const void*>(matvec_kernel<MX, SFG, NT>), kXBytes + kSumBytes);
  if (st != LPQ_OK) return st;
  const int resident = NT == 1 && !MX ? 2 : 2;
  const int64_t tiles = (g.n + kGroup - 1) / kGroup * 8, per = g.cluster > 1 ? kWarps : kWarps / g.segments;
  g.items = (int)((tiles + per - 1) / per);
  const int most = std::max(1, resident * device_sms() / g.cluster);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(std::min(g.items, most) * g.cluster), (unsigned)passes);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)g.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, matvec_kernel<MX, SFG, NT>, g), "matvec launch");
}

}  // namespace

lpq_status launch_matvec(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, void* y, int32_t y_is_fp32,
                         cudaStream_t s) {
  if (m == 0 || w->rows == 0) return LPQ_OK;
  if (w->cols == 0)  // empty reduction: y = 0
    return cuda_check(cudaMemsetAsync(y, 0, (size_t)m * (size_t)w->rows * (y_is_fp32 ? 4 : 2), s), "cudaMemsetAsync(y)");
  const bool mx = w->fmt == LPQ_MXFP4;
  MatvecArgs g{};
  g.codes = static_cast<const uint8_t*>(w->codes);
  g.scales = static_cast<const uint8_t*>(w->scales);
  g.tensor_scale = w->tensor_scale;
  g.ldx = ldx;
  g.n = w->rows;
  g.k = (int)w->cols;
  g.kt = sf_kt_atoms(w->fmt, w->cols);
  g.row_scales = w->cols / (mx ? 32 : 16);
  g.y_fp32 = y_is_fp32;
  g.steps = (g.k + kStep - 1) / kStep;
  g.segments = 1;
  while (g.segments < kSegments && 4 * g.segments <= g.steps) g.segments *= 2;
  // Tokens per pass: 16 or fewer, what fits a CTA's shared memory when a
  // cluster shares K.
  const int seg_bytes = (g.steps + g.segments - 1) / g.segments * kStep * 2;  // of one token's x
  const int most = std::min(16, kXBytes / seg_bytes);
  for (int64_t m0 = 0; m0 < m;) {
    // Passes of equal width share a launch; the rest has one of its own.
    const int64_t left = m - m0;
    g.m = (int)std::min<int64_t>(left, most);
    const int64_t passes = std::min<int64_t>(left / g.m, 65535);
    // Clusters while a group's CTAs all run at once, or when x of all segments
    // takes more than a third of an SM's shared memory.
    const int64_t groups = (g.n + kGroup - 1) / kGroup;
    g.cluster = groups * g.segments <= 3 * device_sms() || g.steps * kStep * 2 * g.m > 60 * 1024 ? g.segments : 1;
    g.x = static_cast<const __nv_bfloat16*>(x) + m0 * ldx;
    g.y = static_cast<uint8_t*>(y) + (size_t)m0 * (size_t)g.n * (y_is_fp32 ? 4 : 2);
    const bool plain = w->sf_layout == LPQ_SF_PLAIN, wide = g.m > 8;
    auto run = mx ? (plain ? (wide ? run_matvec<true, false, 2> : run_matvec<true, false, 1>)
                           : (wide ? run_matvec<true, true, 2> : run_matvec<true, true, 1>))
                  : (plain ? (wide ? run_matvec<false, false, 2> : run_matvec<false, false, 1>)
                           : (wide ? run_matvec<false, true, 2> : run_matvec<false, true, 1>));
    lpq_status st = run(g, (int)passes, s);
    if (st != LPQ_OK) return st;
    m0 += passes * g.m;
  }
  return LPQ_OK;
}

}  // namespace lpq
