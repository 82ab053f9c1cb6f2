// Products of a few bf16 token rows with 4-bit weights and group scales:
// y[i, n] = sum_k x[i, k] w[n, k], w = code * scale (* tensor scale).
//
// The weights are read once and are all the traffic there is, so the kernel is
// built around their stream: every lane copies its own 16 bytes (32 codes) of
// two weight rows, and their scales, some chunks ahead into a ring of its own
// in shared memory with cp.async (no registers, no barriers: a lane reads back
// only what it copied).  What bounds the work is instruction issue: at HBM's
// rate an SM has to take in 40 weights per cycle.  A byte of two E2M1 codes
// becomes an f16 pair in one conversion and is multiplied with its group scale
// (exact: 2 significant bits times 4); the products with x run on mma.m16n8k16
// (weights as the 16 rows, tokens as the 8 columns) with FP32 sums.  tcgen05
// would need the decoded weights written to shared memory first, for a product
// whose tensor work is small.
//
// Measured, weights and scales against the copy bandwidth of 6787 GB/s, NVFP4 at
// k = 4096 unless said: 524288 rows 192 us for one token (93%), 214 us for seven
// (83%); 131073 rows 53 us (83%) and 64 us (70%); 65536 rows 30 us (75%); 12288
// rows 11.4 us and 4096 rows 7 us, of which about 6 us are launch, the
// conversion of x and the join of the segments; MXFP4 4096 x 16384 14.4 us.
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

constexpr int kGroup = 128;         // rows of a group of the tensor-core scale layout: 8 tiles
constexpr int kChunk = 128;         // codes of a row per warp load: 4 lanes x 32
constexpr int kRing = 4;            // chunks in a warp's ring
constexpr int kStep = kRing * kChunk;  // segments of K are whole steps
constexpr int kSegments = 8;        // most parts of K (and CTAs of a cluster)
constexpr int kTokens = 8;          // most tokens of a pass: the columns of an MMA
constexpr int kXBytes = 128 * 1024; // most shared memory for x
constexpr int kSlot = 32 * 40;      // a chunk in a warp's ring: 2 x 16 bytes of codes, 2 x 4 of scales per lane

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
  int items;            // work items of W tiles (cluster > 1) or W / segments tiles
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
// come out 2^-8 down).  MXFP4, scale 2^e: f16 2^min(e, 13) (beyond that callers
// leave groups of zero codes alone, which any finite scale gives: infinity would
// make them NaN); bf16 2^(min(e, 1) + 126) and, where e > 1, the rest by mx_rest.
template <bool MX, bool F16>
__device__ __forceinline__ void scale_pairs(uint32_t s, uint32_t (&o)[2]) {
  if constexpr (MX) {
    if constexpr (F16) {
      const float f = __uint_as_float(min(s, 140u) << 23);
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
// Whether some group of a warp's chunk leaves f16: its scale 2^e outside e in
// [-23, 13] and a code of it not zero, or the scale that is no number.
__device__ __forceinline__ bool mx_far(const Load& l) {
  if (!__any_sync(0xFFFFFFFFu, l.slo - 104u > 36u || l.shi - 104u > 36u)) return false;
  auto outside = [](uint32_t s, const uint4& c) {
    return s - 104u > 36u && (s == 255u || ((c.x | c.y | c.z | c.w) & 0x77777777u));
  };
  return __any_sync(0xFFFFFFFFu, outside(l.slo, l.lo) || outside(l.shi, l.hi));
}
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  uint32_t h2;
  asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h2) : "h"((uint16_t)(code & 15u)));
  return __low2float(*reinterpret_cast<const __half2*>(&h2));
}

// The chunk's products.  e: the lane's x entries (16 bytes per word, words 4 *
// MP entries apart).
template <bool MX, bool F16, int MP>
__device__ __forceinline__ void chunk_products(const Load& l, const uint4* e, float (&acc)[4]) {
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
    const uint4 b = e[w * 4 * MP];
    mma<F16>(acc, pl[0], ph[0], pl[1], ph[1], b.x, b.y);
    mma<F16>(acc, pl[2], ph[2], pl[3], ph[3], b.z, b.w);
  }
}

// A chunk with MXFP4 groups that f16 cannot hold: plain FP32 dot products of
// the lane's 32 codes with each token, joined over the 4 lanes of a row and
// added to the warp's sums in shared memory ([token][row], in x's own scale).
// back: per token 2^-shift of the entries at e.
__device__ __noinline__ void far_chunk(uint4 lo, uint4 hi, uint32_t slo, uint32_t shi, const uint4* e, int mp, int mm,
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
      const uint4 b = e[(w * mp + token) * 4];
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
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool there) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
template <bool MX>
__device__ __forceinline__ uint32_t ld_shared_scale(uint32_t addr) {
  if constexpr (MX) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
  } else {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
  }
}

// MP: tokens that x's place in shared memory is laid out for (g.m or more).
// W warps per CTA: 8, four CTAs on an SM while x is small, else 24 that share x.
template <bool MX, bool SFG, int MP, int W>
__global__ void __launch_bounds__(32 * W, W == 8 ? 4 : 1) matvec_kernel(const MatvecArgs g) {
  constexpr int kThreads = 32 * W;
  extern __shared__ uint4 sx[];
  __shared__ float back_sh[kSegments * kTokens];  // 2^-shift of a segment's x
  __shared__ int fits_sh[kSegments * kTokens];
  let_dependents_start();
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, t = lane & 3;
  const bool shared_k = g.cluster > 1;  // the cluster's CTAs share K
  const int rank = shared_k ? (int)cluster_ctarank() : 0;
  const int first_item = blockIdx.x / g.cluster, item_step = gridDim.x / g.cluster;
  const int seg = shared_k ? rank : warp % g.segments;      // this warp's segment,
  const int slot = shared_k ? warp : warp / g.segments;     // its tile among the item's,
  const int slots = shared_k ? W : W / g.segments;          // and how many those are
  const int64_t m0 = (int64_t)blockIdx.y * g.m;
  const int mm = g.m;  // tokens of this pass
  // segments [seg0, seg1) of this CTA; segment i is steps [i * steps / segments, (i + 1) * steps / segments)
  const int seg0 = shared_k ? rank : 0, seg1 = shared_k ? rank + 1 : g.segments;
  auto seg_begin = [&](int i) { return i * g.steps / g.segments; };
  const int step0 = seg_begin(seg0);
  const int lo = seg_begin(seg), hi = seg_begin(seg + 1);  // this warp's steps
  constexpr int kSums = kTokens * 16;  // a warp's sums: [token][row]
  float* sums = reinterpret_cast<float*>(sx + (size_t)g.x_words * MP);  // two buffers of all warps'
  const uint32_t ring = smem_u32(sums + 2 * W * kSums) + warp * (kRing * kSlot);
  const uint32_t codes_sh = ring + lane * 16, scales_sh = ring + 1024 + lane * 4;  // the lane's places in a slot

  // ---- the weight stream: the lane's place in the step that is copied next
  constexpr int kChunkS = SFG ? (MX ? 512 : 1024) : (MX ? 4 : 8);  // scale bytes per chunk
  const int n_rows = (int)g.n;
  auto row_of = [&](int item, int sl, int r) {  // row r of 16 of an item's tile
    const int tile = item * slots + sl;
    return (tile >> 3) * kGroup + 32 * (r & 3) + 4 * (tile & 7) + (r >> 2);
  };
  const uint8_t *pc = nullptr, *pc2 = nullptr;  // codes of the lane's two rows
  const uint8_t *ps = nullptr, *ps2 = nullptr;  // their scales: a 4-byte word (plain layout: the lane's own bytes)
  int a_item = first_item, a_step = lo;
  enum { kNone, kWhole, kPartial };  // what of the step there is: nothing (no work left), all of it, up to K's end
  int a_kind = kNone;
  auto kind_of = [&]() { return (a_step + 1) * kStep <= g.k ? kWhole : kPartial; };
  auto set_item = [&]() {
    int row = row_of(a_item, slot, gid);
    // rows beyond the matrix read its last row; their results are not stored
    const bool two = row + 2 < n_rows;
    row = min(row, n_rows - 1);
    pc = g.codes + (int64_t)row * (g.k >> 1) + (int64_t)lo * (kStep / 2) + t * 16;
    ps = g.scales + (int64_t)lo * (kRing * kChunkS) +
         (SFG ? sf_gemm_offset(row, 0, g.kt) + (MX ? 0 : (t >> 1) * 512) : row * g.row_scales + (MX ? t : 2 * t));
    pc2 = pc + (two ? g.k : 0);
    ps2 = ps + (two ? (SFG ? 32 : 2 * g.row_scales) : 0);
  };
  auto copy = [&](int h) {  // chunk h of the step
    const uint32_t c = codes_sh + h * kSlot, sc = scales_sh + h * kSlot;
    if (a_kind == kWhole) {
      cp_async<16>(c, pc + h * (kChunk / 2));
      cp_async<16>(c + 512, pc2 + h * (kChunk / 2));
      if constexpr (SFG) {
        cp_async<4>(sc, ps + h * kChunkS);
        cp_async<4>(sc + 128, ps2 + h * kChunkS);
      }
    } else if (a_kind == kPartial) {
      const bool in = a_step * kStep + h * kChunk + t * 32 < g.k;
      cp_async_or_zero<16>(c, in ? pc + h * (kChunk / 2) : g.codes, in);
      cp_async_or_zero<16>(c + 512, in ? pc2 + h * (kChunk / 2) : g.codes, in);
      if constexpr (SFG) {
        cp_async_or_zero<4>(sc, in ? ps + h * kChunkS : g.scales, in);
        cp_async_or_zero<4>(sc + 128, in ? ps2 + h * kChunkS : g.scales, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto next_step = [&]() {
    if (a_kind == kNone) return;
    pc += kStep / 2;
    pc2 += kStep / 2;
    ps += kRing * kChunkS;
    ps2 += kRing * kChunkS;
    if (++a_step == hi) {
      a_step = lo;
      a_item += item_step;
      if (a_item >= g.items) {
        a_kind = kNone;
        return;
      }
      set_item();
    }
    a_kind = kind_of();
  };
  set_item();
  a_kind = kind_of();
#pragma unroll
  for (int h = 0; h < kRing; ++h) copy(h);
  // plain layout: the scales are loaded when the step begins
  const uint8_t *os = ps, *os2 = ps2;
  int o_step = lo;
  next_step();

  // ---- x as operand entries of 16 bytes, ordered by chunk, word, token, lane of
  // four (a warp's reads are contiguous in lane order)
  auto word = [&](int token, int i) {
    const int k = step0 * kStep + i * 8;
    return k < g.k ? __ldg(reinterpret_cast<const uint4*>(g.x + (m0 + token) * g.ldx + k)) : make_uint4(0, 0, 0, 0);
  };
  auto place = [&](int token, int i) { return (((i >> 4) * 4 + (i & 3)) * MP + token) * 4 + ((i >> 2) & 3); };
  // A token's part of a segment takes a warp, or several while there are more
  // warps than parts: each finds the part's range, then converts its share.
  const int parts = (seg1 - seg0) * mm, share = max(1, W / parts);
  for (int p = warp / share; p < parts; p += W / share) {
    const int sg = seg0 + p / mm, token = p % mm;
    const int w0 = (seg_begin(sg) - step0) * (kStep / 8), w1 = (seg_begin(sg + 1) - step0) * (kStep / 8);
    uint32_t top = 0, least = 0xFFFFFFFFu;  // pairs of 16-bit maxima of |x| and minima of |x| - 1 (0 wraps to the top)
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint4 v = word(token, i);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = u[j] & 0x7FFF7FFFu;
        top = __vmaxu2(top, m);
        least = __vminu2(least, __vsub2(m, 0x00010001u));
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, max(top >> 16, top & 0xFFFFu));
    least = __reduce_min_sync(0xFFFFFFFFu, min(least >> 16, least & 0xFFFFu)) + 1u;
    // x * 2^shift: the largest value's exponent field becomes 14 + 127 (at most
    // 126 steps up).  f16 holds a bf16 value exactly down to the field 110 (a
    // subnormal's leading bit lies up to 7 below field 1).
    const int shift = top ? min(141 - (int)max(top >> 7, 1u), 126) : 0;
    if (lane == 0) {
      back_sh[sg * kTokens + token] = __uint_as_float((uint32_t)(127 - shift) << 23);
      fits_sh[sg * kTokens + token] = top < 0x7F80u && (least > 0xFFFFu || (least >> 7 ? (int)(least >> 7) : -6) + shift >= 110);
    }
    const float f = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll 1
    for (int i = w0 + lane + 32 * (warp % share); i < w1; i += 32 * share) {
      const uint4 v = word(token, i);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h2 = __floats2half2_rn(bf16_lo(u[j]) * f, bf16_hi(u[j]) * f);
        r[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      sx[place(token, i)] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  __syncthreads();
  auto fits = [&](int sg) {
    bool all = true;
    for (int token = 0; token < mm; ++token) all = all && fits_sh[sg * kTokens + token];
    return all;
  };
  bool again = false;  // the same in all threads
  for (int sg = seg0; sg < seg1; ++sg) {
    if (fits(sg)) continue;
    again = true;  // x as bf16 pairs instead
    const int w0 = (seg_begin(sg) - step0) * (kStep / 8), w1 = (seg_begin(sg + 1) - step0) * (kStep / 8);
    for (int token = 0; token < mm; ++token)
      for (int i = w0 + threadIdx.x; i < w1; i += kThreads) {
        const uint4 v = word(token, i);
        sx[place(token, i)] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                         __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
      }
  }
  if (again) __syncthreads();

  const float tensor = MX ? 1.0f : *g.tensor_scale;
  auto put = [&](int row, int token, float v) {
    if (row >= n_rows || token >= mm) return;
    const int64_t at = (m0 + token) * g.n + row;
    if (g.y_fp32) static_cast<float*>(g.y)[at] = v * tensor;
    else static_cast<__nv_bfloat16*>(g.y)[at] = __float2bfloat16_rn(v * tensor);
  };
  // operand columns beyond the tokens hold anything: their sums are not stored
  const int col = min(gid, MP - 1) * 4 + t;
  const bool f16 = fits(seg);
  int jbuf = 0;
  for (int item = first_item; item < g.items; item += item_step, jbuf ^= 1) {
    float* mine = sums + (jbuf * W + warp) * kSums;
    float acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i] = 0.f;
      if constexpr (MX) mine[(2 * t + (i & 1)) * 16 + gid + (i >> 1) * 8] = 0.f;  // far_chunk adds to it
    }
    auto steps = [&](auto f16_path) {
      constexpr bool F16 = decltype(f16_path)::value;
      const uint4* e = sx + (size_t)(lo - step0) * (kStep / 8) * MP;
#pragma unroll 1
      for (int s = lo; s < hi; ++s, e += (kStep / 8) * MP) {
#pragma unroll
        for (int h = 0; h < kRing; ++h) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
          Load l;
          l.lo = ld_shared_16(codes_sh + h * kSlot);
          l.hi = ld_shared_16(codes_sh + h * kSlot + 512);
          if constexpr (SFG) {  // the lane's bytes of its word: NVFP4 (t & 1) * 2 on, MXFP4 t on
            const uint32_t at = scales_sh + h * kSlot + (MX ? t : (t & 1) * 2);
            l.slo = ld_shared_scale<MX>(at);
            l.shi = ld_shared_scale<MX>(at + 128);
          } else {
            l.slo = l.shi = 0;
            if (o_step * kStep + h * kChunk + t * 32 < g.k) {
              l.slo = MX ? os[h * kChunkS] : *reinterpret_cast<const uint16_t*>(os + h * kChunkS);
              l.shi = MX ? os2[h * kChunkS] : *reinterpret_cast<const uint16_t*>(os2 + h * kChunkS);
            }
          }
          const uint4* eh = e + h * (kChunk / 8) * MP;
          if (MX && F16 && mx_far(l))
            far_chunk(l.lo, l.hi, l.slo, l.shi, eh + t, MP, mm, back_sh + seg * kTokens, mine);
          else
            chunk_products<MX, F16, MP>(l, eh + col, acc);
          copy(h);  // into the slot whose values have just been used
        }
        if constexpr (!SFG) {  // (the step whose copies have just gone out is the next one)
          os = ps;
          os2 = ps2;
          o_step = a_step;
        }
        next_step();
      }
    };
    if (f16) steps(std::true_type{}); else steps(std::false_type{});
    // back to x's own scale (bf16 NVFP4 sums lie 2^-8 down)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int token = 2 * t + (i & 1);
      acc[i] *= f16 ? back_sh[seg * kTokens + min(token, mm - 1)] : MX ? 1.0f : 256.0f;
      if constexpr (MX) acc[i] += mine[token * 16 + gid + (i >> 1) * 8];
    }
    if (g.segments == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) put(row_of(item, slot, gid + (i >> 1) * 8), 2 * t + (i & 1), acc[i]);
      continue;
    }
    // The segments' sums meet in shared memory (two buffers: one barrier per
    // item) and are added in order; in a cluster each CTA adds its share.
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(2 * t + (i & 1)) * 16 + gid + (i >> 1) * 8] = acc[i];
    __syncwarp();
    if (shared_k) cluster_sync_all(); else __syncthreads();
    const int per = shared_k ? 16 * W / g.cluster : 16 * slots;  // (tile, row) places of this CTA, per token
    for (int e = threadIdx.x; e < per * MP; e += kThreads) {
      const int token = e % MP, r = rank * per + e / MP;
      if (token >= mm) continue;
      const int sl = r >> 4, at = token * 16 + (r & 15);
      float v = 0.f;
      if (shared_k) {
        const uint32_t here = smem_u32(sums + (jbuf * W + sl) * kSums + at);
        for (int c = 0; c < g.segments; ++c) v += ld_shared_cluster(mapa_shared(here, (uint32_t)c));
      } else {
        const float* from = sums + (jbuf * W + sl * g.segments) * kSums + at;
        for (int c = 0; c < g.segments; ++c) v += from[c * kSums];
      }
      put(row_of(item, sl, r & 15), token, v);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (shared_k) cluster_sync_all();  // no CTA leaves while another may still read its sums
}

constexpr int kLayouts[] = {1, 2, kTokens};  // MP
int layout_for(int tokens) {
  for (int mp : kLayouts)
    if (tokens <= mp) return mp;
  return kTokens;
}

template <bool MX, bool SFG, int MP, int W>
lpq_status run_matvec(MatvecArgs g, int passes, cudaStream_t s) {
  constexpr int kSumBytes = 2 * W * kTokens * 16 * 4;
  const int seg_steps = (g.steps + g.segments - 1) / g.segments;
  g.x_words = (g.cluster > 1 ? seg_steps : g.steps) * (kStep / 8);
  const int smem = g.x_words * 16 * MP + kSumBytes + W * kRing * kSlot;
  const void* kernel = reinterpret_cast<const void*>(matvec_kernel<MX, SFG, MP, W>);
  lpq_status st = set_smem_attr(kernel, 222 * 1024);
  if (st != LPQ_OK) return st;
  const int64_t tiles = (g.n + kGroup - 1) / kGroup * 8, per = g.cluster > 1 ? W : W / g.segments;
  g.items = (int)((tiles + per - 1) / per);
  const int resident = std::max(1, std::min(W == 8 ? 4 : 1, 226 * 1024 / (smem + 2048)));
  const int most = std::max(1, resident * device_sms() / g.cluster);
  const dim3 grid((unsigned)(std::min(g.items, most) * g.cluster), (unsigned)passes);
  if (g.cluster == 1)
    return cuda_check(launch_dependent(matvec_kernel<MX, SFG, MP, W>, grid, 32 * W, smem, s, g), "matvec launch");
  // Clusters start when the stream is done: an early start would place them
  // around the kernel ahead and leave the SMs unevenly loaded (16384 -> 4096:
  // 19.9 us, 14.7 us so).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)g.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, matvec_kernel<MX, SFG, MP, W>, g), "matvec launch");
}

template <bool MX>
lpq_status run_tokens(const MatvecArgs& g, int passes, bool plain, bool wide_cta, cudaStream_t s) {
  if (plain) return run_matvec<MX, false, kTokens, 8>(g, passes, s);
  if (wide_cta) return g.m > 2 ? run_matvec<MX, true, kTokens, 24>(g, passes, s) : run_matvec<MX, true, 2, 24>(g, passes, s);
  return g.m > 2 ? run_matvec<MX, true, kTokens, 8>(g, passes, s)
         : g.m == 2 ? run_matvec<MX, true, 2, 8>(g, passes, s) : run_matvec<MX, true, 1, 8>(g, passes, s);
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
  // Tokens per pass: 8 or fewer, what fits a CTA's shared memory when a
  // cluster shares K.
  const bool plain = w->sf_layout == LPQ_SF_PLAIN;
  const int seg_bytes = (g.steps + g.segments - 1) / g.segments * kStep * 2;  // of one token's x
  int most = 1;
  for (int mp : kLayouts)
    if (mp * seg_bytes <= kXBytes) most = mp;
  for (int64_t m0 = 0; m0 < m;) {
    // Passes of equal width share a launch; the rest has one of its own.
    const int64_t left = m - m0;
    g.m = (int)std::min<int64_t>(left, most);
    const int64_t passes = std::min<int64_t>(left / g.m, 65535);
    // Clusters while a group's CTAs all run at once, or when x of all segments
    // is more than a CTA has room for.  Else 8 warps while four CTAs' x fit on
    // an SM, or 24 that share it.
    const int64_t groups = (g.n + kGroup - 1) / kGroup;
    const int mp = layout_for(g.m), token_bytes = g.steps * kStep * 2;
    const bool wide_cta = !plain && token_bytes * mp > 12 * 1024;
    const int x_bytes = token_bytes * (wide_cta ? std::max(mp, 2) : plain ? kTokens : mp);
    g.cluster = groups * g.segments <= 4 * device_sms() || x_bytes > (wide_cta ? 64 : 24) * 1024 ? g.segments : 1;
    g.x = static_cast<const __nv_bfloat16*>(x) + m0 * ldx;
    g.y = static_cast<uint8_t*>(y) + (size_t)m0 * (size_t)g.n * (y_is_fp32 ? 4 : 2);
    lpq_status st = (mx ? run_tokens<true> : run_tokens<false>)(g, (int)passes, plain, wide_cta && g.cluster == 1, s);
    if (st != LPQ_OK) return st;
    m0 += passes * g.m;
  }
  return LPQ_OK;
}

}  // namespace lpq
