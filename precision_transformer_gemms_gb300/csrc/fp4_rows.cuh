// Rows of 4-bit weights in a warp: 16-byte asynchronous loads per lane, decoding,
// and products with a few tokens on mma.m16n8k16 (weights as the 16 rows, tokens
// as the 8 columns).  Shared by the kernels whose traffic is the weights.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kGroup = 128;         // rows of a group of the tensor-core scale layout: 8 tiles
constexpr int kChunk = 128;         // codes of a row per warp load: 4 lanes x 32
constexpr int kTokens = 8;          // most tokens of a pass: the columns of an MMA
constexpr int kSlot = 32 * 40;      // a chunk in a warp's ring: 2 x 16 bytes of codes, 2 x 4 of scales per lane

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
// MP entries apart; of 16 columns, those from 8 on add to the sums of the first 8).
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
    if constexpr (MP > kTokens) {
      const uint4 c = e[w * 4 * MP + kTokens * 4];
      mma<F16>(acc, pl[0], ph[0], pl[1], ph[1], c.x, c.y);
      mma<F16>(acc, pl[2], ph[2], pl[3], ph[3], c.z, c.w);
    }
  }
}

// A chunk with MXFP4 groups that f16 cannot hold: plain FP32 dot products of
// the lane's 32 codes with each token, joined over the 4 lanes of a row and
// added to the warp's sums in shared memory ([token][row], in x's own scale).
// back: per token 2^-shift of the entries at e.  TERMS == 2: x is the sum of the
// columns token and token + mp / 2.
template <int TERMS>
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
      const uint4 b2 = TERMS == 2 ? e[(w * mp + mp / 2 + token) * 4] : b;
      const uint32_t u2[4] = {b2.x, b2.y, b2.z, b2.w};
      const uint32_t cl = w == 0 ? lo.x : w == 1 ? lo.y : w == 2 ? lo.z : lo.w;
      const uint32_t ch = w == 0 ? hi.x : w == 1 ? hi.y : w == 2 ? hi.z : hi.w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[i >> 1]));
        float xv = i & 1 ? p.y : p.x;
        if constexpr (TERMS == 2) {
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&u2[i >> 1]));
          xv += i & 1 ? q.y : q.x;
        }
        xv *= f;
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

}  // namespace
}  // namespace lpq
