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
//
// With adapters, y[i, n] gains s B_e (A_e x_i) for the low-rank pair e of token
// i.  The inner vectors s A_e x_i are a launch of their own in front, of few
// CTAs, which the weights' stream runs beside: the products' kernel waits for
// them only where its sums are done, and adds a row's B there in FP32 before the
// one rounding.  On the device, with and without: 8 x 4096 -> 12288 NVFP4, rank 16 of 32
// adapters, 15.2 and 12.3 us; 5 x 16384 -> 4096 MXFP4, rank 64 of 8, 18.2 and 15.0.  What
// is added is the launch in front and, at the end, B's loads, which the L2 has by then.
#include <algorithm>
#include <type_traits>

#include "fp4_rows.cuh"

namespace lpq {
namespace {

constexpr int kRing = 4;            // chunks in a warp's ring
constexpr int kStep = kRing * kChunk;  // segments of K are whole steps
constexpr int kSegments = 8;        // most parts of K (and CTAs of a cluster)
constexpr int kXBytes = 128 * 1024; // most shared memory for x

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
  // adapters (ADAPTED kernels alone)
  const __nv_bfloat16* b;  // [count, n, rank]
  const float* inner;      // [token, rank]: s A x
  const int64_t* index;    // the token's adapter; outside 0 .. count - 1: none
  int64_t count;
  int rank;
};

// Row `row` of B_e times the token's inner vector.
__device__ __forceinline__ float adapter_row(const MatvecArgs& g, int64_t token, int row) {
  const int64_t e = g.index[token];
  if ((uint64_t)e >= (uint64_t)g.count) return 0.f;
  const uint4* b = reinterpret_cast<const uint4*>(g.b + (e * g.n + row) * g.rank);
  const float4* s = reinterpret_cast<const float4*>(g.inner + token * g.rank);
  float sum = 0.f;
#pragma unroll 2
  for (int i = 0; i < g.rank / 8; ++i) {
    float f[8];
    unpack8(__ldg(b + i), f);
    const float4 p = s[2 * i], q = s[2 * i + 1];
    sum = fmaf(f[0], p.x, sum);
    sum = fmaf(f[1], p.y, sum);
    sum = fmaf(f[2], p.z, sum);
    sum = fmaf(f[3], p.w, sum);
    sum = fmaf(f[4], q.x, sum);
    sum = fmaf(f[5], q.y, sum);
    sum = fmaf(f[6], q.z, sum);
    sum = fmaf(f[7], q.w, sum);
  }
  return sum;
}

// Brings that row of B_e to the L2.
__device__ __forceinline__ void prefetch_adapter_row(const MatvecArgs& g, int64_t token, int row) {
  const int64_t e = g.index[token];
  if ((uint64_t)e >= (uint64_t)g.count || row >= g.n) return;
  const char* b = reinterpret_cast<const char*>(g.b + (e * g.n + row) * g.rank);
  for (int i = 0; i < g.rank * 2; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + i));
}

// inner[token, r] = s A_e[r] . x: a CTA for four rows of a token.
constexpr int kInnerRows = 4, kInnerThreads = 256;
__global__ void __launch_bounds__(kInnerThreads) adapter_inner_kernel(const __nv_bfloat16* a, const float* scale, const int64_t* index,
                                                                      int64_t count, int rank, const __nv_bfloat16* x, int64_t ldx,
                                                                      int k, float* inner) {
  __shared__ float sh[kInnerThreads / 32][kInnerRows];
  wait_for_stream();
  let_dependents_start();  // not before: the products' kernel reads x and the weights without a wait of its own
  const int per = rank / kInnerRows;
  const int64_t token = blockIdx.x / per;
  const int r0 = (int)(blockIdx.x - token * per) * kInnerRows;
  const int64_t e = index[token];
  if ((uint64_t)e >= (uint64_t)count) return;
  const __nv_bfloat16* rows = a + (e * rank + r0) * k;
  const __nv_bfloat16* xr = x + token * ldx;
  float sum[kInnerRows] = {};
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < k; c += kInnerThreads * 8) {
    float xv[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(xr + c)), xv);
#pragma unroll
    for (int r = 0; r < kInnerRows; ++r) {
      float f[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(rows + (int64_t)r * k + c)), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[r] = fmaf(f[i], xv[i], sum[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < kInnerRows; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5][r] = sum[r];
  }
  __syncthreads();
  if (threadIdx.x < kInnerRows) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kInnerThreads / 32; ++w) s += sh[w][threadIdx.x];
    inner[token * rank + r0 + threadIdx.x] = s * (scale ? scale[e] : 1.0f);
  }
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
// MP: tokens that x's place in shared memory is laid out for (g.m or more).
// W warps per CTA: 8, four CTAs on an SM while x is small, else 24 that share x.
template <bool MX, bool SFG, int MP, int W, bool ADAPTED>
__global__ void __launch_bounds__(32 * W, W == 8 ? 4 : 1) matvec_kernel(const MatvecArgs g) {
  constexpr int kThreads = 32 * W;
  extern __shared__ uint4 sx[];
  __shared__ float back_sh[kSegments * kTokens];  // 2^-shift of a segment's x
  __shared__ int fits_sh[kSegments * kTokens];
  let_dependents_start();
  // (the inner vectors' kernel has waited for the stream before it let this one start)
  if constexpr (!ADAPTED) wait_for_stream();
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
    v *= tensor;
    if constexpr (ADAPTED) v += adapter_row(g, m0 + token, row);
    if (g.y_fp32) static_cast<float*>(g.y)[at] = v;
    else static_cast<__nv_bfloat16*>(g.y)[at] = __float2bfloat16_rn(v);
  };
  // operand columns beyond the tokens hold anything: their sums are not stored
  const int col = min(gid, MP - 1) * 4 + t;
  const bool f16 = fits(seg);
  int jbuf = 0;
  for (int item = first_item; item < g.items; item += item_step, jbuf ^= 1) {
    float* mine = sums + (jbuf * W + warp) * kSums;
    if constexpr (ADAPTED) {  // the rows that this CTA finishes, for the end of the item
      const int per = shared_k ? 16 * W / g.cluster : 16 * slots;
      for (int e = threadIdx.x; e < per * mm; e += kThreads) {
        const int r = rank * per + e / mm;
        prefetch_adapter_row(g, m0 + e % mm, row_of(item, r >> 4, r & 15));
      }
    }
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
            far_chunk<1>(l.lo, l.hi, l.slo, l.shi, eh + t, MP, mm, back_sh + seg * kTokens, mine);
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
    if constexpr (ADAPTED) wait_for_stream();  // the inner vectors are there
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

template <bool MX, bool SFG, int MP, int W, bool ADAPTED>
lpq_status run_matvec(MatvecArgs g, int passes, cudaStream_t s) {
  constexpr int kSumBytes = 2 * W * kTokens * 16 * 4;
  const int seg_steps = (g.steps + g.segments - 1) / g.segments;
  g.x_words = (g.cluster > 1 ? seg_steps : g.steps) * (kStep / 8);
  const int smem = g.x_words * 16 * MP + kSumBytes + W * kRing * kSlot;
  const void* kernel = reinterpret_cast<const void*>(matvec_kernel<MX, SFG, MP, W, ADAPTED>);
  lpq_status st = set_smem_attr(kernel, 222 * 1024);
  if (st != LPQ_OK) return st;
  const int64_t tiles = (g.n + kGroup - 1) / kGroup * 8, per = g.cluster > 1 ? W : W / g.segments;
  g.items = (int)((tiles + per - 1) / per);
  const int resident = std::max(1, std::min(W == 8 ? 4 : 1, 226 * 1024 / (smem + 2048)));
  const int most = std::max(1, resident * device_sms() / g.cluster);
  const dim3 grid((unsigned)(std::min(g.items, most) * g.cluster), (unsigned)passes);
  if (g.cluster == 1)
    return cuda_check(launch_dependent(matvec_kernel<MX, SFG, MP, W, ADAPTED>, grid, 32 * W, smem, s, g), "matvec launch");
  // Clusters start when the stream is done: an early start would place them
  // around the kernel ahead and leave the SMs unevenly loaded (16384 -> 4096:
  // 19.9 us, 14.7 us so).  The inner vectors' kernel is too small for that.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)g.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ADAPTED ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, matvec_kernel<MX, SFG, MP, W, ADAPTED>, g), "matvec launch");
}

template <bool MX, bool ADAPTED>
lpq_status run_tokens(const MatvecArgs& g, int passes, bool plain, bool wide_cta, cudaStream_t s) {
  if (plain) return run_matvec<MX, false, kTokens, 8, ADAPTED>(g, passes, s);
  if (wide_cta) return g.m > 2 ? run_matvec<MX, true, kTokens, 24, ADAPTED>(g, passes, s) : run_matvec<MX, true, 2, 24, ADAPTED>(g, passes, s);
  return g.m > 2 ? run_matvec<MX, true, kTokens, 8, ADAPTED>(g, passes, s)
         : g.m == 2 ? run_matvec<MX, true, 2, 8, ADAPTED>(g, passes, s) : run_matvec<MX, true, 1, 8, ADAPTED>(g, passes, s);
}

}  // namespace

lpq_status launch_matvec(const lpq_qview* w, const void* x, int64_t ldx, int64_t m, void* y, int32_t y_is_fp32,
                         const AdapterArgs* ad, cudaStream_t s) {
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
  if (ad) {
    g.count = ad->count;
    g.rank = (int)ad->rank;
    const int64_t ctas = m * (ad->rank / kInnerRows);
    if (ctas > 0x7FFFFFFF) return set_error(LPQ_ERR_SHAPE, "adapters: too many tokens");
    lpq_status st = cuda_check(
        launch_dependent(adapter_inner_kernel, dim3((unsigned)ctas), dim3(kInnerThreads), 0, s, static_cast<const __nv_bfloat16*>(ad->a),
                         ad->scale, ad->index, ad->count, g.rank, static_cast<const __nv_bfloat16*>(x), ldx, g.k, ad->inner),
        "adapter launch");
    if (st != LPQ_OK) return st;
  }
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
    if (ad) {
      g.b = static_cast<const __nv_bfloat16*>(ad->b);
      g.index = ad->index + m0;
      g.inner = ad->inner + m0 * ad->rank;
    }
    const auto run = ad ? (mx ? run_tokens<true, true> : run_tokens<false, true>) : (mx ? run_tokens<true, false> : run_tokens<false, false>);
    lpq_status st = run(g, (int)passes, plain, wide_cta && g.cluster == 1, s);
    if (st != LPQ_OK) return st;
    m0 += passes * g.m;
  }
  return LPQ_OK;
}

}  // namespace lpq
