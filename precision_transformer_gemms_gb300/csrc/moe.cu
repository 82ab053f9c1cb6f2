// A mixture-of-experts layer for a few tokens on 4-bit weights, on sm_103a.
//
//   route:  l = x Wr^T;  the k largest (ties: the lower index);  p = softmax over them
//   layer:  y_i = sum over j of p_ij W2_e (silu(W1g_e x_i) * (W1u_e x_i)),  e = ids_ij
//
// The chosen experts' weights, read once, are the traffic there is; their rows
// stream, decode and multiply as in the plain products of a few tokens.  Two
// launches.  Up: a warp's tile is 8 hidden values of an expert, whose gate and up rows
// share its 16 MMA rows, so that a lane ends with both and stores silu(g) u; the
// MMA's columns are the tokens that chose the expert.  Down: a tile is 16 rows of an
// expert, whose results lie in a workspace until the last expert of those rows has
// come: that warp adds them up per token, in the order of the token's choice.  Which
// experts there are, and for whom, every CTA reads from the ids by itself.  The grid
// is not resident at once: SMs are not equally fast at memory, and runs handed out as
// CTAs end even that out.
//
// Hidden values enter the second product as the sum of two f16 values times a power of
// two per vector (the largest in [2^14, 2^15)), off by 2^-23 of themselves or 2^-39 of the
// largest; one f16 would round to 11 bits what the first product left in FP32.  Up to 4
// tokens the second terms take columns of the MMA that would stand empty, of 8 tokens an
// MMA of their own on the same decoded weights.  The tensor core drops what lies below
// its sum's last bit every 16 products, so it sums a step's 256 columns from 0 and the
// steps' sums are added in FP32 (against one sum of all columns 0 to 2% slower: 8 tokens
// of 8 of 64 experts 116.5 -> 117.3 us, of 32 tokens, 2 of 8 of 2048 x 4096 80.7 -> 82.9).
// Everything else is exact or FP32.
//
// Measured (router, up and down in one graph; in brackets the weights' bytes at the copy
// bandwidth of 6677 GB/s): 8 tokens, 8 of 64 experts of 4096 x 1536 NVFP4 117 us (67),
// MXFP4 124; one token of them 33 (13); 4 tokens, 4 of 32 of 2048 x 768 24 (5.3); 24
// tokens, 2 of 16 of 2048 x 1024 38 (8.5), 200 tokens 214; 5 tokens, 3 of 21 of 2080 x 992 MXFP4 31
// (5.6); one token, 2 of 8 of 512 x 384 12 (0.1), the three launches whose parts wait
// for one another.  The router by itself: 5.8 us for 8 tokens of 64 experts of 4096, of
// which a choice is 0.25 (4.0 with one choice, 11.6 with 32: each is a pass of one warp over
// the keys), 5.0 with 512 columns; the rest is a cluster's chain of loads, two barriers
// and the parts' exchange.  What bounds the large ones: of an earlier state's 126 us the stream
// without a product took 102, the products without the stream 97 and what a CTA does
// before and after its tiles 58 by itself (the plan 15, the vectors' conversion 11, the
// rest launches, the router and the joining of the results); the three overlap in the
// CTAs that share an SM.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp4_rows.cuh"

namespace lpq {
namespace {

// ------------------------------------------------------------------ the router
// A cluster takes up to T tokens, each of its CTAs an eighth of the columns for all
// experts, so that every load is on its way at once; the parts of the logits meet in
// shared memory, and CTA i adds those of token i up, in order, and picks its experts.
// Products are FP32 FMAs: the tensor core's cut of its sum every 16 products would
// move choices between experts that are nearly equal.
constexpr int kRouteCtas = 8, kRouteWarps = 16;
constexpr int kAtOnce = 4;  // experts of a warp

// Floats in the order of their values, from 1 (NaN, below -infinity) up; -0 = +0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? 1u : b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// The warp's sums of N values per lane (N a power of two up to 32): value i lands in
// the lanes i * 32 / N ..; each step halves the values a lane holds.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + n], o);
      v[i] = (up ? v[i + n] : v[i]) + other;
    }
  }
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
  return v[0];
}

template <int T>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const RouteArgs g) {
  extern __shared__ uint4 route_sh[];
  let_dependents_start();
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int64_t m0 = (int64_t)(blockIdx.x / kRouteCtas) * T;
  const int mm = (int)min((int64_t)T, g.m - m0);
  const int words = g.d >> 3, most = (words + kRouteCtas - 1) / kRouteCtas;  // of 8 columns
  const int first = min(rank * most, words), mine = min(most, words - first);
  uint4* xs = route_sh;                                    // [T][most]
  float* parts = reinterpret_cast<float*>(xs + T * most);  // [T][experts], of these columns
  float* row = parts + T * g.experts;                      // [experts]: all of token `rank`'s
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(row + ((g.experts + 1) & ~1) + (T * g.experts & 1));
  for (int i = threadIdx.x; i < T * mine; i += 32 * kRouteWarps) {
    const int t = i / mine, c = i - t * mine;
    xs[t * most + c] = __ldg(reinterpret_cast<const uint4*>(g.x + (m0 + min(t, mm - 1)) * g.ldx) + first + c);
  }
  __syncthreads();
  for (int e0 = warp * kAtOnce; e0 < g.experts; e0 += kRouteWarps * kAtOnce) {
    float sum[kAtOnce * T] = {};
#pragma unroll 2
    for (int c = lane; c < mine; c += 32) {
      uint4 w[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        w[i] = __ldg(reinterpret_cast<const uint4*>(g.w + (int64_t)min(e0 + i, g.experts - 1) * g.ldw) + first + c);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float x[8];
        unpack8(xs[t * most + c], x);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          float f[8];
          unpack8(w[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[i * T + t] = fmaf(f[j], x[j], sum[i * T + t]);
        }
      }
    }
    constexpr int kLanes = 32 / (kAtOnce * T);  // that end with the same value
    const float v = warp_sums(sum);
    const int i = lane / kLanes / T, t = lane / kLanes % T;
    if (lane % kLanes == 0 && e0 + i < g.experts) parts[t * g.experts + e0 + i] = v;
  }
  cluster_sync_all();
  if (rank < mm) {
    for (int e = threadIdx.x; e < g.experts; e += 32 * kRouteWarps) {
      const uint32_t from = smem_u32(parts + rank * g.experts + e);
      float v = 0.f;
#pragma unroll
      for (int p = 0; p < kRouteCtas; ++p) v += ld_shared_cluster(mapa_shared(from, (uint32_t)p));
      row[e] = v;
      keys[e] = (unsigned long long)ordered(v) << 32 | (0xFFFFFFFFu - (uint32_t)e);
    }
  }
  cluster_sync_all();  // (no CTA leaves while another may still read its parts)
  if (rank >= mm || warp != 0) return;
  int pick = 0;
  float value = 0.f, top = 0.f;  // lane j: the j-th choice
  for (int j = 0; j < g.k; ++j) {
    unsigned long long best = 0;
    for (int e = lane; e < g.experts; e += 32) best = max(best, keys[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    const int e = (int)(0xFFFFFFFFu - (uint32_t)best);
    if (j == 0) top = row[e];
    if (lane == j) {
      pick = e;
      value = row[e];
    }
    __syncwarp();
    if (lane == 0) keys[e] = 0;
    __syncwarp();
  }
  float sum = 0.f;
  if (g.renormalize) {
    if (lane < g.k) sum = expf(value - top);
  } else {
    for (int e = lane; e < g.experts; e += 32) sum += expf(row[e] - top);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane < g.k) {
    const int64_t at = (m0 + rank) * g.k + lane;
    g.ids[at] = pick;
    g.probs[at] = __fdiv_rn(expf(value - top), sum);
  }
}

template <int T>
lpq_status route(const RouteArgs& g, cudaStream_t s) {
  const int words = g.d / 8, most = (words + kRouteCtas - 1) / kRouteCtas;
  const int smem = T * most * 16 + (T * g.experts + ((g.experts + 1) & ~1) + (T * g.experts & 1)) * 4 + g.experts * 8;
  const void* kernel = reinterpret_cast<const void*>(moe_route_kernel<T>);
  lpq_status st = set_smem_attr(kernel, 200 * 1024);
  if (st != LPQ_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((g.m + T - 1) / T * kRouteCtas));
  cfg.blockDim = dim3(32 * kRouteWarps);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kRouteCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_check(cudaLaunchKernelEx(&cfg, moe_route_kernel<T>, g), "route launch");
}

// ------------------------------------------------------------------ the experts
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMostPairs = 512;   // (token, choice) pairs of a launch

struct MoeKernelArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;
  int64_t kt;       // scale atoms per 128-row group
  int k;            // columns of the weights
  int rows;         // results of an expert: hidden values (up), rows (down)
  int tiles;        // of an expert: warps' shares of its rows
  int split;        // warps that share a tile's columns
  int m, top, experts;
  const int64_t* ids;    // [m, top]
  const float* probs;    // down
  const __nv_bfloat16* x;  // up: [m, k]
  int64_t ldx;
  float* hidden;    // [pair, hidden values]
  float* results;   // [pair, rows], down
  int* arrived;     // [tiles], down; set to 0 by up
  int down_tiles;
  __nv_bfloat16* y;  // [m, rows], down
  int x_words;      // 16-byte words of a vector's window in shared memory
};

// Which experts a launch reads, and for which pairs: entries of up to MP pairs of one
// expert, in the order of their first pairs.  All CTAs make the same.
struct Plan {
  alignas(16) int16_t id[kMostPairs];  // of a pair: its expert, or -1
  uint16_t next[kMostPairs];   // the expert's next pair
  uint16_t first[kMostPairs];  // of an entry: its first pair
  uint8_t count[kMostPairs];   // and how many it has
  uint8_t heads[kMostPairs / 32];  // entries that begin in 32 pairs
  int entries;
};

template <int MP>
__device__ __forceinline__ void make_plan(Plan& p, const MoeKernelArgs& g) {
  const int pairs = g.m * g.top, tid = threadIdx.x;
  for (int i = tid; i < ((pairs + 31) & ~31); i += kThreads) {
    const int64_t e = i < pairs ? g.ids[i] : -1;
    p.id[i] = (uint64_t)e < (uint64_t)g.experts ? (int16_t)e : -1;
  }
  __syncthreads();
  constexpr int kEach = kMostPairs / kThreads;  // pairs of a thread
  int before[kEach], total[kEach];
  uint32_t begin[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = k * kThreads + tid;
    before[k] = total[k] = 0;
    const int16_t e = i < pairs ? p.id[i] : -1;
    if (e >= 0) {
      int next = 0;
      const uint32_t both = (uint32_t)e * 0x00010001u;
      for (int w = (pairs - 1) >> 5; w >= 0; --w) {  // 32 pairs: which of them have the expert
        const uint4* ids = reinterpret_cast<const uint4*>(p.id) + w * 4;
        uint32_t same = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v = ids[q];
          const uint32_t u[4] = {v.x ^ both, v.y ^ both, v.z ^ both, v.w ^ both};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (!(u[h] & 0xFFFFu)) same |= 1u << (8 * q + 2 * h);
            if (!(u[h] >> 16)) same |= 2u << (8 * q + 2 * h);
          }
        }
        total[k] += __popc(same);
        const int at = i - 32 * w;  // below 0: the pair comes before these; above 31: after them
        before[k] += at > 31 ? __popc(same) : at > 0 ? __popc(same & ((1u << at) - 1)) : 0;
        const uint32_t later = at < 0 ? same : at < 31 ? same & (0xFFFFFFFEu << at) : 0u;
        if (later) next = 32 * w + __ffs(later) - 1;
      }
      p.next[i] = (uint16_t)next;
    }
    begin[k] = __ballot_sync(0xFFFFFFFFu, e >= 0 && before[k] % MP == 0);
    if ((tid & 31) == 0) p.heads[i >> 5] = (uint8_t)__popc(begin[k]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = k * kThreads + tid;
    int at = __popc(begin[k] & ((1u << (tid & 31)) - 1));
    for (int c = 0; c < i >> 5; ++c) at += p.heads[c];
    if (begin[k] >> (tid & 31) & 1) {
      p.first[at] = (uint16_t)i;
      p.count[at] = (uint8_t)min(MP, total[k] - before[k]);
    }
    if (i == kMostPairs - 1) p.entries = at + (begin[k] >> 31);
  }
  __syncthreads();
}

// A step is 256 codes of a tile's 16 rows: whole lines of memory, whose copies take half
// the L1's time that two chunks' half lines take.  A row has 128 bytes of codes in a
// ring's slot, their 16-byte units exchanged across the middle in odd rows (eight lanes
// read two rows' units without a conflict), and behind them a word of scales for every
// 4 blocks.
constexpr int kStepCodes = 2 * kChunk;
constexpr int kRing = 2;  // steps of a warp on their way
constexpr int slot_bytes(bool mx) { return 16 * 128 + 16 * (mx ? 8 : 16); }

// Two values as two f16 terms each: what the first leaves of a number goes to the second.
__device__ __forceinline__ void two_terms(float a, float b, uint32_t& first, uint32_t& second) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(fabsf(f.x) < 0x1p16f ? a - f.x : 0.f, fabsf(f.y) < 0x1p16f ? b - f.y : 0.f);
  first = *reinterpret_cast<const uint32_t*>(&h);
  second = *reinterpret_cast<const uint32_t*>(&l);
}

// Operand columns of an entry of mp pairs: the first terms of the vectors, then (down) the second ones.
constexpr int columns_of(bool up, int mp) { return up ? mp : 2 * mp; }

template <bool MX, int MP, bool UP, bool SPLIT, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) moe_kernel(const MoeKernelArgs g) {
  constexpr int kStepSlot = slot_bytes(MX), kRingBytes = kRing * kStepSlot;
  constexpr int C = columns_of(UP, MP);
  extern __shared__ uint4 sx[];
  __shared__ Plan plan;
  __shared__ uint32_t red[2][kWarps];
  __shared__ float back_sh[kTokens];
  constexpr int kSums = MX ? kTokens * 16 : 0;
  float* sums = reinterpret_cast<float*>(sx + (size_t)g.x_words * C);  // of chunks that f16 cannot hold
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int gid = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(sums + kWarps * kSums) + warp * kRingBytes;
  if constexpr (UP) {
    wait_for_stream();
    let_dependents_start();  // not before: down reads the ids and the weights without a wait of its own
    if (blockIdx.x == 0)
      for (int i = tid; i < g.down_tiles; i += kThreads) g.arrived[i] = 0;
  } else {
    let_dependents_start();
  }
  make_plan<MP>(plan, g);
  // This CTA's run of tiles, which its warps take in turn.  The grid has a CTA for
  // every run that there may be; those beyond the entries have none.
  const int64_t all_tiles = (int64_t)plan.entries * g.tiles;
  const int split = SPLIT ? g.split : 1;
  const int slots = kWarps / split, slot = warp / split, part = SPLIT ? warp % split : 0;  // tiles at once, this warp's, its part of it
  const int begin = (int)min(all_tiles, (int64_t)blockIdx.x * slots), end = (int)min(all_tiles, (int64_t)begin + slots);
  const int chunks = (g.k + kChunk - 1) / kChunk;
  const int steps = (chunks + 1) / 2, step0 = part * steps / split, step1 = (part + 1) * steps / split;

  // ---- the weight stream
  constexpr int kScaleStep = MX ? 1024 : 2048;  // bytes of scales per step: 2 or 4 atoms
  // The tile's 16 rows: up, 8 gate rows and their up rows; down, 16 rows.  They are
  // runs of 2 or 4 neighbours 32 apart, whose scales of 4 blocks lie side by side where
  // the expert begins with a 128-row group.
  auto value_of = [&](int tile, int r) {  // place in the expert's results of row r of 16 (up: of 8)
    return UP ? (tile >> 4) * 128 + 32 * (r & 3) + 2 * (tile & 15) + (r >> 2) : (tile >> 3) * 128 + 32 * (r & 3) + 4 * (tile & 7) + (r >> 2);
  };
  const uint8_t *pc = nullptr, *ps = nullptr, *ps2 = nullptr;
  uint32_t next_row[3] = {};  // from the lane's first row of codes to its others
  int a_item = begin + slot, a_step = step0;
  uint32_t a_slot = 0;
  auto set_item = [&]() {
    const int entry = a_item / g.tiles, tile = a_item - entry * g.tiles;
    const int64_t e = plan.id[plan.first[entry]];
    auto row_of = [&](int r) {  // rows beyond the expert read its last one; their results are not stored
      if constexpr (UP) return e * 2 * g.rows + min(value_of(tile, r & 7), g.rows - 1) + (r >> 3) * g.rows;
      else return e * g.rows + min(value_of(tile, r), g.rows - 1);
    };
    const int64_t first = row_of(lane >> 3);
    pc = g.codes + first * (g.k >> 1) + step0 * (kStepCodes / 2) + (lane & 7) * 16;
#pragma unroll
    for (int q = 1; q < 4; ++q) next_row[q - 1] = (uint32_t)(row_of((lane >> 3) + 4 * q) - first) * (uint32_t)(g.k >> 1);
    ps = g.scales + sf_gemm_offset(row_of(MX ? lane >> 1 : gid), 0, g.kt) + step0 * kScaleStep + (MX ? lane & 1 : t) * 512;
    if constexpr (!MX) ps2 = g.scales + sf_gemm_offset(row_of(gid + 8), 0, g.kt) + step0 * kScaleStep + t * 512;
  };
  const uint32_t codes_to = ring + (lane >> 3) * 128 + ((lane & 7) ^ ((lane >> 3 & 1) << 2)) * 16, scales_to = ring + 2048 + lane * 4;
  auto copy = [&]() {  // the next step of the stream
    if (a_item < end) {
      const uint32_t c = codes_to + a_slot;
      if ((a_step + 1) * kStepCodes <= g.k) {
        cp_async<16>(c, pc);
#pragma unroll
        for (int q = 1; q < 4; ++q) cp_async<16>(c + q * 512, pc + next_row[q - 1]);
      } else {
        const bool in = a_step * kStepCodes + (lane & 7) * 32 < g.k;
        cp_async_or_zero<16>(c, in ? pc : g.codes, in);
#pragma unroll
        for (int q = 1; q < 4; ++q) cp_async_or_zero<16>(c + q * 512, in ? pc + next_row[q - 1] : g.codes, in);
      }
      cp_async<4>(scales_to + a_slot, ps);
      if constexpr (!MX) cp_async<4>(scales_to + a_slot + 128, ps2);
      pc += kStepCodes / 2;
      ps += kScaleStep;
      ps2 += kScaleStep;
      if (++a_step == step1) a_item = end;  // (a tile a warp)
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    a_slot = a_slot == (kRing - 1) * kStepSlot ? 0 : a_slot + kStepSlot;
  };
  if (a_item < end) set_item();
#pragma unroll
  for (int i = 0; i < kRing; ++i) copy();
  if constexpr (!UP) {
    wait_for_stream();  // the hidden values are there
    if (all_tiles == 0)  // no token has an expert
      for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < (int64_t)g.m * g.rows; i += (int64_t)gridDim.x * kThreads)
        g.y[i] = __float2bfloat16_rn(0.f);
  }

  const float tensor = MX ? 1.0f : *g.tensor_scale;
  const int words = g.k >> 3, all_words = chunks * (kChunk / 8);
  auto place = [&](int c, int i) { return (((i >> 4) * 4 + (i & 3)) * C + c) * 4 + ((i >> 2) & 3); };
  float* mine = sums + warp * kSums;
  uint32_t place_at = 0;
  bool f16 = true;
  float up_by = 1.f;
  int item = begin + slot;  // this warp's tile
  for (int entry = begin / g.tiles; begin < end && entry * (int64_t)g.tiles < end; ++entry) {
    const int n = plan.count[entry];
    auto pair_of = [&](int c) {
      int p = plan.first[entry];
      for (int i = 0; i < c; ++i) p = plan.next[p];
      return p;
    };
    // ---- the entry's vectors as operand entries: their range, then their values.  The
    // warps share the vectors out, so that all loads are on their way together.
    const int lg = MP <= 1 || n <= 1 ? 0 : MP <= 2 || n <= 2 ? 1 : MP <= 4 || n <= 4 ? 2 : 3;
    const int vec = warp & ((1 << lg) - 1), first = (warp >> lg) * 32 + lane, step = kThreads >> lg;
    const uint4* xs = nullptr;
    if (vec < n) {
      const int p = pair_of(vec);
      xs = UP ? reinterpret_cast<const uint4*>(g.x + (int64_t)(p / g.top) * g.ldx)
              : reinterpret_cast<const uint4*>(g.hidden + (int64_t)p * g.k);
    }
    uint32_t top = 0, least = 0xFFFFFFFFu;
    if (vec < n) {
#pragma unroll 4
      for (int i = first; i < words; i += step) {
        if constexpr (UP) {
          const uint4 v = __ldg(xs + i);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a = u[j] & 0x7FFF7FFFu;
            top = __vmaxu2(top, a);
            least = __vminu2(least, __vsub2(a, 0x00010001u));
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = xs[2 * i + h];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a = u[j] & 0x7FFFFFFFu;
              if (a < 0x7F800000u) top = max(top, a);  // (no number keeps what it is)
            }
          }
        }
      }
    }
    if constexpr (UP) {
      top = max(top >> 16, top & 0xFFFFu);
      least = min(least >> 16, least & 0xFFFFu);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    if (lane == 0) {
      red[0][warp] = top;
      red[1][warp] = least;
    }
    __syncthreads();  // (the products with the vectors that were there are done, too)
    {                 // lane c: vector c
      const int c = lane & ((1 << lg) - 1);
      top = 0, least = 0xFFFFFFFFu;
      for (int w = c; w < kWarps; w += 1 << lg) {
        top = max(top, red[0][w]);
        least = min(least, red[1][w]);
      }
      int shift;
      bool holds = true;
      if constexpr (UP) {  // (bf16 bits; as in the plain products: exact or not in f16)
        least = (least & 0xFFFFu) + 1u;
        shift = top ? min(141 - (int)max(top >> 7, 1u), 126) : 0;
        holds = top < 0x7F80u && (least > 0xFFFFu || (least >> 7 ? (int)(least >> 7) : -6) + shift >= 110);
      } else {
        shift = top ? min(141 - (int)max(top >> 23, 1u), 126) : 0;
      }
      f16 = __all_sync(0xFFFFFFFFu, c >= n || holds);
      up_by = __uint_as_float((uint32_t)(127 + __shfl_sync(0xFFFFFFFFu, shift, vec)) << 23);
      if (tid < n) back_sh[tid] = __uint_as_float((uint32_t)(127 - shift) << 23);
    }
    // The warp's tile, if it is of this entry.
    const bool has = item < min(end, (entry + 1) * g.tiles);
    const int tile = item - entry * g.tiles;
    if (has) item = end;
    const int col = min(gid, C - 1) * 4 + t;  // columns beyond the entry's hold anything: their sums are not stored
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(2 * t + (i & 1)) * 16 + gid + (i >> 1) * 8] = 0.f;  // far_chunk adds to it
    }
    auto stream = [&](auto f16_path, const uint4* e, int from, int to) {  // the products of steps from .. to - 1
      constexpr bool F16 = decltype(f16_path)::value;
      auto read = [&](int h, bool tail, int s) {  // chunk h of the step
        Load l;
        const uint32_t c = ring + place_at + gid * 128 + ((h * 4 + t) ^ ((gid & 1) << 2)) * 16;
        l.lo = ld_shared_16(c);
        l.hi = ld_shared_16(c + 1024);
        const uint32_t at = ring + place_at + 2048 + (MX ? gid * 8 + h * 4 + t : gid * 16 + h * 8 + t * 2);
        l.slo = ld_shared_scale<MX>(at);
        l.shi = ld_shared_scale<MX>(at + (MX ? 64 : 128));
        if (tail && s * kStepCodes + h * kChunk + t * 32 >= g.k) l.slo = l.shi = 0;  // (anything may stand there)
        return l;
      };
      auto products = [&](const Load& l, float (&sum)[4]) {
        if (MX && F16 && mx_far(l))
          far_chunk<C / MP>(l.lo, l.hi, l.slo, l.shi, e + t, C, n, back_sh, mine);
        else
          chunk_products<MX, F16, C>(l, e + col, sum);
        e += (kChunk / 8) * C;
      };
#pragma unroll 1
      for (int s = from; s < to; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();
        const bool tail = (s + 1) * kStepCodes > g.k;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        products(read(0, tail, s), sum);
        const Load l = read(1, tail, s);
        __syncwarp();
        copy();  // into the slot whose values have just been read
        place_at = place_at == (kRing - 1) * kStepSlot ? 0 : place_at + kStepSlot;
        if (2 * s + 1 < chunks) products(l, sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += sum[i];
      }
    };
    // Window by window of the vectors (up: all of them at once): their values, and the products.
    for (int w0 = 0;; w0 += g.x_words) {
      const int w1 = UP ? all_words : min(all_words, w0 + g.x_words);
      if (vec < n) {
#pragma unroll 2
        for (int i = w0 + first; i < w1; i += step) {
          uint32_t r[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
          if (i < words) {
            if constexpr (UP) {
              const uint4 v = __ldg(xs + i);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
              if (f16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __half2 h2 = __floats2half2_rn(bf16_lo(u[j]) * up_by, bf16_hi(u[j]) * up_by);
                  r[j] = *reinterpret_cast<const uint32_t*>(&h2);
                }
              } else {
                r[0] = __byte_perm(v.x, v.z, 0x5410);
                r[1] = __byte_perm(v.x, v.z, 0x7632);
                r[2] = __byte_perm(v.y, v.w, 0x5410);
                r[3] = __byte_perm(v.y, v.w, 0x7632);
              }
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 v = xs[2 * i + h];
                two_terms(__uint_as_float(v.x) * up_by, __uint_as_float(v.y) * up_by, r[2 * h], q[2 * h]);
                two_terms(__uint_as_float(v.z) * up_by, __uint_as_float(v.w) * up_by, r[2 * h + 1], q[2 * h + 1]);
              }
            }
          }
          sx[place(vec, i - w0)] = make_uint4(r[0], r[1], r[2], r[3]);
          if constexpr (!UP) sx[place(vec + MP, i - w0)] = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
      __syncthreads();
      if (has) {
        constexpr int kStepWords = kStepCodes / 8;
        const int from = UP ? step0 : max(step0, w0 / kStepWords), to = UP ? step1 : min(step1, (w1 + kStepWords - 1) / kStepWords);
        const uint4* e = sx + (size_t)(from - w0 / kStepWords) * kStepWords * C;
        if (!UP || f16) stream(std::true_type{}, e, from, to); else stream(std::false_type{}, e, from, to);
      }
      if (UP || w1 == all_words) break;
      __syncthreads();  // the window's products are done
    }
    if (!has) continue;
    if constexpr (!UP) {  // the second terms' sums, in other columns
      if constexpr (MP == 1) {
        acc[0] += acc[1];
        acc[2] += acc[3];
      } else if constexpr (MP < kTokens) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], MP / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 2 * t + (i & 1);
      acc[i] *= !UP || f16 ? back_sh[min(c, n - 1)] : MX ? 1.0f : 256.0f;
      if constexpr (MX) acc[i] += mine[c * 16 + gid + (i >> 1) * 8];
    }
    if constexpr (SPLIT) {  // the parts' sums in order, through their rings, which are done with
      asm volatile("cp.async.wait_all;" ::: "memory");
      float* left = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(sums + kWarps * kSums) + warp * kRingBytes) + lane;
      if (part > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) left[i * 32] = acc[i];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(32 * split) : "memory");
      if (part > 0) continue;
      for (int p = 1; p < split; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += left[p * (kRingBytes / 4) + i * 32];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= tensor;
    if constexpr (UP) {
      const int v = value_of(tile, gid);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 2 * t + i;
        const float gate = acc[i], lin = acc[2 + i];
        if (c < n && v < g.rows) g.hidden[(int64_t)pair_of(c) * g.rows + v] = __fdiv_rn(gate, 1.0f + expf(-gate)) * lin;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 2 * t + (i & 1), v = value_of(tile, gid + (i >> 1) * 8);
        if (c < n && v < g.rows) g.results[(int64_t)pair_of(c) * g.rows + v] = acc[i];
      }
      // The warp that finds all experts' results of its rows there adds them up.
      __syncwarp();
      int before = 0;
      if (lane == 0) {
        __threadfence();
        before = atomicAdd(&g.arrived[tile], 1);
      }
      if (__shfl_sync(0xFFFFFFFFu, before, 0) == plan.entries - 1) {
        __threadfence();
        const int v = value_of(tile, lane & 15);
        if (v < g.rows)
          for (int i = lane >> 4; i < g.m; i += 2) {
            float sum = 0.f;
#pragma unroll 4
            for (int j = i * g.top; j < (i + 1) * g.top; ++j)
              if (plan.id[j] >= 0) sum = fmaf(__ldcg(g.probs + j), __ldcg(g.results + (int64_t)j * g.rows + v), sum);
            g.y[(int64_t)i * g.rows + v] = __float2bfloat16_rn(sum);
          }
        __syncwarp();
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool MX, int MP, bool UP, bool SPLIT, int CTAS>
lpq_status launch(const MoeKernelArgs& g, int64_t tiles, cudaStream_t s) {
  auto kernel = moe_kernel<MX, MP, UP, SPLIT, CTAS>;
  const int smem = g.x_words * 16 * columns_of(UP, MP) + (MX ? kWarps * kTokens * 16 * 4 : 0) + kWarps * kRing * slot_bytes(MX);
  lpq_status st = set_smem_attr(reinterpret_cast<const void*>(kernel), 200 * 1024);
  if (st != LPQ_OK) return st;
  const int slots = kWarps / g.split;
  return cuda_check(launch_dependent(kernel, dim3((unsigned)((tiles + slots - 1) / slots)), dim3(kThreads), smem, s, g),
                    UP ? "moe up launch" : "moe down launch");
}

// Experts that m tokens with `top` of them each choose, if all are equally likely.
double expected_experts(int64_t m, int64_t top, int64_t experts) {
  const double others = 1.0 - std::min(1.0, (double)top / (double)experts);
  return (double)experts * (1.0 - std::pow(others, (double)m));
}

// Most shared memory for a window of the hidden values, whole steps of them.  With 16
// columns small ones, beside which three CTAs fit an SM (64 tokens, 2 of 8 of 4096 x 1536:
// 108.5 us with 32 KB, 113.5 with 64; 32 tokens, 2 of 8 of 2048 x 4096 80.9, 85.5 and 88.4
// with 128); with fewer one window for most sizes, since the warps that share a tile's
// columns work in different ones (4 tokens, 2 of 8 of 2048 x 8192: 65.8, 59.0 and 57.2).
constexpr int window_bytes(int columns) { return (columns > kTokens ? 32 : 128) * 1024; }

template <bool MX, int MP, bool UP>
lpq_status run(MoeKernelArgs& g, cudaStream_t s) {
  const int chunks = (g.k + kChunk - 1) / kChunk;
  g.x_words = chunks * (kChunk / 8);
  if (!UP) g.x_words = std::min(g.x_words, window_bytes(columns_of(UP, MP)) / (16 * columns_of(UP, MP)));
  // Entries, at most: one for every expert, and for every MP pairs beyond the experts'
  // first ones.  (CTAs without an entry cost a plan each: with one for every pair, 200
  // tokens, 2 of 16 of 2048 x 1024, took 427 us, 223 so.)
  const int64_t pairs = (int64_t)g.m * g.top, firsts = std::min<int64_t>(pairs, g.experts);
  const int64_t tiles = (firsts + (pairs - firsts) / MP) * g.tiles;
  const double likely = std::max(expected_experts(g.m, g.top, g.experts), (double)pairs / MP) * g.tiles;
  // Warps share a tile's columns while there are fewer tiles than places for warps (24
  // an SM) and each gets a few chunks: one token of 8 experts of 4096 x 1536 45.5 ->
  // 36.0 us (32.7 now; with the second product split too, beyond that number, 36.3); 5
  // tokens, 3 of 21 of 2080 x 992 37.0 -> 29.8 us.
  const int most = chunks >= 16 ? 4 : chunks >= 8 ? 2 : 1;
  g.split = 1;
  while (g.split < most && likely * g.split * 2 <= 3 * kWarps * device_sms()) g.split *= 2;
  if (g.split > 1) return launch<MX, MP, UP, true, 3>(g, tiles, s);
  // Where two CTAs an SM hold all tiles, each has more registers, which hide more of the
  // loads' time (24 tokens, 2 of 16 of 2048 x 1024 42.0 -> 37.7 us; with more tiles three
  // are better: 8 tokens, 8 of 64 of 4096 x 1536 120 against 131).
  return likely <= 2 * kWarps * device_sms() ? launch<MX, MP, UP, false, 2>(g, tiles, s) : launch<MX, MP, UP, false, 3>(g, tiles, s);
}

template <bool UP>
lpq_status run_tokens(MoeKernelArgs& g, bool mx, int mp, cudaStream_t s) {
  switch (mp) {
    case 1: return mx ? run<true, 1, UP>(g, s) : run<false, 1, UP>(g, s);
    case 2: return mx ? run<true, 2, UP>(g, s) : run<false, 2, UP>(g, s);
    case 4: return mx ? run<true, 4, UP>(g, s) : run<false, 4, UP>(g, s);
    default: return mx ? run<true, 8, UP>(g, s) : run<false, 8, UP>(g, s);
  }
}

constexpr int kXBytes = 128 * 1024;  // most shared memory for an entry's vectors

// Columns of an entry: enough for an expert's tokens as a rule, and what fits.
int columns(int64_t m, int64_t top, int64_t experts, int64_t k) {
  int mp = m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 || m * top <= 2 * experts ? 4 : 8;
  while (mp > 1 && (k + kChunk - 1) / kChunk * kChunk * 2 * mp > kXBytes) mp /= 2;
  return mp;
}
int64_t tokens_of_launch(int64_t top) { return std::max<int64_t>(1, kMostPairs / std::max<int64_t>(top, 1)); }
// Tiles of an expert: those with a row of it (a tile's first row is the lowest).
int64_t up_tiles(int64_t inter) { return inter / 128 * 16 + std::min<int64_t>(16, (inter % 128 + 1) / 2); }
int64_t down_tiles(int64_t hidden) { return hidden / 128 * 8 + std::min<int64_t>(8, (hidden % 128 + 3) / 4); }
size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

lpq_status launch_moe_route(const RouteArgs& g, cudaStream_t s) {
  if (g.m == 0) return LPQ_OK;
  return g.m <= 1 ? route<1>(g, s) : g.m <= 2 ? route<2>(g, s) : route<4>(g, s);
}

size_t moe_workspace(int64_t m, int64_t top, int64_t hidden, int64_t inter) {
  const size_t pairs = (size_t)(std::min(m, tokens_of_launch(top)) * top);
  return round16(pairs * (size_t)inter * 4) + round16(pairs * (size_t)hidden * 4) + round16((size_t)down_tiles(hidden) * 4);
}

lpq_status launch_moe(const MoeArgs& a, cudaStream_t s) {
  if (a.m == 0) return LPQ_OK;
  const int64_t hidden = a.up->cols, inter = a.down->cols;
  if (a.top == 0)  // no expert
    return cuda_check(cudaMemsetAsync(a.y, 0, (size_t)a.m * (size_t)hidden * 2, s), "cudaMemsetAsync(y)");
  for (int64_t m0 = 0; m0 < a.m; m0 += tokens_of_launch(a.top)) {
    MoeKernelArgs g{};
    g.m = (int)std::min(a.m - m0, tokens_of_launch(a.top));
    const size_t pairs = (size_t)g.m * (size_t)a.top;
    g.top = (int)a.top;
    g.experts = (int)a.experts;
    g.ids = a.ids + m0 * a.top;
    g.probs = a.probs + m0 * a.top;
    g.x = static_cast<const __nv_bfloat16*>(a.x) + m0 * a.ldx;
    g.ldx = a.ldx;
    g.y = static_cast<__nv_bfloat16*>(a.y) + m0 * hidden;
    g.hidden = reinterpret_cast<float*>(a.workspace);
    g.results = reinterpret_cast<float*>(a.workspace + round16(pairs * (size_t)inter * 4));
    g.arrived = reinterpret_cast<int*>(a.workspace + round16(pairs * (size_t)inter * 4) + round16(pairs * (size_t)hidden * 4));
    g.down_tiles = (int)down_tiles(hidden);
    const bool mx = a.up->fmt == LPQ_MXFP4;
    auto weights = [&](const lpq_qview* w) {
      g.codes = static_cast<const uint8_t*>(w->codes);
      g.scales = static_cast<const uint8_t*>(w->scales);
      g.tensor_scale = w->tensor_scale;
      g.k = (int)w->cols;
      g.kt = sf_kt_atoms(w->fmt, w->cols);
    };
    weights(a.up);
    g.rows = (int)inter;
    g.tiles = (int)up_tiles(inter);
    lpq_status st = run_tokens<true>(g, mx, columns(g.m, a.top, a.experts, g.k), s);
    if (st != LPQ_OK) return st;
    weights(a.down);
    g.rows = (int)hidden;
    g.tiles = g.down_tiles;
    st = run_tokens<false>(g, a.down->fmt == LPQ_MXFP4, columns(g.m, a.top, a.experts, g.k), s);
    if (st != LPQ_OK) return st;
  }
  return LPQ_OK;
}

}  // namespace lpq
