// Softmax cross entropy of a vocabulary projection and its gradients on
// sm_103a.  The logits l = h w^T exist tile by tile only:
//
//   forward   each tile leaves, for every row, the maximum m and the sum of
//             exp(l - m) over its columns; a second kernel joins them:
//             lse = log sum_j exp(l_j), loss = lse - l[label].
//   backward  per piece of the vocabulary the logits are computed again and
//             turned into dl = (exp(l - lse) - onehot) dloss in bf16; then
//             dh += dl w (FP32 sums across pieces) and dw = dl^T h.
//
// All four products run on one kernel: a CTA pair (cta_group::2) per 256 x 256
// output tile, operands staged by TMA (128-byte swizzle), FP32 accumulators in
// TMEM.  The operand that a product sums along its rows (w in dl w; dl and h
// in dl^T h) is read as it lies, as an MN-major operand: no transposed copies.
//
// The tensor cores bound it: 2 t v d operations forward, 6 t v d backward (the
// logits again).  Measured: 4096 x 4096 x 19456 forward 327 us and dl 343 us, dh
// and dw 670 us together, the tensor pipe 86 to 95% active, 1.90 to 2.00
// PFLOP/s at full clocks (cuBLAS 1.91 burst, 1.71 sustained under the power
// cap); in a loop, 7936 x 4096 x 32000 forward 1.19 ms (1.75 PFLOP/s) and
// backward 3.65 ms (1.71).  With d = 1024 a tile's result weighs on the port
// that feeds it: 1001 x 1024 x 50001 backward 235 us (1.31).
//
// The backward pass works on the rows that have a target alone: they are
// counted and listed on the device, their hidden states copied together where
// there are others, and the kernels take their sizes from the count.  What the
// other rows hold reaches nothing, and costs nothing.
//
// dl is divided by s = max |dloss| before its rounding to bf16 (what the
// tensor cores read) and s multiplies the FP32 sums: with equal dloss, the
// mean over the tokens say, the entry p - 1 of a label is then rounded as it
// is instead of after a product with 1 / t.  Over many tokens the roundings
// average out below those of bf16 gradients; a few tokens' would show, so where
// up to 128 rows have a target, or the caller asks for it, dl is held as the sum
// of two bf16 terms (16 bits).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kTile = 256;   // rows and columns of an output tile (one CTA pair)
constexpr int kHalf = 128;   // of each operand and of the rows, per CTA
constexpr int kStepK = 64;   // one 128-byte swizzle row of bf16
constexpr int kGroupM = 16;  // tiles along M that share a band of B tiles (L2 reuse)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kOperand = kHalf * kStepK * 2;  // bytes of one operand per CTA and step
constexpr int kStgWarp = 32 * 128;            // epilogue staging: 32 rows x 64 bf16 per warp
constexpr int kStg = kEpiWarps * kStgWarp;
constexpr int kStages = (232448 - 2048 - 512 - kStg) / (2 * kOperand);
constexpr int kSmem = kStages * 2 * kOperand + 2048 + 512 + kStg;
constexpr int kNacc = 2;  // accumulators: one tile's epilogue under the next tile's products
static_assert(kStages == 6 && kNacc * kTile <= 512, "shared memory and TMEM budgets");

// The tensor core cuts (does not round) the FP32 sum at every 16 products, so
// a long sum drifts towards zero: measured 2.5e-6 of the loss over d = 4096.
// The logits are therefore summed in TMEM over kChunk steps (1024 values) at a
// time and across chunks in the epilogue's registers: 2% of the time at 7936 x
// 4096 x 32000 (3% backward at 1001 x 1024 x 50001), a fifth to an eighth of the
// drift.  Both passes do so: exp(l - lse) takes the bits that lse was made of, and
// where p is near 1 its p - 1 is not the difference of two drifts.  The gradients'
// sums are cut in full, which stays below dl's bf16 rounding.
constexpr int kChunk = 16;

// Where up to kFew rows have a target (counted on the device) dl is stored as two
// terms, the value in bf16 and in bf16 what that leaves out.  In dh = dl w they are
// the rows of the two CTAs (one of which had none), whose sums are added in the
// end; in dw = dl^T h they follow one another along K, against the same h.  Reading
// w and storing dw bound the pass up to there, so the terms cost little: 32000 x
// 4096, 1, 33 or 128 rows 196, 200 and 193 us; 20 of 512 rows 235 us (224 with one
// term).  Error of bf16 gradients of up to 128 rows against 64 bits: 0.0020 to
// 0.0025 with one term, 0.0017 with two, which is their own rounding.  A caller can
// ask for two terms of any number of rows: they then follow one another in dh too
// (7936 x 4096 x 32000 3.6 -> 6.3 ms).
constexpr int kFew = kHalf;

// What a kernel's epilogue makes of a tile.
//   kStats    row maxima and sums of exponentials of the logits
//   kDlogits  dl in bf16
//   kGrads    of two products: FP32 partial sums of dh (one slab per split of K,
//             added to across pieces), or a finished gradient: times the scale,
//             bf16 or FP32
enum { kStats, kDlogits, kGrads };

// One product C [M, N] = A B^T of a launch.
struct Product {
  int64_t M, N;
  int num_k;  // steps of kStepK along K
  int tiles_m, tiles_n, splits;
  int items;  // tiles * splits
  int a_mn;   // A lies with K along its rows
  int m_rows, k_rows;  // M, or K, is the number of rows with a target (known on the device)
  int scatter;         // rows of the result go to the places of their list
  int part;            // partial sums into acc instead of out
  void* out;
  int64_t ld;          // of the second terms of dl
  int a_box;           // rows of A that a load takes: kHalf, or fewer that are all of them
};

struct alignas(64) CeMaps {
  CUtensorMap a[2], b[2], c[2];
  CUtensorMap a2[2];  // of the second terms of dl
  CUtensorMap alt;  // of the copied rows of h: A of kDlogits, B of dw
};

struct CeTile {
  Product prod[2];  // the second with no items where there is one product
  int extra;        // items of the second for the pairs with fewer of the first, before all share the rest
  int* err;
  int64_t t;        // rows of h
  const int* rows;  // how many of them have a target (backward)
  const int* list;  // which
  const int64_t* labels;
  int64_t vocab;
  int64_t col0;     // first word of the piece
  float2* stats;    // [M][stat_cols] (maximum, sum) per 128 columns
  int64_t stat_cols;
  float* at_label;  // [M]
  const float* lse;
  const float* dloss;
  const float* scale;
  float* acc;  // [splits][M][N]
  int add;     // 1: add to acc
  int two_terms;      // dl in two terms however many rows have a target
  int64_t rest_rows;  // rows that there is room for in dl's second terms
  int out_fp32;
};

// Instruction descriptor: F32 accumulator, BF16 x BF16, MN-major flags, N = 256, M = 256.
constexpr uint32_t instruction_desc(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp(x - y).  The difference comes first: a product of x alone with log2 e
// would be rounded at x's size, and exp(0) would not be 1.
__device__ __forceinline__ float exp_of_difference(float x, float y) { return ex2((x - y) * kLog2e); }
// The same of two x at a time, y given as -y.
__device__ __forceinline__ float2 exp_of_differences(float2 x, float2 minus_y) {
  const float2 d = __fmul2_rn(__fadd2_rn(x, minus_y), make_float2(kLog2e, kLog2e));
  return make_float2(ex2(d.x), ex2(d.y));
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The i-th work item of a pair: product and item, false after the last.  The
// first product's items go round the pairs; the pairs that get one fewer take
// `extra` of the second's, then the rest goes round all pairs.
__device__ __forceinline__ bool item_at(int i, int pair, int npairs, const Product* prod, int extra, int& which, int& w) {
  const int n0 = prod[0].items, left_over = n0 % npairs;
  const int mine = n0 / npairs + (pair < left_over ? 1 : 0);
  which = 0;
  w = pair + i * npairs;
  if (i < mine) return true;
  which = 1;
  i -= mine;
  if (pair >= left_over) {
    w = i * (npairs - left_over) + pair - left_over;
    if (i < extra) return true;
    i -= extra;
  }
  w = extra * (npairs - left_over) + i * npairs + pair;
  return w < prod[1].items;
}
// Work item w -> tile and split; consecutive tiles walk down a band of kGroupM
// m-tiles, all splits of a tile run together.
__device__ __forceinline__ void item_coords(int w, const Product& p, int& mt, int& nt, int& split) {
  split = w % p.splits;
  const int t = w / p.splits;
  const int per_group = kGroupM * p.tiles_n;
  const int group = t / per_group;
  const int first = group * kGroupM;
  const int size = min(kGroupM, p.tiles_m - first);
  const int r = t - group * per_group;
  mt = first + r % size;
  nt = r / size;
}
__device__ __forceinline__ void split_range(int split, const Product& p, int& k0, int& k1) {
  k0 = (int)((int64_t)p.num_k * split / p.splits);
  k1 = (int)((int64_t)p.num_k * (split + 1) / p.splits);
}

// After an abort: wait (bounded) for the loads of ring uses [from, to).
__device__ __forceinline__ void drain(uint64_t* bars, uint32_t from, uint32_t to, int* err) {
  volatile int no_abort = 0;
  for (uint32_t k = from; k < to; ++k) mbar_wait_bounded(&bars[k % kStages], (k / kStages) & 1u, &no_abort, err);
}

// Persistent: each CTA pair takes work items in turn.  Warp 0 (one lane)
// streams the operands into a ring of shared-memory stages, warp 1 of the even
// CTA (one lane) issues the pair MMAs, eight epilogue warps per CTA (two per
// TMEM lane quarter, 128 columns each) finish the tile.
// MN-major operands (A where a_mn, B of kGrads): the matrix lies with K along
// its rows; a stage holds two 64 x 64 blocks (64 k-rows of 128 bytes each).
template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads)
    ce_pair_kernel(const __grid_constant__ CeMaps maps, const __grid_constant__ CeTile g) {
  constexpr bool B_MN = EPI == kGrads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kOperand;
  uint8_t* stage_c = sB + kStages * kOperand;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_c + kStg);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kNacc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + kNacc);
  uint32_t* peer_base = tmem_slot + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kNacc; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.a[0]);
    prefetch_tmap(&maps.b[0]);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Both CTAs must see the same TMEM address; otherwise stop cleanly.
  if (threadIdx.x == 0) st_shared_remote_u32(mapa_shared(smem_u32(peer_base), rank ^ 1u), tmem_base);
  cluster_sync_all();
  if (*peer_base != tmem_base) {
    if (threadIdx.x == 0) atomicCAS(g.err, 0, (int)LPQ_ERR_UNSUPPORTED);
    *abort_flag = 1;
  }
  const bool run = *peer_base == tmem_base;
  let_dependents_start();
  wait_for_stream();
  // the products at their sizes on the device
  __shared__ Product prod[2];
  __shared__ int extra_sh;
  const int rows = EPI == kStats ? 0 : *g.rows;
  const bool some_rows = EPI != kStats && rows < g.t;
  const bool few = EPI != kStats && rows <= kFew;  // dl in two terms, in dh one for each CTA of a pair
  const bool two = few || (EPI != kStats && g.two_terms);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      Product p = g.prod[i];
      if (p.m_rows) {
        p.M = rows;
        p.tiles_m = (rows + kTile - 1) / kTile;
        p.items = p.tiles_m * p.tiles_n * p.splits;
      }
      if (p.k_rows) p.num_k = (rows + kStepK - 1) / kStepK;
      if (EPI == kGrads && few && p.m_rows) {
        p.part = 1;
        p.scatter = 0;
      } else if (EPI == kGrads && two) {
        p.num_k *= 2;  // a term after the other
      }
      prod[i] = p;
    }
    const int left_over = prod[0].items % npairs;
    extra_sh = left_over ? min(g.extra, prod[1].items / (npairs - left_over)) : 0;
  }
  __syncthreads();
  const int extra = extra_sh;
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);

  if (run && warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = true;
      int which, w;
      for (int i = 0; ok && item_at(i, pair, npairs, prod, extra, which, w); ++i) {
        const Product& p = prod[which];
        const CUtensorMap* tmA = EPI == kDlogits && some_rows ? &maps.alt : &maps.a[which];
        const CUtensorMap* tmA2 = EPI == kGrads && two ? &maps.a2[which] : tmA;
        const CUtensorMap* tmB = EPI == kGrads && p.k_rows && some_rows ? &maps.alt : &maps.b[which];
        int mt, nt, split, k0, k1;
        item_coords(w, p, mt, nt, split);
        split_range(split, p, k0, k1);
        const bool terms = EPI == kGrads && few && p.m_rows;  // the CTAs take a term each
        const int32_t arow = mt * kTile + (terms ? 0 : (int32_t)rank * kHalf), brow = nt * kTile + (int32_t)rank * kHalf;
        // the first step with the second terms
        const int second = terms ? (rank ? 0 : INT_MAX) : EPI == kGrads && two ? p.num_k / 2 : INT_MAX;
        const bool has_a = p.a_box == kHalf || terms || leader;
        const uint32_t bytes = 2 * kOperand + (p.a_box == kHalf || terms ? 2 : 1) * p.a_box * (kStepK * 2);
        auto loads = [&](auto a_is_mn) {
          constexpr bool A_MN = decltype(a_is_mn)::value;
          for (int kt = k0; kt < k1; ++kt) {
            if (!(ok = mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag, g.err))) break;
            if (leader) mbar_arrive_expect_tx(&full[s], bytes);
            const uint32_t fb = full_leader + 8 * s;
            uint8_t* da = sA + s * kOperand;
            uint8_t* db = sB + s * kOperand;
            const CUtensorMap* ta = kt < second ? tmA : tmA2;
            const int32_t k = (kt < second ? kt : kt - second) * kStepK;
            if constexpr (A_MN) {
              tma_load_2d_pair(da, ta, arow, k, fb);
              tma_load_2d_pair(da + kOperand / 2, ta, arow + 64, k, fb);
            } else if (has_a) {
              tma_load_2d_pair(da, ta, k, arow, fb);
            }
            if constexpr (B_MN) {
              tma_load_2d_pair(db, tmB, brow, k, fb);
              tma_load_2d_pair(db + kOperand / 2, tmB, brow + 64, k, fb);
            } else {
              tma_load_2d_pair(db, tmB, k, brow, fb);
            }
            ++it;
            if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
          }
        };
        if (EPI == kGrads && p.a_mn) loads(std::true_type{}); else loads(std::false_type{});
      }
      // After an abort, the even CTA lets the pair's loads in flight land
      // (they all signal its full barriers) before either CTA exits.
      if (!ok && leader) drain(full, it > (uint32_t)kStages ? it - kStages : 0u, it, g.err);
    }
  } else if (run && warp == 1) {
    if (lane == 0 && leader) {
      // K-major: 8-row groups of 1024 bytes, 16 values along K = 32 bytes on.
      // MN-major: 64-value blocks kOperand / 2 bytes apart, 8-row groups of K of
      // 1024 bytes, 16 rows along K = 2048 bytes on.
      const uint64_t ad_k = smem_desc(smem_u32(sA), 16, 1024, 2), ad_mn = smem_desc(smem_u32(sA), kOperand / 2, 1024, 2);
      const uint64_t bd0 = smem_desc(smem_u32(sB), B_MN ? kOperand / 2 : 16, 1024, 2);
      uint32_t s = 0, ph = 0, lt = 0;
      bool ok = true;
      // the products of one item; a_mn as a constant
      auto item_products = [&](auto a_is_mn, int k0, int k1) {
        constexpr bool A_MN = decltype(a_is_mn)::value;
        constexpr uint32_t idesc = instruction_desc(A_MN, B_MN);
        int kt = k0;
        do {  // one accumulator per chunk of the sum (a split without steps still hands one over)
          const int kend = EPI != kGrads ? min(k1, kt + kChunk) : k1;
          const uint32_t a = lt % kNacc, aph = (lt / kNacc) & 1u;
          ++lt;
          if (!(ok = mbar_wait_bounded(&acc_empty[a], aph ^ 1u, abort_flag, g.err))) break;
          tc_fence_after();
          const uint32_t tmem_d = tmem_base + a * kTile;
          for (const int first = kt; kt < kend; ++kt) {
            if (!(ok = mbar_wait_bounded(&full[s], ph, abort_flag, g.err))) break;
            tc_fence_after();
            const uint64_t ad = (A_MN ? ad_mn : ad_k) + (uint64_t)(s * (kOperand >> 4)), bd = bd0 + (uint64_t)(s * (kOperand >> 4));
#pragma unroll
            for (int j = 0; j < kStepK / 16; ++j)
              mma_pair<kKindF16>(tmem_d, ad + (uint64_t)(j * (A_MN ? 128 : 2)), bd + (uint64_t)(j * (B_MN ? 128 : 2)), idesc,
                                 (kt > first || j > 0) ? 1u : 0u);
            tc_commit_pair(&empty[s], 0x3);
            if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
          }
          if (ok) tc_commit_pair(&acc_full[a], 0x3);
        } while (ok && kt < k1);
      };
      int which, w;
      for (int i = 0; ok && item_at(i, pair, npairs, prod, extra, which, w); ++i) {
        const Product& p = prod[which];
        int k0, k1;
        split_range(w % p.splits, p, k0, k1);
        if (EPI == kGrads && p.a_mn) item_products(std::true_type{}, k0, k1);
        else item_products(std::false_type{}, k0, k1);
      }
    }
  } else if (run && warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = stage_c + (warp - 2) * kStgWarp;
    float scale = 1.f;
    if constexpr (EPI != kStats) scale = *g.scale;
    uint32_t lt = 0;
    int which, w;
    for (int item = 0; item_at(item, pair, npairs, prod, extra, which, w); ++item) {
      const Product& p = prod[which];
      int mt, nt, split;
      item_coords(w, p, mt, nt, split);
      const bool terms = few && p.m_rows;  // (dl or dh: one tile down)
      const int64_t row = (int64_t)mt * kTile + (EPI == kGrads && terms ? 0 : rank * kHalf) + q * 32 + lane;
      const int64_t c0 = (int64_t)nt * kTile + half * kHalf;
      const bool live = row < p.M;
      const int ncols = (int)max((int64_t)0, min((int64_t)kHalf, p.N - c0));  // columns of this warp inside the matrix
      // what the row needs is fetched before the accumulator is waited for
      int64_t from = row;  // the row of h
      if (EPI == kGrads && p.scatter && live) from = g.list[row];
      int label = -1;  // its column among this warp's 128, -1: not here
      float lse = 0.f, gs = 0.f;
      bool target = false;
      if constexpr (EPI == kStats || EPI == kDlogits) {
        if (EPI == kDlogits && live) from = g.list[row];
        const int64_t word = live ? g.labels[from] : -1;
        target = word >= 0 && word < g.vocab;
        const int64_t col = word - (g.col0 + c0);
        if (target && col >= 0 && col < kHalf) label = (int)col;
      }
      if constexpr (EPI == kDlogits) {
        if (target) {
          lse = g.lse[from];
          gs = g.dloss[from] / scale;
        }
      }
      // Waits for the next accumulator; hands it back once its values are in registers.
      uint32_t tbase = 0, a = 0;
      auto take = [&]() {
        a = lt % kNacc;
        const bool ok = mbar_wait_bounded(&acc_full[a], (lt / kNacc) & 1u, abort_flag, g.err);
        ++lt;
        __syncwarp();
        tc_fence_after();
        tbase = tmem_base + a * kTile + half * kHalf + ((uint32_t)(q * 32) << 16);
        return __all_sync(0xFFFFFFFFu, ok);
      };
      auto give = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&acc_empty[a]); else mbar_arrive_remote_relaxed(acc_empty_leader + 8 * a);
        }
      };
      float l[EPI != kGrads ? kHalf : 1];  // logits
      if constexpr (EPI != kGrads) {
        bool ok = true;
        for (int kt = 0; kt < p.num_k && ok; kt += kChunk) {
          if (!(ok = take())) break;
#pragma unroll
          for (int cc = 0; cc < kHalf / 16; ++cc) {
            uint32_t v[16];
            tmem_ld16(tbase + (uint32_t)(cc * 16), v);
#pragma unroll
            for (int i = 0; i < 16; ++i) l[cc * 16 + i] = (kt ? l[cc * 16 + i] : 0.f) + __uint_as_float(v[i]);
          }
          give();
        }
        if (!ok) break;
      }
      if constexpr (EPI == kStats) {
        if (ncols < kHalf)
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (i >= ncols) l[i] = kNegInf;
        if (label >= 0) {
          float at = 0.f;
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (label == i) at = l[i];
          g.at_label[row] = at;
        }
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) m = max_nan(m, l[i]);
        // all -inf: the differences are taken from 0, and each term is exp(-inf) = 0
        const float base = m == kNegInf ? 0.f : m;
        const float2 minus = make_float2(-base, -base);
        float2 e[kHalf / 2];
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) e[i] = exp_of_differences(make_float2(l[2 * i], l[2 * i + 1]), minus);
        // in pairs: one after the other, 127 small terms would lose their last
        // bits to a running sum of about 1 (a confident token's)
#pragma unroll
        for (int w = kHalf / 4; w > 0; w >>= 1)
#pragma unroll
          for (int i = 0; i < w; ++i) e[i] = __fadd2_rn(e[i], e[i + w]);
        if (live && ncols > 0) g.stats[row * g.stat_cols + nt * 2 + half] = make_float2(m, e[0].x + e[0].y);
        __syncwarp();
        continue;
      }
      if constexpr (EPI == kDlogits) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) l[i] = target ? exp_of_difference(l[i], lse) * gs : 0.f;
        if (label >= 0)
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (label == i) l[i] -= gs;
        // in place of each pair: its bf16 values and, with two terms, in bf16 what
        // those leave out (nothing of an infinity)
        if (two) {
#pragma unroll
          for (int i = 0; i < kHalf; i += 2) {
            const __nv_bfloat162 top = __floats2bfloat162_rn(l[i], l[i + 1]);
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&top);
            const float a0 = bf16_lo(u), a1 = bf16_hi(u);
            const __nv_bfloat162 rest = __floats2bfloat162_rn(fabsf(a0) < -kNegInf ? l[i] - a0 : 0.f,
                                                              fabsf(a1) < -kNegInf ? l[i + 1] - a1 : 0.f);
            l[i] = __uint_as_float(u);
            l[i + 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&rest));
          }
        } else {
#pragma unroll
          for (int i = 0; i < kHalf; i += 2) {
            const __nv_bfloat162 top = __floats2bfloat162_rn(l[i], l[i + 1]);
            l[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&top));
          }
        }
      }
      bool some = true;
      const bool part = EPI == kGrads && p.part;
      if constexpr (EPI == kGrads) {
        // no steps: a split of a ragged last piece (nothing to add), or dw without rows (zeros)
        int k0, k1;
        split_range(split, p, k0, k1);
        some = k0 < k1;
      }
      if (EPI == kGrads && !take()) break;
      // 32 columns: the last of kGrads hands the accumulator back once it is read
      auto block = [&](int cc) {
        uint32_t v[32];
        __syncwarp();
        if constexpr (EPI == kGrads) {
          tmem_ld32(tbase + (uint32_t)(cc * 32), v);
          if (cc == kHalf / 32 - 1) give();
        }
        if (part) {
          if (live && some && cc * 32 < ncols) {
            float* to = g.acc + ((terms ? split * 2 + (int)rank : split) * p.M + row) * p.N + c0 + cc * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (cc * 32 + 4 * i >= ncols) break;
              float4 o = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                     __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
              if (g.add) {
                const float4 b = reinterpret_cast<const float4*>(to)[i];
                o.x += b.x; o.y += b.y; o.z += b.z; o.w += b.w;
              }
              reinterpret_cast<float4*>(to)[i] = o;
            }
          }
        } else if (EPI == kGrads && g.out_fp32) {
          if (live && cc * 32 < ncols) {
            float* to = static_cast<float*>(p.out) + from * p.N + c0 + cc * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (cc * 32 + 4 * i >= ncols) break;
              reinterpret_cast<float4*>(to)[i] =
                  some ? make_float4(__uint_as_float(v[4 * i]) * scale, __uint_as_float(v[4 * i + 1]) * scale,
                                     __uint_as_float(v[4 * i + 2]) * scale, __uint_as_float(v[4 * i + 3]) * scale)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
        } else {
          // bf16 tile: 32 rows x 64 columns staged (128-byte swizzle: 16-byte
          // chunk i of row r at chunk i ^ (r & 7)) and stored by TMA, which
          // clips at the matrix's edges
          uint4 pk[4];
          if constexpr (EPI == kDlogits) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* f = l + cc * 32 + 8 * i;
              pk[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[2]), __float_as_uint(f[4]), __float_as_uint(f[6]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t u[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float lo = __uint_as_float(v[8 * i + 2 * j]) * scale, hi = __uint_as_float(v[8 * i + 2 * j + 1]) * scale;
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(some ? lo : 0.f, some ? hi : 0.f);
                u[j] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              pk[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
          if (EPI == kGrads && p.scatter) {  // (d is a multiple of 8: whole vectors)
            if (live) {
              uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + from * p.N + c0 + cc * 32);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (cc * 32 + 8 * i < ncols) to[i] = pk[i];
            }
            return;
          }
          if (EPI == kDlogits && terms && rank) return;  // (rows of this CTA: none)
          if (EPI == kDlogits && two) {
            uint16_t* to = static_cast<uint16_t*>(p.out) + row * p.ld + c0 + cc * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* f = l + cc * 32 + 8 * i;
              if (row < g.rest_rows && cc * 32 + 8 * i < ncols)
                reinterpret_cast<uint4*>(to)[i] =
                    make_uint4(__float_as_uint(f[1]), __float_as_uint(f[3]), __float_as_uint(f[5]), __float_as_uint(f[7]));
            }
          }
          if ((cc & 1) == 0) {
            if (lane == 0) bulk_wait_group_read0();  // the previous store has read the buffer
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((((cc & 1) * 4 + i) ^ (lane & 7)) << 4)) = pk[i];
          if (cc & 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.c[which], stg, (int32_t)(c0 + (cc - 1) * 32), mt * kTile + (int32_t)rank * kHalf + q * 32);
              bulk_commit_group();
            }
          }
        }
      };
      if constexpr (EPI == kGrads) {
#pragma unroll 1
        for (int cc = 0; cc < kHalf / 32; ++cc) block(cc);
      } else {
#pragma unroll
        for (int cc = 0; cc < kHalf / 32; ++cc) block(cc);
      }
    }
    if (lane == 0) bulk_wait_group0();  // this warp's TMA stores complete before the CTA exits
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Joins (m, s) pairs: the sum of s exp(m - M) under the common maximum M.  A
// maximum that is NaN, +inf or -inf is the result by itself.  c holds what the
// additions' roundings left out of s (exactly, where neither factor rounds).
struct Stats {
  float m, s, c;
};
__device__ __forceinline__ void join_stats(Stats& a, const Stats& b) {
  const float top = max_nan(a.m, b.m);
  const float base = top == kNegInf ? 0.f : top;
  const float fa = exp_of_difference(a.m, base), fb = exp_of_difference(b.m, base);
  const float x = __fmul_rn(a.s, fa), y = __fmul_rn(b.s, fb);
  const float sum = __fadd_rn(x, y), part = __fsub_rn(sum, x);
  const float left = __fadd_rn(__fsub_rn(x, __fsub_rn(sum, part)), __fsub_rn(y, part));
  a.c = a.c * fa + b.c * fb + left;
  a.s = sum;
  a.m = top;
}

// lse and loss of a row from its column blocks' maxima and sums; one warp per row.
__global__ void __launch_bounds__(256) ce_join_kernel(const float2* stats, int64_t cols, const float* at_label,
                                                      const int64_t* labels, int64_t t, int64_t v, float* loss,
                                                      float* lse) {
  let_dependents_start();
  wait_for_stream();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= t) return;
  const int lane = threadIdx.x & 31;
  Stats a{kNegInf, 0.f, 0.f};
#pragma unroll 4
  for (int64_t i = lane; i < cols; i += 32) {
    const float2 x = stats[row * cols + i];
    join_stats(a, {x.x, x.y, 0.f});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join_stats(a, {__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o), __shfl_xor_sync(0xFFFFFFFFu, a.c, o)});
  if (lane == 0) {
    const float m = a.m, s = a.s + a.c;
    // the loss is taken from the maximum, not from lse: a confident token's is
    // far smaller than lse's last bit (and, with s >= 1, never negative)
    const float rest = (m == m && fabsf(m) != -kNegInf) ? logf(s) : 0.f;
    const int64_t label = labels[row];
    lse[row] = m + rest;
    loss[row] = label >= 0 && label < v ? (m - at_label[row]) + rest : 0.f;
  }
}

// The rows with a target in order, their number, and s = max |dloss| over them
// (1 where that is 0 or not finite).  Where there are other rows, the listed
// rows of h are copied together (and zeros up to a whole step of K behind them)
// and the others' rows of dh are set to zero.  Every CTA takes a run of rows and
// counts the labels ahead of it by itself, 8 bytes a row from the L2: one launch.
__global__ void __launch_bounds__(256) ce_rows_kernel(const float* dloss, const int64_t* labels, int64_t t, int64_t v,
                                                      const uint4* h, int64_t ldh8, int d8, uint4* copied, uint4* dh,
                                                      int dh16, float* scale, int* rows_p, int* list) {
  __shared__ float top_sh[8];
  __shared__ int before_sh[8], total_sh[8], count_sh[8], place_sh[256];
  let_dependents_start();
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per = (t + gridDim.x - 1) / gridDim.x, r0 = min(t, blockIdx.x * per), r1 = min(t, r0 + per);
  float m = 0.f;
  int before = 0, total = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < t; i += 256) {
    const int64_t label = labels[i];
    const bool target = label >= 0 && label < v;
    total += target;
    before += target && i < r0;
    if (blockIdx.x == 0 && target) m = absmax_acc(m, dloss[i]);
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  m = warp_max_xor(m, 32);
  if (lane == 0) {
    before_sh[warp] = before;
    total_sh[warp] = total;
    top_sh[warp] = m;
  }
  __syncthreads();
  before = total = 0;
  for (int i = 0; i < 8; ++i) {
    before += before_sh[i];
    total += total_sh[i];
    m = fmaxf(m, top_sh[i]);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *scale = finite_pos(m) ? m : 1.f;
    *rows_p = total;
  }
  const bool all = total == t;
  for (int64_t b = r0; b < r1; b += 256) {
    const int64_t i = b + threadIdx.x;
    const int64_t label = i < r1 ? labels[i] : -1;
    const bool target = label >= 0 && label < v;
    const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, target);
    __syncthreads();  // the last run's places are used
    if (lane == 0) count_sh[warp] = __popc(ballot);
    __syncthreads();
    int place = before + __popc(ballot & ((1u << lane) - 1u));
    for (int j = 0; j < 8; ++j) {
      if (j < warp) place += count_sh[j];
      before += count_sh[j];
    }
    place_sh[threadIdx.x] = target ? place : -1;
    if (target) list[place] = (int)i;
    if (all) continue;
    __syncthreads();
    for (int64_t r = b + warp; r < min(r1, b + 256); r += 8) {  // one warp per row
      const int to = place_sh[r - b];
      if (to >= 0) {
#pragma unroll 8
        for (int j = lane; j < d8; j += 32) copied[(int64_t)to * d8 + j] = h[r * ldh8 + j];
      } else {
        for (int j = lane; j < dh16; j += 32) dh[r * dh16 + j] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (!all && blockIdx.x == gridDim.x - 1) {
    const int64_t padded = min(t, ((int64_t)total + kStepK - 1) / kStepK * kStepK);
    for (int64_t i = (int64_t)total * d8 + threadIdx.x; i < padded * d8; i += 256) copied[i] = make_uint4(0, 0, 0, 0);
  }
}

// dh from its partial sums: the splits in order (and of few rows both terms of
// each), times the scale, to the listed rows.  A warp takes 32 vectors of a row.
__global__ void __launch_bounds__(256) ce_finish_kernel(const float4* acc, int d4, int splits, int direct,
                                                        const float* scale, const int* rows_p, const int* list, void* out,
                                                        int fp32) {
  let_dependents_start();
  wait_for_stream();
  const float s = *scale;
  const int rows = *rows_p, lane = threadIdx.x & 31, runs = (d4 + 31) / 32;
  if (rows <= kFew) splits *= 2;
  else if (direct) return;
  const int64_t slab = (int64_t)rows * d4, items = (int64_t)rows * runs;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < items; w += (int64_t)gridDim.x * 8) {
    const int64_t r = w / runs;
    const int i = (int)(w - r * runs) * 32 + lane;
    if (i >= d4) continue;
    const int64_t at = (int64_t)list[r] * d4 + i;
    float4 a = acc[r * d4 + i];
#pragma unroll 4
    for (int k = 1; k < splits; ++k) {
      const float4 b = acc[k * slab + r * d4 + i];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    if (fp32) {
      static_cast<float4*>(out)[at] = make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * s, a.y * s), hi = __floats2bfloat162_rn(a.z * s, a.w * s);
      static_cast<uint2*>(out)[at] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
}

// ------------------------------------------------------------------ host side
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t cdiv(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Words per piece of the backward pass: dl takes at most 2^28 values (512 MiB)
// unless 64 words of it are more.
int64_t piece_of(int64_t rows, int64_t v, int64_t piece) {
  if (piece == 0) piece = std::max<int64_t>(64, (((int64_t)1 << 28) / std::max<int64_t>(rows, 1)) / 64 * 64);
  return std::min(piece, round_up(v, 64));
}

constexpr double kItemStart = 3;  // a tile's start and end, in steps (it also stores its result over the port that feeds it)

// What a pair with one item fewer of the first product (n0 of c0 steps) takes
// of the second (n1 of c1 steps) instead.
int extra_items(int64_t n0, double c0, int64_t n1, double c1, int pairs) {
  const int64_t fewer = pairs - n0 % pairs;
  return fewer == pairs ? 0 : (int)std::min<int64_t>((int64_t)(c0 / c1 + 0.5), n1 / fewer);
}

// Splits of dh's sum over a piece's words.  dh has few tiles when t is small
// and its sum is long: the split makes items that spread over the pairs beside
// dw's (t steps each), and costs its slab of FP32 partial sums written and read
// once.  The estimate: the longest pair at 0.33 us a step, memory at 6.5 TB/s.
int dh_splits(int64_t t, int64_t d, int64_t width, bool two_terms, int pairs) {
  const bool few = t <= kFew;
  const int64_t tiles = cdiv(t, kTile) * cdiv(d, kTile), steps = cdiv(width, kStepK);
  const int64_t along = two_terms && !few ? 2 * steps : steps;  // (of few rows with a target: `steps` all the same)
  const int64_t n1 = cdiv(width, kTile) * cdiv(d, kTile);
  const int terms = few ? 2 : 1;  // slabs of dh's sums
  const double c1 = (double)((two_terms || few ? 2 : 1) * cdiv(t, kStepK)) + kItemStart;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 64 && s <= steps; ++s) {
    const int64_t n0 = tiles * s;
    const double c0 = (double)cdiv(along, s) + kItemStart;
    const int64_t fewer = pairs - n0 % pairs, extra = extra_items(n0, c0, n1, c1, pairs);
    const double shared = (double)cdiv(n1 - extra * fewer, pairs) * c1;
    const double longest = std::max((double)cdiv(n0, pairs) * c0, (double)(n0 / pairs) * c0 + (double)extra * c1) + shared;
    const double us = longest * 0.33 + (s > 1 ? (double)(s * terms) * (double)t * (double)d * 8.0 / 6.5e6 : 0.0);
    if (s == 1 || us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

// Rows of A in a load.  A K-major A of up to kFew rows takes those alone, in the
// even CTA (or a term in each): a load of rows that are not there costs more
// than one of rows that are.  What the rest of the stage holds enters rows that
// are not stored.  Forward, one row: 32000 x 4096 90 -> 54 us, 131072 x 1024
// 80 -> 53 us; from 64 rows on no difference.
int a_box(bool a_mn, int64_t M) { return !a_mn && M <= kFew ? (int)round_up(M, 8) : kHalf; }

struct Operand {
  const void* p;
  int64_t ld;  // elements
};

// Describes product i of a launch: A [M, K] (K-major) or [K, M] (a_mn), B [N, K]
// or (b_mn) [K, N]; C the bf16 output of the kinds that store one by TMA.
lpq_status set_product(CeTile& g, CeMaps& maps, int i, int64_t M, int64_t N, int64_t K, Operand a, bool a_mn, Operand b,
                       bool b_mn, void* c, int64_t ldc, int splits) {
  lpq_status st;
  if ((st = a_mn ? make_map(&maps.a[i], a.p, true, M, K, a.ld * 2, 64, kStepK)
                 : make_map(&maps.a[i], a.p, true, K, M, a.ld * 2, kStepK, a_box(a_mn, M))) != LPQ_OK) return st;
  if ((st = b_mn ? make_map(&maps.b[i], b.p, true, N, K, b.ld * 2, 64, kStepK)
                 : make_map(&maps.b[i], b.p, true, K, N, b.ld * 2, kStepK, kHalf)) != LPQ_OK) return st;
  if (c && (st = make_map(&maps.c[i], c, true, N, M, ldc * 2, 64, 32)) != LPQ_OK) return st;
  const int64_t tm = cdiv(M, kTile), tn = cdiv(N, kTile);
  if (tm * tn * splits > (int64_t)1 << 30) return set_error(LPQ_ERR_SHAPE, "too many output tiles");
  Product& p = g.prod[i];
  p.M = M;
  p.N = N;
  p.num_k = (int)cdiv(K, kStepK);
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.splits = splits;
  p.items = (int)(tm * tn * splits);
  p.a_mn = a_mn;
  p.a_box = a_box(a_mn, M);
  return LPQ_OK;
}

template <int EPI>
lpq_status run_pair(CeTile& g, const CeMaps& maps, cudaStream_t s) {
  lpq_status st = device_error_word(&g.err);
  if (st != LPQ_OK) return st;
  if ((st = set_smem_attr(reinterpret_cast<const void*>(ce_pair_kernel<EPI>), kSmem)) != LPQ_OK) return st;
  const int64_t items = (int64_t)g.prod[0].items + g.prod[1].items;
  const int pairs = (int)std::min<int64_t>(items, std::max(1, device_sms() / 2));
  if (g.prod[1].items > 0)
    g.extra = extra_items(g.prod[0].items, (double)cdiv(g.prod[0].num_k, g.prod[0].splits) + kItemStart, g.prod[1].items,
                          (double)g.prod[1].num_k + kItemStart, pairs);
  return cuda_check(launch_dependent(ce_pair_kernel<EPI>, 2 * pairs, kThreads, kSmem, s, maps, g), "cross entropy launch");
}

// Workspace of the backward pass: scale and count, list, copied rows of h, dl,
// partial sums of dh.
struct BackwardPlan {
  int64_t piece, dl_ld;
  int splits;
  bool direct;  // one piece, one split: dh is stored by its product (if over kFew rows have a target)
  int64_t rest_rows;  // of dl's second terms
  size_t list_at, h_at, dl_at, acc_at, bytes;
  BackwardPlan(int64_t t, int64_t v, int64_t d, int64_t asked, bool two_terms) {
    const int64_t few = std::min<int64_t>(t, kFew);
    rest_rows = two_terms ? t : few;
    piece = piece_of(two_terms && t > kFew ? 2 * t : t, v, asked);
    dl_ld = std::min(piece, round_up(v, 8));
    // 76 pairs whatever the device has: the workspace and the results depend on the sizes alone
    splits = dh_splits(t, d, std::min(piece, v), two_terms, 76);
    direct = splits == 1 && piece >= v && t > kFew;
    list_at = 256;
    h_at = list_at + (size_t)round_up(t * 4, 256);
    dl_at = h_at + (size_t)round_up(t * d * 2, 256);
    acc_at = dl_at + (size_t)round_up((t + rest_rows) * dl_ld * 2, 256);
    // partial sums of all rows, and two of each of a few
    bytes = acc_at + (size_t)std::max(direct ? 0 : t, 2 * few) * (size_t)splits * (size_t)d * 4;
  }
};

}  // namespace

size_t ce_workspace(int64_t t, int64_t v, int64_t d, bool backward, int64_t piece, bool two_terms) {
  if (t == 0) return 0;
  if (!backward) return (size_t)round_up(t * 4, 256) + (size_t)cdiv(v, kHalf) * (size_t)t * sizeof(float2);
  return BackwardPlan(t, v, d, piece, two_terms).bytes;
}

lpq_status launch_ce(const CeArgs& a, cudaStream_t s) {
  if (a.t == 0) return LPQ_OK;
  CeTile g{};
  CeMaps maps{};
  g.labels = a.labels;
  g.vocab = a.v;
  g.at_label = reinterpret_cast<float*>(a.workspace);
  g.stats = reinterpret_cast<float2*>(a.workspace + round_up(a.t * 4, 256));
  g.stat_cols = cdiv(a.v, kHalf);
  lpq_status st = set_product(g, maps, 0, a.t, a.v, a.d, {a.h, a.ldh}, false, {a.w, a.ldw}, false, nullptr, 0, 1);
  if (st != LPQ_OK) return st;
  if ((st = run_pair<kStats>(g, maps, s)) != LPQ_OK) return st;
  return cuda_check(launch_dependent(ce_join_kernel, (unsigned)cdiv(a.t, 8), 256, 0, s, g.stats, g.stat_cols, g.at_label,
                                     a.labels, a.t, a.v, a.loss, a.lse_out),
                    "cross entropy join launch");
}

lpq_status launch_ce_backward(const CeArgs& a, cudaStream_t s) {
  const size_t elem = a.grads_fp32 ? 4 : 2;
  if (a.t == 0) return cuda_check(cudaMemsetAsync(a.dw, 0, (size_t)a.v * (size_t)a.d * elem, s), "cudaMemsetAsync(dw)");
  const BackwardPlan plan(a.t, a.v, a.d, a.piece, a.two_terms);
  float* scale = reinterpret_cast<float*>(a.workspace);
  int* rows = reinterpret_cast<int*>(a.workspace + 4);
  int* list = reinterpret_cast<int*>(a.workspace + plan.list_at);
  void* dl = a.workspace + plan.dl_at;
  CeTile base{};
  base.t = a.t;
  base.rows = rows;
  base.list = list;
  base.labels = a.labels;
  base.vocab = a.v;
  base.lse = a.lse;
  base.dloss = a.dloss;
  base.scale = scale;
  base.acc = reinterpret_cast<float*>(a.workspace + plan.acc_at);
  base.out_fp32 = a.grads_fp32;
  base.two_terms = a.two_terms;
  base.rest_rows = plan.rest_rows;
  const Operand h{a.h, a.ldh}, copied{a.workspace + plan.h_at, a.d}, l{dl, plan.dl_ld};
  lpq_status st = cuda_check(
      launch_dependent(ce_rows_kernel, (unsigned)std::min<int64_t>(cdiv(a.t, 8), (int64_t)device_sms() * 8), 256, 0, s, a.dloss,
                       a.labels, a.t, a.v, static_cast<const uint4*>(a.h), a.ldh / 8, (int)(a.d / 8),
                       reinterpret_cast<uint4*>(a.workspace + plan.h_at), static_cast<uint4*>(a.dh),
                       (int)(a.d * (int64_t)elem / 16), scale, rows, list),
      "cross entropy rows launch");
  if (st != LPQ_OK) return st;
  for (int64_t v0 = 0; v0 < a.v; v0 += plan.piece) {
    const int64_t width = std::min(plan.piece, a.v - v0);
    const Operand w{static_cast<const uint8_t*>(a.w) + (size_t)v0 * (size_t)a.ldw * 2, a.ldw};
    CeMaps maps{};
    // dl = (exp(h w^T - lse) - onehot) dloss / s
    CeTile g = base;
    g.col0 = v0;
    if ((st = set_product(g, maps, 0, a.t, width, a.d, h, false, w, false, dl, plan.dl_ld, 1)) != LPQ_OK) return st;
    if ((st = make_map(&maps.alt, copied.p, true, a.d, a.t, copied.ld * 2, kStepK, a_box(false, a.t))) != LPQ_OK) return st;
    g.prod[0].m_rows = 1;
    const Operand l2{static_cast<uint8_t*>(dl) + (size_t)a.t * (size_t)plan.dl_ld * 2, plan.dl_ld};
    g.prod[0].out = const_cast<void*>(l2.p);
    g.prod[0].ld = plan.dl_ld;
    if ((st = run_pair<kDlogits>(g, maps, s)) != LPQ_OK) return st;
    // dh (+)= dl w and dw = dl^T h
    g = base;
    g.add = v0 > 0;
    void* dw = static_cast<uint8_t*>(a.dw) + (size_t)v0 * (size_t)a.d * elem;
    if ((st = set_product(g, maps, 0, a.t, a.d, width, l, false, w, true, nullptr, 0, plan.splits)) != LPQ_OK) return st;
    if ((st = make_map(&maps.a2[0], l2.p, true, width, plan.rest_rows, l2.ld * 2, kStepK, a_box(false, a.t))) != LPQ_OK) return st;
    if ((st = make_map(&maps.alt, copied.p, true, a.d, a.t, copied.ld * 2, 64, kStepK)) != LPQ_OK) return st;
    g.prod[0].m_rows = 1;
    g.prod[0].scatter = plan.direct;
    g.prod[0].part = !plan.direct;
    g.prod[0].out = a.dh;
    // in one launch where dh's last round would leave over a tenth of the
    // pairs' time for it idle, which dw's items then fill (1001 x 1024 x 50001:
    // dh and dw 139 us one after the other, 125 us in one); else one after the
    // other, each with the L2 to itself (7936 x 4096 x 32000: 2182 us, in one 2250)
    const int64_t P = std::max(1, device_sms() / 2), n0 = g.prod[0].items, rounds = cdiv(n0, P) * P;
    const int at = 10 * (rounds - n0) > rounds ? 1 : 0;
    if (at == 0) {
      if ((st = run_pair<kGrads>(g, maps, s)) != LPQ_OK) return st;
      g = base;
    }
    if ((st = set_product(g, maps, at, width, a.d, a.t, l, true, h, true, a.grads_fp32 ? nullptr : dw, a.d, 1)) != LPQ_OK) return st;
    if ((st = make_map(&maps.a2[at], l2.p, true, width, plan.rest_rows, l2.ld * 2, 64, kStepK)) != LPQ_OK) return st;
    if (a.t <= kFew) g.prod[at].num_k *= 2;
    g.prod[at].k_rows = 1;
    g.prod[at].out = dw;
    if ((st = run_pair<kGrads>(g, maps, s)) != LPQ_OK) return st;
  }
  const int64_t most = plan.direct ? kFew : a.t;  // rows to join
  const unsigned grid = (unsigned)std::min<int64_t>(cdiv(most * cdiv(a.d, 128), 8), (int64_t)device_sms() * 8);
  return cuda_check(launch_dependent(ce_finish_kernel, grid, 256, 0, s, reinterpret_cast<const float4*>(base.acc),
                                     (int)(a.d / 4), plan.splits, (int)plan.direct, scale, rows, list, a.dh, a.grads_fp32),
                    "cross entropy finish launch");
}

}  // namespace lpq
