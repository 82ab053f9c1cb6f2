// Softmax cross entropy of a vocabulary projection and its gradients on
// sm_103a.  The logits l = h w^T exist tile by tile only:
//
//   forward   each tile leaves every row's maximum m and sum of exp(l - m);
//             a second kernel joins them: lse = log sum_j exp(l_j),
//             loss = lse - l[label].
//   backward  per piece of the vocabulary the logits are computed again and
//             turned into dl = (exp(l - lse) - onehot) dloss in bf16; then
//             dh += dl w (FP32 sums across pieces) and dw = dl^T h.
//
// dl is divided by s = max |dloss| before its rounding to bf16 (what the
// tensor cores read) and s multiplies the FP32 sums: with equal dloss, the
// mean over the tokens say, the entry p - 1 of a label is then rounded as it
// is instead of after a product with 1 / t.
#include <cuda_bf16.h>

#include <algorithm>

#include "lpq_device.cuh"

namespace lpq {
namespace {

constexpr int kTile = 64, kTileK = 16;
constexpr float kNegInf = -__builtin_huge_valf();

enum { kStats, kDlogits, kDh, kDw };

struct CeTile {
  const __nv_bfloat16* a;  // element (i, k) at a[i * ai + k * ak]
  const __nv_bfloat16* b;  // element (j, k) at b[j * bj + k * bk]
  int64_t ai, ak, bj, bk;
  int64_t M, N, K;
  int64_t col0;  // first word of the piece
  const int64_t* labels;
  int64_t vocab;
  float2* stats;    // [tiles_n][M]
  float* at_label;  // [M]
  const float* lse;
  const float* dloss;
  const float* scale;
  __nv_bfloat16* dl;
  int64_t ldl;
  float* acc;  // dh sums [M, N]
  int first;
  void* out;
  int out_fp32;
};

__device__ __forceinline__ void store(void* out, int fp32, int64_t at, float v) {
  if (fp32) static_cast<float*>(out)[at] = v;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

template <int EPI>
__global__ void __launch_bounds__(256) ce_tile_kernel(const CeTile g) {
  __shared__ float sa[kTileK][kTile + 1], sb[kTileK][kTile + 1], sc[kTile][kTile + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < g.K; k0 += kTileK) {
    for (int e = threadIdx.x; e < kTile * kTileK; e += 256) {
      const int i = e / kTileK, k = e % kTileK;
      sa[k][i] = (m0 + i < g.M && k0 + k < g.K) ? __bfloat162float(g.a[(m0 + i) * g.ai + (k0 + k) * g.ak]) : 0.f;
      sb[k][i] = (n0 + i < g.N && k0 + k < g.K) ? __bfloat162float(g.b[(n0 + i) * g.bj + (k0 + k) * g.bk]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kTileK; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
    __syncthreads();
  }
  if constexpr (EPI == kStats) {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) sc[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    const int64_t row = m0 + threadIdx.x;
    if (threadIdx.x < kTile && row < g.M) {
      const int cols = (int)min((int64_t)kTile, g.N - n0);
      float m = kNegInf, s = 0.f;
      bool nan = false;
      for (int j = 0; j < cols; ++j) {
        nan |= sc[threadIdx.x][j] != sc[threadIdx.x][j];
        m = fmaxf(m, sc[threadIdx.x][j]);
      }
      for (int j = 0; j < cols; ++j) s += isinf(m) ? (sc[threadIdx.x][j] == m && m > 0.f) : expf(sc[threadIdx.x][j] - m);
      g.stats[blockIdx.x * g.M + row] = make_float2(nan ? __int_as_float(0x7FC00000) : m, s);
      const int64_t label = g.labels[row];
      if (label >= n0 && label < n0 + cols) g.at_label[row] = sc[threadIdx.x][label - n0];
    }
  } else {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
        if (r >= g.M || c >= g.N) continue;
        if constexpr (EPI == kDlogits) {
          const int64_t label = g.labels[r];
          float v = 0.f;
          if (label >= 0 && label < g.vocab)
            v = (expf(acc[i][j] - g.lse[r]) - (g.col0 + c == label ? 1.f : 0.f)) * (g.dloss[r] / *g.scale);
          g.dl[r * g.ldl + c] = __float2bfloat16_rn(v);
        } else if constexpr (EPI == kDh) {
          float* p = g.acc + r * g.N + c;
          *p = (g.first ? 0.f : *p) + acc[i][j];
        } else {
          store(g.out, g.out_fp32, r * g.N + c, acc[i][j] * *g.scale);
        }
      }
  }
}

// lse and loss of a row from its tiles' maxima and sums; one thread per row.
__global__ void __launch_bounds__(256) ce_join_kernel(const float2* stats, int64_t tiles, const float* at_label,
                                                      const int64_t* labels, int64_t t, int64_t v, float* loss,
                                                      float* lse) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= t) return;
  float m = kNegInf;
  bool nan = false;
  for (int64_t i = 0; i < tiles; ++i) {
    const float x = stats[i * t + row].x;
    nan |= x != x;
    m = fmaxf(m, x);
  }
  float s = 0.f;
  if (!isinf(m))
    for (int64_t i = 0; i < tiles; ++i) {
      const float2 x = stats[i * t + row];
      if (x.y > 0.f) s += x.y * expf(x.x - m);
    }
  const float l = nan ? __int_as_float(0x7FC00000) : isinf(m) ? m : m + logf(s);
  lse[row] = l;
  const int64_t label = labels[row];
  loss[row] = label >= 0 && label < v ? l - at_label[row] : 0.f;
}

// s = max |dloss| over the rows with a target; 1 where that is 0 or not finite.
__global__ void __launch_bounds__(1024) ce_scale_kernel(const float* dloss, const int64_t* labels, int64_t t, int64_t v,
                                                        float* scale) {
  __shared__ float sh[32];
  float m = 0.f;
  for (int64_t i = threadIdx.x; i < t; i += 1024)
    if (labels[i] >= 0 && labels[i] < v) m = absmax_acc(m, dloss[i]);
  m = warp_max_xor(m, 32);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = warp_max_xor(sh[threadIdx.x], 32);
    if (threadIdx.x == 0) *scale = finite_pos(m) ? m : 1.f;
  }
}

__global__ void __launch_bounds__(256) ce_finish_kernel(const float* acc, int64_t n, const float* scale, void* out,
                                                        int fp32) {
  const float s = *scale;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    store(out, fp32, i, acc[i] * s);
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int64_t piece_of(int64_t t, int64_t v, int64_t piece) {
  if (piece == 0) piece = std::max<int64_t>(64, (((int64_t)1 << 28) / std::max<int64_t>(t, 1)) / 64 * 64);
  return std::min(piece, round_up(v, 64));
}

template <int EPI>
lpq_status run_tile(const CeTile& g, cudaStream_t s) {
  const dim3 grid((unsigned)((g.N + kTile - 1) / kTile), (unsigned)((g.M + kTile - 1) / kTile));
  ce_tile_kernel<EPI><<<grid, 256, 0, s>>>(g);
  return cuda_check(cudaGetLastError(), "cross entropy launch");
}

}  // namespace

size_t ce_workspace(int64_t t, int64_t v, int64_t d, bool backward, int64_t piece) {
  if (t == 0) return 0;
  if (!backward) return (size_t)round_up(t * 4, 256) + (size_t)((v + kTile - 1) / kTile) * (size_t)t * sizeof(float2);
  return 256 + (size_t)round_up(t * d * 4, 256) + (size_t)t * (size_t)piece_of(t, v, piece) * 2;
}

lpq_status launch_ce(const CeArgs& a, cudaStream_t s) {
  if (a.t == 0) return LPQ_OK;
  CeTile g{};
  g.a = static_cast<const __nv_bfloat16*>(a.h);
  g.b = static_cast<const __nv_bfloat16*>(a.w);
  g.ai = a.ldh; g.ak = 1; g.bj = a.ldw; g.bk = 1;
  g.M = a.t; g.N = a.v; g.K = a.d;
  g.labels = a.labels;
  g.at_label = reinterpret_cast<float*>(a.workspace);
  g.stats = reinterpret_cast<float2*>(a.workspace + round_up(a.t * 4, 256));
  lpq_status st = run_tile<kStats>(g, s);
  if (st != LPQ_OK) return st;
  ce_join_kernel<<<(unsigned)((a.t + 255) / 256), 256, 0, s>>>(g.stats, (a.v + kTile - 1) / kTile, g.at_label, a.labels,
                                                               a.t, a.v, a.loss, a.lse_out);
  return cuda_check(cudaGetLastError(), "cross entropy join launch");
}

lpq_status launch_ce_backward(const CeArgs& a, cudaStream_t s) {
  const size_t out_elem = a.grads_fp32 ? 4 : 2;
  if (a.t == 0) return cuda_check(cudaMemsetAsync(a.dw, 0, (size_t)a.v * (size_t)a.d * out_elem, s), "cudaMemsetAsync(dw)");
  float* scale = reinterpret_cast<float*>(a.workspace);
  float* acc = reinterpret_cast<float*>(a.workspace + 256);
  __nv_bfloat16* dl = reinterpret_cast<__nv_bfloat16*>(a.workspace + 256 + round_up(a.t * a.d * 4, 256));
  const int64_t piece = piece_of(a.t, a.v, a.piece);
  ce_scale_kernel<<<1, 1024, 0, s>>>(a.dloss, a.labels, a.t, a.v, scale);
  lpq_status st = cuda_check(cudaGetLastError(), "cross entropy scale launch");
  if (st != LPQ_OK) return st;
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(a.h);
  for (int64_t v0 = 0; v0 < a.v; v0 += piece) {
    const int64_t width = std::min(piece, a.v - v0);
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.w) + v0 * a.ldw;
    CeTile g{};
    g.labels = a.labels; g.vocab = a.v; g.lse = a.lse; g.dloss = a.dloss; g.scale = scale; g.col0 = v0;
    g.dl = dl; g.ldl = piece; g.acc = acc; g.first = v0 == 0; g.out_fp32 = a.grads_fp32;
    g.a = h; g.ai = a.ldh; g.ak = 1; g.b = w; g.bj = a.ldw; g.bk = 1;
    g.M = a.t; g.N = width; g.K = a.d;
    if ((st = run_tile<kDlogits>(g, s)) != LPQ_OK) return st;
    g.a = dl; g.ai = piece; g.ak = 1; g.b = w; g.bj = 1; g.bk = a.ldw;
    g.M = a.t; g.N = a.d; g.K = width;
    if ((st = run_tile<kDh>(g, s)) != LPQ_OK) return st;
    g.a = dl; g.ai = 1; g.ak = piece; g.b = h; g.bj = 1; g.bk = a.ldh;
    g.M = width; g.N = a.d; g.K = a.t;
    g.out = static_cast<uint8_t*>(a.dw) + (size_t)v0 * (size_t)a.d * out_elem;
    if ((st = run_tile<kDw>(g, s)) != LPQ_OK) return st;
  }
  ce_finish_kernel<<<device_sms() * 8, 256, 0, s>>>(acc, a.t * a.d, scale, a.dh, a.grads_fp32);
  return cuda_check(cudaGetLastError(), "cross entropy finish launch");
}

}  // namespace lpq
