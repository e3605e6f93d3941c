// A gradient of all the router's scores taken to the tokens, the router's
// weights and its logit offset: with g = dscores s (1 - s) for sigmoid scores,
//
//   dx = g W_r  [T][d],   dW_r = g^T x  [n][d],   d_offset = sum_t g  [n]
//
// Two products of 2 T n d operations each on the bf16 MFMA.  Their operands
// are written K-contiguous first, in one launch (g both ways, W_r and x
// transposed).  dW_r is an fp32 output:
// g enters it as the exact sum of three bf16 parts (24 bits), three segments of
// one contraction against the same bf16 x.  dx is rounded to bf16: two parts of
// g and of W_r (16 bits each) are kept, without the product of the low parts.
//
// T = 4096, d = 7168, n = 896: 428 us; the products take 236 us (dW_r) and 203 us
// (dx) on their own, 158 GFLOP of bf16 each, 0.67 and 0.78 PFLOP/s, and bound it.
#include <algorithm>

#include "common.hpp"
#include "gemm.hpp"
#include "layer_kernels.hpp"

namespace moe {
namespace router {

constexpr int TILE = 64;

// What bf16 rounding left of v, rounded in turn.
__device__ __forceinline__ void split2(float v, bf16_t& hi, bf16_t& lo) {
  hi = f32_to_bf16(v);
  lo = f32_to_bf16(v - bf16_to_f32(hi));
}

// Eight values to one 16-byte store.
__device__ __forceinline__ void store8(bf16_t* p, const bf16_t (&v)[8]) {
  uint4 q;
  q.x = v[0] | (static_cast<uint32_t>(v[1]) << 16);
  q.y = v[2] | (static_cast<uint32_t>(v[3]) << 16);
  q.z = v[4] | (static_cast<uint32_t>(v[5]) << 16);
  q.w = v[6] | (static_cast<uint32_t>(v[7]) << 16);
  *reinterpret_cast<uint4*>(p) = q;
}

struct Prep {
  const float *scores, *dscores, *w;
  const bf16_t* x;
  int T, n, d;
  int64_t np, Tp;
  bf16_t *g_hi, *g_lo, *gt_hi, *gt_mid, *gt_lo, *wt_hi, *wt_lo, *xt;
  float* part;
  // blocks of each kind, in this order: scores, x, W_r
  int score_blocks, x_blocks;
};

// g of 64 tokens x 64 experts: by token [T][np] in two parts, by expert [n][Tp]
// in three, zeros behind the ends, and the tile's sum per expert.
__device__ __forceinline__ void score_tile(const Prep& p, int e0, int tt, float* lds) {
  auto tile = reinterpret_cast<float(*)[TILE + 1]>(lds);
  const int t0 = tt * TILE;
  for (int i = threadIdx.x; i < TILE * TILE; i += 256) {
    const int t = i / TILE, e = i % TILE;
    float g = 0.f;
    if (t0 + t < p.T && e0 + e < p.n) {
      const int64_t at = static_cast<int64_t>(t0 + t) * p.n + e0 + e;
      const float s = p.scores[at];
      g = p.dscores[at] * (s * (1.f - s));
    }
    tile[t][e] = g;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < TILE * TILE / 8; i += 256) {
    const int r = i / 8, c = i % 8 * 8;
    bf16_t hi[8], mid[8], lo[8];
    if (t0 + r < p.T) {
#pragma unroll
      for (int j = 0; j < 8; ++j) split2(tile[r][c + j], hi[j], lo[j]);
      const int64_t at = static_cast<int64_t>(t0 + r) * p.np + e0 + c;
      store8(p.g_hi + at, hi);
      store8(p.g_lo + at, lo);
    }
    if (e0 + r < p.n) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = tile[c + j][r];
        split2(v, hi[j], mid[j]);
        lo[j] = f32_to_bf16((v - bf16_to_f32(hi[j])) - bf16_to_f32(mid[j]));
      }
      const int64_t at = (e0 + r) * p.Tp + t0 + c;
      store8(p.gt_hi + at, hi);
      store8(p.gt_mid + at, mid);
      store8(p.gt_lo + at, lo);
    }
  }
  if (threadIdx.x < TILE) {
    float sum = 0.f;
#pragma unroll 8
    for (int t = 0; t < TILE; ++t) sum += tile[t][threadIdx.x];
    p.part[tt * p.np + e0 + threadIdx.x] = sum;
  }
}

// out[c][r] = in[r][c], zeros from R to ld_out; fp32 input in two parts.  Tiles
// of 128 rows x 64 columns: 16 bytes per lane in, 256 consecutive bytes of an
// output row out.
constexpr int TROWS = 128;

template <typename IN>
__device__ __forceinline__ void transpose_tile(const IN* in, int R, int C, int64_t ld_out,
                                               bf16_t* hi, bf16_t* lo, int c0, int r0, void* lds) {
  constexpr int PER = 16 / sizeof(IN), LPR = TILE / PER;  // elements per load, lanes per row
  auto tile = reinterpret_cast<IN(*)[TILE + 1]>(lds);
#pragma unroll
  for (int i = threadIdx.x; i < TROWS * LPR; i += 256) {
    const int r = i / LPR, c = i % LPR * PER;
    __attribute__((aligned(16))) IN v[PER] = {};
    if (r0 + r < R)
      *reinterpret_cast<uint4*>(v) =
          *reinterpret_cast<const uint4*>(in + static_cast<int64_t>(r0 + r) * C + c0 + c);
#pragma unroll
    for (int j = 0; j < PER; ++j) tile[r][c + j] = v[j];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < TILE * TROWS / 8; i += 256) {
    const int c = i / (TROWS / 8), r = i % (TROWS / 8) * 8;
    if (r0 + r >= ld_out) continue;
    const int64_t at = (c0 + c) * ld_out + r0 + r;
    bf16_t h[8], l[8];
    if constexpr (std::is_same<IN, float>::value) {
#pragma unroll
      for (int j = 0; j < 8; ++j) split2(tile[r + j][c], h[j], l[j]);
      store8(lo + at, l);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = tile[r + j][c];
    }
    store8(hi + at, h);
  }
}

// All operands of the products in one launch: g both ways, x and W_r transposed.
__global__ __launch_bounds__(256) void prepare_k(Prep p) {
  __shared__ __attribute__((aligned(16))) float lds[TROWS * (TILE + 1)];
  int b = blockIdx.x;
  if (b < p.score_blocks) {
    const int tn = static_cast<int>(p.np / TILE);
    score_tile(p, b % tn * TILE, b / tn, lds);
    return;
  }
  b -= p.score_blocks;
  const int td = p.d / TILE;
  if (b < p.x_blocks) {
    transpose_tile<bf16_t>(p.x, p.T, p.d, p.Tp, p.xt, nullptr, b % td * TILE, b / td * TROWS, lds);
    return;
  }
  b -= p.x_blocks;
  transpose_tile<float>(p.w, p.n, p.d, p.np, p.wt_hi, p.wt_lo, b % td * TILE, b / td * TROWS, lds);
}

// A small layer in one launch, in fp32: a block takes CW columns of x, dx, W_r
// and dW_r with all of g in LDS.
constexpr int CW = 16;

constexpr int SMALL_THREADS = 1024;

__global__ __launch_bounds__(SMALL_THREADS) void small_k(
    const bf16_t* __restrict__ x, const float* __restrict__ w, const float* __restrict__ scores,
    const float* __restrict__ dscores, int T, int d, int n, int accumulate,
    bf16_t* __restrict__ dx, float* __restrict__ dw, float* __restrict__ doff) {
  extern __shared__ float lds[];
  float* const g = lds;           // [T][n]
  float* const wc = g + T * n;    // [n][CW]
  float* const xc = wc + n * CW;  // [T][CW]
  const int c0 = blockIdx.x * CW, tid = threadIdx.x;
  for (int i = tid; i < T * n; i += SMALL_THREADS) {
    const float s = scores[i];
    g[i] = dscores[i] * (s * (1.f - s));
  }
  if (c0 >= d) {  // the block behind the columns adds up the offset's gradient
    __syncthreads();
    for (int e = tid >> 6; e < n; e += SMALL_THREADS / 64) {
      double sum = 0.0;
      for (int t = tid & 63; t < T; t += 64) sum += g[t * n + e];
      for (int k = 32; k; k >>= 1) sum += __shfl_xor(sum, k);
      const float v = static_cast<float>(sum);
      if ((tid & 63) == 0) doff[e] = accumulate ? doff[e] + v : v;
    }
    return;
  }
  if (dx)
    for (int i = tid; i < n * CW; i += SMALL_THREADS)
      wc[i] = w[static_cast<int64_t>(i / CW) * d + c0 + i % CW];
  if (dw)
    for (int i = tid; i < T * CW; i += SMALL_THREADS)
      xc[i] = bf16_to_f32(x[static_cast<int64_t>(i / CW) * d + c0 + i % CW]);
  __syncthreads();
  if (dx)
    for (int i = tid; i < T * CW; i += SMALL_THREADS) {
      const int t = i / CW, c = i % CW;
      float sum = 0.f;
#pragma unroll 8
      for (int e = 0; e < n; ++e) sum = fmaf(g[t * n + e], wc[e * CW + c], sum);
      bf16_t* const o = dx + static_cast<int64_t>(t) * d + c0 + c;
      *o = f32_to_bf16(accumulate ? bf16_to_f32(*o) + sum : sum);
    }
  if (dw)
    for (int i = tid; i < n * CW; i += SMALL_THREADS) {
      const int e = i / CW, c = i % CW;
      float sum = 0.f;
#pragma unroll 8
      for (int t = 0; t < T; ++t) sum = fmaf(g[t * n + e], xc[t * CW + c], sum);
      float* const o = dw + static_cast<int64_t>(e) * d + c0 + c;
      *o = accumulate ? *o + sum : sum;
    }
}

static size_t small_bytes(int T, int n) {
  return 4 * (static_cast<size_t>(T) * n + static_cast<size_t>(T + n) * CW);
}

// d_offset from the tiles' sums, in 64 bits and a fixed order
__global__ __launch_bounds__(256) void offset_k(const float* __restrict__ part, int tiles, int n,
                                                int64_t np, int accumulate,
                                                float* __restrict__ out) {
  __shared__ double red[4][64];
  const int e = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  double sum = 0.0;
  if (e < n)
    for (int t = w; t < tiles; t += 4) sum += part[t * np + e];
  red[w][threadIdx.x & 63] = sum;
  __syncthreads();
  if (w == 0 && e < n) {
    sum = red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x];
    out[e] = accumulate ? out[e] + static_cast<float>(sum) : static_cast<float>(sum);
  }
}

template <typename OUT>
__global__ __launch_bounds__(256) void add_k(const float* __restrict__ v, int64_t count,
                                             OUT* __restrict__ out) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * 256)
    out[i] = from_f32<OUT>(to_f32<OUT>(out[i]) + v[i]);
}

struct Workspace {
  bf16_t *g_hi, *g_lo, *gt_hi, *gt_mid, *gt_lo, *wt_hi, *wt_lo, *xt;
  float *part, *sum, *partial;
  size_t partial_bytes;
};

static int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

static size_t layout(int T, int d, int n, Workspace* out, void* base) {
  Carver cv(base);
  Workspace w{};
  const int64_t np = up64(n), Tp = up64(T);
  w.g_hi = cv.take<bf16_t>(T * np);
  w.g_lo = cv.take<bf16_t>(T * np);
  w.gt_hi = cv.take<bf16_t>(n * Tp);
  w.gt_mid = cv.take<bf16_t>(n * Tp);
  w.gt_lo = cv.take<bf16_t>(n * Tp);
  w.wt_hi = cv.take<bf16_t>(d * np);
  w.wt_lo = cv.take<bf16_t>(d * np);
  w.xt = cv.take<bf16_t>(d * Tp);
  w.part = cv.take<float>(Tp / 64 * np);
  w.sum = cv.take<float>(static_cast<int64_t>(std::max(T, n)) * d);
  w.partial_bytes =
      std::max({gemm::splitk_bytes(T, d, static_cast<int>(3 * np), gemm::EPI_BF16),
                gemm::splitk_bytes(T, d, static_cast<int>(3 * np), gemm::EPI_F32),
                gemm::splitk_bytes(n, d, static_cast<int>(3 * Tp), gemm::EPI_F32)});
  w.partial = cv.take<float>(w.partial_bytes / 4);
  if (out) *out = w;
  return cv.bytes();
}

// What one launch of fp32 multiply-adds does sooner than four: 200 tokens x 512 x
// 40 experts take 11.5 us against 32.2, 64 x 512 x 256 23.6 against 29.5, 1024 x
// 256 x 20 33.1 against 33.1.
static bool is_small(int T, int d, int n) {
  return small_bytes(T, n) <= 96 * 1024 && static_cast<int64_t>(T) * n * d <= (8 << 20);
}

static int check(int32_t T, int32_t d, int32_t n) {
  if (T < 0 || d <= 0 || d % 64 || n < 1) return MOE_EINVAL;
  if (n > 1024 || T > MOE_MAX_TOKENS || d > (1 << 20)) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static unsigned grid_of(int64_t count) {
  return static_cast<unsigned>(std::min<int64_t>((count + 255) / 256, 8192));
}

// C = sum of three products A_i B_i^T over one contraction each of K
static int product3(const Workspace& w, const bf16_t* const (&A)[3], const bf16_t* const (&B)[3],
                    int64_t K, int M, int N, void* C, int epi, hipStream_t st) {
  gemm::Params p{};
  p.M = M;
  p.N = N;
  p.nseg = 3;
  for (int i = 0; i < 3; ++i) p.seg[i] = layer::seg(A[i], K, B[i], K, static_cast<int>(K));
  p.C = C;
  p.ldc = N;
  p.partial = w.partial_bytes ? w.partial : nullptr;
  p.partial_bytes = w.partial_bytes;
  return gemm::launch(p, epi, gemm::B_DENSE, true, 128, st);
}

}  // namespace router
}  // namespace moe

extern "C" size_t moe_router_backward_workspace_bytes(int32_t T, int32_t d, int32_t n) {
  if (moe::router::check(T, d, n) != MOE_OK) return 0;
  return std::max<size_t>(moe::router::layout(T, d, n, nullptr, nullptr), 256);
}

extern "C" int moe_router_backward(const void* x, const float* w_router, const float* scores,
                                   const float* dscores, int32_t T, int32_t d, int32_t n,
                                   int accumulate, void* dx, float* d_w_router,
                                   float* d_router_logit_offset, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  using namespace moe;
  using namespace moe::router;
  int rc = check(T, d, n);
  if (rc != MOE_OK) return rc;
  if (T > 0 && (!scores || !dscores || (dx && !w_router) || (d_w_router && !x)))
    return MOE_EINVAL;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % 16 != 0 || reinterpret_cast<uintptr_t>(w_router) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(dx) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(d_w_router) % 16 != 0)
    return MOE_EINVAL;
  Workspace w;
  const bool small = T == 0 || is_small(T, d, n);
  if (!small && (!workspace || workspace_bytes < layout(T, d, n, &w, workspace)))
    return MOE_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t np = up64(n), Tp = up64(T), nd = static_cast<int64_t>(n) * d;
  if (T == 0) {
    if (!accumulate && d_w_router)
      hipLaunchKernelGGL(layer::fill_u32, dim3(grid_of(nd)), dim3(256), 0, st,
                         reinterpret_cast<uint32_t*>(d_w_router), 0u, nd);
    if (!accumulate && d_router_logit_offset)
      hipLaunchKernelGGL(layer::fill_u32, dim3(grid_of(n)), dim3(256), 0, st,
                         reinterpret_cast<uint32_t*>(d_router_logit_offset), 0u,
                         static_cast<int64_t>(n));
    MOE_LAUNCH_CHECK();
    return MOE_OK;
  }
  if (small) {
    hipLaunchKernelGGL(small_k, dim3(d / CW + (d_router_logit_offset ? 1 : 0)),
                       dim3(SMALL_THREADS), small_bytes(T, n), st,
                       static_cast<const bf16_t*>(x), w_router, scores, dscores, T, d, n,
                       accumulate, static_cast<bf16_t*>(dx), d_w_router, d_router_logit_offset);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
  }
  const int64_t tn = np / TILE, tt = Tp / TILE, td = d / TILE;
  Prep p{scores, dscores, w_router, static_cast<const bf16_t*>(x), T, n, d, np, Tp, w.g_hi, w.g_lo,
         w.gt_hi, w.gt_mid, w.gt_lo, w.wt_hi, w.wt_lo, w.xt, w.part, 0, 0};
  p.score_blocks = static_cast<int>(tn * tt);
  p.x_blocks = d_w_router ? static_cast<int>(td * ((tt + 1) / 2)) : 0;
  const int w_blocks = dx ? static_cast<int>(td * ((tn + 1) / 2)) : 0;
  hipLaunchKernelGGL(prepare_k, dim3(p.score_blocks + p.x_blocks + w_blocks), dim3(256), 0, st, p);
  MOE_LAUNCH_CHECK();
  if (d_router_logit_offset) {
    hipLaunchKernelGGL(offset_k, dim3(static_cast<unsigned>(tn)), dim3(256), 0, st, w.part,
                       static_cast<int>(tt), n, np, accumulate, d_router_logit_offset);
    MOE_LAUNCH_CHECK();
  }
  if (d_w_router) {
    rc = product3(w, {w.gt_hi, w.gt_mid, w.gt_lo}, {w.xt, w.xt, w.xt}, Tp, n, d,
                  accumulate ? w.sum : d_w_router, gemm::EPI_F32, st);
    if (rc != MOE_OK) return rc;
    if (accumulate) {
      hipLaunchKernelGGL(add_k<float>, dim3(grid_of(nd)), dim3(256), 0, st, w.sum, nd, d_w_router);
      MOE_LAUNCH_CHECK();
    }
  }
  if (dx) {
    rc = product3(w, {w.g_hi, w.g_hi, w.g_lo}, {w.wt_hi, w.wt_lo, w.wt_hi}, np, T, d,
                  accumulate ? static_cast<void*>(w.sum) : dx,
                  accumulate ? gemm::EPI_F32 : gemm::EPI_BF16, st);
    if (rc != MOE_OK) return rc;
    if (accumulate) {
      const int64_t count = static_cast<int64_t>(T) * d;
      hipLaunchKernelGGL(add_k<bf16_t>, dim3(grid_of(count)), dim3(256), 0, st, w.sum, count,
                         static_cast<bf16_t*>(dx));
      MOE_LAUNCH_CHECK();
    }
  }
  return MOE_OK;
}
