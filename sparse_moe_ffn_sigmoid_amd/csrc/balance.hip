// The sequence-wise balance loss of the router, its per-expert counts and its
// gradient.
//
// Over the counted tokens t of a sequence s (N of them), with the chosen
// experts idx and the scores' shares p_ti = s_ti / S_t, S_t = sum_i s_ti:
//
//   c_i  = how often expert i was chosen,   L = n / (k N^2) sum_t sum_i c_i p_ti
//   dL/ds_tj = n / (k N^2) (c_j - q_t) / S_t,   q_t = sum_i c_i p_ti
//
// The counts depend on the choices alone, so they are taken first (4 k bytes
// a token); after that ONE pass over the scores gives both the loss, as the
// sum of the per-token q_t, and the gradient: no column sums, no second read.
// The pass moves 4 n bytes per token in and 4 n out and is bound by them: 57,344 x
// 896 with the gradient takes 64 us, 6.4 TB/s, and clearing, counting and the
// final sums 20 us beside it; 16,384 x 896 take 14.5 us for the loss alone and 22.4
// us for the gradient alone (out of the 256 MB last-level cache in part).
//
// A row lives in the registers of one wave (n <= 1024: 16 values a lane), so
// S_t and q_t are two wave sums.  Each wave owns a contiguous range of tokens
// and walks the sequences in it; its sum over sequence s goes to the slot
// (wave + s) of the partials, which no other pair of wave and sequence has,
// because every step to the next slot is a step of one or the other.  The
// partials are added in 64 bits in a fixed order: results do not depend on
// the schedule.  Counts are integer atomics, whose order does not matter.
#include <algorithm>

#include "common.hpp"

namespace moe {
namespace balance {

constexpr int MAXN = 1024;
constexpr int WAVES = 4;  // per block of the pass

struct Args {
  const float* scores;
  int64_t ld;
  int T, n, k;
  const int32_t* idx;
  const int32_t* off;   // [S + 1] or null (one sequence, the whole batch)
  int S;
  const uint8_t* mask;  // [T] or null
  const float* dloss;   // [S] or null (ones)
  int32_t* counts;      // [S][n]
  int32_t* tokens;      // [S]
  float* loss;          // [S] or null
  float* dscores;       // [T][n] or null
  float* part;          // [waves + S]
  int rpw;              // tokens per wave
};

// First token of sequence s (s = S: the end of the last one), inside [0, T]
// whatever the offsets hold.
__device__ __forceinline__ int seq_begin(const Args& a, int s) {
  if (!a.off) return s ? a.T : 0;
  return min(max(a.off[s], 0), a.T);
}

// The last sequence that begins at or before token t (0 if none does).
__device__ __forceinline__ int find_seq(const Args& a, int t) {
  if (!a.off) return 0;
  int lo = 0, hi = a.S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_begin(a, mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
#define MOE_DPP_ADD(ctrl, rows)                                                              \
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, rows, 0xf, false))
  MOE_DPP_ADD(0x111, 0xf);  // row_shr:1
  MOE_DPP_ADD(0x112, 0xf);  // row_shr:2
  MOE_DPP_ADD(0x114, 0xf);  // row_shr:4
  MOE_DPP_ADD(0x118, 0xf);  // row_shr:8
  MOE_DPP_ADD(0x142, 0xa);  // row_bcast:15
  MOE_DPP_ADD(0x143, 0xc);  // row_bcast:31
#undef MOE_DPP_ADD
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

__global__ __launch_bounds__(256) void clear_k(Args a) {
  const int64_t total = static_cast<int64_t>(a.S) * a.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t i = i0; i < total; i += step) a.counts[i] = 0;
  for (int64_t i = i0; i < a.S; i += step) a.tokens[i] = 0;
}

// Choices and counted tokens of tokens [b, e), all of one sequence, added to
// hist and *many by the block's threads.
__device__ __forceinline__ void count_range(const Args& a, int b, int e, int32_t* hist,
                                            int32_t* many) {
  const int last = e * a.k;  // at most 2^30
  for (int i = b * a.k + static_cast<int>(threadIdx.x); i < last; i += blockDim.x) {
    if (a.mask && !a.mask[i / a.k]) continue;
    const int v = a.idx[i];
    if (v >= 0 && v < a.n) atomicAdd(hist + v, 1);  // indices outside the experts count nowhere
  }
  int mine = 0;
  for (int t = b + threadIdx.x; t < e; t += blockDim.x) mine += !a.mask || a.mask[t];
  if (mine) atomicAdd(many, mine);
}

// Counts per sequence: a histogram in LDS for each stretch of a block's tokens
// that lies in one sequence, added to global memory.
constexpr int COUNT_THREADS = 1024;

__global__ __launch_bounds__(COUNT_THREADS) void count_k(Args a, int chunk) {
  __shared__ int32_t hist[MAXN + 1];
  int t = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(blockIdx.x) * chunk, a.T));
  const int end = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(t) + chunk, a.T));
  for (int s = find_seq(a, t); s < a.S && t < end; ++s) {
    t = max(t, seq_begin(a, s));
    const int e = min(end, seq_begin(a, s + 1));
    if (e <= t) continue;
    for (int i = threadIdx.x; i <= a.n; i += COUNT_THREADS) hist[i] = 0;
    __syncthreads();
    count_range(a, t, e, hist, hist + a.n);
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += COUNT_THREADS)
      if (hist[i]) atomicAdd(a.counts + static_cast<int64_t>(s) * a.n + i, hist[i]);
    if (threadIdx.x == 0 && hist[a.n]) atomicAdd(a.tokens + s, hist[a.n]);
    __syncthreads();
    t = e;
  }
}

// Column of a lane's value: VEC consecutive columns per lane and step.
template <int VEC>
__device__ __forceinline__ int column(int i, int lane) {
  return (i / VEC) * (64 * VEC) + lane * VEC + i % VEC;
}

template <int VEC, int NV>
__device__ __forceinline__ void load_row(const float* row, int n, int lane, float (&v)[NV]) {
  if constexpr (VEC == 4) {  // n is a multiple of 4 and rows are 16-byte aligned
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int c = column<4>(i, lane);
      const float4 q = c < n ? *reinterpret_cast<const float4*>(row + c)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column<1>(i, lane);
      v[i] = c < n ? row[c] : 0.f;
    }
  }
}

template <int VEC, int NV>
__device__ __forceinline__ void store_row(float* row, int n, int lane, const float (&v)[NV]) {
  if constexpr (VEC == 4) {
    typedef float f32x4_t __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int c = column<4>(i, lane);
      if (c < n)
        __builtin_nontemporal_store(f32x4_t{v[i], v[i + 1], v[i + 2], v[i + 3]},
                                    reinterpret_cast<f32x4_t*>(row + c));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column<1>(i, lane);
      if (c < n) __builtin_nontemporal_store(v[i], row + c);
    }
  }
}

// One counted token: returns q_t, writes its gradient row scaled by coef.  A
// row whose scores sum to zero has no shares: q_t = 0 and a zero gradient.
template <int VEC, int NV, bool GRAD>
__device__ __forceinline__ float token(const Args& a, int t, const float (&v)[NV],
                                       const float (&c)[NV], float coef, int lane) {
#pragma clang fp contract(off)  // every instantiation rounds alike
  float total = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    total += v[i];
    dot = fmaf(c[i], v[i], dot);
  }
  total = wave_sum(total);
  dot = wave_sum(dot);
  // divided by S_t, not multiplied by 1 / S_t, which overflows under 2^-128
  const bool none = total == 0.f;
  const float q = none ? 0.f : dot / total;
  if constexpr (GRAD) {
    const float g = none ? 0.f : coef / total;
    float out[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = g * (c[i] - q);
    store_row<VEC, NV>(a.dscores + static_cast<int64_t>(t) * a.n, a.n, lane, out);
  }
  return q;
}

template <int VEC, int NV>
__device__ __forceinline__ void zero_row(const Args& a, int t, int lane) {
  const float z[NV] = {};
  store_row<VEC, NV>(a.dscores + static_cast<int64_t>(t) * a.n, a.n, lane, z);
}

// n / (k N^2) times the loss's weight
__device__ __forceinline__ float coefficient(const Args& a, int s, int many) {
  const float N = static_cast<float>(max(many, 1));
  const float w = static_cast<float>(a.n) / (static_cast<float>(a.k) * N * N);
  return a.dloss ? w * a.dloss[s] : w;
}

// The pass over the scores: wave w takes tokens [w rpw, (w + 1) rpw), two at a
// time so that the second row's loads cover the first one's sums.
template <int VEC, int NV, bool LOSS, bool GRAD>
__global__ __launch_bounds__(64 * WAVES) void pass_k(Args a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * WAVES + (threadIdx.x >> 6));
  const int64_t first = static_cast<int64_t>(wave) * a.rpw;
  if (first >= a.T) return;
  int t = static_cast<int>(first);
  const int end = static_cast<int>(std::min<int64_t>(first + a.rpw, a.T));
  for (int s = find_seq(a, t); s < a.S && t < end; ++s) {
    const int b = max(t, min(end, seq_begin(a, s)));
    const int e = min(end, seq_begin(a, s + 1));
    if constexpr (GRAD)
      for (; t < b; ++t) zero_row<VEC, NV>(a, t, lane);
    t = b;
    if (e <= t) continue;
    float c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = column<VEC>(i, lane);
      c[i] = col < a.n ? static_cast<float>(a.counts[static_cast<int64_t>(s) * a.n + col]) : 0.f;
    }
    const float coef = GRAD ? coefficient(a, s, a.tokens[s]) : 0.f;
    float sum = 0.f;
    for (; t < e; t += 2) {
      const bool use0 = !a.mask || a.mask[t];
      const bool in1 = t + 1 < e;
      const bool use1 = in1 && (!a.mask || a.mask[t + 1]);
      float v0[NV], v1[NV];
      // rows that do not count are not read: what they hold does not matter
      if (use0) load_row<VEC, NV>(a.scores + t * a.ld, a.n, lane, v0);
      if (use1) load_row<VEC, NV>(a.scores + (t + 1) * a.ld, a.n, lane, v1);
      if (use0)
        sum += token<VEC, NV, GRAD>(a, t, v0, c, coef, lane);
      else if (GRAD)
        zero_row<VEC, NV>(a, t, lane);
      if (use1)
        sum += token<VEC, NV, GRAD>(a, t + 1, v1, c, coef, lane);
      else if (GRAD && in1)
        zero_row<VEC, NV>(a, t + 1, lane);
    }
    t = e;
    if (LOSS && lane == 0) a.part[static_cast<int64_t>(wave) + s] = sum;
  }
  if constexpr (GRAD)
    for (; t < end; ++t) zero_row<VEC, NV>(a, t, lane);  // behind the last sequence
}

// loss_s = n / (k N^2) times the sum of its waves' partials
__global__ __launch_bounds__(256) void finish_k(Args a) {
  __shared__ double red[4];
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    const int b = seq_begin(a, s), e = seq_begin(a, s + 1);
    double sum = 0.0;
    if (e > b)
      for (int w = b / a.rpw + threadIdx.x; w <= (e - 1) / a.rpw; w += 256)
        sum += a.part[static_cast<int64_t>(w) + s];
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      const int many = a.tokens[s];
      const double w = many ? static_cast<double>(a.n) / (static_cast<double>(a.k) * many * many)
                            : 0.0;
      a.loss[s] = static_cast<float>(w * (red[0] + red[1] + red[2] + red[3]));
    }
    __syncthreads();
  }
}

// A small batch in one launch of one block: for each sequence the counts stay
// in LDS and its tokens are dealt to the waves.  The row arithmetic is pass_k's.
constexpr int SMALL_WAVES = 16;

template <int VEC, int NV>
__global__ __launch_bounds__(64 * SMALL_WAVES) void small_k(Args a) {
  __shared__ int32_t hist[MAXN + 1];
  __shared__ float red[SMALL_WAVES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int done = 0;  // tokens before this one have their gradients
  for (int s = 0; s < a.S; ++s) {
    const int b = max(done, seq_begin(a, s)), e = max(b, seq_begin(a, s + 1));
    if (a.dscores)
      for (int t = done + wave; t < b; t += SMALL_WAVES) zero_row<VEC, NV>(a, t, lane);
    done = e;
    for (int i = tid; i <= a.n; i += 64 * SMALL_WAVES) hist[i] = 0;
    __syncthreads();
    count_range(a, b, e, hist, hist + a.n);
    __syncthreads();
    const int many = hist[a.n];
    for (int i = tid; i < a.n; i += 64 * SMALL_WAVES)
      a.counts[static_cast<int64_t>(s) * a.n + i] = hist[i];
    float c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = column<VEC>(i, lane);
      c[i] = col < a.n ? static_cast<float>(hist[col]) : 0.f;
    }
    const float coef = coefficient(a, s, many);
    float sum = 0.f;
    for (int t = b + wave; t < e; t += SMALL_WAVES) {
      if (a.mask && !a.mask[t]) {
        if (a.dscores) zero_row<VEC, NV>(a, t, lane);
        continue;
      }
      float v[NV];
      load_row<VEC, NV>(a.scores + t * a.ld, a.n, lane, v);
      sum += a.dscores ? token<VEC, NV, true>(a, t, v, c, coef, lane)
                       : token<VEC, NV, false>(a, t, v, c, coef, lane);
    }
    if (lane == 0) red[wave] = sum;
    __syncthreads();  // also: everyone is done with hist
    if (tid == 0) {
      double total = 0.0;
      for (int w = 0; w < SMALL_WAVES; ++w) total += red[w];
      a.tokens[s] = many;
      a.loss[s] = many ? static_cast<float>(static_cast<double>(a.n) /
                                            (static_cast<double>(a.k) * many * many) * total)
                       : 0.f;
    }
  }
  if (a.dscores)
    for (int t = done + wave; t < a.T; t += SMALL_WAVES) zero_row<VEC, NV>(a, t, lane);
}

template <int VEC, int NV>
static void launch_pass(const Args& a, int waves, hipStream_t st) {
  const dim3 grid((waves + WAVES - 1) / WAVES), block(64 * WAVES);
  if (a.loss && a.dscores)
    hipLaunchKernelGGL((pass_k<VEC, NV, true, true>), grid, block, 0, st, a);
  else if (a.loss)
    hipLaunchKernelGGL((pass_k<VEC, NV, true, false>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((pass_k<VEC, NV, false, true>), grid, block, 0, st, a);
}

template <int VEC, int NV>
static void launch(const Args& a, bool small, hipStream_t st) {
  if (small)
    hipLaunchKernelGGL((small_k<VEC, NV>), dim3(1), dim3(64 * SMALL_WAVES), 0, st, a);
  else
    launch_pass<VEC, NV>(a, (a.T + a.rpw - 1) / a.rpw, st);
}

static int pass(const Args& a, bool small, hipStream_t st) {
  const bool vec = a.n % 4 == 0 && a.ld % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(a.scores) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.dscores) % 16 == 0;
  if (vec) {
    if (a.n <= 256)
      launch<4, 4>(a, small, st);
    else if (a.n <= 512)
      launch<4, 8>(a, small, st);
    else
      launch<4, 16>(a, small, st);
  } else if (a.n <= 256) {
    launch<1, 4>(a, small, st);
  } else {
    launch<1, 16>(a, small, st);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

// One block's work against three more launches, us a call: 128 x 896 14.3 against
// 26.4, 256 x 512 14.4 against 24.5, in four sequences 25.3 against 24.6; with
// 1024 tokens (33) or 8 sequences (40 to 53) the one block is the slower.
static bool is_small(int T, int n, int S) {
  return T <= 256 && static_cast<int64_t>(T) * n <= 131072 && S <= 4;
}

// Tokens per wave: 16 waves on each of 256 compute units.
static int rows_per_wave(int T) { return std::max(1, (T + 4095) / 4096); }

static int check(int32_t T, int32_t n, int32_t k, int32_t S, const int32_t* off, int64_t ld) {
  if (T < 0 || n < 1 || k < 1 || k > n || S < 1 || ld < n) return MOE_EINVAL;
  if (!off && S != 1) return MOE_EINVAL;
  if (n > MAXN || T > MOE_MAX_TOKENS || S > MOE_MAX_TOKENS) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace balance
}  // namespace moe

extern "C" size_t moe_balance_loss_workspace_bytes(int32_t T, int32_t S) {
  if (T < 0 || S < 1 || T > MOE_MAX_TOKENS || S > MOE_MAX_TOKENS) return 0;
  const int rpw = moe::balance::rows_per_wave(T);
  return moe::align_up(4 * (static_cast<size_t>((T + rpw - 1) / rpw) + S), 256);
}

extern "C" int moe_balance_loss(const float* scores, int64_t ld_scores, int32_t T, int32_t n,
                                int32_t k, const int32_t* topk_idx, const int32_t* seq_offsets,
                                int32_t n_seq, const uint8_t* token_mask, const float* dloss,
                                float* loss, int32_t* counts, int32_t* tokens, float* dscores,
                                void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe::balance;
  const int st = check(T, n, k, n_seq, seq_offsets, ld_scores);
  if (st != MOE_OK) return st;
  if (!loss || !counts || !tokens) return MOE_EINVAL;
  if (T > 0 && (!scores || !topk_idx)) return MOE_EINVAL;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_EINVAL;
  const bool small = is_small(T, n, n_seq);
  if (!small && (!workspace || workspace_bytes < moe_balance_loss_workspace_bytes(T, n_seq)))
    return MOE_EWORKSPACE;
  Args a{scores, ld_scores, T,      n,    k,       topk_idx, seq_offsets, n_seq, token_mask,
         dloss,  counts,    tokens, loss, dscores, static_cast<float*>(workspace),
         rows_per_wave(T)};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (small) return pass(a, true, hs);
  const int64_t cells = static_cast<int64_t>(n_seq) * n;
  hipLaunchKernelGGL(clear_k, dim3(static_cast<unsigned>(std::min<int64_t>((cells + 255) / 256, 4096))),
                     dim3(256), 0, hs, a);
  if (T > 0) {
    // few blocks: each adds up to n counts per sequence to global memory
    const int chunk = std::max(64, (T + 127) / 128);
    hipLaunchKernelGGL(count_k, dim3((T + chunk - 1) / chunk), dim3(COUNT_THREADS), 0, hs, a, chunk);
    MOE_LAUNCH_CHECK();
    const int rc = pass(a, false, hs);
    if (rc != MOE_OK) return rc;
  }
  hipLaunchKernelGGL(finish_k, dim3(std::min(n_seq, 2048)), dim3(256), 0, hs, a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" int moe_balance_loss_backward(const float* scores, int64_t ld_scores, int32_t T,
                                         int32_t n, int32_t k, const int32_t* counts,
                                         const int32_t* tokens, const int32_t* seq_offsets,
                                         int32_t n_seq, const uint8_t* token_mask,
                                         const float* dloss, float* dscores, void* stream) {
  using namespace moe::balance;
  const int st = check(T, n, k, n_seq, seq_offsets, ld_scores);
  if (st != MOE_OK) return st;
  if (!counts || !tokens) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!scores || !dscores) return MOE_EINVAL;
  Args a{scores, ld_scores, T, n, k, nullptr, seq_offsets, n_seq, token_mask, dloss,
         const_cast<int32_t*>(counts), const_cast<int32_t*>(tokens), nullptr, dscores, nullptr,
         rows_per_wave(T)};
  return pass(a, false, static_cast<hipStream_t>(stream));
}
