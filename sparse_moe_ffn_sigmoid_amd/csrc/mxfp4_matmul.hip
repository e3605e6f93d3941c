// Products of MXFP4 operands: C = A B^T with E2M1 codes and one E8M0 scale per
// 32 elements on both sides, multiplied as they are by gfx950's scaled MFMA
// with fp32 accumulation.
//
// One problem, one per row group (the experts: rows [off[g], off[g + 1]) of A
// meet B[g]), or one per range of the contraction (the experts' weight
// gradients).  Two kernels:
//
// * ring_k, for many rows: tiles go from memory straight into LDS through two
//   buffers of 256 K elements (128 bytes per row, whole cache lines), 16-byte
//   chunks XOR-swizzled by the row so that fills and fragment reads are free
//   of bank conflicts, v_mfma_scale_f32_32x32x64_f8f6f4 on 32x32 blocks.
// * skinny_k, for a few rows per problem, where the codes of B are read once
//   and bound the time: no LDS on the way in, each lane loads its own
//   fragments, v_mfma_scale_f32_16x16x128_f8f6f4 on 16 columns at a time, the
//   contraction split over the waves of a block where the columns alone do not
//   fill the chip.  Activations given unpacked are packed in registers: a lane
//   holds whole blocks of 32.
#include <algorithm>

#include "common.hpp"
#include "lds_ring.hpp"
#include "mxfp4_convert.hpp"

namespace moe {
namespace mx {

typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int FP4 = 4;  // E2M1 in the scaled MFMA's format fields

// What a chunk outside the operands reads as: codes of zero.
__device__ __attribute__((aligned(16))) const uint8_t zero_chunk[16] = {};

struct MatArgs {
  const uint8_t *A, *As, *B, *Bs;
  int64_t lda, ldb;            // code bytes per row (scale bytes: one sixteenth)
  int64_t b_stride;            // code bytes between the groups' B
  int M, N;                    // rows of C (all groups), columns
  int64_t K;                   // contraction (elements, a multiple of 32)
  const int32_t* off;          // [G + 1] row groups, or null
  int G;
  const int32_t* a_rows;       // row of C -> row of A, or null
  int a_count;                 // rows of A
  const int32_t* kofs;         // [G + 1] ranges of K, or null
  void* C;
  int64_t ldc, c_stride;       // elements; c_stride between K groups
  int out;                     // MOE_F32, MOE_BF16 or MOE_F16
};

__device__ __forceinline__ void store_one(const MatArgs& a, int64_t at, float v) {
  if (a.out == MOE_F32)
    static_cast<float*>(a.C)[at] = v;
  else if (a.out == MOE_BF16)
    static_cast<bf16_t*>(a.C)[at] = f32_to_bf16(v);
  else
    static_cast<_Float16*>(a.C)[at] = static_cast<_Float16>(v);
}

// First row of group g (g = G: the end), inside [0, M] whatever the offsets hold
__device__ __forceinline__ int group_begin(const MatArgs& a, int g) {
  return min(max(a.off[g], 0), a.M);
}

struct Tile {
  int g, row0, rows, n0;
  int kb0, kb1;  // blocks of 32 along K
};

// Group of row tile m.  Group g owns the indices from off[g] / BM + g on, one
// per tile: the next group's first index is beyond them, because its rows start
// no earlier than this group's end.  No list of tiles is built.
template <int BM>
__device__ __forceinline__ bool find_rows(const MatArgs& a, int m, Tile& t) {
  if (!a.off) {
    t.g = 0;
    t.row0 = m * BM;
    t.rows = min(BM, a.M - t.row0);
    return t.rows > 0;
  }
  int lo = 0, hi = a.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (group_begin(a, mid) / BM + mid <= m)
      lo = mid;
    else
      hi = mid;
  }
  const int beg = group_begin(a, lo), end = group_begin(a, lo + 1);
  const int64_t row = beg + (static_cast<int64_t>(m) - (beg / BM + lo)) * BM;
  if (row < beg || row >= end) return false;
  t.g = lo;
  t.row0 = static_cast<int>(row);
  t.rows = min(BM, end - t.row0);
  return true;
}

// Block -> tile.  Blocks are dealt to the 8 XCDs in turn, so a block's number is
// turned into one that runs through consecutive tiles on one XCD; row tiles
// come fastest within GM of them, so that the tiles an XCD works on at one time
// share their rows of A and B in its L2.
template <int BM, int BN>
__device__ __forceinline__ bool find_tile(const MatArgs& a, int ntm, int ntn, Tile& t) {
  constexpr int GM = 4;
  const int64_t G = gridDim.x, b = blockIdx.x;
  int64_t tau = (b & 7) * (G >> 3) + (b >> 3);
  const int64_t per = static_cast<int64_t>(ntm) * ntn;
  int kg = 0;
  if (a.kofs) {
    if (tau >= per * a.G) return false;
    kg = static_cast<int>(tau / per);
    tau -= kg * per;
  } else if (tau >= per) {
    return false;
  }
  const int64_t grp = tau / (GM * ntn);
  const int gm = static_cast<int>(min(static_cast<int64_t>(GM), ntm - grp * GM));
  const int64_t r = tau - grp * GM * ntn;
  const int m = static_cast<int>(grp * GM + r % gm);
  t.n0 = static_cast<int>(r / gm) * BN;
  t.kb0 = 0;
  t.kb1 = static_cast<int>(a.K / 32);
  if (a.kofs) {
    t.g = kg;
    t.row0 = m * BM;
    t.rows = min(BM, a.M - t.row0);
    // inside the operands whatever the offsets hold
    t.kb0 = static_cast<int>(min(max(static_cast<int64_t>(a.kofs[kg]), int64_t(0)), a.K) / 32);
    t.kb1 = static_cast<int>(min(max(static_cast<int64_t>(a.kofs[kg + 1]), int64_t(0)), a.K) / 32);
    return true;
  }
  return find_rows<BM>(a, m, t);
}

// 8 scale bytes from block kb of a row on; what lies at or behind kb1 reads as
// 127 (one), which leaves zero codes zero.
__device__ __forceinline__ uint2 scales8(const uint8_t* row, int kb, int kb1) {
  uint2 v;
  if (kb + 8 <= kb1) {
    __builtin_memcpy(&v, row + kb, 8);
    return v;
  }
  uint32_t w[2] = {0x7f7f7f7fu, 0x7f7f7f7fu};
  for (int i = 0; kb + i < kb1; ++i)
    w[i >> 2] = (w[i >> 2] & ~(255u << (8 * (i & 3)))) |
                (static_cast<uint32_t>(row[kb + i]) << (8 * (i & 3)));
  return make_uint2(w[0], w[1]);
}

template <int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(64 * WM * WN) void ring_k(MatArgs a, int ntm, int ntn) {
  constexpr int NW = WM * WN, NTH = 64 * NW;
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  constexpr int AI = BM / 8, BI = BN / 8;  // 1 KB copies of 8 rows per buffer
  constexpr int MA = (AI + NW - 1) / NW, MB = (BI + NW - 1) / NW;
  constexpr int MS = (BM + BN + NTH - 1) / NTH;  // scale rows per thread
  __shared__ __attribute__((aligned(1024))) uint8_t sA[2][BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t sB[2][BN * 128];
  __shared__ __attribute__((aligned(16))) uint2 sS[2][BM + BN];

  Tile t;
  if (!find_tile<BM, BN>(a, ntm, ntn, t)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint8_t* B = a.B + (a.kofs ? 0 : t.g * a.b_stride);
  const uint8_t* Bs = a.Bs + (a.kofs ? 0 : t.g * (a.b_stride / 16));

  // row of A for a row of the tile: -1 where the map points outside A
  auto a_row = [&](int r) -> int64_t {
    const int64_t row = t.row0 + (r < t.rows ? r : 0);
    if (!a.a_rows) return row;
    const int at = a.a_rows[row];
    return at >= 0 && at < a.a_count ? at : -1;
  };
  // this lane's chunk of 32 elements within a buffer's row, the same in every copy
  const int chunk = (lane & 7) ^ (lane >> 3);
  const uint8_t* pa[MA];
  const uint8_t* pb[MB];
#pragma unroll
  for (int i = 0; i < MA; ++i) {
    const int64_t row = a_row((wave + NW * i) * 8 + (lane >> 3));
    pa[i] = row < 0 ? nullptr : a.A + row * a.lda + chunk * 16;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t row = min(t.n0 + (wave + NW * i) * 8 + (lane >> 3), a.N - 1);
    pb[i] = B + row * a.ldb + chunk * 16;
  }
  const uint8_t* ps[MS];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int r = tid + NTH * i;
    if (r < BM) {
      const int64_t row = a_row(r);
      ps[i] = a.As + (row < 0 ? 0 : row) * (a.lda / 16);
    } else {
      ps[i] = Bs + static_cast<int64_t>(min(t.n0 + r - BM, a.N - 1)) * (a.ldb / 16);
    }
  }

  uint2 sc[MS];
  auto load_scales = [&](int kb) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
      if (tid + NTH * i < BM + BN) sc[i] = scales8(ps[i], kb, t.kb1);
  };
  auto copy = [&](int kb, int buf) {
    const bool in = kb + chunk < t.kb1;
    const int64_t at = static_cast<int64_t>(kb) * 16;
#pragma unroll
    for (int i = 0; i < MA; ++i) {
      const int c = wave + NW * i;
      if (c < AI && c * 8 < t.rows)
        copy16_to_lds(in && pa[i] ? pa[i] + at : zero_chunk, sA[buf] + c * 1024);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int c = wave + NW * i;
      if (c < BI) copy16_to_lds(in ? pb[i] + at : zero_chunk, sB[buf] + c * 1024);
    }
  };
  auto put_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
      if (tid + NTH * i < BM + BN) sS[buf][tid + NTH * i] = sc[i];
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int hi = lane >> 5, l31 = lane & 31;
  // fragment i of a wave covers tile rows (i WM + wm) 32 ..: a short tile's
  // fragments are spread evenly over the waves
  auto frag = [&](const uint8_t* s, int row, int q) {
    const v4i_t v =
        *reinterpret_cast<const v4i_t*>(s + row * 128 + (((2 * q + hi) ^ (row & 7)) * 16));
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
  };
  auto compute = [&](int buf, int left) {
    uint2 sa[FM], sb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      sa[i] = sS[buf][(i * WM + wm) * 32 + l31];
      sa[i].x >>= 8 * hi;  // this half's block of a 64-element step in bytes 0 and 2
      sa[i].y >>= 8 * hi;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      sb[j] = sS[buf][BM + (wn * FN + j) * 32 + l31];
      sb[j].x >>= 8 * hi;
      sb[j].y >>= 8 * hi;
    }
    auto step = [&](auto qc) {
      constexpr int q = decltype(qc)::value;
      v8i_t b[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = frag(sB[buf], (wn * FN + j) * 32 + l31, q);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if ((i * WM + wm) * 32 >= t.rows) continue;
        const v8i_t x = frag(sA[buf], (i * WM + wm) * 32 + l31, q);
        const int xs = static_cast<int>(q < 2 ? sa[i].x : sa[i].y);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              x, b[j], acc[i][j], FP4, FP4, 2 * (q & 1), xs, 2 * (q & 1),
              static_cast<int>(q < 2 ? sb[j].x : sb[j].y));
      }
    };
    step(std::integral_constant<int, 0>{});
    if (left > 2) step(std::integral_constant<int, 1>{});
    if (left > 4) step(std::integral_constant<int, 2>{});
    if (left > 6) step(std::integral_constant<int, 3>{});
  };

  int buf = 0;
  if (t.kb0 < t.kb1) {
    load_scales(t.kb0);
    copy(t.kb0, 0);
    put_scales(0);
  }
  for (int kb = t.kb0; kb < t.kb1; kb += 8, buf ^= 1) {
    ring_wait<0>();  // this wave's copies of the buffer to be used
    __syncthreads();  // everyone's; and everyone is done with the other buffer
    const bool more = kb + 8 < t.kb1;
    if (more) {
      load_scales(kb + 8);
      copy(kb + 8, buf ^ 1);
    }
    compute(buf, t.kb1 - kb);
    if (more) put_scales(buf ^ 1);
  }

  const int64_t base = a.kofs ? t.g * a.c_stride : 0;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = (i * WM + wm) * 32 + (r >> 2) * 8 + hi * 4 + (r & 3);
      if (row >= t.rows) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int col = t.n0 + (wn * FN + j) * 32 + l31;
        if (col < a.N) store_one(a, base + (t.row0 + static_cast<int64_t>(row)) * a.ldc + col, acc[i][j][r]);
      }
    }
  }
}

// A few rows per problem.  A block takes 16 NT columns per wave group and all of
// a group's rows, 16 MT at a time; WK waves split the contraction into stretches
// of 256 elements dealt in turn and add their sums through LDS in a fixed order.
// Lane (c, h), c = lane mod 16, h = lane / 16, holds elements [32 h, 32 h + 32)
// of a 128-element step of row c: one block with its scale.
struct Unpacked {  // activations to be packed on the way in
  const void* x;
  int64_t stride;
};

template <int DT>  // -1: A is packed
__device__ __forceinline__ void a_fragment(const MatArgs& a, const Unpacked& u, int64_t row,
                                           int kb, int kb1, v4i_t& q, uint32_t& s) {
  q = v4i_t{0, 0, 0, 0};
  s = 127u;
  if (row < 0 || kb >= kb1) return;
  if constexpr (DT < 0) {
    q = *reinterpret_cast<const v4i_t*>(a.A + row * a.lda + static_cast<int64_t>(kb) * 16);
    s = a.As[row * (a.lda / 16) + kb];
  } else {
    float v[4][8];
    uint32_t m = 0;
    const auto* p = static_cast<const typename Elem<DT>::type*>(u.x) + row * u.stride +
                    static_cast<int64_t>(kb) * 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load8<DT>(p + 8 * i, 8, true, v[i]);
      m = max(m, amax8(v[i]));
    }
    s = scale_byte(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = static_cast<int>(encode8(v[i], s));
  }
}

template <int WN, int WK, int NT, int MT, int DT>
__global__ __launch_bounds__(64 * WN * WK) void skinny_k(MatArgs a, Unpacked u) {
  constexpr int NW = WN * WK;
  __shared__ float part[WK > 1 ? WK * WN * NT * MT * 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WK, wk = wave % WK;
  const int c = lane & 15, h = lane >> 4;
  const int g = blockIdx.y;
  int beg = 0, end = a.M;
  if (a.off) {
    beg = group_begin(a, g);
    end = group_begin(a, g + 1);
  }
  if (beg >= end) return;
  const int n0 = (blockIdx.x * WN + wn) * 16 * NT;
  const int kb1 = static_cast<int>(a.K / 32);
  const uint8_t* B = a.B + g * a.b_stride;
  const uint8_t* Bs = a.Bs + g * (a.b_stride / 16);
  const uint8_t* pb[NT];
  const uint8_t* ps[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(n0 + 16 * j + c, a.N - 1);
    pb[j] = B + n * a.ldb + h * 16;
    ps[j] = Bs + n * (a.ldb / 16) + h;
  }
  for (int m0 = beg; m0 < end; m0 += 16 * MT) {
    f32x4_t acc[MT][NT];
    int64_t row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = m0 + 16 * i + c;
      row[i] = r < end ? r : -1;
      if (a.a_rows && r < end) {
        const int at = a.a_rows[r];
        row[i] = at >= 0 && at < a.a_count ? at : -1;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int kb = wk * 8; kb < kb1; kb += WK * 8) {
      v4i_t bq[2][NT];
      uint32_t bs[2][NT];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bool in = kb + 4 * q + h < kb1;
          bq[q][j] = v4i_t{0, 0, 0, 0};
          bs[q][j] = 127u;
          if (in) {
            bq[q][j] = __builtin_nontemporal_load(
                reinterpret_cast<const v4i_t*>(pb[j] + static_cast<int64_t>(kb + 4 * q) * 16));
            bs[q][j] = ps[j][kb + 4 * q];
          }
        }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if (m0 + 16 * i >= end) continue;
          v4i_t aq;
          uint32_t as;
          a_fragment<DT>(a, u, row[i], kb + 4 * q + h, kb1, aq, as);
          const v8i_t x = __builtin_shufflevector(aq, aq, 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const v8i_t y =
                __builtin_shufflevector(bq[q][j], bq[q][j], 0, 1, 2, 3, -1, -1, -1, -1);
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                x, y, acc[i][j], FP4, FP4, 0, static_cast<int>(as), 0,
                static_cast<int>(bs[q][j]));
          }
        }
    }
    if constexpr (WK == 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int m = m0 + 16 * i + h * 4 + r, n = n0 + 16 * j + c;
            if (m < end && n < a.N) store_one(a, m * a.ldc + n, acc[i][j][r]);
          }
    } else {
      if (m0 > beg) __syncthreads();  // the last rows' sums have been read
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            part[((wave * MT + i) * NT + j) * 256 + (h * 4 + r) * 16 + c] = acc[i][j][r];
      __syncthreads();
      for (int o = threadIdx.x; o < WN * MT * NT * 256; o += 64 * NW) {
        const int wo = o / (MT * NT * 256), rest = o % (MT * NT * 256);
        const int i = rest / (NT * 256), j = rest / 256 % NT, at = rest % 256;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w)
          sum += part[(((wo * WK + w) * MT + i) * NT + j) * 256 + at];
        const int m = m0 + 16 * i + at / 16;
        const int n = (blockIdx.x * WN + wo) * 16 * NT + 16 * j + at % 16;
        if (m < end && n < a.N) store_one(a, m * a.ldc + n, sum);
      }
    }
  }
}

template <int WM, int WN, int FM, int FN>
static int launch_ring(const MatArgs& a, hipStream_t st) {
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  // the indices of find_rows reach M / BM + G
  const int64_t ntm = a.off ? a.M / BM + a.G : (static_cast<int64_t>(a.M) + BM - 1) / BM;
  const int64_t ntn = (static_cast<int64_t>(a.N) + BN - 1) / BN;
  const int64_t tiles = ntm * ntn * (a.kofs ? a.G : 1);
  if (tiles + 7 > 0x7fffffff) return MOE_EUNSUPPORTED;
  hipLaunchKernelGGL((ring_k<WM, WN, FM, FN>), dim3(static_cast<unsigned>((tiles + 7) / 8 * 8)),
                     dim3(64 * WM * WN), 0, st, a, static_cast<int>(ntm), static_cast<int>(ntn));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int WN, int WK, int NT, int MT, int DT>
static int launch_skinny(const MatArgs& a, const Unpacked& u, hipStream_t st) {
  const int64_t per = 16ll * NT * WN;
  hipLaunchKernelGGL((skinny_k<WN, WK, NT, MT, DT>),
                     dim3(static_cast<unsigned>((a.N + per - 1) / per),
                          static_cast<unsigned>(a.off ? a.G : 1)),
                     dim3(64 * WN * WK), 0, st, a, u);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int DT>
static int skinny(const MatArgs& a, const Unpacked& u, int64_t per_group, hipStream_t st) {
  // waves that a split over columns alone gives
  const int64_t waves = (static_cast<int64_t>(a.N) + 15) / 16 * (a.off ? a.G : 1);
  if constexpr (DT < 0) {
    if (per_group > 16) {
      if (waves >= 8192) return launch_skinny<4, 1, 1, 4, DT>(a, u, st);
      return launch_skinny<1, 8, 1, 4, DT>(a, u, st);
    }
  }
  if (waves >= 8192) return launch_skinny<4, 1, 1, 1, DT>(a, u, st);
  return launch_skinny<1, 8, 1, 1, DT>(a, u, st);
}

// Rows per problem up to which the codes of B bound the time and the skinny
// kernel is taken.
constexpr int SKINNY_ROWS = 32;

static int product(const MatArgs& a, hipStream_t st) {
  if (a.kofs) return launch_ring<2, 4, 4, 2>(a, st);
  const int64_t per = a.off ? (a.M + a.G - 1) / a.G : a.M;
  if (per <= SKINNY_ROWS) return skinny<-1>(a, Unpacked{}, per, st);
  if (per <= 128) return launch_ring<1, 8, 4, 1>(a, st);
  return launch_ring<2, 4, 4, 2>(a, st);
}

static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

static int check_out(int32_t out_dtype, const void* out, int64_t ldo, int64_t N) {
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16 && out_dtype != MOE_F16)
    return MOE_EUNSUPPORTED;
  if (!out || ldo < N || ldo > (int64_t(1) << 32) ||
      reinterpret_cast<uintptr_t>(out) % (out_dtype == MOE_F32 ? 4 : 2) != 0)
    return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace mx
}  // namespace moe

extern "C" int moe_mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_rows,
                                const uint8_t* b_codes, const uint8_t* b_scales, int64_t M,
                                int64_t N, int64_t K, const int32_t* row_offsets,
                                int32_t n_groups, const int32_t* row_index, void* out,
                                int32_t out_dtype, int64_t ld_out, void* stream) {
  using namespace moe::mx;
  if (M < 0 || N < 1 || K < 32 || K % 32 || a_rows < 0) return MOE_EINVAL;
  if (row_offsets ? n_groups < 1 : n_groups != 1) return MOE_EINVAL;
  if (!row_index && a_rows < M) return MOE_EINVAL;
  if (M > (1 << 30) || N > (1 << 30) || a_rows > (1 << 30) || K > (1 << 30) || n_groups > 1024)
    return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  const int rc = check_out(out_dtype, out, ld_out, N);
  if (rc != MOE_OK) return rc;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !aligned16(a_codes) ||
      !aligned16(b_codes))
    return MOE_EINVAL;
  MatArgs a{};
  a.A = a_codes;
  a.As = a_scales;
  a.B = b_codes;
  a.Bs = b_scales;
  a.lda = a.ldb = K / 2;
  a.b_stride = N * (K / 2);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = K;
  a.off = row_offsets;
  a.G = n_groups;
  a.a_rows = row_index;
  a.a_count = static_cast<int>(a_rows);
  a.C = out;
  a.ldc = ld_out;
  a.out = out_dtype;
  return product(a, static_cast<hipStream_t>(stream));
}

extern "C" int moe_mxfp4_matmul_kgroup(const uint8_t* a_codes, const uint8_t* a_scales,
                                       const uint8_t* b_codes, const uint8_t* b_scales, int64_t M,
                                       int64_t N, int64_t K, const int32_t* k_offsets,
                                       int32_t n_groups, void* out, int32_t out_dtype,
                                       void* stream) {
  using namespace moe::mx;
  if (M < 1 || N < 1 || K < 0 || K % 32) return MOE_EINVAL;
  if (k_offsets ? n_groups < 1 : n_groups != 1) return MOE_EINVAL;
  if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30) || n_groups > 1024) return MOE_EUNSUPPORTED;
  const int rc = check_out(out_dtype, out, N, N);
  if (rc != MOE_OK) return rc;
  if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return MOE_EINVAL;
  if (!aligned16(a_codes) || !aligned16(b_codes)) return MOE_EINVAL;
  MatArgs a{};
  a.A = a_codes;
  a.As = a_scales;
  a.B = b_codes;
  a.Bs = b_scales;
  a.lda = a.ldb = K / 2;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = K;
  a.G = n_groups;
  a.kofs = k_offsets;
  a.a_count = a.M;
  a.C = out;
  a.ldc = N;
  a.c_stride = M * N;
  a.out = out_dtype;
  // one range: an ordinary product (an empty one still writes its zeros)
  return k_offsets || K == 0 ? launch_ring<2, 4, 4, 2>(a, static_cast<hipStream_t>(stream))
                             : product(a, static_cast<hipStream_t>(stream));
}

extern "C" size_t moe_mxfp4_linear_workspace_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 32 || K % 32 || rows > (1 << 30) || K > (1 << 30)) return 0;
  return moe::align_up(rows * (K / 2), 256) + moe::align_up(rows * (K / 32), 256) + 256;
}

extern "C" int moe_mxfp4_linear(const void* x, int32_t x_dtype, int64_t x_rows,
                                int64_t row_stride, const uint8_t* w_codes,
                                const uint8_t* w_scales, int64_t M, int64_t N, int64_t K,
                                const int32_t* row_offsets, int32_t n_groups,
                                const int32_t* row_index, void* out, int32_t out_dtype,
                                int64_t ld_out, void* workspace, size_t workspace_bytes,
                                void* stream) {
  using namespace moe::mx;
  if (M < 0 || N < 1 || K < 32 || K % 32 || x_rows < 0 || row_stride < K) return MOE_EINVAL;
  if (row_offsets ? n_groups < 1 : n_groups != 1) return MOE_EINVAL;
  if (!row_index && x_rows < M) return MOE_EINVAL;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16 && x_dtype != MOE_F16) return MOE_EUNSUPPORTED;
  if (M > (1 << 30) || N > (1 << 30) || x_rows > (1 << 30) || K > (1 << 30) || n_groups > 1024)
    return MOE_EUNSUPPORTED;
  if (row_stride > (int64_t(1) << 56) / (x_rows + 1)) return MOE_EINVAL;
  if (M == 0) return MOE_OK;
  int rc = check_out(out_dtype, out, ld_out, N);
  if (rc != MOE_OK) return rc;
  const int64_t size = x_dtype == MOE_F32 ? 4 : 2;
  if ((!x && x_rows > 0) || reinterpret_cast<uintptr_t>(x) % size != 0 || !w_codes || !w_scales ||
      !aligned16(w_codes))
    return MOE_EINVAL;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_EINVAL;
  if (workspace_bytes < moe_mxfp4_linear_workspace_bytes(x_rows, K)) return MOE_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (!row_offsets && M <= 16 && aligned16(x) && row_stride * size % 16 == 0) {
    MatArgs a{};
    a.B = w_codes;
    a.Bs = w_scales;
    a.ldb = K / 2;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = K;
    a.G = 1;
    a.a_rows = row_index;
    a.a_count = static_cast<int>(x_rows);
    a.C = out;
    a.ldc = ld_out;
    a.out = out_dtype;
    const Unpacked u{x, row_stride};
    if (x_dtype == MOE_F32) return skinny<MOE_F32>(a, u, M, st);
    if (x_dtype == MOE_BF16) return skinny<MOE_BF16>(a, u, M, st);
    return skinny<MOE_F16>(a, u, M, st);
  }
  moe::Carver cv(workspace);
  uint8_t* codes = cv.take<uint8_t>(x_rows * (K / 2));
  uint8_t* scales = cv.take<uint8_t>(x_rows * (K / 32));
  rc = moe_mxfp4_pack(x, x_dtype, 1, x_rows, K, row_stride, 0, codes, scales, nullptr, nullptr,
                      nullptr, 0, nullptr, stream);
  if (rc != MOE_OK) return rc;
  return moe_mxfp4_matmul(codes, scales, x_rows, w_codes, w_scales, M, N, K, row_offsets,
                          n_groups, row_index, out, out_dtype, ld_out, stream);
}
