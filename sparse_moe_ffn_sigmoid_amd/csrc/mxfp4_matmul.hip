// Products of MXFP4 operands: C = A B^T with E2M1 codes and one E8M0 scale per
// 32 elements on both sides, multiplied as they are by gfx950's scaled MFMA
// with fp32 accumulation.
//
// One problem, one per row group (the experts: rows [off[g], off[g + 1]) of A
// meet B[g]), or one per range of the contraction (the experts' weight
// gradients).  Three kernels:
//
// * ring_k, for many rows: tiles go from memory straight into LDS through two
//   buffers of 256 K elements (128 bytes per row, whole cache lines), 16-byte
//   chunks XOR-swizzled by the row so that fills and fragment reads are free
//   of bank conflicts, v_mfma_scale_f32_32x32x64_f8f6f4 on 32x32 blocks, 64 rows
//   to 320 by 256 columns per tile.  8192 x 8192 x 28672: 4.2 PFLOP/s on random
//   operands and 5.5 on zeros, which is the chip's power limit; the matrix
//   instruction alone, out of registers, reaches 8.7.  4096 x 3584 x 7168 (224 tiles):
//   62 us, 3.4 PFLOP/s.  262,144 rows over 896 experts of 2048 x 3584: 1.39 - 1.45
//   ms, 2.7 PFLOP/s, 3.2 TB/s of weights and outputs; its copies alone take 1.13
//   ms, its products with cached weights 1.11.
// * skinny_k, for a few rows per problem, where the codes of B are read once
//   and bound the time: no LDS on the way in, each lane loads its own
//   fragments, v_mfma_scale_f32_16x16x128_f8f6f4 on 16 columns at a time, the
//   contraction split over the waves of a block where the columns alone do not
//   fill the chip.  1024 rows over 896 experts of 2048 x 3584 (about 610 of them
//   used, 2.4 GB of codes): 449 us, 5.3 TB/s.
// * fused_k, for at most 16 rows that are not packed yet: one launch.  One token
//   against 3584 x 7168: 6.5 us.
#include <algorithm>

#include "common.hpp"
#include "lds_ring.hpp"
#include "mxfp4_convert.hpp"

namespace moe {
namespace mx {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int FP4 = 4;  // E2M1 in the scaled MFMA's format fields

typedef const __attribute__((address_space(1))) uint8_t* global_ptr;

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
  int vec_out;                 // rows of C can be written 16 bytes at a time
};

// 32 codes as a matrix operand: E2M1 takes the first four registers, the rest is not read
__device__ __forceinline__ v8i_t fp4_operand(v4i_t v) {
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

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

// Whether row r of C comes from nowhere: its values are zeros.
__device__ __forceinline__ bool absent(const MatArgs& a, int64_t r) {
  if (!a.a_rows) return false;
  const int at = a.a_rows[r];
  return at < 0 || at >= a.a_count;
}

struct Tile {
  int g, row0, rows, n0;
  int kb0, kb1;  // blocks of 32 along K
};

// 16 scale bytes from block kb < kb1 of a row on.  Blocks at or behind kb1 read
// as scale 2^-127 on both sides: whatever codes stand there, their products are
// below 2^-240, nothing next to an fp32 sum.
__device__ __forceinline__ uint4 scales16(global_ptr row, int kb, int kb1) {
  if (kb + 16 <= kb1) {
    struct __attribute__((packed, aligned(1))) Sixteen {
      uint32_t x, y, z, w;
    };
    const auto* p = reinterpret_cast<const __attribute__((address_space(1))) Sixteen*>(row + kb);
    return make_uint4(p->x, p->y, p->z, p->w);
  }
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = row[min(kb + i, kb1 - 1)];
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (kb + i < kb1) w[i >> 2] |= v[i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four consecutive outputs of a row in the output's type.
template <int OUT>
struct Quad;
template <>
struct Quad<MOE_F32> {
  typedef uint4 type;
  static __device__ __forceinline__ uint4 make(float a, float b, float c, float d) {
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                      __float_as_uint(d));
  }
};
template <>
struct Quad<MOE_BF16> {
  typedef uint2 type;
  static __device__ __forceinline__ uint2 make(float a, float b, float c, float d) {
    const bf16x2_t lo = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    const bf16x2_t hi = {static_cast<__bf16>(c), static_cast<__bf16>(d)};
    uint2 v;
    __builtin_memcpy(&v.x, &lo, 4);
    __builtin_memcpy(&v.y, &hi, 4);
    return v;
  }
};
template <>
struct Quad<MOE_F16> {
  typedef uint2 type;
  static __device__ __forceinline__ uint2 make(float a, float b, float c, float d) {
    const f16x2_t lo = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    const f16x2_t hi = {static_cast<_Float16>(c), static_cast<_Float16>(d)};
    uint2 v;
    __builtin_memcpy(&v.x, &lo, 4);
    __builtin_memcpy(&v.y, &hi, 4);
    return v;
  }
};

// WM x WN waves, up to FM x FN fragments of 32 x 32 each.  Fragment i of wave
// row wm covers tile rows (i WM + wm) 32 ..: a short tile's fragments are
// spread evenly over the waves, and a tile of r rows runs the body for
// NF = ceil(r / (32 WM)) fragments, free of branches.  The matrix instruction
// gets the weights as its first operand, so that a lane holds four consecutive
// columns of one output row.
//
// A block stays and takes one tile after another: the next tile's first copies
// and scales are on their way while the finished one is written out.
template <int WM, int WN, int FM, int FN>
struct Ring {
  static constexpr int NW = WM * WN, NTH = 64 * NW;
  static constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  // Copies into the buffers (1 KB, 8 rows) are made by half of the waves, one on
  // each SIMD: a wave is held up until the address unit has taken its copies, and
  // its neighbour has the matrix unit meanwhile.
  static constexpr int LW = NW / 2;
  static constexpr int MB = BN / 8 / LW;
  static_assert(MB * 8 * LW == BN && (WM * 32) % (8 * LW) == 0, "whole copies per wave");
  static constexpr int AC = WM * 4 / LW;  // copies of A per wave, buffer and fragment row
  static constexpr int MS = (BM + BN + NTH - 1) / NTH;  // scale rows per thread
  static constexpr int BUF = (BM + BN) * 128;
  static constexpr int MAXG = 1024;

  struct Shared {
    __attribute__((aligned(1024))) uint8_t buf[2][BUF];  // rows of A, then of B
    uint2 s[2][BN + BM];      // scales of B, then of A
    uint32_t off[BN + BM];    // offsets of the rows of B and A from their bases
    uint8_t absent[2][BM];    // rows of C that come from nowhere, by the tile's parity
    int first[MAXG + 1];      // row tiles before each group
  };
  static_assert(sizeof(Shared) <= 160 * 1024, "LDS of a compute unit");

  // Row tiles before each group, by a scan of the block.
  static __device__ __forceinline__ void count_tiles(const MatArgs& a, int h, Shared& sh) {
    static_assert(NTH * 2 >= MAXG, "two groups per thread");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int g = 2 * tid + i;
      if (g < a.G) n[i] = (max(group_begin(a, g + 1) - group_begin(a, g), 0) + h - 1) / h;
    }
    int sum = n[0] + n[1];
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    int* part = reinterpret_cast<int*>(sh.s);
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += part[w];
    if (2 * tid < a.G) sh.first[2 * tid + 1] = sum - n[1];
    if (2 * tid + 1 < a.G) sh.first[2 * tid + 2] = sum;
    if (tid == 0) sh.first[0] = 0;
    __syncthreads();
  }

  // Tile number tau.  Row tiles come fastest within GM of them, so that the tiles
  // that an XCD works on at one time share their rows of A and B in its L2.
  static __device__ __forceinline__ void find_tile(const MatArgs& a, int h, int ntm, int ntn,
                                                   int tau, const Shared& sh, Tile& t) {
    constexpr int GM = 4;
    t.g = 0;
    t.kb0 = 0;
    t.kb1 = static_cast<int>(a.K / 32);
    if (a.kofs) {
      t.g = tau / (ntm * ntn);
      tau -= t.g * (ntm * ntn);
      // inside the operands whatever the offsets hold
      t.kb0 = static_cast<int>(min(max(static_cast<int64_t>(a.kofs[t.g]), int64_t(0)), a.K) / 32);
      t.kb1 =
          static_cast<int>(min(max(static_cast<int64_t>(a.kofs[t.g + 1]), int64_t(0)), a.K) / 32);
    }
    const int grp = tau / (GM * ntn);
    const int gm = min(GM, ntm - grp * GM);
    const int r = tau - grp * GM * ntn;
    const int m = grp * GM + r % gm;
    t.n0 = r / gm * BN;
    t.row0 = m * h;
    int end = a.M;
    if (a.off) {
      int lo = 0, hi = a.G;  // first[lo] <= m < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.first[mid] <= m)
          lo = mid;
        else
          hi = mid;
      }
      t.g = lo;
      t.row0 = group_begin(a, lo) + (m - sh.first[lo]) * h;
      end = group_begin(a, lo + 1);
    }
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(min(h, end - t.row0));
    t.kb0 = __builtin_amdgcn_readfirstlane(t.kb0);
    t.kb1 = __builtin_amdgcn_readfirstlane(t.kb1);
  }

  // The operands of a tile as the copies and scale loads go through them.
  struct Cursor {
    const uint8_t *base_a, *base_b;
    global_ptr ps[MS];
    uint4 sc[MS];  // scales of two buffers, loaded every other time
  };

  static __device__ __forceinline__ void load_scales(Cursor& cur, const Tile& t, int kb, int rows) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
      if (threadIdx.x + NTH * i < rows) cur.sc[i] = scales16(cur.ps[i], kb, t.kb1);
  }

  // Scales of block kb on into the buffer: the loaded pair's first or second half.
  static __device__ __forceinline__ void put_scales(const Cursor& cur, bool second, int buf,
                                                    int rows, Shared& sh) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
      if (threadIdx.x + NTH * i < rows)
        sh.s[buf][threadIdx.x + NTH * i] = second ? make_uint2(cur.sc[i].z, cur.sc[i].w)
                                                  : make_uint2(cur.sc[i].x, cur.sc[i].y);
  }

  // The copies of the buffer from block kb on, na (at most MA) of them of A.
  // Chunks behind the contraction's end read the first one instead.  A lane's
  // chunk of 32 elements within a row is the same in every copy: a row's chunks
  // are turned by (row / 2) mod 8, so that 16 rows of one chunk fill the 64
  // banks, and a wave's copies are LW, an even number, apart.
  template <int MA>
  static __device__ __forceinline__ void copy(const Cursor& cur, const Tile& t, int kb, int buf,
                                              int na, Shared& sh) {
    static_assert(LW % 2 == 0, "one swizzle for all copies of a wave");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= LW) return;
    const int chunk = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
    const uint32_t at = (kb + chunk < t.kb1 ? chunk : 0) * 16;
    const uint32_t* off = sh.off + wave * 8 + (lane >> 3);
    const uint8_t* from_a = cur.base_a + static_cast<int64_t>(kb - t.kb0) * 16;
    const uint8_t* from_b = cur.base_b + static_cast<int64_t>(kb - t.kb0) * 16;
    const uint32_t to_a = lds_address(sh.buf[0]) + buf * BUF + wave * 1024;
    uint32_t ob[MB], oa[MA];
#pragma unroll
    for (int i = 0; i < MB; ++i) ob[i] = off[LW * i * 8] + at;
#pragma unroll
    for (int i = 0; i < MA; ++i) oa[i] = off[BN + LW * i * 8] + at;
#pragma unroll
    for (int i = 0; i < MB; ++i)
      copy16_to_lds(from_b, ob[i], to_a + BM * 128 + LW * i * 1024);
#pragma unroll
    for (int i = 0; i < MA; ++i)
      if (i < na) copy16_to_lds(from_a, oa[i], to_a + LW * i * 1024);
  }

  // A tile's cursor, row offsets and first copies and scale loads, into buffer
  // buf.  Offsets from the bases fit 32 bits: a tile's rows, or (checked by the
  // launch) all of A where rows are gathered.  A row that the map sends outside A
  // is read as row 0 and written as zeros.
  static __device__ __forceinline__ void begin(const MatArgs& a, const Tile& t, int buf,
                                               uint8_t* gone, Shared& sh, Cursor& cur) {
    const int tid = threadIdx.x;
    const int64_t group = (a.kofs ? 0 : t.g * a.b_stride) + t.n0 * a.ldb;
    const int64_t row0 = a.a_rows ? 0 : t.row0 * a.lda;
    const int64_t k0 = static_cast<int64_t>(t.kb0) * 16;
    cur.base_a = uniform_ptr(a.A + row0 + k0);
    cur.base_b = uniform_ptr(a.B + group + k0);
    const uint8_t* scales_a = uniform_ptr(a.As + row0 / 16);
    const uint8_t* scales_b = uniform_ptr(a.Bs + group / 16);
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      const int r = tid + NTH * i;
      if (r >= BN + BM) break;
      uint32_t row = min(r, a.N - 1 - t.n0);
      if (r >= BN) {
        row = r - BN < t.rows ? r - BN : 0;
        if (a.a_rows) {
          const int at = a.a_rows[t.row0 + row];
          const bool none = at < 0 || at >= a.a_count;
          row = none ? 0 : at;
          gone[r - BN] = none;
        }
      }
      const uint32_t off = row * static_cast<uint32_t>(r < BN ? a.ldb : a.lda);
      sh.off[r] = off;
      cur.ps[i] = (global_ptr)((r < BN ? scales_b : scales_a) + off / 16);
    }
    __syncthreads();
    if (t.kb0 < t.kb1) {
      const int nf = (t.rows + 32 * WM - 1) / (32 * WM);
      load_scales(cur, t, t.kb0, BN + nf * WM * 32);
      copy<FM * AC>(cur, t, t.kb0, buf, nf * AC, sh);
    }
  }

  // The products of one buffer.
  template <int NF>
  static __device__ __forceinline__ void compute(int buf, const Shared& sh,
                                                 f32x16_t (&acc)[NF][FN]) {
    const int lane = threadIdx.x & 63, hi = lane >> 5, l31 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // fragment rows' offsets in a buffer; 64 elements further is an exclusive or
    // with 32 q, because the swizzle only turns the chunk's number.  They are made
    // anew for each buffer rather than kept in registers.
    int oa = (wm * 32 + l31) * 128 + (hi ^ (l31 >> 1 & 7)) * 16;
    int ob = (wn * FN * 32 + l31) * 128 + (hi ^ (l31 >> 1 & 7)) * 16;
    int os = l31;
    asm volatile("" : "+v"(oa), "+v"(ob), "+v"(os));
    uint2 sa[NF], sb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      sb[j] = sh.s[buf][(wn * FN + j) * 32 + os];
      sb[j].x >>= 8 * hi;  // this half's block of a 64-element step in bytes 0 and 2
      sb[j].y >>= 8 * hi;
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      sa[i] = sh.s[buf][BN + (i * WM + wm) * 32 + os];
      sa[i].x >>= 8 * hi;
      sa[i].y >>= 8 * hi;
    }
    // the fragments of the next 64 elements are read under the products of these
    v4i_t b[2][FN], x[2][NF];
    auto read = [&](auto qc) __attribute__((always_inline)) {
      constexpr int q = decltype(qc)::value;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        b[q & 1][j] =
            *reinterpret_cast<const v4i_t*>(sh.buf[buf] + BM * 128 + j * 4096 + (ob ^ 32 * q));
#pragma unroll
      for (int i = 0; i < NF; ++i)
        x[q & 1][i] =
            *reinterpret_cast<const v4i_t*>(sh.buf[buf] + i * WM * 4096 + (oa ^ 32 * q));
    };
    auto step = [&](auto qc) __attribute__((always_inline)) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q < 3) read(std::integral_constant<int, q + 1>{});
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fp4_operand(b[q & 1][j]), fp4_operand(x[q & 1][i]), acc[i][j], FP4, FP4,
              2 * (q & 1), static_cast<int>(q < 2 ? sb[j].x : sb[j].y), 2 * (q & 1),
              static_cast<int>(q < 2 ? sa[i].x : sa[i].y));
      __builtin_amdgcn_sched_barrier(0);
    };
    read(std::integral_constant<int, 0>{});
    __builtin_amdgcn_sched_barrier(0);
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }

  // All of a tile's contraction; buf is the buffer of its first copies, and on
  // return the one that was used last.
  template <int NF>
  static __device__ __forceinline__ void products(const Tile& t, Cursor& cur, int& buf, Shared& sh,
                                                  f32x16_t (&acc)[NF][FN]) {
    const bool copies = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) < LW;
    constexpr int SR = BN + NF * WM * 32;  // scale rows that are used
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    bool second = false;  // of the pair of buffers whose scales were loaded
    for (int kb = t.kb0; kb < t.kb1; kb += 8) {
      if (copies) ring_wait<0>();  // this wave's copies of the buffer to be used
      lds_wait();
      ring_barrier();  // everyone's; and everyone is done with the other buffer
      if (kb + 8 < t.kb1) {
        put_scales(cur, !second, buf ^ 1, SR, sh);
        if (!second && kb + 16 < t.kb1) load_scales(cur, t, kb + 16, SR);
        copy<NF * AC>(cur, t, kb + 8, buf ^ 1, NF * AC, sh);
      }
      compute<NF>(buf, sh, acc);
      second = !second;
      buf ^= 1;
    }
    buf ^= 1;
  }

  // Writes a tile from the accumulators: one row of fragments at a time through
  // the buffer that was used last, then whole rows, 16 bytes per lane.  A thread
  // keeps its column.
  template <int NF, int OUT>
  static __device__ __forceinline__ void write(const MatArgs& a, const Tile& t, int buf,
                                               const uint8_t* gone, Shared& sh,
                                               const f32x16_t (&acc)[NF][FN]) {
    typedef typename Quad<OUT>::type quad_t;
    const int tid = threadIdx.x, lane = tid & 63, hi = lane >> 5, l31 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    constexpr int ESZ = sizeof(quad_t) / 4, ROWS = WM * 32;
    constexpr int PITCH = BN * ESZ + 16, CPR = BN * ESZ / 16, RPS = NTH / CPR;
    constexpr int AREA = ROWS * PITCH, AREAS = 2 * AREA <= BUF ? 2 : 1;
    static_assert(AREA <= BUF, "staging fits a buffer");
    static_assert(NTH % CPR == 0 && ROWS % RPS == 0, "whole rows per step");
    const int trow = tid / CPR, tcol = tid % CPR * (16 / ESZ);
    const int64_t ldc = a.ldc * ESZ;
    uint8_t* dst = static_cast<uint8_t*>(a.C) +
                   ((a.kofs ? t.g * a.c_stride : 0) + (t.row0 + trow) * a.ldc + t.n0 + tcol) * ESZ;
    const bool whole = a.vec_out && !a.a_rows && t.n0 + BN <= a.N;
    const uint8_t* const from = sh.buf[buf] + trow * PITCH + tcol * ESZ;
    uint8_t* const to = sh.buf[buf] + (wm * 32 + l31) * PITCH + (wn * FN * 32 + hi * 4) * ESZ;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int area = i % AREAS * AREA;
      if (AREAS == 1 && i > 0) __syncthreads();  // the rows before have been read
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<quad_t*>(to + area + (j * 32 + r * 2) * ESZ) =
              Quad<OUT>::make(acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]);
      __syncthreads();
      if (whole) {
#pragma unroll
        for (int s = 0; s < ROWS; s += RPS, dst += RPS * ldc) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(from + area + s * PITCH);
          if (i * ROWS + s + trow < t.rows)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(dst));
        }
      } else {
#pragma unroll 1
        for (int s = 0; s < ROWS; s += RPS, dst += RPS * ldc) {
          u32x4_t v = *reinterpret_cast<const u32x4_t*>(from + area + s * PITCH);
          const int row = i * ROWS + s + trow, left = a.N - t.n0 - tcol;
          if (row >= t.rows || left <= 0) continue;
          if (a.a_rows && gone[row]) v = u32x4_t{0, 0, 0, 0};
          if (a.vec_out && left >= 16 / ESZ) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(dst));
          } else {
#pragma unroll
            for (int e = 0; e < 16 / ESZ; ++e)
              if (e < left) {
                if constexpr (ESZ == 4)
                  reinterpret_cast<uint32_t*>(dst)[e] = v[e];
                else
                  reinterpret_cast<uint16_t*>(dst)[e] =
                      static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
              }
          }
        }
      }
    }
  }
};

// ntm row tiles of h rows (counted here where there are row groups), ntn column
// tiles, problems ranges of K.  Blocks are dealt to the 8 XCDs in turn; each XCD
// takes a consecutive eighth of the tiles, its blocks side by side.
template <int WM, int WN, int FM, int FN, int OUT>
__global__ __launch_bounds__(64 * WM * WN) void ring_k(MatArgs a, int h, int ntm, int ntn) {
  typedef Ring<WM, WN, FM, FN> R;
  __shared__ typename R::Shared sh;
  if (a.off) {
    R::count_tiles(a, h, sh);
    ntm = __builtin_amdgcn_readfirstlane(sh.first[a.G]);
  }
  // offsets that fall could name more tiles than the launch allowed for
  if (static_cast<int64_t>(ntm) * ntn * (a.kofs ? a.G : 1) > 0x7fff0000) return;
  const int tiles = ntm * ntn * (a.kofs ? a.G : 1);
  const int per = (tiles + 7) >> 3, step = gridDim.x >> 3;
  const int last = min(tiles, static_cast<int>(blockIdx.x & 7) * per + per);
  int tau = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (tau >= last) return;
  Tile t;
  typename R::Cursor cur;
  int buf = 0, parity = 0;
  R::find_tile(a, h, ntm, ntn, tau, sh, t);
  R::begin(a, t, buf, sh.absent[0], sh, cur);
  bool more = true;
  auto body = [&](auto nfc) __attribute__((always_inline)) {
    constexpr int NF = decltype(nfc)::value;
    f32x16_t acc[NF][FN];
    if (t.kb0 < t.kb1) R::put_scales(cur, false, buf, R::BN + NF * WM * 32, sh);
    R::template products<NF>(t, cur, buf, sh, acc);
    const Tile done = t;
    tau += step;
    more = tau < last;
    if (more) {
      // its barrier also sees every wave out of the buffer that was used last
      R::find_tile(a, h, ntm, ntn, tau, sh, t);
      R::begin(a, t, buf ^ 1, sh.absent[parity ^ 1], sh, cur);
    } else {
      __syncthreads();
    }
    R::template write<NF, OUT>(a, done, buf, sh.absent[parity], sh, acc);
    buf ^= 1;
    parity ^= 1;
  };
  while (more) {
    const int nf = (t.rows + 32 * WM - 1) / (32 * WM);
    if (nf <= 1)
      body(std::integral_constant<int, 1>{});
    else if (FM >= 2 && nf == 2)
      body(std::integral_constant<int, FM >= 2 ? 2 : 1>{});
    else if (FM >= 3 && nf == 3)
      body(std::integral_constant<int, FM >= 3 ? 3 : 1>{});
    else if (FM >= 4 && nf == 4)
      body(std::integral_constant<int, FM >= 4 ? 4 : 1>{});
    else
      body(std::integral_constant<int, FM>{});
  }
}

// A few rows per problem.  A block takes 16 NT columns per wave group and all of
// a group's rows, 16 MT at a time; WK waves split the contraction into stretches
// of 256 elements dealt in turn and add their sums through LDS in a fixed order.
// The matrix instruction multiplies 128 elements, lane (c, h), c = lane mod 16,
// h = lane / 16, holding one block of 32 of row c with its scale.  Which blocks
// meet in one instruction is free as long as both operands agree: lane h takes
// blocks 2 h and 2 h + 1 of a stretch, so that its codes are 32 consecutive bytes,
// four lanes read a whole cache line and the scales are two bytes.  U stretches
// are loaded before the first is multiplied.
// Two blocks of a row from block kb on: codes and scales (in bytes 0 and 1).
// Blocks at or behind kb1, and a row that is not there, are codes of zero.
__device__ __forceinline__ void load_pair(const uint8_t* codes, const uint8_t* scales, int kb,
                                          int kb1, bool there, v4i_t (&q)[2], uint32_t& s) {
  q[0] = q[1] = v4i_t{0, 0, 0, 0};
  s = 0x7f7fu;
  if (!there || kb >= kb1) return;
  const v4i_t* p = reinterpret_cast<const v4i_t*>(codes + static_cast<int64_t>(kb) * 16);
  q[0] = p[0];
  if (kb + 1 < kb1) {
    struct __attribute__((packed, aligned(1))) Two {
      uint16_t v;
    };
    q[1] = p[1];
    s = reinterpret_cast<const Two*>(scales + kb)->v;
  } else {
    s = 0x7f00u | scales[kb];
  }
}

template <int WN, int WK, int NT, int MT, int U>
__global__ __launch_bounds__(64 * WN * WK) void skinny_k(MatArgs a) {
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
    pb[j] = B + n * a.ldb;
    ps[j] = Bs + n * (a.ldb / 16);
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
    for (int k0 = wk * 8; k0 < kb1; k0 += WK * U * 8) {
      v4i_t bq[U][NT][2], aq[U][MT][2];
      uint32_t bs[U][NT], as[U][MT];
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          load_pair(pb[j], ps[j], k0 + v * WK * 8 + 2 * h, kb1, true, bq[v][j], bs[v][j]);
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int64_t r = row[i] < 0 ? 0 : row[i];
          load_pair(a.A + r * a.lda, a.As + r * (a.lda / 16), k0 + v * WK * 8 + 2 * h, kb1,
                    row[i] >= 0, aq[v][i], as[v][i]);
        }
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fp4_operand(aq[v][i][0]), fp4_operand(bq[v][j][0]), acc[i][j], FP4, FP4, 0,
                static_cast<int>(as[v][i]), 0, static_cast<int>(bs[v][j]));
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fp4_operand(aq[v][i][1]), fp4_operand(bq[v][j][1]), acc[i][j], FP4, FP4, 1,
                static_cast<int>(as[v][i]), 1, static_cast<int>(bs[v][j]));
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
            if (m < end && n < a.N)
              store_one(a, m * a.ldc + n, absent(a, m) ? 0.f : acc[i][j][r]);
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
        if (m < end && n < a.N) store_one(a, m * a.ldc + n, absent(a, m) ? 0.f : sum);
      }
    }
  }
}

// At most 16 rows of activations as they are: the block packs them into LDS while
// its first codes of the weights are on the way, then goes on as skinny_k.  One
// launch for a token, whose time is the launch and one trip to memory.
constexpr int FUSED_WAVES = 8, FUSED_U = 4;

template <int DT>
__global__ __launch_bounds__(64 * FUSED_WAVES) void fused_k(MatArgs a, const void* x,
                                                            int64_t stride) {
  constexpr int WK = FUSED_WAVES, U = FUSED_U;
  __shared__ float part[WK * 256];
  // codes of the rows, each followed by 32 bytes that keep rows off one
  // another's banks, then their scales
  extern __shared__ __attribute__((aligned(16))) uint8_t packed[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int kb1 = static_cast<int>(a.K / 32), pitch = kb1 * 16 + 32;
  uint8_t* const scales = packed + a.M * pitch;
  const int n0 = blockIdx.x * 16;
  const int64_t n = min(n0 + c, a.N - 1);
  const uint8_t *pb = a.B + n * a.ldb, *ps = a.Bs + n * (a.ldb / 16);
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  v4i_t bq[U][2];
  uint32_t bs[U];
  auto load = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < U; ++v)
      load_pair(pb, ps, k0 + v * WK * 8 + 2 * h, kb1, true, bq[v], bs[v]);
  };
  load(wave * 8);
  // eight elements a thread, four threads a block of 32
  for (int i = tid; i < a.M * kb1 * 4; i += 64 * WK) {
    const int m = i / (kb1 * 4), e = i - m * (kb1 * 4);
    const int at = a.a_rows ? a.a_rows[m] : m;
    const int64_t row = at >= 0 && at < a.a_count ? at : 0;
    float v[8];
    load8<DT>(static_cast<const typename Elem<DT>::type*>(x) + row * stride + e * 8, 8, true, v);
    const uint32_t sb = scale_byte(max4(amax8(v)));
    *reinterpret_cast<uint32_t*>(packed + m * pitch + e * 4) = encode8(v, sb);
    if ((e & 3) == 0) scales[m * kb1 + (e >> 2)] = static_cast<uint8_t>(sb);
  }
  __syncthreads();
  for (int k0 = wave * 8;;) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
      v4i_t aq[2] = {v4i_t{0, 0, 0, 0}, v4i_t{0, 0, 0, 0}};
      uint32_t as = 0x7f7fu;
      const int kb = k0 + v * WK * 8 + 2 * h;
      if (c < a.M && kb < kb1) {
        const int second = min(kb + 1, kb1 - 1);  // its partner's codes are zero there
        aq[0] = *reinterpret_cast<const v4i_t*>(packed + c * pitch + kb * 16);
        aq[1] = *reinterpret_cast<const v4i_t*>(packed + c * pitch + second * 16);
        as = scales[c * kb1 + kb] | (static_cast<uint32_t>(scales[c * kb1 + second]) << 8);
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          fp4_operand(aq[0]), fp4_operand(bq[v][0]), acc, FP4, FP4, 0, static_cast<int>(as), 0,
          static_cast<int>(bs[v]));
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          fp4_operand(aq[1]), fp4_operand(bq[v][1]), acc, FP4, FP4, 1, static_cast<int>(as), 1,
          static_cast<int>(bs[v]));
    }
    k0 += WK * U * 8;
    if (k0 >= kb1) break;
    load(k0);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) part[wave * 256 + (h * 4 + r) * 16 + c] = acc[r];
  __syncthreads();
  if (tid < a.M * 16 && n0 + tid % 16 < a.N) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) sum += part[w * 256 + tid];
    const int m = tid / 16;
    store_one(a, m * a.ldc + n0 + tid % 16, absent(a, m) ? 0.f : sum);
  }
}

// LDS of fused_k's packed rows; it takes what leaves a second block room.
static int64_t fused_bytes(int64_t M, int64_t K) { return M * (K / 2 + 32 + K / 32); }
constexpr int64_t FUSED_BYTES = 64 << 10;
constexpr int64_t FUSED_N = 1 << 26;  // 32 threads a column, fewer than 2^32

template <int DT>
static int launch_fused(const MatArgs& a, const void* x, int64_t stride, hipStream_t st) {
  hipLaunchKernelGGL(fused_k<DT>, dim3(static_cast<unsigned>((a.N + 15ll) / 16)),
                     dim3(64 * FUSED_WAVES), static_cast<unsigned>(fused_bytes(a.M, a.K)), st, a, x,
                     stride);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

// h: rows per tile, at most the kernel's
template <int WM, int WN, int FM, int FN>
static int launch_ring(MatArgs a, int h, hipStream_t st) {
  constexpr int BN = WN * FN * 32;
  const int64_t ntm = a.off ? a.M / h + a.G : (static_cast<int64_t>(a.M) + h - 1) / h;  // at most
  const int64_t ntn = (static_cast<int64_t>(a.N) + BN - 1) / BN;
  const int64_t tiles = ntm * ntn * (a.kofs ? a.G : 1);
  if (tiles > 0x7fff0000) return MOE_EUNSUPPORTED;
  const int esz = a.out == MOE_F32 ? 4 : 2;
  a.vec_out = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && a.ldc * esz % 16 == 0 &&
              a.c_stride * esz % 16 == 0;
  // one block per compute unit, or per tile where there are fewer
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(256, (tiles + 7) / 8 * 8)));
  const dim3 block(64 * WM * WN);
  const int tm = static_cast<int>(ntm), tn = static_cast<int>(ntn);
  if (a.out == MOE_F32)
    hipLaunchKernelGGL((ring_k<WM, WN, FM, FN, MOE_F32>), grid, block, 0, st, a, h, tm, tn);
  else if (a.out == MOE_BF16)
    hipLaunchKernelGGL((ring_k<WM, WN, FM, FN, MOE_BF16>), grid, block, 0, st, a, h, tm, tn);
  else
    hipLaunchKernelGGL((ring_k<WM, WN, FM, FN, MOE_F16>), grid, block, 0, st, a, h, tm, tn);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int WN, int WK, int NT, int MT, int U>
static int launch_skinny(const MatArgs& a, hipStream_t st) {
  const int64_t per = 16ll * NT * WN;
  hipLaunchKernelGGL((skinny_k<WN, WK, NT, MT, U>),
                     dim3(static_cast<unsigned>((a.N + per - 1) / per),
                          static_cast<unsigned>(a.off ? a.G : 1)),
                     dim3(64 * WN * WK), 0, st, a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

static int skinny(const MatArgs& a, int64_t per_group, hipStream_t st) {
  // waves that a split over columns alone gives
  const int64_t waves = (static_cast<int64_t>(a.N) + 15) / 16 * (a.off ? a.G : 1);
  if (per_group > 16)
    return waves >= 8192 ? launch_skinny<4, 1, 1, 4, 1>(a, st) : launch_skinny<1, 8, 1, 4, 1>(a, st);
  return waves >= 8192 ? launch_skinny<4, 1, 1, 1, 4>(a, st) : launch_skinny<1, 8, 1, 1, 4>(a, st);
}

// Rows per problem up to which the skinny kernel is the faster.  One problem, K =
// 7168: 64 rows 14.7 us against the ring kernel's 25.5 at N = 3584 and 26.6
// against 28.5 at N = 7168; 128 rows 27.4 against 25.9 and 50.5 against 28.9.  64
// groups of 2048 x 3584: past 16 rows each it reads the weights' codes once more
// per 64 rows without the others' sharing them, 17 rows 75.9 us against 45.1.
constexpr int SKINNY_ROWS = 64, SKINNY_GROUP_ROWS = 16;

// Tile height: the multiple of 64 up to 320 whose tiles cover the rows of a
// problem soonest, a tile of h rows costing h and the 128 rows' worth that every
// tile's weights and start take; the taller one on a tie (fewer reads of B).
static int tile_height(int64_t rows, int64_t problems, int64_t N) {
  int best = 64;
  int64_t cost = 0;
  for (int h = 64; h <= 320; h += 64) {
    const int64_t tiles = (rows + h - 1) / h * ((N + 255) / 256) * problems;
    const int64_t c = (tiles + 255) / 256 * (h + 128);
    if (h == 64 || c <= cost) {
      best = h;
      cost = c;
    }
  }
  return best;
}

// The ring kernel's offsets: 320 rows of A or B, or all of A if its rows are
// gathered, within 4 GiB.
static bool ring_fits(const MatArgs& a) {
  const int64_t limit = int64_t(1) << 32;
  return 320 * std::max(a.lda, a.ldb) < limit &&
         (!a.a_rows || static_cast<int64_t>(a.a_count) * a.lda < limit);
}

static int product(const MatArgs& a, hipStream_t st) {
  if (a.kofs)
    return ring_fits(a) ? launch_ring<2, 4, 5, 2>(a, tile_height(a.M, a.G, a.N), st)
                        : MOE_EUNSUPPORTED;
  const int64_t per = a.off ? (a.M + a.G - 1) / a.G : a.M;
  if (per <= (a.off ? SKINNY_GROUP_ROWS : SKINNY_ROWS) || !ring_fits(a)) return skinny(a, per, st);
  return launch_ring<2, 4, 5, 2>(a, tile_height(per, a.off ? a.G : 1, a.N), st);
}

// Rows of C: tile counts of any row offsets stay within 32 bits.
constexpr int64_t MAX_ROWS = 1 << 30, MAX_GROUPED_ROWS = 1 << 24;
// Columns of C: skinny_k's grid has 4 threads a column, fewer than 2^32.
constexpr int64_t MAX_N = 1 << 29;

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
  if (row_index ? M > 0 && a_rows < 1 : a_rows < M) return MOE_EINVAL;
  if (M > (row_offsets ? MAX_GROUPED_ROWS : MAX_ROWS) || N > MAX_N || a_rows > (1 << 30) ||
      K > (1 << 30) || n_groups > 1024)
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
  // an empty contraction still writes its zeros
  if (K == 0) return launch_ring<2, 4, 5, 2>(a, 64, static_cast<hipStream_t>(stream));
  return product(a, static_cast<hipStream_t>(stream));
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
  if (row_index ? M > 0 && x_rows < 1 : x_rows < M) return MOE_EINVAL;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16 && x_dtype != MOE_F16) return MOE_EUNSUPPORTED;
  if (M > (row_offsets ? MAX_GROUPED_ROWS : MAX_ROWS) || N > MAX_N || x_rows > (1 << 30) ||
      K > (1 << 30) || n_groups > 1024)
    return MOE_EUNSUPPORTED;
  if (row_stride > (int64_t(1) << 56) / (x_rows + 1)) return MOE_EINVAL;
  if (M == 0) return MOE_OK;
  int rc = check_out(out_dtype, out, ld_out, N);
  if (rc != MOE_OK) return rc;
  const int64_t size = x_dtype == MOE_F32 ? 4 : 2;
  if ((!x && x_rows > 0) || reinterpret_cast<uintptr_t>(x) % size != 0 || !w_codes || !w_scales ||
      !aligned16(w_codes))
    return MOE_EINVAL;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (!row_offsets && M <= 16 && N <= FUSED_N && fused_bytes(M, K) <= FUSED_BYTES &&
      aligned16(x) && row_stride * size % 16 == 0) {
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
    if (x_dtype == MOE_F32) return launch_fused<MOE_F32>(a, x, row_stride, st);
    if (x_dtype == MOE_BF16) return launch_fused<MOE_BF16>(a, x, row_stride, st);
    return launch_fused<MOE_F16>(a, x, row_stride, st);
  }
  if (!workspace || workspace_bytes < moe_mxfp4_linear_workspace_bytes(x_rows, K))
    return MOE_EWORKSPACE;
  moe::Carver cv(workspace);
  uint8_t* codes = cv.take<uint8_t>(x_rows * (K / 2));
  uint8_t* scales = cv.take<uint8_t>(x_rows * (K / 32));
  rc = moe_mxfp4_pack(x, x_dtype, 1, x_rows, K, row_stride, 0, codes, scales, nullptr, nullptr,
                      nullptr, 0, nullptr, stream);
  if (rc != MOE_OK) return rc;
  return moe_mxfp4_matmul(codes, scales, x_rows, w_codes, w_scales, M, N, K, row_offsets,
                          n_groups, row_index, out, out_dtype, ld_out, stream);
}
