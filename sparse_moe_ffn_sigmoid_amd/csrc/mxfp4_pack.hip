// MXFP4 packing along rows and along columns, and unpacking.
//
// A block of 32 consecutive elements v gets the shared exponent
// X = floor(log2 max|v|) - 2 (2 = E2M1's largest exponent), stored as X + 127
// clamped to [0, 254] (0 for an all-zero block), and each element becomes the
// E2M1 value nearest to v / 2^X, ties to the even code, at most 6 in
// magnitude.  A block that holds an infinity or a NaN has no such exponent:
// its scale byte is 255 (NaN in the format) and its codes are 0, so that the
// value is not lost silently.
//
// Along a row the blocks run with the columns (the contraction of x W^T);
// along a column they run with the rows, and the codes come out transposed
// ([columns][rows/2]), K-contiguous again: the operands of a product that
// contracts over the rows (dx and dW of a linear layer).  One read of the
// input serves both.  Everything here is bound by memory: 2 or 4 bytes per
// element in and 17/32 of a byte out per direction.  bf16 16,384 x 7168 both ways:
// 105 us for 360 MB (3.4 TB/s); 24 x 2048 x 3584 both ways: 118 us for 539 MB (4.6
// TB/s, a large copy's rate); unpacking 16,384 x 7168: 50 us for 297 MB (5.9 TB/s).
#include <algorithm>

#include "common.hpp"
#include "mxfp4_convert.hpp"

namespace moe {
namespace mx {

struct PackArgs {
  const void* x;
  int64_t rows, cols, row_stride, batch_stride;  // strides in elements
  int vec;                                       // rows can be read 16 bytes at a time
  uint8_t *codes, *scales;                       // [batch][rows][cb * 16], [batch][rows][cb]
  uint8_t *codes_t, *scales_t;                   // [batch][cols][rb * 16], [batch][cols][rb]
  int64_t cb, rb;                                // blocks along a row, along a column
  const int32_t* off;                            // [G + 1] row groups or null
  const int32_t* poff;                           // [G + 1] their padded starts
  int G;
};

// Rows only: a wave takes 512 consecutive elements of a row (8 per lane, four
// lanes to a block) and ROWS_PER rows one after the other.
constexpr int ROWS_PER = 4;
template <int DT>
__global__ __launch_bounds__(256) void pack_rows_k(PackArgs a) {
  typedef typename Elem<DT>::type E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 512 + lane * 8;
  const int64_t b = blockIdx.z;
  if (c >= a.cb * 32) return;
  const E* x = static_cast<const E*>(a.x) + b * a.batch_stride + c;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 4 * ROWS_PER;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.y) * 4 + wave) * ROWS_PER; r0 < a.rows;
       r0 += step) {
    float v[ROWS_PER][8];
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i)
      if (r0 + i < a.rows) load8<DT>(x + (r0 + i) * a.row_stride, a.cols - c, a.vec, v[i]);
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      if (r0 + i >= a.rows) break;
      const uint32_t sb = scale_byte(max4(amax8(v[i])));
      const int64_t row = b * a.rows + r0 + i;
      *reinterpret_cast<uint32_t*>(a.codes + row * a.cb * 16 + (c >> 1)) = encode8(v[i], sb);
      if ((lane & 3) == 0) a.scales[row * a.cb + (c >> 5)] = static_cast<uint8_t>(sb);
    }
  }
}

// Columns, with or without rows: a block takes 256 rows (eight blocks of 32 of
// each column) by TC columns.  The rows come in as in pack_rows_k, are packed
// from registers if wanted and laid down in LDS; then each thread packs the 32
// rows of one block for each of its columns.  The LDS words of the row blocks
// are turned by 8 words against each other, so that 8 columns by eight row
// blocks, one wave's read, hit 64 different banks, and eight neighbouring lanes
// write 128 consecutive bytes of a column.
constexpr int PACK_ROWS = 256;  // rows of a tile, half its threads

template <int DT, bool WITH_ROWS>
__global__ __launch_bounds__(2 * PACK_ROWS) void pack_cols_k(PackArgs a) {
  typedef typename Elem<DT>::type E;
  constexpr int PER = 4 / sizeof(E);  // elements per LDS word
  constexpr int TR = PACK_ROWS, NTH = 2 * TR, TC = 64 * PER;
  constexpr int LPR = TC / 8;          // lanes per row while loading
  constexpr int RPP = NTH / LPR;       // rows per step
  __shared__ uint32_t tile[TR * 64];
  __shared__ int32_t src[TR];          // input row of each row of the tile, -1: none
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.z;
  const int64_t p0 = static_cast<int64_t>(blockIdx.y) * TR;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * TC;
  if (tid < TR) {
    const int64_t p = p0 + tid;
    int64_t r = p < a.rows ? p : -1;
    if (a.off) {  // the group whose padded rows hold p
      r = -1;
      if (p < a.poff[a.G]) {
        int lo = 0, hi = a.G;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.poff[mid] <= p)
            lo = mid;
          else
            hi = mid;
        }
        const int64_t beg = min(max(static_cast<int64_t>(a.off[lo]), int64_t(0)), a.rows);
        const int64_t end = min(max(static_cast<int64_t>(a.off[lo + 1]), beg), a.rows);
        r = beg + (p - a.poff[lo]);
        if (r >= end) r = -1;
      }
    }
    src[tid] = static_cast<int32_t>(r);
  }
  __syncthreads();
  const E* x = static_cast<const E*>(a.x) + b * a.batch_stride;
  const int lc = (tid % LPR) * 8;
  const int64_t c = c0 + lc;
  // all of the tile's loads are under way before the first value is used
  Raw8<DT> raw8[TR / RPP];
#pragma unroll
  for (int i = 0; i < TR / RPP; ++i) {
    const int64_t row = src[i * RPP + tid / LPR];
    if (row >= 0 && c < a.cols)
      raw8[i].load(x + row * a.row_stride + c, a.cols - c, a.vec);
    else
      raw8[i] = Raw8<DT>{};
  }
#pragma unroll
  for (int i = 0; i < TR / RPP; ++i) {
    const int r = i * RPP + tid / LPR;
    if constexpr (WITH_ROWS) {
      const int64_t row = src[r];
      float v[8];
      raw8[i].values(v);
      const uint32_t sb = scale_byte(max4(amax8(v)));
      if (row >= 0 && c < a.cb * 32) {
        const int64_t o = b * a.rows + row;
        *reinterpret_cast<uint32_t*>(a.codes + o * a.cb * 16 + (c >> 1)) = encode8(v, sb);
        if ((tid & 3) == 0) a.scales[o * a.cb + (c >> 5)] = static_cast<uint8_t>(sb);
      }
    }
    // LDS holds the input's own bits
    const int w0 = lc / PER;
#pragma unroll
    for (int w = 0; w < 8 / PER; ++w) tile[r * 64 + ((w0 + w + 8 * (r >> 5)) & 63)] = raw8[i].w[w];
  }
  __syncthreads();
  const int rb = tid % (TR / 32), word = tid / (TR / 32);
  const int64_t blk = (p0 >> 5) + rb;
  if (blk >= a.rb || (a.off && p0 + rb * 32 >= a.poff[a.G])) return;
  uint32_t raw[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) raw[i] = tile[(rb * 32 + i) * 64 + ((word + 8 * rb) & 63)];
#pragma unroll
  for (int h = 0; h < PER; ++h) {
    const int64_t col = c0 + word * PER + h;
    if (col >= a.cols) return;
    uint32_t amax = 0;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float f;
      if constexpr (PER == 1) {
        f = __uint_as_float(raw[i]);
      } else if constexpr (DT == MOE_BF16) {
        f = __uint_as_float(h ? raw[i] & 0xffff0000u : raw[i] << 16);
      } else {
        f16x2_t p;
        __builtin_memcpy(&p, &raw[i], 4);
        f = static_cast<float>(p[h]);
      }
      v[i >> 3][i & 7] = f;
      amax = max(amax, __float_as_uint(f) & 0x7fffffffu);
    }
    const uint32_t sb = scale_byte(amax);
    const int64_t o = (b * a.cols + col) * a.rb + blk;
    *reinterpret_cast<uint4*>(a.codes_t + o * 16) =
        make_uint4(encode8(v[0], sb), encode8(v[1], sb), encode8(v[2], sb), encode8(v[3], sb));
    a.scales_t[o] = static_cast<uint8_t>(sb);
  }
}

// Padded starts of the row groups: every group begins at a multiple of 32.
__global__ __launch_bounds__(1024) void pad_groups_k(const int32_t* __restrict__ off, int G,
                                                     int64_t rows, int32_t* __restrict__ poff) {
  __shared__ int64_t part[16];
  const int g = threadIdx.x, lane = g & 63, wave = g >> 6;
  int64_t len = 0;
  if (g < G) {
    const int64_t beg = min(max(static_cast<int64_t>(off[g]), int64_t(0)), rows);
    const int64_t end = min(max(static_cast<int64_t>(off[g + 1]), beg), rows);
    len = (end - beg + 31) / 32 * 32;
  }
  int64_t sum = len;
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 63) part[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += part[w];
  // groups that overlap (offsets that fall) could pass the room there is: held inside it
  const int64_t room = (rows + 31ll * G) / 32 * 32;
  if (g == 0) poff[0] = 0;
  if (g < G) poff[g + 1] = static_cast<int32_t>(min(sum, room));
}

// Codes 2 j and 2 j + 1 of a word times the scale, in the output's type.
template <int DT, int J>
__device__ __forceinline__ auto decode2(uint32_t q, float scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (DT == MOE_F32)
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, J);
  else if constexpr (DT == MOE_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, J);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, J);
#else
  return 0;
#endif
}

// Codes back to values: a wave takes 512 elements of a row, 8 per lane.
template <int DT>
__global__ __launch_bounds__(256) void unpack_k(const uint8_t* __restrict__ codes,
                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                int64_t cols, int64_t cb, void* __restrict__ outv,
                                                int64_t row_stride, int vec) {
  typedef typename Elem<DT>::type E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 512 + lane * 8;
  if (c >= cols) return;
  E* out = static_cast<E*>(outv) + c;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 4 * ROWS_PER;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.y) * 4 + wave) * ROWS_PER; r0 < rows;
       r0 += step) {
    uint32_t q[ROWS_PER], s[ROWS_PER];
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      const int64_t r = min(r0 + i, rows - 1);
      q[i] = *reinterpret_cast<const uint32_t*>(codes + r * cb * 16 + (c >> 1));
      s[i] = scales[r * cb + (c >> 5)];
    }
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      if (r0 + i >= rows) break;
      // the hardware conversion takes the scale's exponent field as it is: 2^-127
      // at 0, NaN at 255
      const float sc = __uint_as_float(s[i] << 23);
      __attribute__((aligned(16))) E e[8];
#if defined(__HIP_DEVICE_COMPILE__)
#define MOE_UNPACK2(j)                                                          \
  {                                                                             \
    const auto v = decode2<DT, j>(q[i], sc);                                    \
    __builtin_memcpy(e + 2 * (j), &v, 2 * sizeof(E));                           \
  }
      MOE_UNPACK2(0)
      MOE_UNPACK2(1)
      MOE_UNPACK2(2)
      MOE_UNPACK2(3)
#undef MOE_UNPACK2
#endif
      E* dst = out + (r0 + i) * row_stride;
      if (vec && c + 8 <= cols) {
#pragma unroll
        for (int j = 0; j < static_cast<int>(8 * sizeof(E)) / 16; ++j)
          reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(e)[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) dst[j] = e[j];
      }
    }
  }
}

static int64_t blocks32(int64_t v) { return (v + 31) / 32; }

template <int DT>
static void launch_pack(const PackArgs& a, int64_t batch, hipStream_t st) {
  if (!a.codes_t) {
    const dim3 grid(static_cast<unsigned>((a.cb * 32 + 511) / 512),
                    static_cast<unsigned>(std::min<int64_t>((a.rows + 4 * ROWS_PER - 1) /
                                                                (4 * ROWS_PER), 32768)),
                    static_cast<unsigned>(batch));
    hipLaunchKernelGGL(pack_rows_k<DT>, grid, dim3(256), 0, st, a);
    return;
  }
  constexpr int TC = DT == MOE_F32 ? 64 : 128;
  const dim3 grid(static_cast<unsigned>((a.cols + TC - 1) / TC),
                  static_cast<unsigned>((a.rb * 32 + PACK_ROWS - 1) / PACK_ROWS),
                  static_cast<unsigned>(batch));
  if (a.codes)
    hipLaunchKernelGGL((pack_cols_k<DT, true>), grid, dim3(2 * PACK_ROWS), 0, st, a);
  else
    hipLaunchKernelGGL((pack_cols_k<DT, false>), grid, dim3(2 * PACK_ROWS), 0, st, a);
}

}  // namespace mx
}  // namespace moe

extern "C" int64_t moe_mxfp4_padded_rows(int64_t rows, int32_t n_groups) {
  if (rows < 0 || n_groups < 0 || n_groups > 1024 || rows > (int64_t(1) << 30)) return -1;
  if (n_groups == 0) return moe::mx::blocks32(rows) * 32;
  return (rows + 31ll * n_groups) / 32 * 32;
}

extern "C" int moe_mxfp4_pack(const void* x, int32_t dtype, int64_t batch, int64_t rows,
                              int64_t cols, int64_t row_stride, int64_t batch_stride,
                              uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                              uint8_t* scales_t, const int32_t* row_offsets, int32_t n_groups,
                              int32_t* padded_offsets, void* stream) {
  using namespace moe::mx;
  if (batch < 0 || rows < 0 || cols < 1 || row_stride < cols || batch_stride < 0)
    return MOE_EINVAL;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return MOE_EINVAL;
  if (row_offsets ? (n_groups < 1 || !padded_offsets || batch != 1 || !codes_t)
                  : n_groups != 0)
    return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16) return MOE_EUNSUPPORTED;
  if (batch > 65535 || rows > (int64_t(1) << 30) || cols > (int64_t(1) << 30) ||
      n_groups > 1024)
    return MOE_EUNSUPPORTED;
  const int64_t padded = moe_mxfp4_padded_rows(rows, n_groups);
  if (codes_t && (padded + PACK_ROWS - 1) / PACK_ROWS > 65535) return MOE_EUNSUPPORTED;
  if (row_stride > (int64_t(1) << 56) / (rows + 1) ||
      batch_stride > (int64_t(1) << 56) / (batch + 1))
    return MOE_EINVAL;
  if (batch == 0 || (rows == 0 && !row_offsets)) return MOE_OK;
  if (!codes && !codes_t) return MOE_EINVAL;
  if (rows > 0 && !x) return MOE_EINVAL;
  const int64_t size = dtype == MOE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size != 0 || reinterpret_cast<uintptr_t>(codes) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(codes_t) % 16 != 0)
    return MOE_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  PackArgs a{x, rows, cols, row_stride, batch_stride, 0, codes, scales, codes_t, scales_t,
             blocks32(cols), padded / 32, row_offsets, padded_offsets, n_groups};
  a.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && row_stride * size % 16 == 0 &&
          (batch == 1 || batch_stride * size % 16 == 0);
  if (row_offsets) {
    hipLaunchKernelGGL(pad_groups_k, dim3(1), dim3(1024), 0, st, row_offsets, n_groups, rows,
                       padded_offsets);
    MOE_LAUNCH_CHECK();
    if (rows == 0) return MOE_OK;
  }
  if (dtype == MOE_F32)
    launch_pack<MOE_F32>(a, batch, st);
  else if (dtype == MOE_BF16)
    launch_pack<MOE_BF16>(a, batch, st);
  else
    launch_pack<MOE_F16>(a, batch, st);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" int moe_mxfp4_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, int32_t dtype, void* out, int64_t row_stride,
                                void* stream) {
  using namespace moe::mx;
  if (rows < 0 || cols < 1 || row_stride < cols) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16) return MOE_EUNSUPPORTED;
  if (rows > (int64_t(1) << 36) || cols > (int64_t(1) << 30)) return MOE_EUNSUPPORTED;
  if (row_stride > (int64_t(1) << 56) / (rows + 1)) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !out) return MOE_EINVAL;
  const int64_t size = dtype == MOE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(codes) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % size != 0)
    return MOE_EINVAL;
  const int vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && row_stride * size % 16 == 0;
  const dim3 grid(static_cast<unsigned>((cols + 511) / 512),
                  static_cast<unsigned>(std::min<int64_t>((rows + 4 * ROWS_PER - 1) /
                                                              (4 * ROWS_PER), 32768)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(unpack_k<MOE_F32>, grid, dim3(256), 0, st, codes, scales, rows, cols,
                       blocks32(cols), out, row_stride, vec);
  else if (dtype == MOE_BF16)
    hipLaunchKernelGGL(unpack_k<MOE_BF16>, grid, dim3(256), 0, st, codes, scales, rows, cols,
                       blocks32(cols), out, row_stride, vec);
  else
    hipLaunchKernelGGL(unpack_k<MOE_F16>, grid, dim3(256), 0, st, codes, scales, rows, cols,
                       blocks32(cols), out, row_stride, vec);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
