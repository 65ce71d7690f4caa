// fp8_quant.cu -- bf16 to 8-bit floating point with one power-of-two scale for each block
// of 128 along the contracted dimension.
//
// For a block with largest finite magnitude m = 1.f 2^(E - 127) the scale 2^(byte - 127) is
// the smallest with m <= 2^(byte - 127) fmax. fmax is 1.75 2^8 (e4m3) or 1.75 2^15 (e5m2),
// so byte = E - 8 (or 15) + (1.f > 1.75), read from m's bits: no logarithm, no rounding.
// x 2^(127 - byte) is exact in fp32, and one conversion rounds it.
//
// Both kernels are bound by HBM (2 bytes read and 129/128 written a value and layout) and
// keep every value in registers between its one reading and its writing.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "internal.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct QuantParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* gamma;           // [rows] or NULL
  uint8_t *q, *sf, *qt, *sft;           // either pair may be NULL
  int64_t rows, cols, ldx, gstride;
  int64_t pitch, pitch_t;               // of q, qt
  int64_t kt, kt_t;                     // scale tiles along the columns, along the rows
  int64_t plane, plane_t;               // bytes of one matrix's scales
};

constexpr uint32_t kInf = 0x7f80u;      // bf16 infinity

// The larger magnitude in each half of a pair of magnitudes; a NaN gives way.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Magnitudes of a pair, infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  uint32_t m = w & 0x7fff7fffu;
  if ((m & kInf) == kInf) m &= 0xffff0000u;
  if ((m & kInf << 16) == kInf << 16) m &= 0xffffu;
  return m;
}

__device__ __forceinline__ uint32_t larger_half(uint32_t w) {
  return max(w & 0xffffu, w >> 16);     // magnitudes order as integers
}

// Scale byte of a block whose largest finite magnitude has the bf16 bits m.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if (m == 0) return 127;
  const int e = static_cast<int>(m >> 7) - (FMT == BOOST_E4M3 ? 8 : 15) + ((m & 0x7f) > 0x60);
  return e < 0 ? 0 : e;
}

// 2^(127 - byte), the factor that takes the block's values to 8 bits (byte <= 247, so the
// exponent field 254 - byte is that of a normal number).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two values to 8 bits, nearest even. A scaled finite value never exceeds fmax, so
// saturation only meets infinities, which the caller mends (mend_inf).
template <int FMT>
__device__ __forceinline__ uint32_t to8(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE,
                                  FMT == BOOST_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// One bf16 value's 8 bits where it is an infinity: NaN in e4m3, infinity in e5m2.
template <int FMT>
__device__ __forceinline__ uint32_t mend_inf(uint32_t bits16, uint32_t q8) {
  if ((bits16 & 0x7fffu) != kInf) return q8;
  return ((bits16 >> 8) & 0x80u) | (FMT == BOOST_E4M3 ? 0x7fu : 0x7cu);
}

// 8 values (a vector's four words) times `inv` to 8 bytes.
template <int FMT>
__device__ __forceinline__ uint2 quant8(const uint32_t (&w)[4], float inv, bool inf) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = to8<FMT>(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  if (inf) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = mend_inf<FMT>(w[i] & 0xffffu, p[i] & 0xffu) |
             mend_inf<FMT>(w[i] >> 16, p[i] >> 8) << 8;
  }
  return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
}

// ------------------------------------------------------------------- rows alone
// A warp takes rows of 512 columns: 8 lanes a block of 128, 16 values a lane, four rows in
// flight. A block of 8 warps covers 32 rows. grid = (scale tiles along the columns,
// 4 x row tiles of 128, matrices).
template <int FMT>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const QuantParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 512 + lane * 16;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 32 + warp * 4;
  const int64_t blocks = (p.cols + 127) / 128;
  const __nv_bfloat16* x = p.x + blockIdx.z * p.gstride;
  uint32_t w[4][2][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row0 + r < p.rows && col + 8 * h < p.cols)
        v = __ldg(reinterpret_cast<const uint4*>(x + (row0 + r) * p.ldx + col + 8 * h));
      w[r][h][0] = v.x; w[r][h][1] = v.y; w[r][h][2] = v.z; w[r][h][3] = v.w;
    }
  }
  // largest magnitudes over a block's 8 lanes, two rows in the halves of a word
  uint32_t top[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max2(m, w[r][i >> 2][i & 3] & 0x7fff7fffu);
    top[r] = larger_half(m);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
      const uint32_t both = top[r] | top[r + 1] << 16;
      const uint32_t m = max2(both, __shfl_xor_sync(0xffffffffu, both, o));
      top[r] = m & 0xffffu;
      top[r + 1] = m >> 16;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t row = row0 + r;
    const bool inf = top[r] == kInf;
    if (__any_sync(0xffffffffu, inf)) {          // again over the finite values
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max2(m, finite2(w[r][i >> 2][i & 3]));
      m = larger_half(m);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (inf) top[r] = m;
    }
    const uint32_t byte = scale_byte<FMT>(top[r]);
    if (row < p.rows && col < p.pitch) {
      const float inv = scale_inverse(byte);
      const uint2 a = quant8<FMT>(w[r][0], inv, inf), b = quant8<FMT>(w[r][1], inv, inf);
      *reinterpret_cast<uint4*>(p.q + (blockIdx.z * p.rows + row) * p.pitch + col) =
          make_uint4(a.x, a.y, b.x, b.y);
    }
    // the four blocks' bytes, 127 outside the operand
    const bool in = row < p.rows && static_cast<int64_t>(blockIdx.x) * 4 + (lane >> 3) < blocks;
    uint32_t word = (in ? byte : 127u) << (lane & 24);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(p.sf + blockIdx.z * p.plane +
                                   scale_at(row, static_cast<int64_t>(blockIdx.x) * 4, p.kt)) = word;
  }
}

// ---------------------------------------------------------------- 128 x 128 tiles
// A block holds one tile in registers: thread (rg, cg), rg = threadIdx.x / 16, has rows
// 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7, so that 16 lanes read a row's 256 bytes. The
// transposed bytes go through shared memory: column c's 128 bytes lie at 128 c, the 8 bytes
// of row group rg in slot rg ^ (c / 8), which keeps both sides free of bank conflicts.
// grid = (column tiles, row tiles, matrices).
template <int FMT, bool SQUARE>
__global__ void __launch_bounds__(kThreads) quant_tile_kernel(const QuantParams p) {
  pdl_enter();
  __shared__ __align__(16) uint8_t bytes[128 * 128];
  __shared__ uint32_t part[2][16][64];  // a row group's column maxima, in pairs:
                                        // of all magnitudes, of the finite ones
  __shared__ uint32_t col_all[64], col_top[64];         // the tile's
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int64_t col = col0 + cg * 8;
  const __nv_bfloat16* x = p.x + blockIdx.z * p.gstride;
  uint32_t w[8][4];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t row = row0 + rg * 8 + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < p.rows && col < p.cols)
      v = __ldg(reinterpret_cast<const uint4*>(x + row * p.ldx + col));
    w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
  }
  if (p.gamma != nullptr) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t row = row0 + rg * 8 + r;
      if (row < p.rows) {
        const float g = __bfloat162float(p.gamma[row]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col < p.cols) w[r][i] = pack_bf16x2(g * bf16_lo(w[r][i]), g * bf16_hi(w[r][i]));
      }
    }
  }

  if (SQUARE || p.qt != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) m = max2(m, w[r][i] & 0x7fff7fffu);
      uint32_t f = m;
      if ((m & 0xffffu) == kInf || (m >> 16) == kInf) {
        f = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) f = max2(f, finite2(w[r][i]));
      }
      part[0][rg][cg * 4 + i] = m;
      part[1][rg][cg * 4 + i] = f;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      const int which = threadIdx.x >> 6, c2 = threadIdx.x & 63;
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < 16; ++g) m = max2(m, part[which][g][c2]);
      (which == 0 ? col_all : col_top)[c2] = m;
    }
    __syncthreads();
  }
  uint32_t tile_top = 0;
  bool tile_inf = false;
  if constexpr (SQUARE) {
    const int lane = threadIdx.x & 31;
    uint32_t m = max2(col_all[lane], col_all[lane + 32]);
    uint32_t f = max2(col_top[lane], col_top[lane + 32]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
      f = max2(f, __shfl_xor_sync(0xffffffffu, f, o));
    }
    tile_top = larger_half(f);
    tile_inf = larger_half(m) == kInf;
  }

  if (p.q != nullptr) {
    const int64_t blocks = (p.cols + 127) / 128;
    const bool last = blockIdx.x + 1 == gridDim.x;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t row = row0 + rg * 8 + r;
      uint32_t top = tile_top;
      bool inf = tile_inf;
      if constexpr (!SQUARE) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max2(top, w[r][i] & 0x7fff7fffu);
        top = larger_half(top);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        inf = top == kInf;
        if (__any_sync(0xffffffffu, inf)) {      // again over the finite values
          uint32_t f = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) f = max2(f, finite2(w[r][i]));
          f = larger_half(f);
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, o));
          if (inf) top = f;
        }
      }
      const uint32_t byte = scale_byte<FMT>(top);
      if (row < p.rows && col < p.pitch)
        *reinterpret_cast<uint2*>(p.q + (blockIdx.z * p.rows + row) * p.pitch + col) =
            quant8<FMT>(w[r], scale_inverse(byte), inf);
      // one byte a block; the last column tile fills its scale tile
      const int64_t b = static_cast<int64_t>(blockIdx.x) + cg;
      if (cg == 0 || (last && b < 4 * p.kt))
        p.sf[blockIdx.z * p.plane + scale_at(row, b, p.kt)] =
            static_cast<uint8_t>(row < p.rows && b < blocks ? byte : 127u);
    }
  }

  if (p.qt != nullptr) {
    const int64_t blocks = (p.rows + 127) / 128;
    const bool last = blockIdx.y + 1 == gridDim.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = cg * 8 + 2 * i + h;
        uint32_t top = tile_top;
        bool inf = tile_inf;
        if constexpr (!SQUARE) {
          const uint32_t t = col_top[cg * 4 + i], a = col_all[cg * 4 + i];
          top = h ? t >> 16 : t & 0xffffu;
          inf = (h ? a >> 16 : a & 0xffffu) == kInf;
        }
        const uint32_t byte = scale_byte<FMT>(top);
        uint32_t v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)     // rows 2 r and 2 r + 1 of this column
          v[r] = h ? (w[2 * r][i] >> 16) | (w[2 * r + 1][i] & 0xffff0000u)
                   : (w[2 * r][i] & 0xffffu) | (w[2 * r + 1][i] << 16);
        *reinterpret_cast<uint2*>(bytes + c * 128 + ((rg ^ cg) * 8)) =
            quant8<FMT>(v, scale_inverse(byte), inf);
        // one byte a block; the last row tile fills its scale tile
        const int64_t b = static_cast<int64_t>(blockIdx.y) + rg;
        if (rg == 0 || (last && b < 4 * p.kt_t))
          p.sft[blockIdx.z * p.plane_t + scale_at(col0 + c, b, p.kt_t)] =
              static_cast<uint8_t>(col0 + c < p.cols && b < blocks ? byte : 127u);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {       // 8 lanes a column, 16 bytes a lane
      const int c = k * 32 + (threadIdx.x >> 3), piece = threadIdx.x & 7;
      const uint8_t* at = bytes + c * 128;
      const uint2 a = *reinterpret_cast<const uint2*>(at + (((2 * piece) ^ (c >> 3)) * 8));
      const uint2 b = *reinterpret_cast<const uint2*>(at + (((2 * piece + 1) ^ (c >> 3)) * 8));
      if (col0 + c < p.cols && row0 + piece * 16 < p.pitch_t)
        *reinterpret_cast<uint4*>(p.qt + (blockIdx.z * p.cols + col0 + c) * p.pitch_t + row0 +
                                  piece * 16) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(const boost_fp8_quant_desc& d, const void* x, const void* gamma,
                                void* q, void* sf, void* qt, void* sft, cudaStream_t stream) {
  QuantParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.q = static_cast<uint8_t*>(q);
  p.sf = static_cast<uint8_t*>(sf);
  p.qt = static_cast<uint8_t*>(qt);
  p.sft = static_cast<uint8_t*>(sft);
  p.rows = d.rows;
  p.cols = d.cols;
  p.ldx = d.ldx;
  p.gstride = d.gstride;
  p.pitch = (d.cols + 15) / 16 * 16;
  p.pitch_t = (d.rows + 15) / 16 * 16;
  p.kt = scale_tiles_k(d.cols);
  p.kt_t = scale_tiles_k(d.rows);
  p.plane = scale_plane(d.rows, d.cols);
  p.plane_t = scale_plane(d.cols, d.rows);
  const unsigned G = static_cast<unsigned>(d.G);
  const bool e4m3 = d.fmt == BOOST_E4M3;
  const unsigned row_tiles = static_cast<unsigned>((d.rows + 127) / 128);
  if (d.block_rows == 1 && qt == nullptr) {
    const dim3 grid(static_cast<unsigned>(p.kt), row_tiles * 4, G);
    return launch_grid(e4m3 ? quant_rows_kernel<BOOST_E4M3> : quant_rows_kernel<BOOST_E5M2>, grid,
                       stream, p);
  }
  const dim3 grid(static_cast<unsigned>((d.cols + 127) / 128), row_tiles, G);
  if (d.block_rows == 128)
    return launch_grid(e4m3 ? quant_tile_kernel<BOOST_E4M3, true>
                            : quant_tile_kernel<BOOST_E5M2, true>, grid, stream, p);
  return launch_grid(e4m3 ? quant_tile_kernel<BOOST_E4M3, false>
                          : quant_tile_kernel<BOOST_E5M2, false>, grid, stream, p);
}

}  // namespace boost_gb300
