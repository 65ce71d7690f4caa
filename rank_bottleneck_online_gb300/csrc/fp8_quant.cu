// fp8_quant.cu -- bf16 to 8-bit floating point with one power-of-two scale for each block
// of 128 along the contracted dimension.
//
// For a block with largest finite magnitude m = 1.f 2^(E - 127) the scale 2^(byte - 127) is
// the smallest with m <= 2^(byte - 127) fmax. fmax is 1.75 2^8 (e4m3) or 1.75 2^15 (e5m2),
// so byte = E - 8 (or 15) + (1.f > 1.75), read from m's bits: no logarithm, no rounding.
// x 2^(127 - byte) is exact in fp32, and one conversion rounds it.
//
// Both kernels keep every value in registers between its one reading and its writing, so they
// move what they must: 2 bytes read and 129/128 written a value and layout. Rows alone run near
// the copy rate; what holds the tiles back stands beside their kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "fp8_values.cuh"
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

constexpr int64_t kMaxLines = 65535;    // of 32 rows: a grid's limit, and the most of an operand

// ------------------------------------------------------------------- rows alone
// A warp takes rows of 512 columns: 8 lanes a block of 128, 16 values a lane, four rows in
// flight. A block of 8 warps covers 32 rows. grid = (scale tiles along the columns, lines of
// 32 rows of the whole row tiles, matrices). The most rows have 65536 lines, one more than a
// grid: the last is behind the operand, and the block before it fills its scales (MOST: asked in
// the kernel of every size, it cost up to 0.09 us of 1024 x 4096's 2.7).
template <int FMT, bool MOST>
__global__ void __launch_bounds__(kThreads, 4) quant_rows_kernel(const QuantParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 512 + lane * 16;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 32 + warp * 4;
  const int rows = static_cast<int>(min(max(p.rows - row0, static_cast<int64_t>(0)),
                                        static_cast<int64_t>(4)));
  const __nv_bfloat16* x = p.x + blockIdx.z * p.gstride + row0 * p.ldx + col;
  uint32_t w[4][8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows && col + 8 * h < p.cols)
        v = __ldg(reinterpret_cast<const uint4*>(x + r * p.ldx + 8 * h));
      w[r][4 * h] = v.x; w[r][4 * h + 1] = v.y; w[r][4 * h + 2] = v.z; w[r][4 * h + 3] = v.w;
    }
  }
  uint32_t top[4];
  const bool mend = block_tops<4, 8, 8>(w, top);
  uint8_t* q = p.q + (blockIdx.z * p.rows + row0) * p.pitch + col;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 4;      // block of lane 0
  uint8_t* sf = p.sf + blockIdx.z * p.plane + scale_at(row0, first, p.kt);
  const bool in_cols = first + (lane >> 3) < (p.cols + 127) / 128;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t byte = scale_byte<FMT>(top[r]);
    if (r < rows && col < p.pitch) {
      const float inv = scale_inverse(byte);
      const uint2 a = quant8<FMT>(w[r], inv, mend), b = quant8<FMT>(w[r] + 4, inv, mend);
      *reinterpret_cast<uint4*>(q + r * p.pitch) = make_uint4(a.x, a.y, b.x, b.y);
    }
    // the four blocks' bytes, 127 outside the operand
    uint32_t word = static_cast<uint32_t>(stored_byte(byte, top[r], in_cols && r < rows)) << (lane & 24);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    // (four rows of one quarter of a scale tile lie 16 bytes apart, the quarters 4)
    if (lane == 0) *reinterpret_cast<uint32_t*>(sf + 16 * r) = word;
    if (MOST && lane == 0 && blockIdx.y + 1 == kMaxLines)
      *reinterpret_cast<uint32_t*>(sf + 16 * r + 4) = 0x7f7f7f7fu;
  }
}

// ---------------------------------------------------------------- 128 x 128 tiles
// A block holds one tile in registers: thread (rg, cg), rg = threadIdx.x / 16, has rows
// 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7, so that 16 lanes read a row's 256 bytes. The
// transposed bytes go through shared memory: column c's 128 bytes lie at 128 c, the 8 bytes
// of row group rg in slot rg ^ (c / 8), which keeps both sides free of bank conflicts. Every
// address is a base and a small stride, and tiles that lie inside x and are finite, by far the
// most, skip the checks of both: at 28 instructions a value the pass was bound by them, at 15.5
// (both ways) they take 55% of the issue slots. (A persistent form with the next tile on its way
// by cp.async was slower, 67 us against 57 before that last step: its shared memory leaves three
// blocks an SM, not four.) 16384 x 4096 both ways: 48 us, 5.6 TB/s, 83% of the measured copy rate;
// what is left is the latency of a tile's three barriers at four blocks an SM.
// grid = (column tiles, row tiles, matrices).

// Thread c < 64 stores the scales of the tile's columns 2 c and 2 c + 1, whose largest finite
// magnitudes are `top`: one byte a block; the last row tile fills its scale tile.
template <int FMT>
__device__ __forceinline__ void column_scales(const QuantParams& p, uint32_t top) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 128 + 2 * threadIdx.x;
  const int64_t b0 = blockIdx.y, blocks = (p.rows + 127) / 128;
  const int64_t end = b0 + 1 == gridDim.y ? 4 * p.kt_t : b0 + 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t m = h ? top >> 16 : top & 0xffffu;
    const uint8_t byte = stored_byte(scale_byte<FMT>(m), m, col < p.cols);
    for (int64_t b = b0; b < end; ++b)
      p.sft[blockIdx.z * p.plane_t + scale_at(col + h, b, p.kt_t)] = b < blocks ? byte : 127;
  }
}

// What follows a tile's column maxima: both layouts' values and scales. PLAIN: the tile lies
// inside x and holds finite values alone.
template <int FMT, bool SQUARE, bool PLAIN>
__device__ __forceinline__ void write_tile(const QuantParams& p, const uint32_t (&w)[8][4],
                                           const uint32_t* col_top, uint8_t* bytes) {
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int64_t row = row0 + rg * 8, col = col0 + cg * 8;          // this thread's first
  const int rows = PLAIN ? 8 : static_cast<int>(min(max(p.rows - row, static_cast<int64_t>(0)),
                                                    static_cast<int64_t>(8)));
  uint32_t tile_top = 0, tile_byte = 0;
  if constexpr (SQUARE) {
    const int lane = threadIdx.x & 31;
    uint32_t m = max2(col_top[lane], col_top[lane + 32]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
    tile_top = larger_half(m);
    tile_byte = scale_byte<FMT>(tile_top);
  }

  if (p.q != nullptr) {
    const int64_t b0 = static_cast<int64_t>(blockIdx.x), blocks = (p.cols + 127) / 128;
    uint8_t* q = p.q + (blockIdx.z * p.rows + row) * p.pitch + col;
    uint32_t top[8];
    if constexpr (!SQUARE) block_tops<8, 4, 16, !PLAIN>(w, top);
    // one byte a block; the last column tile fills its scale tile
    const int64_t b = b0 + cg;
    const bool writes = cg == 0 || (b0 + 1 == gridDim.x && b < 4 * p.kt);
    uint8_t* sf = p.sf + blockIdx.z * p.plane + scale_at(row, b, p.kt);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if constexpr (SQUARE) top[r] = tile_top;
      const uint32_t byte = SQUARE ? tile_byte : scale_byte<FMT>(top[r]);
      // (eight rows of one quarter of a scale tile lie 16 bytes apart)
      if (writes) sf[16 * r] = stored_byte(byte, top[r], r < rows && b < blocks);
      if (PLAIN || (r < rows && col < p.pitch))
        *reinterpret_cast<uint2*>(q) = quant8<FMT>(w[r], scale_inverse(byte), !PLAIN);
      q += p.pitch;
    }
  }

  if (p.qt != nullptr) {
    uint8_t* slot = bytes + cg * 1024 + ((rg ^ cg) * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = SQUARE ? 0 : col_top[cg * 4 + i];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 2 * i + h;
        const uint32_t byte =
            SQUARE ? tile_byte : scale_byte<FMT>(h ? t >> 16 : t & 0xffffu);
        uint32_t v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)     // rows 2 r and 2 r + 1 of this column
          v[r] = __byte_perm(w[2 * r][i], w[2 * r + 1][i], h ? 0x7632 : 0x5410);
        *reinterpret_cast<uint2*>(slot + c * 128) = quant8<FMT>(v, scale_inverse(byte), !PLAIN);
      }
    }
    if (SQUARE && threadIdx.x < 64) column_scales<FMT>(p, tile_top | tile_top << 16);
    __syncthreads();
    // 8 lanes a column, 16 bytes a lane
    const int c0 = threadIdx.x >> 3, piece = threadIdx.x & 7;
    const bool in_pitch = PLAIN || row0 + piece * 16 < p.pitch_t;
    uint8_t* qt = p.qt + (blockIdx.z * p.cols + col0 + c0) * p.pitch_t + row0 + piece * 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = k * 32 + c0;
      const uint8_t* at = bytes + c * 128;
      const uint2 lo = *reinterpret_cast<const uint2*>(at + (((2 * piece) ^ (c >> 3)) * 8));
      const uint2 hi = *reinterpret_cast<const uint2*>(at + (((2 * piece + 1) ^ (c >> 3)) * 8));
      if (PLAIN || (col0 + c < p.cols && in_pitch))
        *reinterpret_cast<uint4*>(qt) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      qt += 32 * p.pitch_t;
    }
  }
}

template <int FMT, bool SQUARE>
__global__ void __launch_bounds__(kThreads, 4) quant_tile_kernel(const QuantParams p) {
  pdl_enter();
  __shared__ __align__(16) uint8_t bytes[128 * 128];
  __shared__ uint32_t part[16][64];     // a row group's largest finite column magnitudes, in pairs
  __shared__ uint32_t col_top[64];      // the tile's
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t row = static_cast<int64_t>(blockIdx.y) * 128 + rg * 8;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 128 + cg * 8;
  const bool inside = row + 8 <= p.rows && col < p.cols;
  uint32_t w[8][4];
  {
    const __nv_bfloat16* x = p.x + blockIdx.z * p.gstride + row * p.ldx + col;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (inside || (row + r < p.rows && col < p.cols)) v = __ldg(reinterpret_cast<const uint4*>(x));
      x += p.ldx;
      w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
    }
  }
  if (p.gamma != nullptr) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (row + r < p.rows && col < p.cols) {
        const float g = __bfloat162float(p.gamma[row + r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[r][i] = pack_bf16x2(g * bf16_lo(w[r][i]), g * bf16_hi(w[r][i]));
      }
    }
  }

  bool other = !inside;                 // than PLAIN
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m = w[0][i] & 0x7fff7fffu;
#pragma unroll
    for (int r = 1; r < 8; ++r) m = max2_nan(m, w[r][i] & 0x7fff7fffu);
    if (not_finite2(m)) {
      other = true;
      m = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) m = max2(m, finite2(w[r][i]));
    }
    part[rg][cg * 4 + i] = m;
  }
  const bool plain = __syncthreads_or(other) == 0;
  if (threadIdx.x < 64) {
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < 16; ++g) m = max2(m, part[g][threadIdx.x]);
    col_top[threadIdx.x] = m;
    if (!SQUARE && p.qt != nullptr) column_scales<FMT>(p, m);
  }
  __syncthreads();
  if (plain) write_tile<FMT, SQUARE, true>(p, w, col_top, bytes);
  else write_tile<FMT, SQUARE, false>(p, w, col_top, bytes);
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
  // Rows alone take the kernel without barriers: 16384 x 4096 in 33 us, 6.1 TB/s, against 35 for
  // the rows of square blocks and 37 for the columns alone, both of the tile kernel.
  if (d.block_rows == 1 && qt == nullptr) {
    const int64_t lines = (d.rows + 127) / 128 * 4;
    const bool most = lines > kMaxLines;
    const dim3 grid(static_cast<unsigned>(p.kt), static_cast<unsigned>(most ? kMaxLines : lines), G);
    if (most)
      return launch_grid(e4m3 ? quant_rows_kernel<BOOST_E4M3, true>
                              : quant_rows_kernel<BOOST_E5M2, true>, grid, stream, p);
    return launch_grid(e4m3 ? quant_rows_kernel<BOOST_E4M3, false>
                            : quant_rows_kernel<BOOST_E5M2, false>, grid, stream, p);
  }
  const dim3 grid(static_cast<unsigned>((d.cols + 127) / 128),
                  static_cast<unsigned>((d.rows + 127) / 128), G);
  if (d.block_rows == 128)
    return launch_grid(e4m3 ? quant_tile_kernel<BOOST_E4M3, true>
                            : quant_tile_kernel<BOOST_E5M2, true>, grid, stream, p);
  return launch_grid(e4m3 ? quant_tile_kernel<BOOST_E4M3, false>
                          : quant_tile_kernel<BOOST_E5M2, false>, grid, stream, p);
}

}  // namespace boost_gb300
