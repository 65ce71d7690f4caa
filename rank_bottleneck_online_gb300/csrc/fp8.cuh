// fp8.cuh -- 8-bit operands with a power-of-two scale for each block of 128: the layout of
// their scales, and the kernels' launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "boost_ops.h"

namespace boost_gb300 {

constexpr int kScaleBlock = 128;        // values of K that share a scale
constexpr int kScaleTile = 512;         // bytes of the scales of 128 rows x 4 blocks

// Tiles of 4 blocks along K.
__host__ __device__ __forceinline__ int64_t scale_tiles_k(int64_t K) {
  return (K + 4 * kScaleBlock - 1) / (4 * kScaleBlock);
}

// Bytes of one plane of scales.
__host__ __device__ __forceinline__ int64_t scale_plane(int64_t rows, int64_t K) {
  return (rows + 127) / 128 * scale_tiles_k(K) * kScaleTile;
}

// Offset of the scale of row r, block b in a plane whose rows hold kt tiles.
__host__ __device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t kt) {
  return ((r >> 7) * kt + (b >> 2)) * kScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

cudaError_t launch_fp8_quantize(const boost_fp8_quant_desc& d, const void* x, const void* gamma,
                                void* q, void* sf, void* qt, void* sft, cudaStream_t stream);

struct Fp8GemmParams {
  boost_fp8_matmul_desc d;
  const uint8_t *a, *a_sf, *b, *b_sf;
  const float* row_scale;
  void* out;
  void* ws;                             // the workspace, error word first
};

size_t fp8_gemm_workspace(const boost_fp8_matmul_desc& d);
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, cudaStream_t stream);

}  // namespace boost_gb300
