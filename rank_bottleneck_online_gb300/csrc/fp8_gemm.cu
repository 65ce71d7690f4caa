// fp8_gemm.cu -- out = act(row_scale (.) (A B^T)) for 8-bit operands with a power-of-two
// scale for each block of 128 along K.
//
// One thread an output element: the products of a block of 128 are summed in fp32 and
// joined with the block's two scales, 2^(ea + eb - 254), which is exact.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "internal.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

__device__ __forceinline__ float from8(uint8_t v, int fmt) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(v, fmt == BOOST_E4M3 ? __NV_E4M3 : __NV_E5M2);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ float scale_of(uint8_t byte) {
  if (byte == 255) return __uint_as_float(0x7fc00000u);
  return byte == 0 ? 0x1p-127f : __uint_as_float(static_cast<uint32_t>(byte) << 23);
}

__global__ void __launch_bounds__(kThreads) fp8_gemm_kernel(const Fp8GemmParams p) {
  pdl_enter();
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t n = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x & 15);
  const int64_t g = blockIdx.z;
  if (m >= p.d.M || n >= p.d.N) return;
  const uint8_t* a = p.a + (g * p.d.M + m) * p.d.a_pitch;
  const uint8_t* b = p.b + (g * p.d.N + n) * p.d.b_pitch;
  const uint8_t* sa = p.a_sf + g * scale_plane(p.d.M, p.d.K);
  const uint8_t* sb = p.b_sf + g * scale_plane(p.d.N, p.d.K);
  const int64_t kt = scale_tiles_k(p.d.K);
  float acc = 0.0f;
  for (int64_t k0 = 0; k0 < p.d.K; k0 += kScaleBlock) {
    float part = 0.0f;
    const int64_t end = min(k0 + kScaleBlock, p.d.K);
    for (int64_t k = k0; k < end; ++k)
      part = fmaf(from8(a[k], p.d.a_fmt), from8(b[k], p.d.b_fmt), part);
    acc += part * scale_of(sa[scale_at(m, k0 / kScaleBlock, kt)]) *
           scale_of(sb[scale_at(n, k0 / kScaleBlock, kt)]);
  }
  if (p.row_scale != nullptr) acc *= p.row_scale[m];
  if (p.d.act == BOOST_ACT_SILU) acc = act_fwd(acc, 1);
  static_cast<__nv_bfloat16*>(p.out)[(g * p.d.M + m) * p.d.N + n] = __float2bfloat16_rn(acc);
}

}  // namespace

size_t fp8_gemm_workspace(const boost_fp8_matmul_desc&) { return 256; }

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.d.M + 15) / 16), static_cast<unsigned>((p.d.N + 15) / 16),
                  static_cast<unsigned>(p.d.G));
  return launch_grid(fp8_gemm_kernel, grid, stream, p);
}

}  // namespace boost_gb300
