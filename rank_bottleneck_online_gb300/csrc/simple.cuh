// simple.cuh -- what the CUDA-core kernels share: 16-byte bf16 vectors, the warp sum, the
// programmatic-dependent-launch entry and the launch helper.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "internal.h"

namespace boost_gb300 {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x);
  f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z);
  f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The first statement of every kernel launched with launch_k: wait for the kernel before
// it on the stream (a no-op unless the launch carried a programmatic dependency), then let
// the next one be scheduled. Both precede any global memory access.
__device__ __forceinline__ void pdl_enter() {
  griddep_wait();
  griddep_launch_dependents();
}

// Launch `kern` on `stream` with a grid of `grid` and blocks of kThreads, with the
// programmatic-stream-serialisation attribute when enabled.
template <typename... KArgs, typename... Args>
cudaError_t launch_grid(void (*kern)(KArgs...), dim3 grid, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kern)(KArgs...), int64_t grid, cudaStream_t stream, Args&&... args) {
  return launch_grid(kern, dim3(static_cast<unsigned>(grid), 1, 1), stream,
                     std::forward<Args>(args)...);
}

}  // namespace boost_gb300
