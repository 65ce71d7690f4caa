// attention.cuh -- what the attention kernels share: their parameters, the sequences' bounds and
// the launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "boost_ops.h"

namespace boost_gb300 {

// One [T, heads, dim] operand (strides in elements).
template <typename T>
struct Heads {
  T* at;
  int64_t ts, hs;
  __host__ __device__ __forceinline__ T* row(int64_t t, int64_t h) const {
    return at + t * ts + h * hs;
  }
};
using HeadsIn = Heads<const __nv_bfloat16>;
using HeadsOut = Heads<__nv_bfloat16>;

struct AttentionArgs {
  boost_attention_desc d;
  HeadsIn q, k, v, o, dout;              // o, dout: of the backward
  HeadsOut out, dq, dk, dv;
  float* lse;                            // [hq, Tq], or NULL in the forward
  const int32_t *q_starts, *k_starts;    // or NULL
  void* ws;                              // error word first
};

size_t attention_workspace(const boost_attention_desc& d);
cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t stream);
cudaError_t launch_attention_bwd(const AttentionArgs& a, cudaStream_t stream);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Bounds of sequence s: starts[s] and starts[s + 1] inside 0..T, and in order.
__device__ __forceinline__ void sequence_bounds(const int32_t* starts, int64_t T, int s,
                                                int32_t& at, int32_t& n) {
  if (starts == nullptr) {
    at = 0;
    n = static_cast<int32_t>(T);
    return;
  }
  const int32_t top = static_cast<int32_t>(T);
  at = min(max(starts[s], 0), top);
  n = max(min(max(starts[s + 1], 0), top) - at, 0);
}

}  // namespace boost_gb300
