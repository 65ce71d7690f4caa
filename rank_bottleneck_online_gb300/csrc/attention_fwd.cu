// attention_fwd.cu -- softmax attention over packed sequences, one warp a row.
#include <math_constants.h>

#include "attention.cuh"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct SimpleParams {
  AttentionArgs a;
};

// Sequence that row t lies in (the last whose start is not behind it), or -1.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int n, int64_t T, int64_t t) {
  if (starts == nullptr) return t < T ? 0 : -1;
  for (int s = 0; s < n; ++s)
    if (t >= starts[s] && t < min(static_cast<int64_t>(starts[s + 1]), T)) return s;
  return -1;
}

__device__ __forceinline__ float dot(const __nv_bfloat16* a, const __nv_bfloat16* b, int dim) {
  float s = 0.0f;
  for (int e = 0; e < dim; e += 8) {
    float x[8], y[8];
    unpack8(*reinterpret_cast<const uint4*>(a + e), x);
    unpack8(*reinterpret_cast<const uint4*>(b + e), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  }
  return s;
}

__global__ void __launch_bounds__(kThreads) attention_row_kernel(const SimpleParams p) {
  pdl_enter();
  const AttentionArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / a.d.hq;
  const int h = static_cast<int>(item % a.d.hq);
  if (t >= a.d.Tq) return;
  const int s = sequence_of(a.q_starts, a.d.sequences, a.d.Tq, t);
  if (s < 0) return;
  int32_t q0, nq, k0, nk;
  sequence_bounds(a.q_starts, a.d.Tq, s, q0, nq);
  sequence_bounds(a.k_starts, a.d.Tk, s, k0, nk);
  const int64_t sees = a.d.causal ? min(static_cast<int64_t>(nk), t - q0 + 1 + nk - nq) : nk;
  const int hk = h / (a.d.hq / a.d.hk);
  float m = -CUDART_INF_F, l = 0.0f, o[4] = {};
  for (int64_t j0 = 0; j0 < sees; j0 += 32) {
    const bool in = j0 + lane < sees;
    const float x = in ? a.d.scale * dot(a.q.row(t, h), a.k.row(k0 + j0 + lane, hk), a.d.dim) : -CUDART_INF_F;
    float top = x;
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float next = fmaxf(m, top), f = m == -CUDART_INF_F ? 0.0f : __expf(m - next);
    const float w = in ? __expf(x - next) : 0.0f;
    l = l * f + warp_sum(w);
    m = next;
    for (int i = 0; i < 4; ++i) o[i] *= f;
    for (int j = 0; j < 32 && j0 + j < sees; ++j) {
      const float pj = __shfl_sync(0xffffffffu, w, j);
      const __nv_bfloat16* v = a.v.row(k0 + j0 + j, hk);
      for (int i = 0; i < 4; ++i)
        if (i * 32 + lane < a.d.dim) o[i] = fmaf(pj, __bfloat162float(v[i * 32 + lane]), o[i]);
    }
  }
  for (int i = 0; i < 4; ++i)
    if (i * 32 + lane < a.d.dim)
      a.out.row(t, h)[i * 32 + lane] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[i] / l);
  if (lane == 0 && a.lse != nullptr) a.lse[h * a.d.Tq + t] = m + logf(l);
}

}  // namespace

size_t attention_workspace(const boost_attention_desc& d) {
  return 256 + 8 * static_cast<size_t>(d.hq) * d.Tq;
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t stream) {
  return launch_k(attention_row_kernel, (a.d.Tq * a.d.hq + 7) / 8, stream, SimpleParams{a});
}

}  // namespace boost_gb300
