// attention_bwd.cu -- gradients of attention, one warp a row of dq or of dk and dv.
#include <math_constants.h>

#include "attention.cuh"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct SimpleBwdParams {
  AttentionArgs a;
  float* delta;                          // [hq, Tq]
};

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

__global__ void __launch_bounds__(kThreads) attention_dq_row_kernel(const SimpleBwdParams p) {
  pdl_enter();
  const AttentionArgs& a = p.a;
  const int lane = threadIdx.x & 31, dim = a.d.dim;
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
  const float delta = dot(a.dout.row(t, h), a.o.row(t, h), dim), lse = a.lse[h * a.d.Tq + t];
  if (lane == 0) p.delta[h * a.d.Tq + t] = delta;
  float g[4] = {};
  for (int64_t j0 = 0; j0 < sees; j0 += 32) {
    float ds = 0.0f;
    if (j0 + lane < sees) {
      const float w = __expf(a.d.scale * dot(a.q.row(t, h), a.k.row(k0 + j0 + lane, hk), dim) - lse);
      ds = w * (dot(a.dout.row(t, h), a.v.row(k0 + j0 + lane, hk), dim) - delta);
    }
    for (int j = 0; j < 32 && j0 + j < sees; ++j) {
      const float d = __shfl_sync(0xffffffffu, ds, j);
      const __nv_bfloat16* k = a.k.row(k0 + j0 + j, hk);
      for (int i = 0; i < 4; ++i)
        if (i * 32 + lane < dim) g[i] = fmaf(d, __bfloat162float(k[i * 32 + lane]), g[i]);
    }
  }
  for (int i = 0; i < 4; ++i)
    if (i * 32 + lane < dim) a.dq.row(t, h)[i * 32 + lane] = __float2bfloat16_rn(g[i] * a.d.scale);
}

__global__ void __launch_bounds__(kThreads) attention_dkv_row_kernel(const SimpleBwdParams p) {
  pdl_enter();
  const AttentionArgs& a = p.a;
  const int lane = threadIdx.x & 31, dim = a.d.dim;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / a.d.hk;
  const int hk = static_cast<int>(item % a.d.hk), group = a.d.hq / a.d.hk;
  if (t >= a.d.Tk) return;
  const int s = sequence_of(a.k_starts, a.d.sequences, a.d.Tk, t);
  if (s < 0) return;
  int32_t q0, nq, k0, nk;
  sequence_bounds(a.q_starts, a.d.Tq, s, q0, nq);
  sequence_bounds(a.k_starts, a.d.Tk, s, k0, nk);
  const int64_t first = a.d.causal ? max(static_cast<int64_t>(0), t - k0 - (nk - nq)) : 0;
  float gk[4] = {}, gv[4] = {};
  for (int h = hk * group; h < (hk + 1) * group; ++h)
    for (int64_t i0 = first; i0 < nq; i0 += 32) {
      float w = 0.0f, ds = 0.0f;
      if (i0 + lane < nq) {
        const int64_t q = q0 + i0 + lane;
        w = __expf(a.d.scale * dot(a.q.row(q, h), a.k.row(t, hk), dim) - a.lse[h * a.d.Tq + q]);
        ds = w * (dot(a.dout.row(q, h), a.v.row(t, hk), dim) - p.delta[h * a.d.Tq + q]);
      }
      for (int j = 0; j < 32 && i0 + j < nq; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j), dj = __shfl_sync(0xffffffffu, ds, j);
        for (int i = 0; i < 4; ++i)
          if (i * 32 + lane < dim) {
            gv[i] = fmaf(wj, __bfloat162float(a.dout.row(q0 + i0 + j, h)[i * 32 + lane]), gv[i]);
            gk[i] = fmaf(dj, __bfloat162float(a.q.row(q0 + i0 + j, h)[i * 32 + lane]), gk[i]);
          }
      }
    }
  for (int i = 0; i < 4; ++i)
    if (i * 32 + lane < dim) {
      a.dk.row(t, hk)[i * 32 + lane] = __float2bfloat16_rn(gk[i] * a.d.scale);
      a.dv.row(t, hk)[i * 32 + lane] = __float2bfloat16_rn(gv[i]);
    }
}

}  // namespace

cudaError_t launch_attention_bwd(const AttentionArgs& a, cudaStream_t stream) {
  SimpleBwdParams p{a, reinterpret_cast<float*>(static_cast<char*>(a.ws) + 256)};
  if (a.d.Tq > 0) {
    const cudaError_t e = launch_k(attention_dq_row_kernel, (a.d.Tq * a.d.hq + 7) / 8, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (a.d.Tk == 0) return cudaSuccess;
  return launch_k(attention_dkv_row_kernel, (a.d.Tk * a.d.hk + 7) / 8, stream, p);
}

}  // namespace boost_gb300
