// grad_clip.cu -- the norm over a model's gradients and their scaling to it.
//
// Two passes over the gradients. The first leaves one sum of squares a block in the workspace;
// every block of the second adds those up, in the same order, and has the norm without a launch
// between. The first pass goes through the gradients from front to back, the second from back to
// front, so that what the first read last is still in L2. A table of the tensors travels in the
// launch parameters; more tensors than fit take more launches, which add to the same sums.
// Squares are summed in fp32 over a thread's 32 values and in fp64 beyond, so that many small
// ones do not vanish beside the sum; a thread whose 32 leave fp32's range takes them again in fp64
// (at 1.25 TFLOP/s all of a layer's 125 million values would take 0.2 ms). A sum of 0 may be squares
// too small for fp32, or zeros (rows of an embedding that no token has): the values' bits tell, and
// zeros are not read again. (125 million of them: 60 us, as any values; read again one by one 510.
// Bits taken only where a sum is 0 kept the values in registers: 48 in place of 32, 64 us.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "boost_ops.h"
#include "internal.h"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

// Eight an SM, and as many sums in the workspace. (125 million bf16 values: 132 us, of which the first
// pass takes 46, at 70% of HBM's peak, and the second 84; with four an SM 161.) Adding up the sums is
// what small calls wait for: 6.3 million values take 27 us, in a replayed graph too, with the fp64 pipe
// busy for 70% of the first pass and 75% of the second.
constexpr int kBlocks = 1216;
constexpr int kChunk = 8192;             // elements of one block's step

// The tensors of one launch: 28 bytes each, in the 4 KB of parameters that any launch may have, or,
// for more of them, in the 32 KB of a large one.
constexpr int kFew = 120, kMany = 1100;

template <int kTensors>
struct ClipParams {
  const void* g[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  uint32_t end[kTensors];                // chunks up to and with this tensor's
  uint32_t wide[(kTensors + 31) / 32];
  int32_t tensors, first;                // first: the sums begin here
  double* sums;
  float* norm;                           // of the last scaling launch, or NULL
  double max_norm;
};
static_assert(sizeof(ClipParams<kFew>) <= 4096 && sizeof(ClipParams<kMany>) <= 32764, "parameters");

// The tensor of a chunk, and the chunk's place in it.
template <int N>
__device__ __forceinline__ int tensor_of(const ClipParams<N>& p, uint32_t chunk, int64_t& at) {
  int lo = 0, hi = p.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (chunk < p.end[mid]) hi = mid; else lo = mid + 1;
  }
  at = static_cast<int64_t>(chunk - (lo == 0 ? 0 : p.end[lo - 1])) * kChunk;
  return lo;
}

template <int N>
__device__ __forceinline__ bool is_wide(const ClipParams<N>& p, int t) {
  return p.wide[t >> 5] >> (t & 31) & 1u;
}

// Sum over the block's threads, in a fixed order, for all of them.
__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kThreads / 32; ++i) v += shared[i];
  return v;
}

// Whether fp32 holds a sum of squares: not beyond its range (or NaN), and no square that counts
// has lost bits below 2^-126.
__device__ __forceinline__ bool holds(float sum) { return sum >= 0x1p-90f && sum < CUDART_INF_F; }

// This thread's squares of a chunk in fp64, `V` values side by side where the chunk is whole.
template <int V, typename T>
__device__ __noinline__ double squares64(const T* g, int n) {
  const int side = n == kChunk ? V : 1;
  double sum = 0.0;
  for (int i = threadIdx.x * side; i < n; i += kThreads * side)
    for (int e = 0; e < side; ++e) {
      const double x = static_cast<double>(static_cast<float>(g[i + e]));
      if (x != 0.0) sum = fma(x, x, sum);
    }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ ClipParams<N> p) {
  pdl_enter();
  __shared__ double shared[kThreads / 32];
  double sum = 0.0;
  const uint32_t chunks = p.end[p.tensors - 1];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    int64_t at;
    const int t = tensor_of(p, c, at);
    const int64_t n = min(p.n[t] - at, static_cast<int64_t>(kChunk));
    float s0 = 0.0f, s1 = 0.0f;
    uint32_t bits = 0u;                    // of this thread's magnitudes
    if (is_wide(p, t)) {
      const float* g = static_cast<const float*>(p.g[t]) + at;
      if (n == kChunk) {
        float4 v[kChunk / 4 / kThreads];
#pragma unroll
        for (int i = 0; i < kChunk / 4 / kThreads; ++i)
          v[i] = __ldg(reinterpret_cast<const float4*>(g) + i * kThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kChunk / 4 / kThreads; ++i) {
          s0 = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, s0));
          s1 = fmaf(v[i].z, v[i].z, fmaf(v[i].w, v[i].w, s1));
          bits |= __float_as_uint(v[i].x) | __float_as_uint(v[i].y);
          bits |= __float_as_uint(v[i].z) | __float_as_uint(v[i].w);
        }
      } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          s0 = fmaf(g[i], g[i], s0);
          bits |= __float_as_uint(g[i]);
        }
      }
      bits &= 0x7fffffffu;
    } else {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(p.g[t]) + at;
      if (n == kChunk) {
        uint4 v[kChunk / 8 / kThreads];
#pragma unroll
        for (int i = 0; i < kChunk / 8 / kThreads; ++i)
          v[i] = __ldg(reinterpret_cast<const uint4*>(g) + i * kThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kChunk / 8 / kThreads; ++i) {
          float f[8];
          unpack8(v[i], f);
          bits |= v[i].x | v[i].y;
          bits |= v[i].z | v[i].w;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            s0 = fmaf(f[e], f[e], s0);
            s1 = fmaf(f[e + 1], f[e + 1], s1);
          }
        }
      } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const float f = __bfloat162float(g[i]);
          s0 = fmaf(f, f, s0);
          bits |= __float_as_uint(f);
        }
      }
      bits &= 0x7fff7fffu;
    }
    if (holds(s0 + s1))
      sum += static_cast<double>(s0) + static_cast<double>(s1);
    else if (bits == 0u)
      continue;                            // (zeros, of either sign)
    else if (is_wide(p, t))
      sum += squares64<4>(static_cast<const float*>(p.g[t]) + at, static_cast<int>(n));
    else
      sum += squares64<8>(static_cast<const __nv_bfloat16*>(p.g[t]) + at, static_cast<int>(n));
  }
  sum = block_sum(sum, shared);
  if (threadIdx.x == 0) p.sums[blockIdx.x] = (p.first ? 0.0 : p.sums[blockIdx.x]) + sum;
}

// What scales. A factor below fp32's normal numbers would have few bits, or none: then the values go
// down first, by a power of two, which is exact for all that do not become 0, and the factor goes
// up. (By its exponent's bits: fp64 instructions are what small calls wait for.)
struct Factor {
  float down, f;
  __device__ __forceinline__ explicit Factor(double by) {
    const int hi = __double2hiint(by), exponent = (hi >> 20 & 0x7ff) - 1023;
    const int up = exponent < -180 ? 149 : exponent < -100 ? 64 : 0;
    down = up == 149 ? 0x1p-149f : up == 64 ? 0x1p-64f : 1.0f;
    f = static_cast<float>(__hiloint2double(hi + (up << 20), __double2loint(by)));
  }
  template <int N>
  __device__ __forceinline__ void operator()(float (&x)[N]) const {
    if (down != 1.0f) {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= down;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] *= f;
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ ClipParams<N> p) {
  pdl_enter();
  __shared__ double shared[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < kBlocks; i += kThreads) sum += p.sums[i];
  const double norm = sqrt(block_sum(sum, shared));
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.norm != nullptr) *p.norm = static_cast<float>(norm);
  const double by = p.max_norm / (norm + 1e-6);
  const bool whole = by >= 1.0;            // (a NaN scales)
  const Factor scale(whole ? 1.0 : by);
  const uint32_t chunks = p.tensors > 0 ? p.end[p.tensors - 1] : 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    int64_t at;
    const int t = tensor_of(p, chunks - 1 - c, at);
    if (p.out[t] == nullptr || (whole && p.out[t] == p.g[t])) continue;
    const int64_t n = min(p.n[t] - at, static_cast<int64_t>(kChunk));
    if (is_wide(p, t)) {
      const float* g = static_cast<const float*>(p.g[t]) + at;
      float* out = static_cast<float*>(p.out[t]) + at;
      if (n == kChunk) {
        float4 v[kChunk / 4 / kThreads];
#pragma unroll
        for (int i = 0; i < kChunk / 4 / kThreads; ++i)
          v[i] = *(reinterpret_cast<const float4*>(g) + i * kThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kChunk / 4 / kThreads; ++i) {
          float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          scale(x);
          __stcs(reinterpret_cast<float4*>(out) + i * kThreads + threadIdx.x,
                 make_float4(x[0], x[1], x[2], x[3]));
        }
      } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          float x[1] = {g[i]};
          scale(x);
          out[i] = x[0];
        }
      }
    } else {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(p.g[t]) + at;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[t]) + at;
      if (n == kChunk) {
        uint4 v[kChunk / 8 / kThreads];
#pragma unroll
        for (int i = 0; i < kChunk / 8 / kThreads; ++i)
          v[i] = *(reinterpret_cast<const uint4*>(g) + i * kThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kChunk / 8 / kThreads; ++i) {
          float x[8];
          unpack8(v[i], x);
          scale(x);
          __stcs(reinterpret_cast<uint4*>(out) + i * kThreads + threadIdx.x, pack8(x));
        }
      } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          float x[1] = {__bfloat162float(g[i])};
          scale(x);
          out[i] = __float2bfloat16_rn(x[0]);
        }
      }
    }
  }
}

struct Span {
  uintptr_t at, end;
  bool output;
};

// Whether an output shares a byte with another tensor (its own g apart).
bool outputs_meet(const boost_grad* grads, int64_t count) {
  std::vector<Span> spans;
  spans.reserve(2 * static_cast<size_t>(count));
  for (int64_t i = 0; i < count; ++i) {
    const uintptr_t bytes = static_cast<uintptr_t>(grads[i].n) * (grads[i].wide ? 4 : 2);
    if (bytes == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i].g);
    const uintptr_t o = reinterpret_cast<uintptr_t>(grads[i].out);
    spans.push_back({g, g + bytes, o == g});
    if (o != 0 && o != g) spans.push_back({o, o + bytes, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
  uintptr_t any = 0, written = 0;          // how far the spans so far reach
  for (const Span& s : spans) {
    if (s.at < written || (s.output && s.at < any)) return true;
    any = std::max(any, s.end);
    if (s.output) written = std::max(written, s.end);
  }
  return false;
}

// The two passes over the tensors, N of them a launch.
template <int N>
cudaError_t launch(int64_t count, const boost_grad* grads, double max_norm, float* norm, double* sums,
                   cudaStream_t s) {
  std::vector<ClipParams<N>> launches;
  for (int64_t i = 0; i < count; ++i) {
    if (grads[i].n == 0) continue;
    if (launches.empty() || launches.back().tensors == N) {
      launches.emplace_back();
      ClipParams<N>& p = launches.back();
      std::fill(std::begin(p.wide), std::end(p.wide), 0u);
      p.tensors = 0;
      p.sums = sums;
      p.max_norm = max_norm;
      p.norm = nullptr;
      p.first = launches.size() == 1;
    }
    ClipParams<N>& p = launches.back();
    const int t = p.tensors++;
    p.g[t] = grads[i].g;
    p.out[t] = grads[i].out;
    p.n[t] = grads[i].n;
    p.end[t] = (t == 0 ? 0 : p.end[t - 1]) +
               static_cast<uint32_t>((grads[i].n + kChunk - 1) / kChunk);
    if (grads[i].wide) p.wide[t >> 5] |= 1u << (t & 31);
  }
  if (launches.empty()) {
    prof_note_kernels(-1);
    return cudaMemsetAsync(norm, 0, 4, s);
  }
  // (every launch of the first pass has all blocks: each leaves its sum)
  for (const ClipParams<N>& p : launches) {
    const cudaError_t e = launch_k(grad_norm_kernel<N>, kBlocks, s, p);
    if (e != cudaSuccess) return e;
  }
  launches.front().norm = norm;            // the last of the second pass
  int kernels = static_cast<int>(launches.size());
  for (size_t i = launches.size(); i-- > 0;) {
    ClipParams<N>& p = launches[i];
    const bool writes = std::any_of(p.out, p.out + p.tensors, [](void* q) { return q != nullptr; });
    if (!writes && i > 0) continue;
    if (!writes) p.tensors = 0;
    const int64_t grid = p.tensors == 0 ? 1 : std::min<int64_t>(p.end[p.tensors - 1], kBlocks);
    const cudaError_t e = launch_k(grad_scale_kernel<N>, grid, s, p);
    if (e != cudaSuccess) return e;
    ++kernels;
  }
  prof_note_kernels(kernels - 1);
  return cudaSuccess;
}

}  // namespace

}  // namespace boost_gb300

using namespace boost_gb300;

extern "C" {

size_t boost_grad_clip_workspace_bytes(void) { return 256 + sizeof(double) * kBlocks; }

boost_status boost_grad_clip(int64_t count, const boost_grad* grads, double max_norm, float* norm,
                             void* ws, size_t ws_bytes, void* stream) try {
  if (count < 0 || (count > 0 && grads == nullptr) || !(max_norm >= 0.0) || norm == nullptr)
    return BOOST_ERR_INVALID_ARG;
  if (count > (1 << 24)) return BOOST_ERR_UNSUPPORTED_SHAPE;
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return BOOST_ERR_ALIGNMENT;
  double values = 0.0, bytes = 0.0;
  for (int64_t i = 0; i < count; ++i) {
    const boost_grad& t = grads[i];
    if (t.n < 0 || (t.wide != 0 && t.wide != 1) || (t.n > 0 && t.g == nullptr))
      return BOOST_ERR_INVALID_ARG;
    if (t.n > (int64_t{1} << 40)) return BOOST_ERR_UNSUPPORTED_SHAPE;
    if ((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & 15u)
      return BOOST_ERR_ALIGNMENT;
    values += static_cast<double>(t.n);
    bytes += static_cast<double>(t.n) * (t.wide ? 4 : 2) * (t.out ? 2 : 1);
  }
  if (values > 0x1p44) return BOOST_ERR_UNSUPPORTED_SHAPE;   // 31 bits of chunks
  const size_t need = boost_grad_clip_workspace_bytes();
  const uintptr_t w = reinterpret_cast<uintptr_t>(ws), o = reinterpret_cast<uintptr_t>(norm);
  if (ws == nullptr || (w & 255u) || ws_bytes < need) return BOOST_ERR_WORKSPACE;
  if (o < w + need && w < o + 4) return BOOST_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    const uintptr_t n = static_cast<uintptr_t>(grads[i].n) * (grads[i].wide ? 4 : 2);
    for (const void* t : {grads[i].g, static_cast<const void*>(grads[i].out)}) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(t);
      if (t != nullptr && ((a < w + need && w < a + n) || (a < o + 4 && o < a + n)))
        return BOOST_ERR_INVALID_ARG;
    }
  }
  if (outputs_meet(grads, count)) return BOOST_ERR_INVALID_ARG;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, K_GRAD_CLIP, 3.0 * values, bytes);
  double* sums = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  const cudaError_t e = count <= kFew ? launch<kFew>(count, grads, max_norm, norm, sums, s)
                                      : launch<kMany>(count, grads, max_norm, norm, sums, s);
  return e == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
} catch (...) {
  return BOOST_ERR_CUDA;                   // (host memory for the tables)
}

}  // extern "C"
