// norm_quant.cu -- the residual's addition, the row scale of the root-mean-square norm behind it
// and the sum in 8 bits, from one reading.
//
// The norm's 1 / rms is a factor of the row and the 8-bit product applies it in its epilogue, so
// that a block's scale depends on its 128 values alone and nothing waits for the row's sum. A
// lane holds 16 values of two rows, a warp 512 columns (four scale bytes, one word of the scales'
// layout); the warps of a row join their sums of squares in shared memory, in a fixed order. The
// pass moves 4 bytes in and 3 out a value and is bound by HBM: 16384 x 4096 takes 72 us (6.5 TB/s).
// Without a residual the issue rate counts too: 8191 x 5120 with weights, e5m2, 31 us (4.1 TB/s; 66% of
// the issue slots).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "boost_ops.h"
#include "fp8.cuh"
#include "fp8_values.cuh"
#include "internal.h"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct NormQuantParams {
  const __nv_bfloat16 *x, *res, *gamma;  // res, gamma or NULL
  __nv_bfloat16* h;                      // or NULL
  float* rstd;
  uint8_t *q, *sf;
  int64_t T, d, pitch, kt;
  int32_t warps;                         // of a row
  float eps;
};

constexpr int kRows = 2;                 // of a warp
// Warps of a block at most. (A residual's values take registers: 80 a thread in three blocks of
// eight warps an SM, 16384 x 4096 in 71 us; 64 in blocks of up to sixteen, 75 us, and 128, 85 us.)
constexpr int most_warps(bool residual) { return residual ? 8 : 16; }

__device__ __forceinline__ void words_of(const uint4& v, uint32_t* w) {
  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}

// Squares of two values added to two sums, in one instruction.
__device__ __forceinline__ float2 square_sum2(float a, float b, float2 s) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "fma.rn.f32x2 y, x, x, y;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(s.x), "f"(s.y));
  return r;
}

// x + residual of 8 values, rounded once.
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  float x[8], y[8];
  unpack8(a, x);
  unpack8(b, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] += y[e];
  return pack8(x);
}

// gamma h of 8 values, rounded once (a product of two bf16 values is exact before that).
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

__device__ __forceinline__ uint4 mul8(const uint4& a, const uint4& b) {
  return make_uint4(mul2_bf16(a.x, b.x), mul2_bf16(a.y, b.y), mul2_bf16(a.z, b.z),
                    mul2_bf16(a.w, b.w));
}

template <int FMT, bool RES>
__global__ void __launch_bounds__(32 * most_warps(RES), RES ? 3 : 2)
    norm_quant_kernel(const NormQuantParams p) {
  pdl_enter();
  __shared__ float sums[most_warps(RES)][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % p.warps, lines = blockDim.x / 32 / p.warps;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * lines + warp / p.warps) * kRows;
  const int rows = static_cast<int>(min(max(p.T - row0, static_cast<int64_t>(0)),
                                        static_cast<int64_t>(kRows)));
  float2 sum[kRows] = {};
  const int64_t tiles = p.kt;                          // of 512 columns
  const int64_t first_at = row0 * p.d + lane * 16;
  for (int64_t tile = part; tile < tiles; tile += p.warps) {
    const int64_t col = tile * 512 + lane * 16;
    // (d is a multiple of 8: a lane's second vector may lie behind the columns, or both)
    const bool in[2] = {col < p.d, col + 8 < p.d};
    const int64_t at = first_at + tile * 512;
    uint4 v[kRows][2], r[RES ? kRows : 1][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        v[i][k] = make_uint4(0, 0, 0, 0);
        if (RES) r[i][k] = v[i][k];
        if (i < rows && in[k]) {
          v[i][k] = *reinterpret_cast<const uint4*>(p.x + at + i * p.d + 8 * k);
          if (RES) r[i][k] = *reinterpret_cast<const uint4*>(p.res + at + i * p.d + 8 * k);
        }
      }
    uint4 g[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (p.gamma != nullptr && in[k])
        g[k] = __ldg(reinterpret_cast<const uint4*>(p.gamma + col + 8 * k));
    uint32_t w[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (RES) v[i][k] = add8(v[i][k], r[i][k]);
        words_of(v[i][k], w[i] + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[i] = square_sum2(bf16_lo(w[i][4 * k + e]), bf16_hi(w[i][4 * k + e]), sum[i]);
        if (p.h != nullptr && i < rows && in[k])
          *reinterpret_cast<uint4*>(p.h + at + i * p.d + 8 * k) = v[i][k];
        if (p.gamma != nullptr) words_of(mul8(v[i][k], g[k]), w[i] + 4 * k);
      }
    }
    uint32_t top[kRows];
    const bool mend = block_tops<kRows, 8, 8>(w, top);
    const int64_t first = tile * 4;                    // block of lane 0
    const bool in_cols = first + (lane >> 3) < (p.d + 127) / 128;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t byte = scale_byte<FMT>(top[i]);
      if (i < rows && col < p.pitch) {
        const float inv = scale_inverse(byte);
        const uint2 a = quant8<FMT>(w[i], inv, mend), b = quant8<FMT>(w[i] + 4, inv, mend);
        *reinterpret_cast<uint4*>(p.q + (row0 + i) * p.pitch + col) = make_uint4(a.x, a.y, b.x, b.y);
      }
      uint32_t word = static_cast<uint32_t>(stored_byte(byte, top[i], in_cols && i < rows))
                      << (lane & 24);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      word |= __shfl_xor_sync(0xffffffffu, word, 16);
      // (the scales of rows behind the last, up to a whole row tile, are 127)
      if (lane == 0 && row0 + i < (p.T + 127) / 128 * 128)
        *reinterpret_cast<uint32_t*>(p.sf + scale_at(row0 + i, first, p.kt)) = word;
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float all = warp_sum(sum[i].x + sum[i].y);
    if (lane == 0) sums[warp][i] = all;
  }
  __syncthreads();
  if (part == 0 && lane < kRows && row0 + lane < p.T) {
    float total = 0.0f;
    for (int i = 0; i < p.warps; ++i) total += sums[warp + i][lane];
    p.rstd[row0 + lane] = 1.0f / sqrtf(total / static_cast<float>(p.d) + p.eps);
  }
}

bool meets(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != 0 && y != 0 && x < y + nb && y < x + na;
}

}  // namespace

}  // namespace boost_gb300

using namespace boost_gb300;

extern "C" boost_status boost_norm_quantize(int64_t T, int64_t d, int32_t fmt, float eps,
                                            const void* x, const void* residual,
                                            const void* gamma, void* h, float* rstd, void* q,
                                            void* sf, void* stream) {
  if (T < 0 || d < 1 || (fmt != BOOST_E4M3 && fmt != BOOST_E5M2) || !(eps >= 0.0f))
    return BOOST_ERR_INVALID_ARG;
  if (d % 8) return BOOST_ERR_UNSUPPORTED_SHAPE;
  // the grid stays within 31 bits, offsets within 50
  if (T > 0x7fffffff || d > (int64_t{1} << 24)) return BOOST_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return BOOST_OK;
  if (x == nullptr || rstd == nullptr || q == nullptr || sf == nullptr)
    return BOOST_ERR_INVALID_ARG;
  for (const void* p : {x, residual, gamma, static_cast<const void*>(h),
                        static_cast<const void*>(rstd), static_cast<const void*>(q),
                        static_cast<const void*>(sf)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return BOOST_ERR_ALIGNMENT;
  NormQuantParams p{};
  p.pitch = (d + 15) / 16 * 16;
  p.kt = scale_tiles_k(d);
  const uint64_t bytes = 2ull * T * d;
  struct { const void* at; uint64_t n; } out[] = {
      {h, bytes}, {rstd, 4ull * T}, {q, static_cast<uint64_t>(T) * p.pitch},
      {sf, static_cast<uint64_t>(scale_plane(T, d))}}, in[] = {
      {x, bytes}, {residual, bytes}, {gamma, 2ull * d}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (!(i == 0 && j < 2 && out[i].at == in[j].at) && meets(out[i].at, out[i].n, in[j].at, in[j].n))
        return BOOST_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meets(out[i].at, out[i].n, out[j].at, out[j].n)) return BOOST_ERR_INVALID_ARG;
  }
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.res = static_cast<const __nv_bfloat16*>(residual);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.h = static_cast<__nv_bfloat16*>(h);
  p.rstd = rstd;
  p.q = static_cast<uint8_t*>(q);
  p.sf = static_cast<uint8_t*>(sf);
  p.T = T;
  p.d = d;
  p.eps = eps;
  // A warp for each of a row's tiles, if a block can have as many: then nobody waits for a turn's
  // loads after another's; else as few turns as that takes, shared evenly. Blocks of eight warps
  // where rows are short. (8191 x 5120, ten tiles: eight warps in two turns took 43 us.)
  const bool res = residual != nullptr;
  const int64_t turns = (p.kt + most_warps(res) - 1) / most_warps(res);
  p.warps = static_cast<int32_t>((p.kt + turns - 1) / turns);
  const int lines = p.warps >= 8 ? 1 : 8 / p.warps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double n = static_cast<double>(T) * d;
  ProfScope ps(s, K_NORM_QUANT, 0.0,
               n * (2.0 + (residual ? 2.0 : 0.0) + (h ? 2.0 : 0.0) + 129.0 / 128.0));
  const auto kern = fmt == BOOST_E4M3
      ? (res ? norm_quant_kernel<BOOST_E4M3, true> : norm_quant_kernel<BOOST_E4M3, false>)
      : (res ? norm_quant_kernel<BOOST_E5M2, true> : norm_quant_kernel<BOOST_E5M2, false>);
  const int64_t block_rows = lines * kRows;
  const int64_t grid = ((T + 127) / 128 * 128 + block_rows - 1) / block_rows;
  const cudaError_t e = launch_blocks(kern, dim3(static_cast<unsigned>(grid), 1, 1),
                                      dim3(32 * p.warps * lines, 1, 1), s, p);
  return e == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}
