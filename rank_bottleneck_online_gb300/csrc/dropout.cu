// dropout.cu -- dropout of a branch added to its residual, with a mask regenerated from a
// counter and never stored.
//
// One Philox4x32-10 block (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011) gives the 16-bit draws of 8 elements, one 16-byte vector: 40
// instructions for the ten rounds (the rounds' keys are launch parameters) and about 15 an
// element in all. With a residual the pass is bound by HBM (6 bytes an element; 16384 x 4096:
// 57 us, 7.0 TB/s, the measured copy rate). The gradient moves 4 bytes an element and issue slots
// are 56% busy (8191 x 5120: 28 us, 6.0 TB/s, 88%), which is why a word gives two draws: with
// one, the rounds would cost twice as much and bind it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "boost_ops.h"
#include "internal.h"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct DropoutParams {
  const uint4* x;
  const uint4* res;            // or NULL
  uint4* out;
  const uint64_t* counter;     // or NULL
  int64_t count;
  uint64_t offset;
  uint32_t key[10][2];         // the seed's words, raised by the generator's steps each round
  uint32_t drop;               // 65536 times the draw below which an element is dropped
  float scale;                 // 65536 / (65536 - drop)
};

// The Philox4x32-10 block of vector g.
__device__ __forceinline__ void draw(const DropoutParams& p, uint64_t offset, int64_t g,
                                     uint32_t (&c)[4]) {
  c[0] = static_cast<uint32_t>(g);
  c[1] = static_cast<uint32_t>(g >> 32);
  c[2] = static_cast<uint32_t>(offset);
  c[3] = static_cast<uint32_t>(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
    const uint32_t n0 = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ p.key[r][0];
    const uint32_t n2 = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ p.key[r][1];
    c[1] = static_cast<uint32_t>(p1);
    c[3] = static_cast<uint32_t>(p0);
    c[0] = n0;
    c[2] = n2;
  }
}

// A word's two bf16 values with the dropped ones zero: a draw is compared as the upper half of
// a word, whose lower half cannot change the answer.
__device__ __forceinline__ uint32_t kept(uint32_t word, uint32_t c, uint32_t drop) {
  if (c << 16 < drop) word &= 0xffff0000u;
  if (c < drop) word &= 0xffffu;
  return word;
}

// Vectors in flight a thread. With 1 to 4 (and the keys still formed here) the gradient took
// 33.6, 30.2, 29.5, 29.5 us, a short batch (77 x 2048, both ways) 4.9, 4.9, 5.6, 6.3 us.
constexpr int kBatch = 2;

template <bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
  pdl_enter();
  const uint64_t offset = p.offset + (p.counter != nullptr ? *p.counter : 0);
  const int64_t vectors = p.count / 8;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kBatch * kThreads) + threadIdx.x;
  uint4 x[kBatch], r[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t g = first + b * kThreads;
    if (g < vectors) {
      x[b] = p.x[g];
      if (RES) r[b] = p.res[g];
    }
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t g = first + b * kThreads;
    if (g < vectors) {
      float f[8], s[8];
      uint32_t c[4];
      draw(p, offset, g, c);
      unpack8(make_uint4(kept(x[b].x, c[0], p.drop), kept(x[b].y, c[1], p.drop),
                         kept(x[b].z, c[2], p.drop), kept(x[b].w, c[3], p.drop)), f);
      if (RES) unpack8(r[b], s);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = RES ? fmaf(f[e], p.scale, s[e]) : f[e] * p.scale;
      p.out[g] = pack8(f);
    }
  }
  // the last, partly filled vector
  const int tail = static_cast<int>(p.count & 7);
  if (blockIdx.x == 0 && threadIdx.x < tail) {
    uint32_t c[4];
    draw(p, offset, vectors, c);
    const int j = threadIdx.x >> 1;
    const uint32_t word = j == 0 ? c[0] : j == 1 ? c[1] : j == 2 ? c[2] : c[3];
    const bool keep = (threadIdx.x & 1 ? word : word << 16) >= p.drop;
    const int64_t e = vectors * 8 + threadIdx.x;
    const float f = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.x)[e]);
    const float s = RES ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.res)[e]) : 0.0f;
    const float v = keep ? f : 0.0f;
    reinterpret_cast<__nv_bfloat16*>(p.out)[e] =
        __float2bfloat16_rn(RES ? fmaf(v, p.scale, s) : v * p.scale);
  }
}

// Two buffers of `bytes` each that overlap without being the same buffer.
bool partial_overlap(const void* a, const void* b, uint64_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && x < y + bytes && y < x + bytes;
}

}  // namespace

}  // namespace boost_gb300

using namespace boost_gb300;

extern "C" boost_status boost_dropout(int64_t count, const void* x, const void* res, void* out,
                                      double p, uint64_t seed, uint64_t offset,
                                      const uint64_t* counter, void* stream) {
  if (count < 0 || !(p >= 0.0 && p < 1.0)) return BOOST_ERR_INVALID_ARG;
  const double drop = std::floor(p * 65536.0 + 0.5);
  if (drop >= 65536.0 || (drop == 0.0 && p > 0.0)) return BOOST_ERR_INVALID_ARG;
  if (count > (int64_t{1} << 38)) return BOOST_ERR_UNSUPPORTED_SHAPE;   // 31 bits of blocks
  if (count == 0) return BOOST_OK;
  if (x == nullptr || out == nullptr) return BOOST_ERR_INVALID_ARG;
  for (const void* q : {x, res, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(q) & 15u) return BOOST_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(counter) & 7u) return BOOST_ERR_ALIGNMENT;
  const uint64_t bytes = 2ull * static_cast<uint64_t>(count);
  if (partial_overlap(x, out, bytes) || (res != nullptr && partial_overlap(res, out, bytes)))
    return BOOST_ERR_INVALID_ARG;
  const uintptr_t c = reinterpret_cast<uintptr_t>(counter), o = reinterpret_cast<uintptr_t>(out);
  if (counter != nullptr && c < o + bytes && o < c + 8) return BOOST_ERR_INVALID_ARG;

  DropoutParams d{};
  d.x = static_cast<const uint4*>(x);
  d.res = static_cast<const uint4*>(res);
  d.out = static_cast<uint4*>(out);
  d.counter = counter;
  d.count = count;
  for (uint32_t r = 0; r < 10; ++r) {
    d.key[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
    d.key[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
  }
  d.offset = offset;
  d.drop = static_cast<uint32_t>(drop) << 16;
  d.scale = static_cast<float>(65536.0 / (65536.0 - drop));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t grid = (count / 8 + kBatch * kThreads - 1) / (kBatch * kThreads);
  ProfScope ps(s, K_DROPOUT, 0.0, (res != nullptr ? 6.0 : 4.0) * count);
  const cudaError_t e =
      launch_k(res != nullptr ? dropout_kernel<true> : dropout_kernel<false>, grid < 1 ? 1 : grid,
               s, d);
  return e == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}
