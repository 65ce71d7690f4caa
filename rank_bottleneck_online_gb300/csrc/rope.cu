// rope.cu -- rotary positions of q and k with one or more position axes, and their inverse.
//
// Per token and pair one angle serves every head, so a block first forms the cosines and
// sines of its tokens in shared memory (one (token, pair) a thread) and then streams the
// heads through 16-byte vectors, the next ones in flight while the last are turned. The pass is
// bound by HBM: 4 bytes of traffic a value and 3 fp32 operations (16384 tokens of 32 + 32 heads
// of 128: 82 us, 6.5 TB/s, 96% of the measured copy rate).
//
// The angle: phi = p w with p a 64-bit integer and w an fp64 frequency. In turns,
// p w / (2 pi) mod 1 is wanted. F = floor(2^64 w / (2 pi)) mod 2^64 holds the frequency as a
// 64-bit fixed-point fraction of a turn, and p F mod 2^64, the integer product's own wrap,
// is the fraction of a turn to 2^-63 |p|, whatever the size of p: F loses its floor, and
// |w| 2^-64 for the 128 bits that 1 / (2 pi) is held to, so frequencies are taken below 2^64.
// Its upper 32 bits go to sincospif. No fp64 arithmetic is used (its rate is a 60th of fp32's
// here).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "boost_ops.h"
#include "internal.h"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

constexpr int kMaxAngles = 2048;   // (token, pair) angles of one block: 16 KB of shared memory

struct RopeParams {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *qo, *ko;
  const void* positions;
  const double* inv_freq;
  boost_rope_desc d;
  int tok;                         // tokens of one block
  int units;                       // units of a head
  int head_step, tok_step;         // heads and tokens that a block turns at a time
};

// Exponent field of a frequency; from kNoAngle on (2^64, infinities and NaN) there is no angle.
constexpr int kNoAngle = 1023 + 64;
__device__ __forceinline__ int exponent_field(double w) {
  return static_cast<int>((__double_as_longlong(w) >> 52) & 0x7ff);
}

// 2^64 w / (2 pi) mod 2^64, from the bits of w (0 where it has no angle).
__device__ __forceinline__ uint64_t turns_fixed(double w) {
  // 2^128 / (2 pi), upper and lower word
  constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
  const uint64_t b = __double_as_longlong(w);
  const int e = exponent_field(w);
  // (zero and subnormals turn by nothing at any 64-bit position)
  if (e == 0 || e >= kNoAngle) return 0;
  const uint64_t m = (b & 0xfffffffffffffull) | (1ull << 52);
  // m 2^128 / (2 pi) in three words, upper one first
  const uint64_t low = m * kHigh, w1 = low + __umul64hi(m, kLow), w0 = m * kLow;
  const uint64_t w2 = __umul64hi(m, kHigh) + (w1 < low ? 1 : 0);
  const int sh = 52 - (e - 1023);  // w = m 2^-sh, so the words go down by 64 + sh bits
  uint64_t f;
  if (sh < 0) f = (w1 << -sh) | (w0 >> (64 + sh));
  else if (sh == 0) f = w1;
  else if (sh < 64) f = (w2 << (64 - sh)) | (w1 >> sh);
  else f = sh < 128 ? w2 >> (sh - 64) : 0;
  return (b >> 63) ? 0 - f : f;
}

// Where the pairs lie, and how many a thread turns at a time: kHalf pairs i with i + rot / 2
// (a vector of each half), kAdjacent pairs 2 i with 2 i + 1 (adjacent values).
enum Pairing { kHalf, kAdjacent };

// N pairs (8, or 4 where a head's pairs are no multiple of 8) of one head as N words of two
// bf16 values.
template <Pairing P, int N>
struct Unit {
  uint32_t w[N];

  // word i of the unit's first (kHalf: N / 2 words of each half)
  template <int kWords>
  static __device__ __forceinline__ void words(const __nv_bfloat16* from, uint32_t* to) {
    if constexpr (kWords == 2) {
      const uint2 a = *reinterpret_cast<const uint2*>(from);
      to[0] = a.x; to[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(from + 2 * i);
        to[i] = a.x; to[i + 1] = a.y; to[i + 2] = a.z; to[i + 3] = a.w;
      }
    }
  }
  template <int kWords>
  static __device__ __forceinline__ void put(__nv_bfloat16* to, const uint32_t* from) {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(to) = make_uint2(from[0], from[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(to + 2 * i) = make_uint4(from[i], from[i + 1], from[i + 2], from[i + 3]);
    }
  }

  __device__ __forceinline__ void load(const __nv_bfloat16* h, int u, int half) {
    if constexpr (P == kHalf) {
      words<N / 2>(h + N * u, w);
      words<N / 2>(h + half + N * u, w + N / 2);
    } else {
      words<N>(h + 2 * N * u, w);
    }
  }

  __device__ __forceinline__ void turn(const float (&c)[N], const float (&s)[N]) {
    if constexpr (P == kAdjacent) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
        w[i] = pack_bf16x2(a * c[i] - b * s[i], b * c[i] + a * s[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const uint32_t x = w[i], y = w[N / 2 + i];
        const float a0 = bf16_lo(x), a1 = bf16_hi(x), b0 = bf16_lo(y), b1 = bf16_hi(y);
        w[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
        w[N / 2 + i] =
            pack_bf16x2(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
      }
    }
  }

  __device__ __forceinline__ void store(__nv_bfloat16* h, int u, int half) const {
    if constexpr (P == kHalf) {
      put<N / 2>(h + N * u, w);
      put<N / 2>(h + half + N * u, w + N / 2);
    } else {
      put<N>(h + 2 * N * u, w);
    }
  }
};

// Head `h` of token `t`: query heads first.
__device__ __forceinline__ const __nv_bfloat16* head_in(const RopeParams& p, int64_t t, int h) {
  return h < p.d.hq ? p.q + t * p.d.q_ts + h * p.d.q_hs
                    : p.k + t * p.d.k_ts + (h - p.d.hq) * p.d.k_hs;
}
__device__ __forceinline__ __nv_bfloat16* head_out(const RopeParams& p, int64_t t, int h) {
  return h < p.d.hq ? p.qo + t * p.d.qo_ts + h * p.d.qo_hs
                    : p.ko + t * p.d.ko_ts + (h - p.d.hq) * p.d.ko_hs;
}

template <Pairing P, int N>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  pdl_enter();
  __shared__ __align__(16) float cs[kMaxAngles], sn[kMaxAngles];
  const int pairs = p.d.rot / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tok;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tok), p.d.T - t0));
  // A thread keeps its unit of a head, and so its angles, over a token's heads: no division and
  // few multiplications in the loop (with both, the pass was bound by integer instructions).
  const int heads = p.d.hq + p.d.hk;
  const int slot = threadIdx.x / p.units, u = threadIdx.x - slot * p.units;
  const int ts = slot / p.head_step, h0 = slot - ts * p.head_step;
  constexpr int kBatch = 2;                             // units in flight a thread, twice
  Unit<P, N> now[kBatch], next[kBatch];
  auto load = [&](Unit<P, N> (&v)[kBatch], int t, int h) {
    const __nv_bfloat16* qi = p.q + (t0 + t) * p.d.q_ts;
    const __nv_bfloat16* ki = p.k + (t0 + t) * p.d.k_ts;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int hb = h + b * p.head_step;
      if (t < tokens && hb < heads)
        v[b].load(hb < p.d.hq ? qi + hb * p.d.q_hs : ki + (hb - p.d.hq) * p.d.k_hs, u, pairs);
    }
  };
  // (threads past the last whole slot have no token)
  int t = ts < p.tok_step ? ts : tokens, h = h0;
  load(now, t, h);

  for (int a = threadIdx.x; a < tokens * pairs; a += kThreads) {
    const int ta = a / pairs, i = a - ta * pairs;
    const int64_t at = p.d.pos_at + p.d.axis[i] * p.d.pos_as + t0 + ta;
    const int64_t pos = p.d.pos64 ? static_cast<const int64_t*>(p.positions)[at]
                                  : static_cast<const int32_t*>(p.positions)[at];
    const double w = p.inv_freq[i];
    const uint64_t phase = turns_fixed(w) * static_cast<uint64_t>(pos);
    // half turns in [-1, 1): the phase's upper 32 bits as a signed fraction
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
    if (exponent_field(w) >= kNoAngle) s = c = nanf("");
    cs[a] = c;
    sn[a] = p.d.inverse ? -s : s;
  }
  __syncthreads();

  while (t < tokens) {
    int tn = t, hn = h + kBatch * p.head_step;
    if (hn >= heads) {
      hn = h0;
      tn += p.tok_step;
    }
    load(next, tn, hn);
    float c[N], s[N];
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + t * pairs + u * N + i);
      *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + t * pairs + u * N + i);
    }
    __nv_bfloat16* qo = p.qo + (t0 + t) * p.d.qo_ts;
    __nv_bfloat16* ko = p.ko + (t0 + t) * p.d.ko_ts;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int hb = h + b * p.head_step;
      if (hb < heads) {
        now[b].turn(c, s);
        now[b].store(hb < p.d.hq ? qo + hb * p.d.qo_hs : ko + (hb - p.d.hq) * p.d.ko_hs, u, pairs);
      }
      now[b] = next[b];
    }
    t = tn;
    h = hn;
  }

  // values that do not turn
  const int rest = (p.d.dim - p.d.rot) / 8;
  for (int item = threadIdx.x; item < tokens * heads * rest; item += kThreads) {
    const int th = item / rest, t = th / heads, h = th - t * heads;
    const int at = p.d.rot + 8 * (item - th * rest);
    const __nv_bfloat16* src = head_in(p, t0 + t, h);
    __nv_bfloat16* dst = head_out(p, t0 + t, h);
    if (src != dst)
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
  }
}

cudaError_t launch_rope(const RopeParams& p_in, cudaStream_t stream) {
  RopeParams p = p_in;
  const int pairs = p.d.rot / 2;
  const int n = pairs % 8 == 0 ? 8 : 4;
  // A block has room for `slots` units' worth of heads: all heads of one or more tokens, or a
  // part of one token's heads at a time. It takes tokens until each thread has eight units: a
  // block waits for its positions before it has angles, and its first loads come before that.
  // (16384 tokens of 32 + 32 heads of 128: 85, 81, 82, 85 us with 2, 4, 8, 16 units; 12007 of
  // 40 + 8, adjacent pairs, three axes: 60, 53, 49, 53 us.)
  const int heads = p.d.hq + p.d.hk;
  p.units = pairs / n;
  const int slots = kThreads / p.units;
  p.head_step = std::min(heads, slots);
  p.tok_step = slots / p.head_step;
  const int64_t passes = (heads + p.head_step - 1) / p.head_step;
  int64_t tok = std::max<int64_t>(1, 8 * p.tok_step / passes);
  tok = std::min<int64_t>({tok, kMaxAngles / pairs, std::max<int64_t>(1, p.d.T / 304)});
  p.tok = static_cast<int>(tok);
  const int64_t grid = (p.d.T + tok - 1) / tok;
  if (p.d.interleaved)
    return launch_k(n == 8 ? rope_kernel<kAdjacent, 8> : rope_kernel<kAdjacent, 4>, grid, stream, p);
  return launch_k(n == 8 ? rope_kernel<kHalf, 8> : rope_kernel<kHalf, 4>, grid, stream, p);
}

// ------------------------------------------------------------------ host checks
// One [T, heads, dim] operand as it lies in memory (strides in elements).
struct Slice {
  uintptr_t base;
  int64_t T, heads, dim, ts, hs;
  // bytes from the first to behind the last element
  uint64_t extent() const {
    return T * heads == 0 ? 0 : 2ull * ((T - 1) * ts + (heads - 1) * hs + dim);
  }
  bool same(const Slice& o) const {
    return base == o.base && heads == o.heads && (T == 1 || ts == o.ts) &&
           (heads == 1 || hs == o.hs);
  }
  // no two elements coincide: tokens apart by more than a token's heads, or heads by more
  // than a head's tokens
  bool one_to_one() const {
    const int64_t token = (heads - 1) * hs + dim, head = (T - 1) * ts + dim;
    return (heads == 1 || hs >= dim) && (T == 1 || ts >= dim) &&
           (T == 1 || heads == 1 || ts >= token || hs >= head);
  }
};

// Whether |x + i step| >= apart for every i from -times to times.
bool stays_away(int64_t x, int64_t step, int64_t times, int64_t apart) {
  if (step == 0) times = 0;
  const int64_t n = times == 0 ? 0 : -x / step;        // the nearest is one of n - 1 .. n + 1
  for (int64_t i = n - 1; i <= n + 1; ++i)
    if (std::abs(x + std::clamp(i, -times, times) * step) < apart) return false;
  return true;
}

// Whether two operands share no element: disjoint ranges; heads side by side in the rows of one
// packed buffer (the same token stride, and spans that do not meet modulo it); or heads that lie
// between each other's (the same strides, and no pair of heads and tokens that meet).
bool disjoint(const Slice& a, const Slice& b) {
  if (a.extent() == 0 || b.extent() == 0) return true;
  if (a.base + a.extent() <= b.base || b.base + b.extent() <= a.base) return true;
  if (a.T > 1 && a.ts != b.ts) return false;
  const int64_t away = static_cast<int64_t>(b.base) - static_cast<int64_t>(a.base);   // bytes
  if (a.T > 1 && a.ts > 0) {
    const int64_t sa = 2 * ((a.heads - 1) * a.hs + a.dim), sb = 2 * ((b.heads - 1) * b.hs + b.dim);
    const int64_t row = 2 * a.ts;
    // where b's span begins within a's rows
    const int64_t o = (away % row + row) % row;
    if (o >= sa && o + sb <= row) return true;
  }
  if (a.heads > 1 && b.heads > 1 && a.hs != b.hs) return false;
  const int64_t hs = a.heads > 1 ? a.hs : b.hs;
  for (int64_t h = 1 - a.heads; h < b.heads; ++h)      // b's head less a's
    if (!stays_away(away / 2 + h * hs, a.ts, a.T - 1, a.dim)) return false;
  return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

}  // namespace boost_gb300

using namespace boost_gb300;

extern "C" boost_status boost_rope(const boost_rope_desc* desc, const void* q, const void* k,
                                   const void* positions, const double* inv_freq, void* q_out,
                                   void* k_out, void* stream) {
  if (desc == nullptr) return BOOST_ERR_INVALID_ARG;
  const boost_rope_desc& D = *desc;
  if (D.T < 0 || D.hq < 1 || D.hk < 0 || D.dim < 1 || D.rot < 1 || D.rot > D.dim || D.axes < 1 ||
      D.axes > BOOST_ROPE_MAX_AXES)
    return BOOST_ERR_INVALID_ARG;
  if ((D.interleaved | D.inverse | D.pos64) & ~1) return BOOST_ERR_INVALID_ARG;
  if (D.dim % 8 || D.rot % 8 || D.dim > BOOST_ROPE_MAX_DIM) return BOOST_ERR_UNSUPPORTED_SHAPE;
  // the grid and a block's heads x pairs stay within 31 bits; offsets take 64
  if (D.T > 0x7fffffff || D.hq > 65536 || D.hk > 65536) return BOOST_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < D.rot / 2; ++i)
    if (D.axis[i] >= D.axes) return BOOST_ERR_INVALID_ARG;
  const int64_t strides[8] = {D.q_ts, D.q_hs, D.k_ts, D.k_hs, D.qo_ts, D.qo_hs, D.ko_ts, D.ko_hs};
  for (int i = 0; i < 8; ++i) {
    if (D.hk == 0 && (i & 2)) continue;
    if (strides[i] < 0) return BOOST_ERR_INVALID_ARG;
    if (strides[i] % 8) return BOOST_ERR_UNSUPPORTED_SHAPE;
    // (every offset below 2^50 elements, so that sums of them fit)
    const double n = i % 2 == 0 ? static_cast<double>(D.T) : (i & 2) ? D.hk : D.hq;
    if (n * static_cast<double>(strides[i]) > 0x1p50) return BOOST_ERR_UNSUPPORTED_SHAPE;
  }
  if (D.pos_at < 0 || D.pos_as < 0 || (D.pos_as > 0 && D.pos_as < D.T)) return BOOST_ERR_INVALID_ARG;
  if (D.pos_at > (int64_t{1} << 50) || D.pos_as > (int64_t{1} << 50))
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  if (D.hk == 0 && (k != nullptr || k_out != nullptr)) return BOOST_ERR_INVALID_ARG;
  if (D.T == 0) return BOOST_OK;
  if (q == nullptr || positions == nullptr || inv_freq == nullptr || q_out == nullptr)
    return BOOST_ERR_INVALID_ARG;
  if (D.hk > 0 && (k == nullptr || k_out == nullptr)) return BOOST_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(positions) || !aligned16(inv_freq))
    return BOOST_ERR_ALIGNMENT;
  auto slice = [&](const void* ptr, int64_t heads, int64_t ts, int64_t hs) {
    return Slice{reinterpret_cast<uintptr_t>(ptr), D.T, heads, D.dim, ts, hs};
  };
  const Slice sq = slice(q, D.hq, D.q_ts, D.q_hs), sk = slice(k, D.hk, D.k_ts, D.k_hs);
  const Slice qo = slice(q_out, D.hq, D.qo_ts, D.qo_hs), ko = slice(k_out, D.hk, D.ko_ts, D.ko_hs);
  if (!qo.one_to_one() || (D.hk > 0 && !ko.one_to_one())) return BOOST_ERR_INVALID_ARG;
  if (!(sq.same(qo) || disjoint(sq, qo)) || !(sk.same(ko) || disjoint(sk, ko)) ||
      !disjoint(sq, ko) || !disjoint(sk, qo) || !disjoint(qo, ko))
    return BOOST_ERR_INVALID_ARG;
  // positions and frequencies are read while the outputs are written: nothing shared there
  const uint64_t pos_size = D.pos64 ? 8 : 4, freq_bytes = 4ull * D.rot;
  const int64_t pos_as = D.pos_as > 0 ? D.pos_as : D.T;
  const uint64_t pos_bytes = pos_size * ((D.axes - 1) * pos_as + D.T);
  const void* first_pos = static_cast<const char*>(positions) + pos_size * D.pos_at;
  auto meets = [](const Slice& o, const void* in, uint64_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(in);
    return o.extent() > 0 && b < o.base + o.extent() && o.base < b + bytes;
  };
  if (meets(qo, first_pos, pos_bytes) || meets(ko, first_pos, pos_bytes) ||
      meets(qo, inv_freq, freq_bytes) || meets(ko, inv_freq, freq_bytes))
    return BOOST_ERR_INVALID_ARG;

  RopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.d = D;
  p.d.pos_as = pos_as;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double values = static_cast<double>(D.T) * (D.hq + D.hk) * D.dim;
  ProfScope ps(s, K_ROPE, 0.0, 4.0 * values + static_cast<double>(pos_size * D.axes * D.T));
  return launch_rope(p, s) == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}
