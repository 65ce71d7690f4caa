// fp8.cu -- C ABI of the 8-bit quantiser and matrix product: argument checks.
#include "fp8.cuh"

#include "boost_ops.h"
#include "internal.h"
#include "profile.h"

using namespace boost_gb300;

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1;

bool misaligned(const void* p, uintptr_t to = 16) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

struct Range {
  const void* at;
  uint64_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x != 0 && y != 0 && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}

// Whether an output shares a byte with an input or another output.
template <int NI, int NO>
bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

boost_status validate(const boost_fp8_matmul_desc* D) {
  if (D == nullptr) return BOOST_ERR_INVALID_ARG;
  if (D->G < 1 || D->M < 0 || D->N < 1 || D->K < 0) return BOOST_ERR_INVALID_ARG;
  for (int f : {D->a_fmt, D->b_fmt})
    if (f != BOOST_E4M3 && f != BOOST_E5M2) return BOOST_ERR_INVALID_ARG;
  if (D->act != BOOST_ACT_IDENTITY && D->act != BOOST_ACT_SILU) return BOOST_ERR_INVALID_ARG;
  if (D->a_pitch < D->K || D->b_pitch < D->K) return BOOST_ERR_INVALID_ARG;
  if (D->a_pitch % 16 || D->b_pitch % 16 || D->N % 8) return BOOST_ERR_UNSUPPORTED_SHAPE;
  if (D->M > kMaxDim || D->N > 65535ll * 16 || D->K > kMaxDim || D->G > 65535 ||
      D->a_pitch > kMaxDim || D->b_pitch > kMaxDim)
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  // a tensor map's matrix stride is below 2^40 bytes; tiles, times 8 for a shared K, and grids
  // stay within 31 bits
  constexpr double kStride = 0x1p40;
  if (static_cast<double>(D->M) * D->a_pitch >= kStride ||
      static_cast<double>(D->N) * D->b_pitch >= kStride || 2.0 * D->M * D->N >= kStride)
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  const double tiles = static_cast<double>((D->M + 127) / 128) * ((D->N + 127) / 128) * D->G;
  if (tiles > 0x1p28 - 1) return BOOST_ERR_UNSUPPORTED_SHAPE;
  return BOOST_OK;
}

}  // namespace

extern "C" {

size_t boost_fp8_scale_bytes(int64_t rows, int64_t K) {
  if (rows <= 0 || K <= 0 || rows > kMaxDim || K > kMaxDim) return 0;
  return static_cast<size_t>(scale_plane(rows, K));
}

boost_status boost_fp8_quantize(const boost_fp8_quant_desc* desc, const void* x,
                                const void* gamma, void* q, void* sf, void* qt, void* sft,
                                void* stream) {
  if (desc == nullptr) return BOOST_ERR_INVALID_ARG;
  const boost_fp8_quant_desc& D = *desc;
  if (D.G < 1 || D.rows < 0 || D.cols < 1 || D.ldx < 0 || D.gstride < 0)
    return BOOST_ERR_INVALID_ARG;
  if (D.fmt != BOOST_E4M3 && D.fmt != BOOST_E5M2) return BOOST_ERR_INVALID_ARG;
  if (D.block_rows != 1 && D.block_rows != 128) return BOOST_ERR_INVALID_ARG;
  if (D.cols % 8 || D.ldx % 8 || D.gstride % 8) return BOOST_ERR_UNSUPPORTED_SHAPE;
  // one grid line of 32 rows each; offsets of x below 2^50 elements
  if (D.G > 65535 || D.rows > 65535ll * 32 || D.cols > kMaxDim || D.ldx > (1ll << 28) ||
      D.gstride > (1ll << 33))
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  if ((q == nullptr) != (sf == nullptr) || (qt == nullptr) != (sft == nullptr))
    return BOOST_ERR_INVALID_ARG;
  if (gamma != nullptr && D.block_rows == 1 && qt == nullptr) return BOOST_ERR_INVALID_ARG;
  if (D.rows == 0) return BOOST_OK;
  if (x == nullptr || (q == nullptr && qt == nullptr)) return BOOST_ERR_INVALID_ARG;
  for (const void* p : {x, gamma, static_cast<const void*>(q), static_cast<const void*>(sf),
                        static_cast<const void*>(qt), static_cast<const void*>(sft)})
    if (misaligned(p)) return BOOST_ERR_ALIGNMENT;
  const uint64_t pitch = (D.cols + 15) / 16 * 16, pitch_t = (D.rows + 15) / 16 * 16;
  const uint64_t G = D.G;
  const Range in[] = {{x, 2ull * ((D.G - 1) * D.gstride + (D.rows - 1) * D.ldx + D.cols)},
                      {gamma, 2ull * D.rows}};
  const Range out[] = {{q, G * D.rows * pitch}, {sf, G * scale_plane(D.rows, D.cols)},
                       {qt, G * D.cols * pitch_t}, {sft, G * scale_plane(D.cols, D.rows)}};
  if (any_overlap(in, out)) return BOOST_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double n = static_cast<double>(D.G) * D.rows * D.cols;
  const int layouts = (q != nullptr) + (qt != nullptr);
  ProfScope ps(s, K_FP8_QUANT, 0.0, n * (2.0 + layouts * 129.0 / 128.0));
  return launch_fp8_quantize(D, x, gamma, q, sf, qt, sft, s) == cudaSuccess ? BOOST_OK
                                                                            : BOOST_ERR_CUDA;
}

size_t boost_fp8_matmul_workspace_bytes(const boost_fp8_matmul_desc* desc) {
  return validate(desc) == BOOST_OK ? fp8_gemm_workspace(*desc) : 0;
}

boost_status boost_fp8_matmul(const boost_fp8_matmul_desc* desc, const void* a, const void* a_sf,
                              const void* b, const void* b_sf, const float* row_scale, void* out,
                              void* ws, size_t ws_bytes, void* stream) {
  boost_status st = validate(desc);
  if (st != BOOST_OK) return st;
  const boost_fp8_matmul_desc& D = *desc;
  const bool empty = D.K == 0;            // the operands and their scales may be NULL
  if (D.M > 0) {
    if (out == nullptr) return BOOST_ERR_INVALID_ARG;
    if (!empty && (a == nullptr || a_sf == nullptr || b == nullptr || b_sf == nullptr))
      return BOOST_ERR_INVALID_ARG;
  }
  for (const void* p : {a, a_sf, b, b_sf, static_cast<const void*>(row_scale),
                        static_cast<const void*>(out)})
    if (misaligned(p)) return BOOST_ERR_ALIGNMENT;
  const size_t need = fp8_gemm_workspace(D);
  if (ws == nullptr || misaligned(ws, 256) || ws_bytes < need) return BOOST_ERR_WORKSPACE;
  if (D.M == 0) return BOOST_OK;
  const uint64_t G = D.G, values = G * D.M * D.N;
  const Range in[] = {{a, empty ? 0 : G * D.M * D.a_pitch},
                      {a_sf, empty ? 0 : G * scale_plane(D.M, D.K)},
                      {b, empty ? 0 : G * D.N * D.b_pitch},
                      {b_sf, empty ? 0 : G * scale_plane(D.N, D.K)},
                      {row_scale, 4ull * D.M}};
  const Range outs[] = {{out, 2 * values}, {ws, need}};
  if (any_overlap(in, outs)) return BOOST_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return cudaMemsetAsync(out, 0, 2 * values, s) == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
  Fp8GemmParams p{};
  p.d = D;
  p.a = static_cast<const uint8_t*>(a);
  p.a_sf = static_cast<const uint8_t*>(a_sf);
  p.b = static_cast<const uint8_t*>(b);
  p.b_sf = static_cast<const uint8_t*>(b_sf);
  p.row_scale = row_scale;
  p.out = out;
  p.ws = ws;
  ProfScope ps(s, K_FP8_GEMM, 2.0 * values * D.K,
               D.G * static_cast<double>(D.M + D.N) * D.K * 129.0 / 128.0 + 2.0 * values);
  return launch_fp8_gemm(p, s) == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}

}  // extern "C"
