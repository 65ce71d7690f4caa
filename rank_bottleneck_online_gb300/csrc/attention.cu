// attention.cu -- C ABI of attention and its gradients: argument checks.
#include "attention.cuh"

#include "boost_ops.h"
#include "heads.h"
#include "internal.h"
#include "profile.h"

using namespace boost_gb300;

namespace {

bool stride_ok(int64_t stride, int64_t times) {
  return stride >= 0 && (times <= 1 || stride > 0);
}

boost_status validate(const boost_attention_desc* desc) {
  if (desc == nullptr) return BOOST_ERR_INVALID_ARG;
  const boost_attention_desc& D = *desc;
  if (D.Tq < 0 || D.Tk < 0 || D.hq < 1 || D.hk < 1 || D.dim < 1 || D.sequences < 1 ||
      (D.causal & ~1) || D.hq % D.hk || !(D.scale > 0.0f) || D.scale > 0x1p127f)
    return BOOST_ERR_INVALID_ARG;
  if (D.dim % 8 || D.dim > BOOST_ATTENTION_MAX_DIM) return BOOST_ERR_UNSUPPORTED_SHAPE;
  // token and tile numbers, and tiles times heads, stay within 31 bits
  if (D.Tq > (1 << 30) || D.Tk > (1 << 30) || D.sequences > (1 << 20) || D.hq > 65535)
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  const double tiles = (D.Tq > D.Tk ? D.Tq : D.Tk) / 64.0 + D.sequences;
  if (tiles * D.hq > 0x1p30) return BOOST_ERR_UNSUPPORTED_SHAPE;
  return BOOST_OK;
}

// Strides of one operand: multiples of 8, bytes within a tensor map's 40 bits.
boost_status strides(int64_t T, int64_t heads, int64_t ts, int64_t hs) {
  if (!stride_ok(ts, T) || !stride_ok(hs, heads)) return BOOST_ERR_INVALID_ARG;
  if (ts % 8 || hs % 8 || ts >= (int64_t{1} << 38) || hs >= (int64_t{1} << 38))
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<double>(T) * ts + static_cast<double>(heads) * hs > 0x1p50)
    return BOOST_ERR_UNSUPPORTED_SHAPE;
  return BOOST_OK;
}

Slice slice(const void* p, int64_t T, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  return Slice{reinterpret_cast<uintptr_t>(p), T, heads, dim, ts, hs};
}

bool meets(const Slice& o, const void* p, uint64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return p != nullptr && bytes > 0 && o.extent() > 0 && b < o.base + o.extent() && o.base < b + bytes;
}

bool meet(const void* p, uint64_t n, const void* q, uint64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p != nullptr && q != nullptr && a < b + m && b < a + n;
}

// What both calls check of the starts, the workspace and where the operands lie: outputs share
// no byte with anything else; lse is one of them where `writes_lse`.
template <int NI, int NO>
boost_status placed(const boost_attention_desc& D, const Slice (&in)[NI], const Slice (&out)[NO],
                    const int32_t* q_starts, const int32_t* k_starts, const float* lse,
                    bool writes_lse, void* ws, size_t ws_bytes) {
  if (D.sequences > 1 && (q_starts == nullptr || k_starts == nullptr)) return BOOST_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(q_starts), static_cast<const void*>(k_starts),
                        static_cast<const void*>(lse)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return BOOST_ERR_ALIGNMENT;
  const size_t need = attention_workspace(D);
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < need)
    return BOOST_ERR_WORKSPACE;
  const uint64_t n_starts = 4ull * (D.sequences + 1), n_lse = 4ull * D.hq * D.Tq;
  for (int i = 0; i < NO; ++i) {
    if (!out[i].one_to_one()) return BOOST_ERR_INVALID_ARG;
    for (int j = 0; j < NI; ++j)
      if (!disjoint(out[i], in[j])) return BOOST_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (!disjoint(out[i], out[j])) return BOOST_ERR_INVALID_ARG;
    if (meets(out[i], q_starts, n_starts) || meets(out[i], k_starts, n_starts) ||
        meets(out[i], lse, n_lse) || meets(out[i], ws, need))
      return BOOST_ERR_INVALID_ARG;
  }
  for (int j = 0; j < NI; ++j)
    if (meets(in[j], ws, need) || (writes_lse && meets(in[j], lse, n_lse)))
      return BOOST_ERR_INVALID_ARG;
  if (meet(ws, need, lse, n_lse) || meet(ws, need, q_starts, n_starts) ||
      meet(ws, need, k_starts, n_starts))
    return BOOST_ERR_INVALID_ARG;
  if (writes_lse && (meet(lse, n_lse, q_starts, n_starts) || meet(lse, n_lse, k_starts, n_starts)))
    return BOOST_ERR_INVALID_ARG;
  return BOOST_OK;
}

// Work of `products` products over all pairs of queries and keys (the lengths are on the device:
// half of them with a causal mask, as if the sequences were of one length).
double flops(const boost_attention_desc& D, int products) {
  return 2.0 * products * D.Tq * D.Tk / D.sequences * D.hq * D.dim * (D.causal ? 0.5 : 1.0);
}

}  // namespace

extern "C" {

size_t boost_attention_workspace_bytes(const boost_attention_desc* desc) {
  return validate(desc) == BOOST_OK ? attention_workspace(*desc) : 0;
}

boost_status boost_attention(const boost_attention_desc* desc, const void* q, const void* k,
                             const void* v, const int32_t* q_starts, const int32_t* k_starts,
                             void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  boost_status st = validate(desc);
  if (st != BOOST_OK) return st;
  const boost_attention_desc& D = *desc;
  const int64_t T[4] = {D.Tq, D.Tk, D.Tk, D.Tq}, heads[4] = {D.hq, D.hk, D.hk, D.hq};
  const int64_t ts[4] = {D.q_ts, D.k_ts, D.v_ts, D.o_ts}, hs[4] = {D.q_hs, D.k_hs, D.v_hs, D.o_hs};
  for (int i = 0; i < 4; ++i)
    if ((st = strides(T[i], heads[i], ts[i], hs[i])) != BOOST_OK) return st;
  const void* at[4] = {q, k, v, out};
  for (int i = 0; i < 4; ++i) {
    if (T[i] > 0 && at[i] == nullptr) return BOOST_ERR_INVALID_ARG;
    if (!aligned16(at[i])) return BOOST_ERR_ALIGNMENT;
  }
  auto of = [&](int i) { return slice(at[i], T[i], heads[i], D.dim, ts[i], hs[i]); };
  const Slice in[] = {of(0), of(1), of(2)}, outs[] = {of(3)};
  st = placed(D, in, outs, q_starts, k_starts, lse, true, ws, ws_bytes);
  if (st != BOOST_OK || D.Tq == 0) return st;
  AttentionArgs a{};
  a.d = D;
  a.q = {static_cast<const __nv_bfloat16*>(q), D.q_ts, D.q_hs};
  a.k = {static_cast<const __nv_bfloat16*>(k), D.k_ts, D.k_hs};
  a.v = {static_cast<const __nv_bfloat16*>(v), D.v_ts, D.v_hs};
  a.out = {static_cast<__nv_bfloat16*>(out), D.o_ts, D.o_hs};
  a.lse = lse;
  a.q_starts = q_starts;
  a.k_starts = k_starts;
  a.ws = ws;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, K_ATTENTION, flops(D, 2),
               4.0 * D.dim * (static_cast<double>(D.Tq) * D.hq + static_cast<double>(D.Tk) * D.hk));
  return launch_attention(a, s) == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}

boost_status boost_attention_bwd(const boost_attention_desc* desc, const void* q, const void* k,
                                 const void* v, const void* out, const float* lse,
                                 const void* dout, const int32_t* q_starts,
                                 const int32_t* k_starts, void* dq, void* dk, void* dv, void* ws,
                                 size_t ws_bytes, void* stream) {
  boost_status st = validate(desc);
  if (st != BOOST_OK) return st;
  const boost_attention_desc& D = *desc;
  const int64_t T[8] = {D.Tq, D.Tk, D.Tk, D.Tq, D.Tq, D.Tq, D.Tk, D.Tk};
  const int64_t heads[8] = {D.hq, D.hk, D.hk, D.hq, D.hq, D.hq, D.hk, D.hk};
  const int64_t ts[8] = {D.q_ts, D.k_ts, D.v_ts, D.o_ts, D.do_ts, D.dq_ts, D.dk_ts, D.dv_ts};
  const int64_t hs[8] = {D.q_hs, D.k_hs, D.v_hs, D.o_hs, D.do_hs, D.dq_hs, D.dk_hs, D.dv_hs};
  for (int i = 0; i < 8; ++i)
    if ((st = strides(T[i], heads[i], ts[i], hs[i])) != BOOST_OK) return st;
  const void* at[8] = {q, k, v, out, dout, dq, dk, dv};
  for (int i = 0; i < 8; ++i) {
    if (T[i] > 0 && at[i] == nullptr) return BOOST_ERR_INVALID_ARG;
    if (!aligned16(at[i])) return BOOST_ERR_ALIGNMENT;
  }
  if (D.Tq > 0 && lse == nullptr) return BOOST_ERR_INVALID_ARG;
  auto of = [&](int i) { return slice(at[i], T[i], heads[i], D.dim, ts[i], hs[i]); };
  const Slice in[] = {of(0), of(1), of(2), of(3), of(4)}, outs[] = {of(5), of(6), of(7)};
  st = placed(D, in, outs, q_starts, k_starts, lse, false, ws, ws_bytes);
  if (st != BOOST_OK || (D.Tq == 0 && D.Tk == 0)) return st;
  AttentionArgs a{};
  a.d = D;
  a.q = {static_cast<const __nv_bfloat16*>(q), D.q_ts, D.q_hs};
  a.k = {static_cast<const __nv_bfloat16*>(k), D.k_ts, D.k_hs};
  a.v = {static_cast<const __nv_bfloat16*>(v), D.v_ts, D.v_hs};
  a.o = {static_cast<const __nv_bfloat16*>(out), D.o_ts, D.o_hs};
  a.dout = {static_cast<const __nv_bfloat16*>(dout), D.do_ts, D.do_hs};
  a.dq = {static_cast<__nv_bfloat16*>(dq), D.dq_ts, D.dq_hs};
  a.dk = {static_cast<__nv_bfloat16*>(dk), D.dk_ts, D.dk_hs};
  a.dv = {static_cast<__nv_bfloat16*>(dv), D.dv_ts, D.dv_hs};
  a.lse = const_cast<float*>(lse);
  a.q_starts = q_starts;
  a.k_starts = k_starts;
  a.ws = ws;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, K_ATTENTION_BWD, flops(D, 5),
               8.0 * D.dim * (static_cast<double>(D.Tq) * D.hq + static_cast<double>(D.Tk) * D.hk));
  return launch_attention_bwd(a, s) == cudaSuccess ? BOOST_OK : BOOST_ERR_CUDA;
}

}  // extern "C"
