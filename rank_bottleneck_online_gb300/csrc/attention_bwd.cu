// attention_bwd.cu -- gradients of attention on the tensor cores, in two passes of one kernel.
//
//     P = exp(scale S - lse), S = q k^T      dP = dout v^T      dS = P (dP - delta)
//     dv = P^T dout        dk = scale dS^T q        dq = scale dS k,   delta = sum_j P dP
//
// Both passes keep two tiles of 128 rows (X0, X1) and go through tiles of 128 rows of the other
// side (Y0, Y1), forming S = X0 Y0^T and dP = X1 Y1^T in TMEM; threads turn them into P and dS,
// written back over them as bf16, which are the first operands of two more products, summed in
// TMEM. The first pass keeps q and dout of 128 queries and sums dS k; the second keeps k and v of
// 128 keys (S and dP transposed), goes through the queries of all heads that share the key head,
// and sums P^T dout and dS^T q. So no sum leaves the SM, none is taken in another order from call
// to call, and S and dP are formed twice (8 products of 128^3 a pair of tiles instead of 5) where
// one pass would add dq to memory by atomics.
//
// delta: sum_d dout out is its value but for the rounding of out, which is of the size of dS
// where a row's probability lies on few keys (a row of one key: dS = 0). The first pass takes
// delta from out and sums what is missing, e = sum_j P (dP - delta), beside sum_j P k in TMEM;
// dq = scale (sum dS k - e sum P k), and the second pass reads delta + e. (Without that the
// gradients of 77 tokens were off by 0.0030, relative to all, with it by the 0.002 of a bf16
// result and bf16 dS.)
//
// Warp 0 loads the tiles through a ring, warp 1 issues the products, warp 2 fetches the second
// pass's lse and delta, sixteen warps are the rows of a tile, four threads a row. The products of
// one kind run while the threads work on the other's scores: acc1 += P B and the next S during dS,
// acc2 += dS Y0 and the next dP during P.
#include <math_constants.h>

#include <atomic>
#include <cstring>

#include "attention.cuh"
#include "attention_tc.cuh"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

enum Pass : int { kDq = 0, kDkv = 1 };

struct BwdParams {
  CUtensorMap tmX0, tmX1, tmY0, tmY1;    // boxes of 64 values x 128 rows of one head
  HeadsIn o, dout;                       // kDq
  HeadsOut g1, g2;                       // kDq: -, dq; kDkv: dv, dk
  const float* lse;                      // [hq, Tq]
  float* delta;                          // [hq, Tq]: written by kDq, read by kDkv
  const int32_t *q_starts, *k_starts;
  int64_t Tq, Tk;
  int32_t heads, group;                  // of the tiles' side; query heads of a key head
  int32_t dim, sequences, causal;
  float scale, scale_log2;
  DeviceError* err;
  uint64_t wait_limit_ns;
};

template <int HD>
struct BwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = HD == 128 ? 4 : 8;      // Y0(0), Y1(0), Y0(1), ...
  static constexpr int kBars = 2 * kStages + 11;
  static constexpr int kStatOffset = (2 + kStages) * kTileBytes;
  static constexpr int kParts = 4;                       // threads of a row
  static constexpr int kCols = kTile / kParts;           // of its scores, each
  static constexpr int kStatBytes = 4 * 4 * kTile;       // two buffers of lse and delta
  static constexpr int kBarOffset = kStatOffset + kStatBytes;
  static constexpr int kSmemBytes = 1024 + kBarOffset + 8 * kBars + 16;
  static constexpr int kWarps = 4 * kParts;              // that work on the scores
  static constexpr int kThreads = 128 + 32 * kWarps;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

// Sum of a row's products over `n` values (a multiple of 8).
__device__ __forceinline__ float dot_row(const __nv_bfloat16* a, const __nv_bfloat16* b, int n) {
  float s = 0.0f;
  for (int e = 0; e < n; e += 8) {
    float x[8], y[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(a + e)), x);
    unpack8(__ldg(reinterpret_cast<const uint4*>(b + e)), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  }
  return s;
}

template <int HD, int PASS>
__global__ void __launch_bounds__(BwdCfg<HD>::kThreads, 1)
    attention_bwd_kernel(const __grid_constant__ BwdParams p) {
  using Cfg = BwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = smem;                                   // X0, X1
  uint8_t* sY = smem + 2 * Cfg::kTileBytes;
  float* stat = reinterpret_cast<float*>(smem + Cfg::kStatOffset);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOffset);
  uint64_t* empty_bar = full_bar + Cfg::kStages;
  uint64_t* x_bar = empty_bar + Cfg::kStages;
  uint64_t* s_bar = x_bar + 1;                          // S is complete
  uint64_t* d_bar = s_bar + 1;                          // dP is complete
  uint64_t* p_bar = d_bar + 1;                          // P is written
  uint64_t* ds_bar = p_bar + 1;                         // dS is written
  uint64_t* acc_bar = ds_bar + 1;                       // the sums are complete
  uint64_t* stat_full = acc_bar + 1;                    // [2]
  uint64_t* stat_empty = stat_full + 2;                 // [2]
  uint64_t* done_bar = stat_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(x_bar, 1);
    mbar_init(s_bar, 1);
    mbar_init(d_bar, 1);
    mbar_init(p_bar, Cfg::kWarps);
    mbar_init(ds_bar, Cfg::kWarps);
    mbar_init(acc_bar, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&stat_full[b], 1);
      mbar_init(&stat_empty[b], Cfg::kWarps);
    }
    mbar_init(done_bar, 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmX0);
    tma_prefetch_desc(&p.tmX1);
    tma_prefetch_desc(&p.tmY0);
    tma_prefetch_desc(&p.tmY1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tS = tmem, tD = tmem + 128, tAcc1 = tmem + 256, tAcc2 = tmem + 256 + HD;
  griddep_wait();
  griddep_launch_dependents();

  // This CTA's tile of queries (kDq, longest rows first) or keys, and the tiles [first, first +
  // count) of the other side that its rows see; kDkv has those once for each head of the group.
  const int32_t head = static_cast<int32_t>(blockIdx.x) % p.heads;
  Place at = find_tile(p.q_starts, p.k_starts, p.Tq, p.Tk, p.sequences,
                       static_cast<int32_t>(blockIdx.x) / p.heads, kTile, PASS == kDkv);
  const int32_t off = at.nk - at.nq;                     // keys before the first query
  const int32_t x0 = (PASS == kDq ? at.tiles - 1 - at.tile : at.tile) * kTile;
  const int32_t nx = PASS == kDq ? at.nq : at.nk, ny = PASS == kDq ? at.nk : at.nq;
  int32_t first = 0, count = 0;
  if (at.tiles > 0) {
    if (PASS == kDq) {
      const int32_t keys = p.causal ? min(at.nk, min(x0 + kTile, at.nq) + off) : at.nk;
      count = keys > 0 ? (keys + kTile - 1) / kTile : 0;
    } else {
      first = p.causal ? max(x0 - off, 0) / kTile : 0;
      count = max((at.nq + kTile - 1) / kTile - first, 0);
    }
  }
  const int32_t steps = PASS == kDq ? count : count * p.group;
  const int32_t x_row = (PASS == kDq ? at.q0 : at.k0) + x0;
  const int32_t y_row = PASS == kDq ? at.k0 : at.q0;
  const int32_t y_head = PASS == kDq ? head / p.group : head * p.group;
  const int ksteps = (p.dim + 15) / 16;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t armed = 0, parities = 0;
    if (steps > 0) {
      if (elect_one()) {
        mbar_arrive_expect_tx(x_bar, 2 * Cfg::kTileBytes);
        for (int b = 0; b < Cfg::kBoxes; ++b) {
          tma_load_3d(sX + b * kBoxBytes, &p.tmX0, x_bar, 64 * b, head, x_row);
          tma_load_3d(sX + Cfg::kTileBytes + b * kBoxBytes, &p.tmX1, x_bar, 64 * b, head, x_row);
        }
      }
      __syncwarp();
      int stage = 0;
      uint32_t phase = 0;
      int32_t tile = first, h = y_head;
      for (int32_t i = 0; i < 2 * steps; ++i) {
        if (!warp_wait_all(&empty_bar[stage], phase ^ 1u, p.err, 61, p.wait_limit_ns)) break;
        armed |= 1u << stage;
        parities = (parities & ~(1u << stage)) | (phase << stage);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full_bar[stage], Cfg::kTileBytes);
          for (int b = 0; b < Cfg::kBoxes; ++b)
            tma_load_3d(sY + stage * Cfg::kTileBytes + b * kBoxBytes, i & 1 ? &p.tmY1 : &p.tmY0,
                        &full_bar[stage], 64 * b, h, y_row + tile * kTile);
        }
        __syncwarp();
        if ((i & 1) && ++tile == first + count) {
          tile = first;
          ++h;
        }
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the copies started here have landed before the CTA exits
      for (int s = 0; s < Cfg::kStages; ++s)
        if (armed >> s & 1u)
          warp_wait_all(&full_bar[s], parities >> s & 1u, nullptr, 67, p.wait_limit_ns);
      warp_wait_all(x_bar, 0, nullptr, 67, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t id_s = idesc_bf16_f32(kTile, kTile, 0, 0);
    const uint32_t id_acc = idesc_bf16_f32(kTile, 16 * ksteps, 0, 1);
    const uint64_t x0_desc = desc_k_major(smem_u32(sX));
    const uint64_t x1_desc = desc_k_major(smem_u32(sX) + Cfg::kTileBytes);
    const uint64_t yk_desc = desc_k_major(smem_u32(sY)), ymn_desc = desc_mn_major(smem_u32(sY));
    auto slot = [&](int32_t u) { return u % Cfg::kStages * (Cfg::kTileBytes >> 4); };
    // Wait for tile `u` of the ring; rows behind the sequence become 0.
    auto take = [&](int32_t u, int32_t step) {
      const int s = u % Cfg::kStages;
      if (!warp_wait_all(&full_bar[s], u / Cfg::kStages & 1, p.err, 63, p.wait_limit_ns))
        return false;
      const int32_t left = ny - (first + step % max(count, 1)) * kTile;
      if (left < kTile) zero_rows(sY + s * Cfg::kTileBytes, Cfg::kBoxes, left, lane);
      tc_fence_after();
      return true;
    };
    bool ok = steps > 0 && warp_wait_all(x_bar, 0, p.err, 62, p.wait_limit_ns) && take(0, 0);
    if (ok) {
      if (elect_one()) {
        issue_scores<HD / 16>(tS, x0_desc, yk_desc, id_s, ksteps);
        tc_commit(s_bar);
      }
      __syncwarp();
      ok = take(1, 0);
    }
    if (ok) {
      const uint64_t y = yk_desc + slot(1);
      if (elect_one()) {
        issue_scores<HD / 16>(tD, x1_desc, y, id_s, ksteps);
        tc_commit(d_bar);
        if (PASS == kDq) tc_commit(&empty_bar[1]);
      }
      __syncwarp();
    }
    for (int32_t i = 0; i < steps && ok; ++i) {
      const int32_t y0 = 2 * i, y1 = 2 * i + 1;
      const bool more = i + 1 < steps;
      ok = warp_wait_all(p_bar, i & 1, p.err, 64, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      const uint64_t b1 = ymn_desc + slot(PASS == kDq ? y0 : y1), b2 = ymn_desc + slot(y0);
      const uint64_t next0 = yk_desc + slot(y0 + 2), next1 = yk_desc + slot(y1 + 2);
      if (elect_one()) {
        issue_sums<Cfg::kCols>(tAcc1, tS, b1, id_acc, i > 0);
        if (PASS == kDkv) tc_commit(&empty_bar[y1 % Cfg::kStages]);
      }
      __syncwarp();
      if (more) {
        ok = take(y0 + 2, i + 1);
        if (!ok) break;
        if (elect_one()) {
          issue_scores<HD / 16>(tS, x0_desc, next0, id_s, ksteps);
          tc_commit(s_bar);
        }
        __syncwarp();
      }
      ok = warp_wait_all(ds_bar, i & 1, p.err, 65, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        issue_sums<Cfg::kCols>(tAcc2, tD, b2, id_acc, i > 0);
        tc_commit(more ? &empty_bar[y0 % Cfg::kStages] : acc_bar);
      }
      __syncwarp();
      if (more) {
        ok = take(y1 + 2, i + 1);
        if (!ok) break;
        if (elect_one()) {
          issue_scores<HD / 16>(tD, x1_desc, next1, id_s, ksteps);
          tc_commit(d_bar);
          if (PASS == kDq) tc_commit(&empty_bar[(y1 + 2) % Cfg::kStages]);
        }
        __syncwarp();
      }
    }
    // every MMA issued here is complete before TMEM is released
    if (elect_one()) tc_commit(done_bar);
    __syncwarp();
    warp_wait_all(done_bar, 0, nullptr, 68, p.wait_limit_ns);
  } else if (warp == 2 && PASS == kDkv) {
    // ----------------------------------------------- lse and delta of the queries
    // (loaded a step ahead, all at once: the threads wait for these as for the scores)
    int32_t tile = first, h = y_head;
    float l[4], d[4];
    auto fetch = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t q = tile * kTile + k * 32 + lane;
        const int64_t t = static_cast<int64_t>(h) * p.Tq + at.q0 + q;
        l[k] = q < at.nq ? p.lse[t] : -CUDART_INF_F;
        d[k] = q < at.nq ? p.delta[t] : 0.0f;
      }
      if (++tile == first + count) {
        tile = first;
        ++h;
      }
    };
    if (steps > 0) fetch();
    for (int32_t i = 0; i < steps; ++i) {
      const int b = i & 1;
      if (!warp_wait_all(&stat_empty[b], (i >> 1 & 1) ^ 1, p.err, 66, p.wait_limit_ns)) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // (a query that is none, or sees no key, has no probabilities)
        const bool none = l[k] == -CUDART_INF_F;
        stat[b * 2 * kTile + k * 32 + lane] = none ? CUDART_INF_F : l[k] * kLog2e;
        stat[b * 2 * kTile + kTile + k * 32 + lane] = none ? 0.0f : d[k];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[b]);
      if (i + 1 < steps) fetch();
    }
  } else if (warp >= 4 && at.tiles > 0) {
    // ------------------------------------------------------ probabilities, dS
    constexpr int kCols = Cfg::kCols, kDims = HD / Cfg::kParts;
    const int part = (warp >> 2) - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tS + lane_base + kCols * part, d_at = tD + lane_base + kCols * part;
    const int32_t x = x0 + row;                           // in the sequence
    const bool valid = x < nx;
    const int64_t token = x_row + static_cast<int64_t>(row);
    // sum over a row's parts, in order
    auto over_parts = [&](float v) {
      stat[part * kTile + row] = v;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * Cfg::kWarps) : "memory");
      v = stat[row];
#pragma unroll
      for (int i = 1; i < Cfg::kParts; ++i) v += stat[i * kTile + row];
      asm volatile("bar.sync 1, %0;" ::"n"(32 * Cfg::kWarps) : "memory");
      return v;
    };
    float lse = 0.0f, delta = 0.0f, e = 0.0f;             // kDq: of this row; what delta lacks
    if (PASS == kDq) {
      if (valid) {
        lse = p.lse[head * p.Tq + token] * kLog2e;
        const int32_t c0 = part * kDims;
        delta = dot_row(p.dout.row(token, head) + c0, p.o.row(token, head) + c0,
                        min(max(p.dim - c0, 0), kDims));
      }
      delta = over_parts(delta);
    }
    // kDq: keys that this row sees; kDkv: the first query that sees this row
    const int32_t bound = PASS == kDq ? (p.causal ? min(at.nk, x + off + 1) : at.nk)
                                      : (p.causal ? x - off : 0);
    bool ok = true;
    int32_t tile = first;
    for (int32_t i = 0; i < steps; ++i) {
      const float* st = stat + (i & 1) * 2 * kTile + part * kCols;
      if (PASS == kDkv) ok = warp_wait_all(&stat_full[i & 1], i >> 1 & 1, p.err, 69, p.wait_limit_ns);
      ok = ok && warp_wait_all(s_bar, i & 1, p.err, 70, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      float s[kCols];
      tmem_ld_32x32b_x32(s_at, s);
      tmem_ld_wait();
      const int32_t lim = bound - tile * kTile - kCols * part;   // of this part's columns
      if (PASS == kDq) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) s[c] = exp2_fast(fmaf(s[c], p.scale_log2, -lse));
        if (__any_sync(0xffffffffu, lim < kCols)) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = c < lim ? s[c] : 0.0f;
        }
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 l = *reinterpret_cast<const float4*>(st + c);
          s[c] = exp2_fast(fmaf(s[c], p.scale_log2, -l.x));
          s[c + 1] = exp2_fast(fmaf(s[c + 1], p.scale_log2, -l.y));
          s[c + 2] = exp2_fast(fmaf(s[c + 2], p.scale_log2, -l.z));
          s[c + 3] = exp2_fast(fmaf(s[c + 3], p.scale_log2, -l.w));
        }
        if (__any_sync(0xffffffffu, lim > 0)) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = c >= lim ? s[c] : 0.0f;
        }
      }
      uint32_t w[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) w[c] = pack_bf16x2(s[2 * c], s[2 * c + 1]);
      tmem_st_32x32b_x16(s_at, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_bar);

      ok = warp_wait_all(d_bar, i & 1, p.err, 71, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      float d[kCols];
      tmem_ld_32x32b_x32(d_at, d);
      tmem_ld_wait();
      if (PASS == kDq) {
        float sum[4] = {};
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          d[c] = s[c] * (d[c] - delta);
          sum[c & 3] += d[c];
        }
        e += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 l = *reinterpret_cast<const float4*>(st + kTile + c);
          d[c] = s[c] * (d[c] - l.x);
          d[c + 1] = s[c + 1] * (d[c + 1] - l.y);
          d[c + 2] = s[c + 2] * (d[c + 2] - l.z);
          d[c + 3] = s[c + 3] * (d[c + 3] - l.w);
        }
      }
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) w[c] = pack_bf16x2(d[2 * c], d[2 * c + 1]);
      tmem_st_32x32b_x16(d_at, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_bar);
        if (PASS == kDkv) mbar_arrive(&stat_empty[i & 1]);
      }
      if (++tile == first + count) tile = first;
    }
    if (ok && steps > 0) ok = warp_wait_all(acc_bar, 0, p.err, 72, p.wait_limit_ns);
    tc_fence_after();
    if (PASS == kDq) {
      e = over_parts(e);
      if (valid && part == 0) p.delta[head * p.Tq + token] = delta + e;
    }
    if (ok) {
#pragma unroll
      for (int c = part * kDims; c < (part + 1) * kDims; c += 16) {
        float a1[16], a2[16];
        if (steps > 0) {
          tmem_ld_32x32b_x16(tAcc1 + lane_base + c, a1);
          tmem_ld_32x32b_x16(tAcc2 + lane_base + c, a2);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) a1[k] = a2[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 8) {
          if (valid && c + k < p.dim) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              f[j] = p.scale * (PASS == kDq ? fmaf(-e, a1[k + j], a2[k + j]) : a2[k + j]);
            *reinterpret_cast<uint4*>(p.g2.row(token, head) + c + k) = pack8(f);
            if (PASS == kDkv) {
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = a1[k + j];
              *reinterpret_cast<uint4*>(p.g1.row(token, head) + c + k) = pack8(f);
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, int PASS>
cudaError_t launch_pass(const BwdParams& p, int64_t tiles, cudaStream_t stream) {
  using Cfg = BwdCfg<HD>;
  const auto kern = attention_bwd_kernel<HD, PASS>;
  static std::atomic<bool> ready[64];    // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.heads), 1, 1);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_attention_bwd(const AttentionArgs& a, cudaStream_t stream) {
  const boost_attention_desc& d = a.d;
  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  CUtensorMap q, k, v, dout;
  if (!heads_map(&q, a.q.at, a.ws, d.Tq, d.hq, d.dim, d.q_ts, d.q_hs, 1, kTile) ||
      !heads_map(&k, a.k.at, a.ws, d.Tk, d.hk, d.dim, d.k_ts, d.k_hs, 1, kTile) ||
      !heads_map(&v, a.v.at, a.ws, d.Tk, d.hk, d.dim, d.v_ts, d.v_hs, 1, kTile) ||
      !heads_map(&dout, a.dout.at, a.ws, d.Tq, d.hq, d.dim, d.do_ts, d.do_hs, 1, kTile))
    return cudaErrorInvalidValue;
  p.lse = a.lse;
  p.delta = reinterpret_cast<float*>(static_cast<char*>(a.ws) + 256);
  p.q_starts = a.q_starts;
  p.k_starts = a.k_starts;
  p.Tq = d.Tq;
  p.Tk = d.Tk;
  p.group = d.hq / d.hk;
  p.dim = d.dim;
  p.sequences = d.sequences;
  p.causal = d.causal;
  p.scale = d.scale;
  p.scale_log2 = d.scale * kLog2e;
  p.err = static_cast<DeviceError*>(a.ws);
  p.wait_limit_ns = wait_limit_ns();
  if (d.Tq > 0) {
    p.tmX0 = q;
    p.tmX1 = dout;
    p.tmY0 = k;
    p.tmY1 = v;
    p.o = a.o;
    p.dout = a.dout;
    p.g2 = a.dq;
    p.heads = d.hq;
    const int64_t tiles = most_tiles(d.Tq, kTile, d.sequences);
    const cudaError_t e = d.dim <= 64 ? launch_pass<64, kDq>(p, tiles, stream)
                                      : launch_pass<128, kDq>(p, tiles, stream);
    if (e != cudaSuccess) return e;
  }
  if (d.Tk == 0) return cudaSuccess;
  p.tmX0 = k;
  p.tmX1 = v;
  p.tmY0 = q;
  p.tmY1 = dout;
  p.g1 = a.dv;
  p.g2 = a.dk;
  p.heads = d.hk;
  const int64_t tiles = most_tiles(d.Tk, kTile, d.sequences);
  return d.dim <= 64 ? launch_pass<64, kDkv>(p, tiles, stream)
                     : launch_pass<128, kDkv>(p, tiles, stream);
}

}  // namespace boost_gb300
