// attention_fwd.cu -- softmax attention over packed sequences on the tensor cores.
//
// A CTA has two tiles of 128 query rows of a head (A and B) and goes once through the keys they
// see, 128 at a time: S = Q K^T into TMEM, one thread a row takes its scores, keeps the running
// maximum and sum, and writes P = 2^(c S - c m) back over them as bf16, which the second product
// reads from there (O += P V, in TMEM too). While one tile's softmax runs, the tensor core has the
// other's products. Warp 0 loads K and V tiles through a ring, warp 1 issues, warps 4..7 and 8..11
// are the rows of A and of B.
//
// The maximum that P is taken against only moves when a row's true maximum passes it by more than
// 2^8 (in the exponent's units: P <= 256, sums in fp32 and a bf16 P lose nothing by that), so O is
// hardly ever rescaled. P is rounded to bf16 as the second product's operand; the sum takes it
// before that.
//
// Query heads that share a key head share a tile: its rows are `pack` heads of 128 / pack tokens.
// Where the tiles leave SMs idle, a tile's keys are split, and the parts (fp32, with their own
// sums) joined in order by a second kernel: into equal parts, or, where all queries are a
// single tile's (a decoding step), into parts of a fixed number of key tiles, so that long and
// short sequences fill the SMs alike. There A and B are the same queries, A with the even and B
// with the odd tiles of a part: two steps of a chain of load, product, softmax, product at a time.
//
// Measured: 16384 tokens in four sequences, 16 heads of 128, 379 us (1.45 PFLOP/s), causal 225 (1.22),
// in bursts at 2070 MHz, as all times here (one after another, at the 1920 MHz that the power cap
// leaves, 397 and 233). A step of both tiles takes the tensor core 2048 cycles and lasts about 3000: what bounds it is each
// tile's chain (scores, softmax of a row in one thread, product) and the issuing warp's waits for
// both (tensor pipe 53-60% busy, issue slots 35%). Not faster: CTAs that go from tile to tile (290-320
// us causal), CTA pairs, two threads a row (spills), an issuing warp for each tile (567 us), the next
// K and V awaited behind queued products (409), P handed over whole (405) or its second half's
// exponents begun before the first is handed over (377). Decoding: a token of eight sequences of 1 to
// 16384 keys, 40 heads over 8: 53 us, 4.6 TB/s of their keys and values.
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "attention.cuh"
#include "attention_tc.cuh"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

struct FwdParams {
  CUtensorMap tmQ, tmK, tmV;             // boxes of 64 values x (pack heads x tok tokens, 128 rows)
  HeadsOut out;
  float* lse;                            // [hq, Tq] or NULL
  const int32_t *q_starts, *k_starts;
  float *part, *part_lse;                // of the splits: [splits, Tq, hq, dim], [splits, Tq, hq]
  int64_t Tq, Tk;
  int32_t hq, dim, sequences, causal;
  int32_t pack, tok;                     // heads and tokens of a tile
  Order order;                           // of hq / pack heads
  int32_t group;                         // of them that share a key head
  int32_t splits, chunk;                 // equal parts of a tile's keys; or key tiles of a part (or 0)
  float scale_log2;
  DeviceError* err;
  uint64_t wait_limit_ns;
};

template <int HD>
struct FwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = HD == 128 ? 5 : 8;
  static constexpr int kBars = 2 * kStages + 10;
  static constexpr int kBarOffset = (2 + kStages) * kTileBytes;
  static constexpr int kSmemBytes = 1024 + kBarOffset + 8 * kBars + 16;
  static constexpr int kThreads = 384;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

constexpr float kSlack = 8.0f;           // log2 of the largest P

template <int HD, bool OWN>
__global__ void __launch_bounds__(FwdCfg<HD>::kThreads, 1)
    attention_fwd_kernel(const __grid_constant__ FwdParams p) {
  using Cfg = FwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                   // A, B
  uint8_t* sKV = smem + 2 * Cfg::kTileBytes;            // K(0), V(0), K(1), ...
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOffset);
  uint64_t* empty_bar = full_bar + Cfg::kStages;
  uint64_t* q_bar = empty_bar + Cfg::kStages;
  uint64_t* s_bar = q_bar + 1;                          // [2] scores are complete
  uint64_t* p_bar = s_bar + 2;                          // [2][2] a half of P is written
  uint64_t* o_bar = p_bar + 4;                          // [2] the last product is complete
  uint64_t* done_bar = o_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(q_bar, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_bar[x], 1);
      mbar_init(&p_bar[2 * x], 4);
      mbar_init(&p_bar[2 * x + 1], 4);
      mbar_init(&o_bar[x], 1);
    }
    mbar_init(done_bar, 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmQ);
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 256 + HD};
  griddep_wait();
  griddep_launch_dependents();

  // This CTA's pair of tiles, longest rows first.
  const int32_t span = p.order.set * p.order.tiles;
  const int32_t first_head = static_cast<int32_t>(blockIdx.x) / span * p.order.set;
  const int32_t set = min(p.order.set, p.order.heads - first_head);
  const int32_t in_set = static_cast<int32_t>(blockIdx.x) % span, head = first_head + in_set % set;
  constexpr bool own = OWN;                                       // A and B have keys of their own
  Place at = find_tile(p.q_starts, p.k_starts, p.Tq, p.Tk, p.sequences, in_set / set,
                       own ? p.chunk * kTile : 2 * p.tok, own);
  const int32_t t0 = own ? 0 : (at.tiles - 1 - at.tile) * 2 * p.tok;   // first token in the sequence
  const int32_t apart = own ? 0 : p.tok;                          // from A's to B's
  const int32_t off = at.nk - at.nq;                              // keys before the first query
  // key tiles [first, first + n) of each, and of this split alone
  int32_t n[2], first = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int32_t begin = t0 + x * apart, last = min(begin + p.tok, at.nq) - 1;
    int32_t keys = 0;
    if (at.tiles > 0 && last >= begin) keys = p.causal ? min(at.nk, last + off + 1) : at.nk;
    n[x] = keys > 0 ? (keys + kTile - 1) / kTile : 0;
  }
  if (own) {
    first = at.tile * p.chunk;
    const int32_t all = max(min(n[0] - first, p.chunk), 0);
    n[0] = (all + 1) / 2;
    n[1] = all / 2;
  } else if (p.splits > 1) {
    const int32_t most = max(n[0], n[1]), each = (most + p.splits - 1) / p.splits;
    first = static_cast<int32_t>(blockIdx.y) * each;
    n[0] = max(min(n[0] - first, each), 0);
    n[1] = max(min(n[1] - first, each), 0);
  }
  const int32_t steps = own ? n[0] + n[1] : max(n[0], n[1]);      // key tiles
  const int ksteps = (p.dim + 15) / 16;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t armed = 0, parities = 0;
    if (steps > 0) {
      const int32_t kh = head / p.group;
      const uint32_t q_bytes = Cfg::kBoxes * 128 * p.pack * p.tok;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_bar, ((n[0] > 0) + (n[1] > 0)) * q_bytes);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (n[x] > 0)
            for (int b = 0; b < Cfg::kBoxes; ++b)
              tma_load_3d(sQ + x * Cfg::kTileBytes + b * kBoxBytes, &p.tmQ, q_bar, 64 * b,
                          head * p.pack, at.q0 + t0 + x * apart);
      }
      __syncwarp();
      int stage = 0;
      uint32_t phase = 0;
      // K of the first step (of A's and B's); then V and the K that comes next
      const int32_t ahead = own ? min(2, steps) : 1;
      for (int32_t i = 0; i < 2 * steps; ++i) {
        int32_t tile = i;
        bool v = false;
        if (i >= ahead) {
          const int32_t r = i - ahead, whole = 2 * (steps - ahead);
          v = r >= whole || !(r & 1);
          tile = r >= whole ? steps - ahead + r - whole : (r >> 1) + (v ? 0 : ahead);
        }
        if (!warp_wait_all(&empty_bar[stage], phase ^ 1u, p.err, 41, p.wait_limit_ns)) break;
        armed |= 1u << stage;
        parities = (parities & ~(1u << stage)) | (phase << stage);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full_bar[stage], Cfg::kTileBytes);
          for (int b = 0; b < Cfg::kBoxes; ++b)
            tma_load_3d(sKV + stage * Cfg::kTileBytes + b * kBoxBytes, v ? &p.tmV : &p.tmK,
                        &full_bar[stage], 64 * b, kh, at.k0 + (first + tile) * kTile);
        }
        __syncwarp();
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the copies started here have landed before the CTA exits
      for (int s = 0; s < Cfg::kStages; ++s)
        if (armed >> s & 1u)
          warp_wait_all(&full_bar[s], parities >> s & 1u, nullptr, 47, p.wait_limit_ns);
      warp_wait_all(q_bar, 0, nullptr, 47, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t id_s = idesc_bf16_f32(kTile, kTile, 0, 0);
    const uint32_t id_o = idesc_bf16_f32(kTile, 16 * ksteps, 0, 1);
    const uint64_t q_desc[2] = {desc_k_major(smem_u32(sQ)),
                                desc_k_major(smem_u32(sQ) + Cfg::kTileBytes)};
    const uint64_t k_desc = desc_k_major(smem_u32(sKV)), v_desc = desc_mn_major(smem_u32(sKV));
    constexpr uint32_t kStep = Cfg::kTileBytes >> 4;
    int stage = 0;
    uint32_t phase = 0;
    auto next = [&]() {
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    bool ok = steps > 0 && warp_wait_all(q_bar, 0, p.err, 42, p.wait_limit_ns) &&
              warp_wait_all(&full_bar[0], 0, p.err, 43, p.wait_limit_ns);
    // tiles of their own: tile i is A's or B's in turn
    for (int32_t i = -2; own && ok && i < steps; ++i) {
      const int x = i & 1;
      const uint32_t s_tm = tS[0] + kTile * x;
      if (i >= 0) {                                      // O_x += P_x V
        const int32_t left = at.nk - (first + i) * kTile;
        ok = warp_wait_all(&full_bar[stage], phase, p.err, 44, p.wait_limit_ns);
        if (ok && left < kTile)
          zero_rows(sKV + stage * Cfg::kTileBytes, Cfg::kBoxes, kTile, left, lane);
        ok = ok && warp_wait_all(&p_bar[2 * x], i >> 1 & 1, p.err, 46, p.wait_limit_ns) &&
             warp_wait_all(&p_bar[2 * x + 1], i >> 1 & 1, p.err, 46, p.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = v_desc + stage * kStep;
        if (elect_one()) {
          issue_sums<1, kTile>(tO[0] + HD * x, s_tm, vd, id_o, i > 1);
          tc_commit(&empty_bar[stage]);
          if (i + 2 >= steps) tc_commit(&o_bar[x]);
        }
        __syncwarp();
        next();
      }
      if (i + 2 < steps) {                               // S_x = Q K^T
        ok = warp_wait_all(&full_bar[stage], phase, p.err, 45, p.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = k_desc + stage * kStep;
        if (elect_one()) {
          issue_scores<1, HD / 16>(s_tm, q_desc[0], kd, id_s, ksteps);
          tc_commit(&s_bar[x]);
          tc_commit(&empty_bar[stage]);
        }
        __syncwarp();
        next();
      }
    }
    if (ok && !own) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (n[x] > 0) {
            issue_scores<1, HD / 16>(tS[x], q_desc[x], k_desc, id_s, ksteps);
            tc_commit(&s_bar[x]);
          }
        tc_commit(&empty_bar[0]);
      }
      __syncwarp();
      next();
    }
    for (int32_t j = 0; j < steps && ok && !own; ++j) {
      const int v_stage = stage;
      ok = warp_wait_all(&full_bar[stage], phase, p.err, 44, p.wait_limit_ns);
      next();
      const bool more = j + 1 < steps;
      if (ok && more) ok = warp_wait_all(&full_bar[stage], phase, p.err, 45, p.wait_limit_ns);
      if (!ok) break;
      const int32_t left = at.nk - (first + j) * kTile;
      if (left < kTile) zero_rows(sKV + v_stage * Cfg::kTileBytes, Cfg::kBoxes, kTile, left, lane);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j < n[x]) {
          // O_x += P_x V; the first half's products run while the threads work on the second
          const uint64_t vd = v_desc + v_stage * kStep, kd = k_desc + stage * kStep;
          ok = warp_wait_all(&p_bar[2 * x], j & 1, p.err, 46, p.wait_limit_ns);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) issue_sums<1, kTile, 0, 1, 4>(tO[x], tS[x], vd, id_o, j > 0);
          __syncwarp();
          ok = warp_wait_all(&p_bar[2 * x + 1], j & 1, p.err, 46, p.wait_limit_ns);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_sums<1, kTile, 4>(tO[x], tS[x], vd, id_o, true);
            if (j + 1 < n[x]) {
              issue_scores<1, HD / 16>(tS[x], q_desc[x], kd, id_s, ksteps);
              tc_commit(&s_bar[x]);
            } else {
              tc_commit(&o_bar[x]);
            }
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      if (elect_one()) {
        tc_commit(&empty_bar[v_stage]);
        if (more) tc_commit(&empty_bar[stage]);
      }
      __syncwarp();
      if (more) next();
    }
    // every MMA issued here is complete before TMEM is released
    if (elect_one()) tc_commit(done_bar);
    __syncwarp();
    warp_wait_all(done_bar, 0, nullptr, 48, p.wait_limit_ns);
  } else if (warp >= 4 && at.tiles > 0) {
    // -------------------------------------------------------------- softmax
    const int x = (warp >> 2) - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tS[x] + lane_base, o_at = tO[x] + lane_base;
    const int32_t tq = t0 + x * apart + row / p.pack;     // token in the sequence
    const bool valid = row < p.pack * p.tok && tq < at.nq;
    // keys that this row sees, from its first tile, and how far its tiles are apart
    const int32_t sees =
        (p.causal ? min(at.nk, tq + off + 1) : at.nk) - (first + (own ? x : 0)) * kTile;
    const int32_t step = own ? 2 * kTile : kTile;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    float m = -CUDART_INF_F, l = 0.0f;                    // reference in S's units, sum of P
    bool ok = true;
    for (int32_t j = 0; j < n[x]; ++j) {
      if (!warp_wait_all(&s_bar[x], j & 1, p.err, 49, p.wait_limit_ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld_32x32b_x32(s_at + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
      tmem_ld_wait();
      const int32_t lim = sees - j * step;
      if (__any_sync(0xffffffffu, lim < kTile)) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < lim ? s[c] : -CUDART_INF_F;
      }
      float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 128; c += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = fmaxf(t[i], s[c + i]);
      const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
      const bool raise = (top - m) * p.scale_log2 > kSlack || (m == -CUDART_INF_F && top > m);
      if (__any_sync(0xffffffffu, raise)) {
        const float to = raise ? top : m;
        const float f = to == m ? 1.0f : exp2_fast((m - to) * p.scale_log2);
        m = to;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < 16 * ksteps; c += 16) {
            float o[16];
            tmem_ld_32x32b_x16(o_at + c, o);
            tmem_ld_wait();
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * f);
            tmem_st_32x32b_x16(o_at + c, w);
          }
        }
      }
      // (a row that sees nothing yet: all its scores are -inf, and so are their exponents)
      const float shift = m == -CUDART_INF_F ? 0.0f : -m * p.scale_log2;
      const float2 shift2 = make_float2(shift, shift);
      float2 sum[2] = {};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const int c = 64 * half + k;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float2 x = fma2(make_float2(s[c + i], s[c + i + 1]), scale2, shift2);
            s[c + i] = exp2_fast(x.x);
            s[c + i + 1] = exp2_fast(x.y);
            sum[i / 2] = add2(sum[i / 2], make_float2(s[c + i], s[c + i + 1]));
          }
          w[k / 2] = pack_bf16x2(s[c], s[c + 1]);
          w[k / 2 + 1] = pack_bf16x2(s[c + 2], s[c + 3]);
        }
        tmem_st_32x32b_x32(s_at + 32 * half, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_bar[2 * x + half]);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // O / l, and the logarithm of the sum
    if (ok && n[x] > 0) ok = warp_wait_all(&o_bar[x], 0, p.err, 50, p.wait_limit_ns);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // (NaN stays)
      const float lse2 = l == 0.0f ? -CUDART_INF_F : fmaf(m, p.scale_log2, __log2f(l));
      const int64_t token = at.q0 + static_cast<int64_t>(tq);
      const int32_t h = head * p.pack + row % p.pack;
      __nv_bfloat16* dst = p.out.row(token, h);
      const bool parts = own || p.splits > 1;
      const int32_t part_index = own ? 2 * at.tile + x : static_cast<int32_t>(blockIdx.y);
      const int64_t item = (static_cast<int64_t>(part_index) * p.Tq + token) * p.hq + h;
      float* part = p.part + item * p.dim;
      if (valid) {
        if (parts)
          p.part_lse[item] = lse2;
        else if (p.lse != nullptr)
          p.lse[h * p.Tq + token] = lse2 * kLn2;
      }
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        if (n[x] > 0) {
          tmem_ld_32x32b_x32(o_at + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          if (valid && c + i < p.dim) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = inv == 0.0f ? 0.0f : o[i + e] * inv;
            if (parts) {
              *reinterpret_cast<float4*>(part + c + i) = make_float4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<float4*>(part + c + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
            } else {
              *reinterpret_cast<uint4*>(dst + c + i) = pack8(f);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a row's keys: WARPS of a block take a row of one head, each parts in turn, and
// the warps' sums are added in their order. (Many parts, a block a row: a warp alone took 22 us for
// the 100 parts of the longest of eight rows of 40 heads, one load after another, a block 4. Few
// parts of many rows, a warp a row: 2048 tokens of 4 heads in four parts take 25 us in all, with a
// block a row 47.)
template <int WARPS>
__global__ void __launch_bounds__(kThreads) attention_join_kernel(const FwdParams p) {
  pdl_enter();
  constexpr int kWarps = kThreads / 32;
  static_assert(WARPS == 1 || WARPS == kWarps, "a warp or a block");
  __shared__ float4 sums[WARPS][32];
  __shared__ float tops[WARPS], totals[WARPS];
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const int64_t rows = p.Tq * p.hq;
  const int64_t item = WARPS == 1 ? static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)
                                  : static_cast<int64_t>(blockIdx.x);
  if (item >= rows) return;
  const int32_t token = static_cast<int32_t>(item / p.hq), h = static_cast<int32_t>(item % p.hq);
  int32_t keys = -1;                                     // rows of no sequence stay
  for (int s = lane; s < p.sequences; s += 32) {
    int32_t q0, nq, k0, nk;
    sequence_bounds(p.q_starts, p.Tq, s, q0, nq);
    sequence_bounds(p.k_starts, p.Tk, s, k0, nk);
    if (token >= q0 && token < q0 + nq) keys = nk;
  }
  keys = __reduce_max_sync(0xffffffffu, keys);
  if (keys < 0) return;                                  // (all of the row's warps)
  // (a sequence has two parts for each `chunk` tiles of its keys)
  const int32_t step = p.chunk * kTile, parts = step > 0 ? 2 * ((keys + step - 1) / step) : p.splits;
  float top = -CUDART_INF_F, sum = 0.0f, o[4] = {};
  const int c = lane * 4;
  for (int i0 = warp; i0 < parts; i0 += 4 * WARPS) {
    float l[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * WARPS;
      l[k] = -CUDART_INF_F;
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < parts) {
        l[k] = p.part_lse[i * rows + item];
        if (c < p.dim) v[k] = *reinterpret_cast<const float4*>(p.part + (i * rows + item) * p.dim + c);
      }
    }
    float next = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) next = fmaxf(next, l[k]);
    const float base = next == -CUDART_INF_F ? 0.0f : next, f = exp2_fast(top - base);
    sum *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= f;
    top = next;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = exp2_fast(l[k] - base);
      sum += w;
      if (w != 0.0f) {                                   // (a part of no keys counts nothing)
        o[0] = fmaf(w, v[k].x, o[0]); o[1] = fmaf(w, v[k].y, o[1]);
        o[2] = fmaf(w, v[k].z, o[2]); o[3] = fmaf(w, v[k].w, o[3]);
      }
    }
  }
  if constexpr (WARPS > 1) {
    sums[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) {
      tops[warp] = top;
      totals[warp] = sum;
    }
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int i = 1; i < WARPS; ++i) top = fmaxf(top, tops[i]);
    const float base = top == -CUDART_INF_F ? 0.0f : top;
    sum = o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const float w = exp2_fast(tops[i] - base);
      const float4 v = sums[i][lane];
      sum = fmaf(w, totals[i], sum);
      if (w != 0.0f) {
        o[0] = fmaf(w, v.x, o[0]); o[1] = fmaf(w, v.y, o[1]);
        o[2] = fmaf(w, v.z, o[2]); o[3] = fmaf(w, v.w, o[3]);
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (c < p.dim)
    *reinterpret_cast<uint2*>(p.out.row(token, h) + c) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[h * p.Tq + token] = (top + __log2f(sum)) * kLn2;
}

// Heads that share a tile's rows.
int packed_heads(const boost_attention_desc& d) {
  const int group = d.hq / d.hk;
  // (128 / 33 tokens would leave a fifth of the rows idle. A token of 32 sequences of 4096 keys, heads
  // over one: 32 heads 19 us; 48 heads, each with a tile of its own, 367.)
  return group <= 32 ? group : 1;
}

// How a call's work is cut.
struct FwdPlan {
  int pack, tok, splits, chunk, parts;
  int64_t tiles;                         // of a head: pairs of tiles of queries, or parts of keys
};

FwdPlan plan(const boost_attention_desc& d) {
  FwdPlan f{};
  f.pack = packed_heads(d);
  f.tok = kTile / f.pack;
  f.splits = f.parts = 1;
  const int64_t heads = d.hq / f.pack, keys = (d.Tk + kTile - 1) / kTile;
  // All queries are a tile's: parts of the keys of a fixed length, two for each SM, but long
  // enough that the parts' own traffic stays below half of the keys' and values'. (A token of eight
  // sequences of 1 to 16384 keys, 40 heads, 8 of keys: 54 us, in equal parts 68; with three parts an
  // SM 55, with one 62. 32 x 2048 keys, 8 heads: 60, three 62, one 55.) Queries of more than a tile
  // go on below, where a sequence's keys are one CTA's: 25 tokens of 40 heads over 8, contexts of up to
  // 16384 keys of any length, 87 us (4.9 TB/s), 26 such tokens 168 (2.4); of 4096 keys each 79 and 95.
  if (d.Tq <= f.tok) {
    const int64_t rows = d.Tq / d.sequences * f.pack;
    const int64_t chunk = std::max<int64_t>({4, rows / 16, (keys * heads + 303) / 304});
    if (keys > chunk) {
      f.chunk = static_cast<int>(std::min<int64_t>(chunk, 1 << 20));
      f.parts = static_cast<int>(2 * ((keys + f.chunk - 1) / f.chunk));
      f.tiles = most_tiles(d.Tk, static_cast<int64_t>(f.chunk) * kTile, d.sequences);
      return f;
    }
  }
  // Else as many equal parts as an SM each takes at once, with four tiles of an average sequence's
  // keys or more. (512 queries over 8192 keys, 8 heads: 30 us, in one part 100; 300 over 6000, 2
  // heads: 23, one 76, parts of two tiles 21; 512 over 512, 8 heads: 14.5 in one part, 18.6 in parts
  // of two tiles.)
  f.tiles = most_tiles(d.Tq, 2 * f.tok, d.sequences);
  const int64_t each = (d.Tq + d.sequences - 1) / d.sequences;
  const int64_t ctas = (each + 2 * f.tok - 1) / (2 * f.tok) * d.sequences * heads;
  if (ctas > 0)
    f.splits = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>({152 / ctas, d.Tk / d.sequences / kTile / 4, 64})));
  f.parts = f.splits;
  return f;
}

template <int HD, bool OWN>
cudaError_t launch_fwd(const FwdParams& p, cudaStream_t stream) {
  using Cfg = FwdCfg<HD>;
  const auto kern = attention_fwd_kernel<HD, OWN>;
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
  cfg.gridDim = dim3(static_cast<unsigned>(p.order.tiles * p.order.heads), p.splits, 1);
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

size_t attention_workspace(const boost_attention_desc& d) {
  const FwdPlan f = plan(d);
  const size_t rows = static_cast<size_t>(d.hq) * d.Tq;
  const size_t fwd = f.parts > 1 ? 4 * f.parts * rows * (d.dim + 1) : 0;
  return 256 + std::max(fwd, 4 * rows);                  // (the backward keeps a value a row)
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t stream) {
  const boost_attention_desc& d = a.d;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  const FwdPlan f = plan(d);
  p.pack = f.pack;
  p.tok = f.tok;
  p.group = d.hq / p.pack / d.hk;
  // With a causal mask a set of heads ends with its shortest tiles, and the next begins with long ones:
  // few and equal sets, of about 96 MB. (16384 tokens in four sequences, causal: 16 heads 222 us in one
  // set, 254 in sets of three heads; 32 heads 437 in three sets, 457 in one. Without the mask, where
  // all tiles have as much, 16 heads 418 in one set and 402 in sets of 32 MB.)
  p.order = grid_order(d.hq / p.pack, f.tiles, 4.0 * d.dim * d.Tk / p.group, d.causal ? 96e6 : 32e6);
  if (!heads_map(&p.tmQ, a.q.at, a.ws, d.Tq, d.hq, d.dim, d.q_ts, d.q_hs, p.pack, p.tok) ||
      !heads_map(&p.tmK, a.k.at, a.ws, d.Tk, d.hk, d.dim, d.k_ts, d.k_hs, 1, kTile) ||
      !heads_map(&p.tmV, a.v.at, a.ws, d.Tk, d.hk, d.dim, d.v_ts, d.v_hs, 1, kTile))
    return cudaErrorInvalidValue;
  p.out = a.out;
  p.lse = a.lse;
  p.q_starts = a.q_starts;
  p.k_starts = a.k_starts;
  p.Tq = d.Tq;
  p.Tk = d.Tk;
  p.hq = d.hq;
  p.dim = d.dim;
  p.sequences = d.sequences;
  p.causal = d.causal;
  p.splits = f.splits;
  p.chunk = f.chunk;
  p.scale_log2 = d.scale * kLog2e;
  p.err = static_cast<DeviceError*>(a.ws);
  p.wait_limit_ns = wait_limit_ns();
  const int64_t rows = d.Tq * d.hq;
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + 256);
  p.part_lse = p.part + f.parts * rows * d.dim;
  cudaError_t e = cudaSuccess;
  if (f.tiles > 0 && f.chunk > 0)
    e = d.dim <= 64 ? launch_fwd<64, true>(p, stream) : launch_fwd<128, true>(p, stream);
  else if (f.tiles > 0)
    e = d.dim <= 64 ? launch_fwd<64, false>(p, stream) : launch_fwd<128, false>(p, stream);
  if (e != cudaSuccess || f.parts == 1) return e;
  prof_note_kernels(1);
  constexpr int kWarps = kThreads / 32;
  if (f.parts > 2 * kWarps) return launch_k(attention_join_kernel<kWarps>, rows, stream, p);
  return launch_k(attention_join_kernel<1>, (rows + kWarps - 1) / kWarps, stream, p);
}

}  // namespace boost_gb300
