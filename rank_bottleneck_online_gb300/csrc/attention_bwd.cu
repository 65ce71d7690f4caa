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
// delta from out and sums what is missing, e = sum_j P (dP - delta), beside sum_j P k in TMEM, and
// the second pass reads delta + e. (Without that the gradients of 77 tokens were off by 0.0030,
// relative to all, with it by the 0.002 of a bf16 result and bf16 dS.) A row's dS sum to 0, so what
// its keys have in common has no part in dq, but has in the sum's error by dS's rounding: dq = scale
// (sum dS k - r sum P k) with r, e's sum over dS as rounded, in place of e. (Heads of 40
// values, scores spread by up to 4, 6641 tokens: dq off by 1.50 times a bf16 result's rounding with
// e, 1.32 with r; it costs 1%.)
//
// A tile of 128 x 128 products takes 512 cycles of the tensor core, and reads 128 bytes a cycle of
// shared memory while both operands lie there, which is all that there is: the loads' writes cost
// time. So with heads of more than 64 values a pair of CTAs works on 256 rows: each has half of
// the other side's tile, once split along its rows (for S and dP) and once along its values (for
// the sums), and half the reads. Shorter sequences, whose last rows leave a CTA of the pair idle
// and which wait for their pair at each end of a work, take single CTAs.
//
// Warp 0 loads the tiles, each through two buffers, warp 1 issues the products, warp 2 fetches lse
// and delta (the first pass's a work ahead, the second's a step), warp 3 the next work, sixteen
// warps are the rows of a tile, four threads a row. The products of one kind run while the threads
// work on the other's scores: acc1 += P B and the next S during dS, acc2 += dS Y0 and the next dP
// during P.
//
// Measured, both passes: 16384 tokens in four sequences, 16 heads of 128, 1280 us (1.07 PFLOP/s by the
// formula's 5 products, 1.72 by the 8 done), causal 736, in bursts at 2070 MHz, as all times here;
// one after another the power cap leaves 1700 to 1850 MHz, and they take 1390 and 790. A step of four products takes the tensor
// core 2048 cycles and lasts about 2800 in the first pass and 2600 in the second (tensor pipe 66%
// and 72% busy): the chain from a product over the threads' work to the next one. Between works pass
// about 9000 cycles. Not faster: P handed over whole (826 us causal, 797 then in halves), dS in halves
// (769, 753 then), a half's exponents begun before the one before is handed over (784), two sets of 64
// columns in turns (995, 961 then), two buffers of S for heads of 64 (416 us for 426, and 685 for
// 678).
#include <math_constants.h>

#include <atomic>
#include <cstring>

#include "attention.cuh"
#include "attention_tc.cuh"
#include "profile.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

enum Pass : int { kDq = 0, kDkv = 1 };

struct BwdParams {
  CUtensorMap tmX0, tmX1, tmY0, tmY1;    // boxes of 64 values x 64 rows of one head
  HeadsIn o, dout;                       // kDq
  HeadsOut g1, g2;                       // kDq: -, dq; kDkv: dv, dk
  const float* lse;                      // [hq, Tq]
  float* delta;                          // [hq, Tq]: written by kDq, read by kDkv
  const int32_t *q_starts, *k_starts;
  int64_t Tq, Tk;
  Order order;                           // of the tiles' side
  int32_t group;                         // query heads of a key head
  int32_t dim, sequences, causal;
  float scale, scale_log2;
  DeviceError* err;
  uint64_t wait_limit_ns;
};

// Tiles of the other side, as first met in a step: Y0 and Y1 as K-major operands, Y1 and Y0 as
// MN-major ones. A single CTA has both in one.
enum Kind : int { kY0k = 0, kY1k, kY1m, kY0m, kKinds };

template <int HD, int CG>
struct BwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kSlotBytes = kTileBytes / CG;     // of a loaded tile
  static constexpr int kSlotKinds = CG == 2 ? 4 : 2;
  static constexpr int kBars = 4 * kSlotKinds + 16;
  static constexpr int kStatOffset = 2 * kTileBytes + 2 * kSlotKinds * kSlotBytes;
  static constexpr int kParts = 4;                       // threads of a row
  static constexpr int kCols = kTile / kParts;           // of its scores, each
  // two buffers of lse and delta; kDq: and two of the parts of e and r
  static constexpr int kStatBytes = (4 + 4 * kParts) * 4 * kTile;
  static constexpr int kWarps = 4 * kParts;              // that work on the scores
  static constexpr int kStageOffset = kStatOffset + kStatBytes;   // 16 rows of 64 bytes a warp
  static constexpr int kSchedOffset = kStageOffset + kWarps * 1024;
  static constexpr int kBarOffset = kSchedOffset + 256;
  static constexpr int kSmemBytes = 1024 + kBarOffset + 8 * kBars + 16;
  static_assert(sizeof(Schedule) <= 256, "its place");
  static constexpr int kThreads = 128 + 32 * kWarps;
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(CG == 1 || HD == 128, "a half of a tile's values is a box");
};

// A work's rows of X (queries for kDq, longest rows first; keys for kDkv), and the tiles [first,
// first + count) of the other side that they see; kDkv has those once for each head of the group.
template <int CG, int PASS>
struct Tile {
  int32_t x0, nx, ny, off;               // first row, rows in the sequence; keys before its queries
  int32_t x_row, y_row, y_head;          // in the tensors
  int32_t first, count, steps;
  __device__ __forceinline__ Tile(const Work& w, const BwdParams& p, int rank) {
    const Place& at = w.at;
    off = at.nk - at.nq;
    const int32_t pair0 = (PASS == kDq ? at.tiles - 1 - at.tile : at.tile) * (CG * kTile);
    x0 = pair0 + rank * kTile;
    nx = PASS == kDq ? at.nq : at.nk;
    ny = PASS == kDq ? at.nk : at.nq;
    x_row = (PASS == kDq ? at.q0 : at.k0) + x0;
    y_row = PASS == kDq ? at.k0 : at.q0;
    y_head = PASS == kDq ? w.head / p.group : w.head * p.group;
    first = count = 0;
    if (w.head < 0 || at.tiles < 0) {
      nx = x0;                           // no rows
    } else if (PASS == kDq) {
      const int32_t keys = p.causal ? min(at.nk, min(pair0 + CG * kTile, at.nq) + off) : at.nk;
      count = keys > 0 ? (keys + kTile - 1) / kTile : 0;
    } else {
      first = p.causal ? max(pair0 - off, 0) / kTile : 0;
      count = max((at.nq + kTile - 1) / kTile - first, 0);
    }
    steps = PASS == kDq ? count : count * p.group;
  }
};

// Store 32 rows of a warp, each lane's DIMS values of its row (from value `col`, of `dim`), rows
// [row, row + rows) of a head: through 16 rows of shared memory at a time, so that neighbouring
// lanes store neighbouring bytes (16 bytes of 32 rows a store took about 4000 cycles a tile).
template <int DIMS>
__device__ __forceinline__ void store_rows(const HeadsOut& out, int32_t head, int32_t row,
                                           int32_t rows, int32_t col, int32_t dim,
                                           const uint32_t (&v)[DIMS / 2], uint8_t* stage, int lane) {
  constexpr int kPieces = DIMS / 8;      // of 16 bytes a row: 2 or 4
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncwarp();
    if (lane >> 4 == half) {
      const int r = lane & 15;
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        *reinterpret_cast<uint4*>(stage + r * 64 + ((c ^ (r >> 1)) & (kPieces - 1)) * 16) =
            make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPieces / 2; ++i) {
      const int r = i * (32 / kPieces) + lane / kPieces, c = lane % kPieces;
      const uint4 x =
          *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ (r >> 1)) & (kPieces - 1)) * 16);
      if (half * 16 + r < rows && col + c * 8 < dim)
        *reinterpret_cast<uint4*>(out.row(row + half * 16 + r, head) + col + c * 8) = x;
    }
  }
}

// Adds a pair of bf16 values to two sums, an instruction each.
__device__ __forceinline__ void add_bf16x2(float2& sum, uint32_t pair) {
  asm("{\n\t.reg .b16 x, y;\n\t"
      "mov.b32 {x, y}, %2;\n\t"
      "add.f32.bf16 %0, x, %0;\n\t"
      "add.f32.bf16 %1, y, %1;\n\t}"
      : "+f"(sum.x), "+f"(sum.y)
      : "r"(pair));
}

// Rounds s to bf16 as an operand in TMEM, pairs of columns a word: N / 2 words from `to` on; what that
// rounds off, where `fine`, as another operand `apart` words behind it. The rounded values are added
// to `kept`, if it is given.
template <int N>
__device__ __forceinline__ void store_operand(uint32_t to, uint32_t apart, const float* s, bool fine,
                                              float2* kept = nullptr) {
  static_assert(N == 16 || N == 32, "");
  uint32_t w[N / 2];
#pragma unroll
  for (int c = 0; c < N; c += 2) w[c / 2] = pack_bf16x2(s[c], s[c + 1]);
  if (kept != nullptr) {
#pragma unroll
    for (int c = 0; c < N / 2; ++c) add_bf16x2(kept[c & 1], w[c]);
  }
  if constexpr (N == 16) tmem_st_32x32b_x8(to, w); else tmem_st_32x32b_x16(to, w);
  if (fine) {
#pragma unroll
    for (int c = 0; c < N; c += 2)
      w[c / 2] = pack_bf16x2(s[c] - bf16_lo(w[c / 2]), s[c + 1] - bf16_hi(w[c / 2]));
    if constexpr (N == 16) tmem_st_32x32b_x8(to + apart, w); else tmem_st_32x32b_x16(to + apart, w);
  }
}

// Whether a call has few scores, of all heads and of up to 32 sequences: P and dS are two operands each
// then. Rounded once they put the gradients off by 1.3 to 1.4 times what a bf16 result alone is, at
// any size; but over few values that scatters (6 tokens of one head of 16: 1.14 to 1.61 times in nine
// draws of ten, up to 2; 200 tokens: 1.36 to 1.42), and the tensor cores have little else to do (77
// tokens, 16 heads, forward and backward: 35 us, 32 without). A short sequence among many is rounded
// once, as a long one: what is bounded here is a whole call's error. By a whole warp.
__device__ __forceinline__ bool few_scores(const BwdParams& p, int32_t heads) {
  if (p.sequences > 32) return false;
  constexpr int64_t kMost = 1 << 18;
  const int lane = threadIdx.x & 31;
  int64_t pairs = 0;
  if (lane < p.sequences) {
    int32_t q0, nq, k0, nk;
    sequence_bounds(p.q_starts, p.Tq, lane, q0, nq);
    sequence_bounds(p.k_starts, p.Tk, lane, k0, nk);
    const int64_t m = min(nq, nk);
    pairs = p.causal ? m * nk - m * (m - 1) / 2 : static_cast<int64_t>(nq) * nk;
  }
  const uint32_t all = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(min(pairs, kMost + 1)));
  return static_cast<int64_t>(all) * heads <= kMost;
}

template <int HD, int CG, int PASS, bool FINE>
__global__ void __launch_bounds__(BwdCfg<HD, CG>::kThreads, 1)
    attention_bwd_kernel(const __grid_constant__ BwdParams p) {
  using Cfg = BwdCfg<HD, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = smem;                                   // X0, X1
  uint8_t* sY = smem + 2 * Cfg::kTileBytes;             // two slots of each kind
  float* stat = reinterpret_cast<float*>(smem + Cfg::kStatOffset);
  // (full, x, p, ds and acc_free: the even CTA's of a pair, for both; the others: each CTA's own)
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOffset);
  uint64_t* empty_bar = full_bar + 2 * Cfg::kSlotKinds;
  uint64_t* x_bar = empty_bar + 2 * Cfg::kSlotKinds;
  uint64_t* s_bar = x_bar + 1;                          // S is complete
  uint64_t* d_bar = s_bar + 1;                          // dP is complete
  uint64_t* p_bar = d_bar + 1;                          // [2] P is written, half by half
  uint64_t* ds_bar = p_bar + 2;                         // dS is written
  uint64_t* acc_bar = ds_bar + 1;                       // the sums are complete
  uint64_t* stat_full = acc_bar + 1;                    // [2]
  uint64_t* stat_empty = stat_full + 2;                 // [2]
  uint64_t* tail_bar = stat_empty + 2;                  // a tile that ends inside
  uint64_t* x_empty = tail_bar + 1;                     // X0 and X1 are used up
  uint64_t* acc_free = x_empty + 1;                     // the sums have been read
  uint64_t* sync_bar = acc_free + 1;
  uint64_t* done_bar = sync_bar + 1;
  Schedule* sched = reinterpret_cast<Schedule*>(smem + Cfg::kSchedOffset);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * Cfg::kSlotKinds; ++s) {
      mbar_init(&full_bar[s], CG);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(x_bar, CG);
    mbar_init(s_bar, 1);
    mbar_init(d_bar, 1);
    mbar_init(&p_bar[0], CG * Cfg::kWarps);
    mbar_init(&p_bar[1], CG * Cfg::kWarps);
    mbar_init(ds_bar, CG * Cfg::kWarps);
    mbar_init(acc_bar, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&stat_full[b], 1);
      mbar_init(&stat_empty[b], Cfg::kWarps);
    }
    mbar_init(tail_bar, 1);
    mbar_init(x_empty, 1);
    mbar_init(acc_free, CG * Cfg::kWarps);
    mbar_init(sync_bar, Cfg::kWarps);
    mbar_init(done_bar, 1);
    schedule_init<CG>(sched, Cfg::kWarps + 2 + (rank == 0));
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmX0);
    tma_prefetch_desc(&p.tmX1);
    tma_prefetch_desc(&p.tmY0);
    tma_prefetch_desc(&p.tmY1);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_holder, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tS = tmem, tD = tmem + 128, tAcc1 = tmem + 256, tAcc2 = tmem + 256 + HD;
  // the address of the even CTA's barrier
  auto lead = [&](uint64_t* bar) {
    return CG == 2 ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar);
  };
  griddep_wait();
  griddep_launch_dependents();

  const bool fine = FINE && few_scores(p, PASS == kDq ? p.order.heads : p.order.heads * p.group);
  const int ksteps = (p.dim + 15) / 16;
  const int32_t width = CG == 2 ? (p.dim + 31) / 32 * 32 : 16 * ksteps;   // columns of the sums
  uint32_t works = 0;                                    // of this warp so far
  Work w;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    constexpr int kHalf = kBoxBytes / 2;                 // a box of 64 rows
    constexpr uint32_t kTailBytes =
        (PASS == kDq && CG == 2 ? Cfg::kSlotKinds - 1 : Cfg::kSlotKinds) * Cfg::kSlotBytes;
    int32_t last[Cfg::kSlotKinds];                       // the last load of each, of all steps
    uint32_t tails = 0, tiles = 0;                       // tiles that had steps
    int32_t u = 0;                                       // steps
    bool ok = true;
#pragma unroll
    for (int kind = 0; kind < Cfg::kSlotKinds; ++kind) last[kind] = -1;
    while (ok && next_work(sched, works, w, p.err, p.wait_limit_ns)) {
      const Tile<CG, PASS> t(w, p, rank);
      if (t.steps == 0) {
        if (rank == 0) want_work(sched);
        continue;
      }
      ok = warp_wait_all(x_empty, (tiles & 1) ^ 1, p.err, 60, p.wait_limit_ns);
      if (!ok) break;
      ++tiles;
      if (elect_one()) {
        const uint32_t bar = lead(x_bar);
        if constexpr (CG == 2) mbar_arrive_expect_tx_cluster(bar, 2 * Cfg::kTileBytes);
        else mbar_arrive_expect_tx(x_bar, 2 * Cfg::kTileBytes);
        for (int b = 0; b < 2 * Cfg::kBoxes; ++b) {
          uint8_t* dst = sX + b * kHalf;
          const int32_t col = 64 * (b >> 1), row = t.x_row + (b & 1) * (kTile / 2);
          if constexpr (CG == 2) {
            tma_load_3d_pair(dst, &p.tmX0, bar, col, w.head, row);
            tma_load_3d_pair(dst + Cfg::kTileBytes, &p.tmX1, bar, col, w.head, row);
          } else {
            tma_load_3d(dst, &p.tmX0, x_bar, col, w.head, row);
            tma_load_3d(dst + Cfg::kTileBytes, &p.tmX1, x_bar, col, w.head, row);
          }
        }
      }
      __syncwarp();
      int32_t tile = t.first, h = t.y_head;
      for (int32_t i = 0; i < t.steps && ok; ++i, ++u) {
        // (the next work's row sums take warp 2 about as long as eight steps)
        if (rank == 0 && i == max(t.steps - 8, 0)) want_work(sched);
        const int32_t left = t.ny - tile * kTile, row = t.y_row + tile * kTile;
        // a tile in which the sequence ends lands on this CTA's own barrier first
        const bool tail = left < kTile;
#pragma unroll
        for (int kind = 0; kind < Cfg::kSlotKinds; ++kind) {
          if (PASS == kDq && kind == kY1m) continue;
          const int s = 2 * kind + (u & 1);
          ok = ok && warp_wait_all(&empty_bar[s], (u >> 1 & 1) ^ 1, p.err, 61, p.wait_limit_ns);
          if (!ok) break;
          last[kind] = u;
          const CUtensorMap* map = kind == kY0k || kind == kY0m ? &p.tmY0 : &p.tmY1;
          uint8_t* dst = sY + s * Cfg::kSlotBytes;
          if (elect_one()) {
            if constexpr (CG == 2) {
              const uint32_t bar = tail ? mapa_shared(smem_u32(tail_bar), rank) : lead(&full_bar[s]);
              const uint32_t bytes = tail ? (kind == 0 ? kTailBytes : 0) : Cfg::kSlotBytes;
              if (bytes > 0) mbar_arrive_expect_tx_cluster(bar, bytes);
              for (int b = 0; b < 2; ++b) {
                if (kind == kY0k || kind == kY1k)        // half of the rows
                  tma_load_3d_pair(dst + b * kHalf, map, bar, 64 * b, h, row + rank * (kTile / 2));
                else                                     // half of the values
                  tma_load_3d_pair(dst + b * kHalf, map, bar, rank * (width / 2), h,
                                   row + b * (kTile / 2));
              }
            } else {
              uint64_t* bar = tail ? tail_bar : &full_bar[s];
              const uint32_t bytes = tail ? (kind == 0 ? kTailBytes : 0) : Cfg::kSlotBytes;
              if (bytes > 0) mbar_arrive_expect_tx(bar, bytes);
              for (int b = 0; b < 2 * Cfg::kBoxes; ++b)
                tma_load_3d(dst + b * kHalf, map, bar, 64 * (b >> 1), h,
                            row + (b & 1) * (kTile / 2));
            }
          }
          __syncwarp();
        }
        if (ok && tail) {                                // its rows behind the sequence become 0
          ok = warp_wait_all(tail_bar, tails++ & 1, p.err, 67, p.wait_limit_ns);
#pragma unroll
          for (int kind = 0; kind < Cfg::kSlotKinds; ++kind) {
            if (PASS == kDq && kind == kY1m) continue;
            const int s = 2 * kind + (u & 1);
            uint8_t* dst = sY + s * Cfg::kSlotBytes;
            if (CG == 2 && (kind == kY0k || kind == kY1k))
              zero_rows(dst, 2, kTile / 2, min(max(left - rank * (kTile / 2), 0), kTile / 2), lane);
            else
              zero_rows(dst, Cfg::kBoxes / CG, kTile, left, lane);
            if (elect_one()) {
              if constexpr (CG == 2) mbar_arrive_release(lead(&full_bar[s]));
              else mbar_arrive(&full_bar[s]);
            }
            __syncwarp();
          }
        }
        if (++tile == t.first + t.count) {
          tile = t.first;
          ++h;
        }
      }
    }
    // the copies started here have landed before the CTA (or the pair) exits
    if (rank == 0) {
      if (tiles > 0) warp_wait_all(x_bar, (tiles - 1) & 1, nullptr, 67, p.wait_limit_ns);
#pragma unroll
      for (int kind = 0; kind < Cfg::kSlotKinds; ++kind)
        for (int32_t i = max(last[kind] - 1, 0); i <= last[kind]; ++i)
          warp_wait_all(&full_bar[2 * kind + (i & 1)], i >> 1 & 1, nullptr, 67, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    if (rank == 0) {
      const uint32_t id_s = idesc_bf16_f32(CG * kTile, kTile, 0, 0);
      const uint32_t id_acc = idesc_bf16_f32(CG * kTile, width, 0, 1);
      const uint64_t x0_desc = desc_k_major(smem_u32(sX));
      const uint64_t x1_desc = desc_k_major(smem_u32(sX) + Cfg::kTileBytes);
      const uint64_t yk_desc = desc_k_major(smem_u32(sY)), ymn_desc = desc_mn_major(smem_u32(sY));
      constexpr int kYBox = kBoxBytes / CG;
      constexpr int k1m = CG == 2 ? kY1m : kY1k, k0m = CG == 2 ? kY0m : kY0k;
      constexpr int kB1 = PASS == kDq ? k0m : k1m;       // of the first sum
      auto slot = [&](int kind, int32_t i) {
        return static_cast<uint32_t>(2 * kind + (i & 1)) * (Cfg::kSlotBytes >> 4);
      };
      auto take = [&](int kind, int32_t i) {
        uint64_t* bar = &full_bar[2 * kind + (i & 1)];
        const uint32_t parity = i >> 1 & 1;
        const bool there = CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, there)) return true;
        bool ok = warp_wait_all(bar, parity, p.err, 63, p.wait_limit_ns);
        if (CG == 2) ok = ok && __all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity));
        return ok;
      };
      auto written = [&](uint64_t* bar, int32_t i, uint32_t where) {
        return warp_wait_all(bar, i & 1, p.err, where, p.wait_limit_ns);
      };
      auto commit = [&](uint64_t* bar) {
        if constexpr (CG == 2) tc_commit_pair_mc(bar, static_cast<uint16_t>(3));
        else tc_commit(bar);
      };
      auto free_slot = [&](int kind, int32_t i) { commit(&empty_bar[2 * kind + (i & 1)]); };
      bool ok = true;
      uint32_t tiles = 0;
      int32_t u0 = 0;                                    // step that this tile begins with
      while (ok && next_work(sched, works, w, p.err, p.wait_limit_ns)) {
        const Tile<CG, PASS> t(w, p, rank);
        if (t.steps == 0) continue;
        ok = warp_wait_all(x_bar, tiles & 1, p.err, 62, p.wait_limit_ns) && take(kY0k, u0);
        if (!ok) break;
        tc_fence_after();
        const uint64_t y0 = yk_desc + slot(kY0k, u0), y1 = yk_desc + slot(kY1k, u0);
        if (elect_one()) {
          issue_scores<CG, HD / 16, kYBox>(tS, x0_desc, y0, id_s, ksteps);
          commit(s_bar);
          if (CG == 2) free_slot(kY0k, u0);
        }
        __syncwarp();
        ok = take(kY1k, u0);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_scores<CG, HD / 16, kYBox>(tD, x1_desc, y1, id_s, ksteps);
          commit(d_bar);
          if (CG == 2 || PASS == kDq) free_slot(kY1k, u0);
          if (t.steps == 1) commit(x_empty);
        }
        __syncwarp();
        // the last tile's sums have been read
        ok = warp_wait_all(acc_free, (tiles & 1) ^ 1, p.err, 59, p.wait_limit_ns);
        ++tiles;
        for (int32_t i = 0; i < t.steps && ok; ++i) {
          const int32_t u = u0 + i;
          const bool more = i + 1 < t.steps;
          const uint64_t b1 = ymn_desc + slot(kB1, u), b2 = ymn_desc + slot(k0m, u);
          const uint64_t next0 = yk_desc + slot(kY0k, u + 1), next1 = yk_desc + slot(kY1k, u + 1);
          // (the first half's products run while the threads work on the second's P)
          ok = (CG == 1 || take(kB1, u)) && written(&p_bar[0], u, 64);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_sums<CG, Cfg::kCols, 0, 2>(tAcc1, tS, b1, id_acc, i > 0);
            if (fine) issue_sums<CG, Cfg::kCols, 0, 2>(tAcc1, tS + Cfg::kCols / 2, b1, id_acc, true);
          }
          __syncwarp();
          ok = written(&p_bar[1], u, 64);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_sums<CG, Cfg::kCols, 1, 2>(tAcc1, tS, b1, id_acc, true);
            if (fine) issue_sums<CG, Cfg::kCols, 1, 2>(tAcc1, tS + Cfg::kCols / 2, b1, id_acc, true);
            if (PASS == kDkv) free_slot(k1m, u);
          }
          __syncwarp();
          if (more) {
            ok = take(kY0k, u + 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_scores<CG, HD / 16, kYBox>(tS, x0_desc, next0, id_s, ksteps);
              commit(s_bar);
              if (CG == 2) free_slot(kY0k, u + 1);
            }
            __syncwarp();
          }
          ok = (CG == 1 || PASS == kDq || take(k0m, u)) && written(ds_bar, u, 65);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_sums<CG, Cfg::kCols>(tAcc2, tD, b2, id_acc, i > 0);
            if (fine) issue_sums<CG, Cfg::kCols>(tAcc2, tD + Cfg::kCols / 2, b2, id_acc, true);
            free_slot(k0m, u);
            if (!more) commit(acc_bar);
          }
          __syncwarp();
          if (more) {
            ok = take(kY1k, u + 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_scores<CG, HD / 16, kYBox>(tD, x1_desc, next1, id_s, ksteps);
              commit(d_bar);
              if (CG == 2 || PASS == kDq) free_slot(kY1k, u + 1);
              if (i + 2 == t.steps) commit(x_empty);
            }
            __syncwarp();
          }
        }
        u0 += t.steps;
      }
      // every MMA issued here is complete before TMEM is released
      if (elect_one()) {
        if constexpr (CG == 2) tc_commit_pair(done_bar); else tc_commit(done_bar);
      }
      __syncwarp();
      warp_wait_all(done_bar, 0, nullptr, 68, p.wait_limit_ns);
    }
  } else if (warp == 2 && PASS == kDq) {
    // ------------------------- lse of the tile's rows, and delta from out: a work ahead
    bool ok = true;
    for (uint32_t n = 0; ok && next_work(sched, works, w, p.err, p.wait_limit_ns); ++n) {
      const Tile<CG, PASS> t(w, p, rank);
      float* to = stat + (n & 1) * 2 * kTile;
      ok = warp_wait_all(&stat_empty[n & 1], (n >> 1 & 1) ^ 1, p.err, 66, p.wait_limit_ns);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < kTile; k += 32)
        to[k + lane] = t.x0 + k + lane < t.nx
                           ? p.lse[w.head * p.Tq + t.x_row + k + lane] * kLog2e : 0.0f;
      // 16 lanes a row, 8 rows at a time
      const int c = (lane & 15) * 8;
#pragma unroll 1
      for (int r0 = lane >> 4; r0 < kTile; r0 += 16) {
        uint4 a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + 2 * k;
          a[k] = b[k] = make_uint4(0, 0, 0, 0);
          if (t.x0 + r < t.nx && c < p.dim) {
            a[k] = *reinterpret_cast<const uint4*>(p.o.row(t.x_row + r, w.head) + c);
            b[k] = *reinterpret_cast<const uint4*>(p.dout.row(t.x_row + r, w.head) + c);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[8], y[8], s = 0.0f;
          unpack8(a[k], x);
          unpack8(b[k], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if ((lane & 15) == 0) to[kTile + r0 + 2 * k] = s;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[n & 1]);
    }
  } else if (warp == 2) {
    // ----------------------------------- lse and delta of the queries, less than zero
    // (loaded a step ahead, all at once: the threads wait for these as for the scores)
    int32_t u = 0;
    bool ok = true;
    while (ok && next_work(sched, works, w, p.err, p.wait_limit_ns)) {
      const Tile<CG, PASS> t(w, p, rank);
      int32_t tile = t.first, h = t.y_head;
      float l[4], d[4];
      auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int32_t q = tile * kTile + k * 32 + lane;
          const int64_t at = static_cast<int64_t>(h) * p.Tq + w.at.q0 + q;
          l[k] = q < w.at.nq ? p.lse[at] : -CUDART_INF_F;
          d[k] = q < w.at.nq ? p.delta[at] : 0.0f;
        }
        if (++tile == t.first + t.count) {
          tile = t.first;
          ++h;
        }
      };
      if (t.steps > 0) fetch();
      for (int32_t i = 0; i < t.steps; ++i, ++u) {
        const int b = u & 1;
        ok = warp_wait_all(&stat_empty[b], (u >> 1 & 1) ^ 1, p.err, 66, p.wait_limit_ns);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // (a query that is none, or sees no key, has no probabilities)
          const bool none = l[k] == -CUDART_INF_F;
          stat[b * 2 * kTile + k * 32 + lane] = none ? -CUDART_INF_F : l[k] * -kLog2e;
          stat[b * 2 * kTile + kTile + k * 32 + lane] = none ? 0.0f : -d[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&stat_full[b]);
        if (i + 1 < t.steps) fetch();
      }
    }
  } else if (warp == 3) {
    schedule<CG>(sched, p.q_starts, p.k_starts, p.Tq, p.Tk, p.sequences, p.order, CG * kTile,
                 PASS == kDkv, rank, p.err, p.wait_limit_ns);
  } else if (warp >= 4) {
    // ------------------------------------------------------ probabilities, dS
    constexpr int kCols = Cfg::kCols, kDims = HD / Cfg::kParts;
    const int part = (warp >> 2) - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tS + lane_base + kCols * part, d_at = tD + lane_base + kCols * part;
    uint8_t* stage = smem + Cfg::kStageOffset + (warp - 4) * 1024;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    int32_t u = 0;
    uint32_t tiles = 0, stats = 0;                        // works with steps; works
    bool ok = true;
    bool have = next_work(sched, works, w, p.err, p.wait_limit_ns);
    Tile<CG, PASS> t(w, p, rank);
    while (have) {
      const int32_t x = t.x0 + row;                       // in the sequence
      const bool valid = x < t.nx;
      // kDq: of this row; what delta lacks, and the same sum over dS as rounded
      float lse = 0.0f, delta = 0.0f, e = 0.0f, rounded = 0.0f;
      if (PASS == kDq) {
        const float* st = stat + (stats & 1) * 2 * kTile;
        ok = warp_wait_all(&stat_full[stats & 1], stats >> 1 & 1, p.err, 69, p.wait_limit_ns);
        lse = st[row];
        delta = st[kTile + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&stat_empty[stats & 1]);
      }
      // kDq: keys that this row sees; kDkv: the first query that sees this row
      const int32_t bound = PASS == kDq ? (p.causal ? min(w.at.nk, x + t.off + 1) : w.at.nk)
                                        : (p.causal ? x - t.off : 0);
      int32_t tile = t.first;
      for (int32_t i = 0; i < t.steps; ++i, ++u) {
        const float* st = stat + (u & 1) * 2 * kTile + part * kCols;
        if (PASS == kDkv)
          ok = ok && warp_wait_all(&stat_full[u & 1], u >> 1 & 1, p.err, 69, p.wait_limit_ns);
        ok = ok && warp_wait_all(s_bar, u & 1, p.err, 70, p.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        float s[kCols];
        tmem_ld_32x32b_x32(s_at, s);
        tmem_ld_wait();
        const int32_t lim = bound - tile * kTile - kCols * part;   // of this part's columns
        const bool cut = __any_sync(0xffffffffu, PASS == kDq ? lim < kCols : lim > 0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          constexpr int kHalf = kCols / 2;
#pragma unroll
          for (int c = half * kHalf; c < (half + 1) * kHalf; c += 4) {
            float4 l = make_float4(-lse, -lse, -lse, -lse);
            if (PASS == kDkv) l = *reinterpret_cast<const float4*>(st + c);
            const float2 x = fma2(make_float2(s[c], s[c + 1]), scale2, make_float2(l.x, l.y));
            const float2 y = fma2(make_float2(s[c + 2], s[c + 3]), scale2, make_float2(l.z, l.w));
            s[c] = exp2_fast(x.x);
            s[c + 1] = exp2_fast(x.y);
            s[c + 2] = exp2_fast(y.x);
            s[c + 3] = exp2_fast(y.y);
          }
          if (cut) {
#pragma unroll
            for (int c = half * kHalf; c < (half + 1) * kHalf; ++c)
              s[c] = (PASS == kDq ? c < lim : c >= lim) ? s[c] : 0.0f;
          }
          store_operand<kHalf>(s_at + half * (kHalf / 2), kCols / 2, s + half * kHalf, fine);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_cluster(lead(&p_bar[half]));
            else mbar_arrive(&p_bar[half]);
          }
        }

        ok = warp_wait_all(d_bar, u & 1, p.err, 71, p.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        float d[kCols];
        tmem_ld_32x32b_x32(d_at, d);
        tmem_ld_wait();
        float2 sum[2] = {};
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          float2 l = make_float2(-delta, -delta);
          if (PASS == kDkv) l = *reinterpret_cast<const float2*>(st + kTile + c);
          const float2 x = mul2(make_float2(s[c], s[c + 1]), add2(make_float2(d[c], d[c + 1]), l));
          if (PASS == kDq) sum[c / 2 & 1] = add2(sum[c / 2 & 1], x);
          d[c] = x.x;
          d[c + 1] = x.y;
        }
        if (PASS == kDq) e += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        float2 kept[2] = {};
        store_operand<kCols>(d_at, kCols / 2, d, fine, PASS == kDq ? kept : nullptr);
        if (PASS == kDq) rounded += (kept[0].x + kept[0].y) + (kept[1].x + kept[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_cluster(lead(ds_bar)); else mbar_arrive(ds_bar);
          if (PASS == kDkv) mbar_arrive(&stat_empty[u & 1]);
        }
        if (++tile == t.first + t.count) tile = t.first;
      }
      if (PASS == kDq) {                                  // over the row's parts, in order
        float* parts = stat + 4 * kTile + (stats & 1) * 2 * Cfg::kParts * kTile;
        float* others = parts + Cfg::kParts * kTile;
        parts[part * kTile + row] = e;
        others[part * kTile + row] = rounded;
        __syncwarp();
        if (lane == 0) mbar_arrive(sync_bar);
        ok = ok && warp_wait_all(sync_bar, stats & 1, p.err, 73, p.wait_limit_ns);
        e = parts[row];
        rounded = others[row];
#pragma unroll
        for (int i = 1; i < Cfg::kParts; ++i) {
          e += parts[i * kTile + row];
          rounded += others[i * kTile + row];
        }
        if (fine) rounded = e;
        if (ok && valid && part == 0) p.delta[w.head * p.Tq + t.x_row + row] = delta + e;
        ++stats;
      }
      // (the softmax of a single key is constant: the gradients of its score are 0, to the bit)
      const float scale = (PASS == kDq ? bound : w.at.nk) == 1 ? 0.0f : p.scale;
      const Tile<CG, PASS> done = t;
      const int32_t head = w.head;
      have = ok && next_work(sched, works, w, p.err, p.wait_limit_ns);
      t = Tile<CG, PASS>(w, p, rank);
      if (done.steps > 0) {
        ok = ok && warp_wait_all(acc_bar, tiles++ & 1, p.err, 72, p.wait_limit_ns);
        if (!ok) break;
      }
      tc_fence_after();
      uint32_t g1[kDims / 2], g2[kDims / 2];
#pragma unroll
      for (int c = 0; c < kDims; c += 16) {
        float a1[16], a2[16];
        if (done.steps > 0) {
          tmem_ld_32x32b_x16(tAcc1 + lane_base + part * kDims + c, a1);
          tmem_ld_32x32b_x16(tAcc2 + lane_base + part * kDims + c, a2);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) a1[k] = a2[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          if (PASS == kDq) {
            a2[k] = fmaf(-rounded, a1[k], a2[k]);
            a2[k + 1] = fmaf(-rounded, a1[k + 1], a2[k + 1]);
          }
          g2[(c + k) / 2] = pack_bf16x2(scale * a2[k], scale * a2[k + 1]);
          if (PASS == kDkv) g1[(c + k) / 2] = pack_bf16x2(a1[k], a1[k + 1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && done.steps > 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(lead(acc_free)); else mbar_arrive(acc_free);
      }
      store_rows<kDims>(p.g2, head, done.x_row + quarter * 32, done.nx - done.x0 - quarter * 32,
                        part * kDims, p.dim, g2, stage, lane);
      if (PASS == kDkv)
        store_rows<kDims>(p.g1, head, done.x_row + quarter * 32, done.nx - done.x0 - quarter * 32,
                          part * kDims, p.dim, g1, stage, lane);
    }
  }
  if constexpr (CG == 2) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem, 512); else tmem_dealloc(tmem, 512);
  }
}

template <int HD, int CG, int PASS, bool FINE>
cudaError_t launch_pass(BwdParams p, int64_t T, cudaStream_t stream) {
  using Cfg = BwdCfg<HD, CG>;
  const auto kern = attention_bwd_kernel<HD, CG, PASS, FINE>;
  // the other side: k and v of a key head, or q and dout of its query heads
  const double bytes = 4.0 * p.dim * (PASS == kDq ? static_cast<double>(p.Tk) / p.group
                                                  : static_cast<double>(p.Tq) * p.group);
  // (16 x 1024 tokens, 16 heads, causal: four sets of four heads 354 us, five of three and one of one
  // 371; sets of 96 MB 381)
  p.order = grid_order(p.order.heads, most_tiles(T, CG * kTile, p.sequences), bytes, 32e6);
  // (some waits last as long as a tile's work: 4 us a step at most, on top of the limit)
  const int64_t steps = PASS == kDq ? p.Tk / kTile + 1 : (p.Tq / kTile + 1) * p.group;
  p.wait_limit_ns += 4000 * static_cast<uint64_t>(steps);
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
  cfg.gridDim = dim3(static_cast<unsigned>(p.order.tiles * p.order.heads * CG), 1, 1);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int PASS>
cudaError_t launch(const BwdParams& p, int64_t T, cudaStream_t stream) {
  // Where the rows bound the scores by 2^24 (sequences of one length), the kernels that look how many
  // there are: in the others that would cost 3% (16384 tokens: 735 us, 757).
  const double heads = static_cast<double>(p.order.heads) * (PASS == kDq ? 1 : p.group);
  if (static_cast<double>(p.Tq) * p.Tk / p.sequences * heads <= 0x1p24)
    return p.dim <= 64 ? launch_pass<64, 1, PASS, true>(p, T, stream)
                       : launch_pass<128, 1, PASS, true>(p, T, stream);
  if (p.dim <= 64) return launch_pass<64, 1, PASS, false>(p, T, stream);
  // Pairs where sequences are long. (16384 tokens, 16 heads, us of both passes, singles and pairs: 32 x
  // 512 321 and 344 causal, 357 and 366 without; 24 x 640 306 and 353, 363 and 400; 16 x 1024 355 and
  // 367, 452 and 444; 10 x 1664 428 and 451, 636 and 651; 8 x 2048 471 and 483, 752 and 723; 6 x 2816
  // 604 and 615, 1015 and 965; 4 x 4096 788 and 778, 1411 and 1336.)
  if (T / p.sequences >= 2048) return launch_pass<128, 2, PASS, false>(p, T, stream);
  return launch_pass<128, 1, PASS, false>(p, T, stream);
}

}  // namespace

cudaError_t launch_attention_bwd(const AttentionArgs& a, cudaStream_t stream) {
  const boost_attention_desc& d = a.d;
  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  CUtensorMap q, k, v, dout;
  if (!heads_map(&q, a.q.at, a.ws, d.Tq, d.hq, d.dim, d.q_ts, d.q_hs, 1, kTile / 2) ||
      !heads_map(&k, a.k.at, a.ws, d.Tk, d.hk, d.dim, d.k_ts, d.k_hs, 1, kTile / 2) ||
      !heads_map(&v, a.v.at, a.ws, d.Tk, d.hk, d.dim, d.v_ts, d.v_hs, 1, kTile / 2) ||
      !heads_map(&dout, a.dout.at, a.ws, d.Tq, d.hq, d.dim, d.do_ts, d.do_hs, 1, kTile / 2))
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
    p.order.heads = d.hq;
    const cudaError_t e = launch<kDq>(p, d.Tq, stream);
    if (e != cudaSuccess) return e;
  }
  if (d.Tk == 0) return cudaSuccess;
  if (d.Tq > 0) prof_note_kernels(1);
  p.tmX0 = k;
  p.tmX1 = v;
  p.tmY0 = q;
  p.tmY1 = dout;
  p.g1 = a.dv;
  p.g2 = a.dk;
  p.order.heads = d.hk;
  return launch<kDkv>(p, d.Tk, stream);
}

}  // namespace boost_gb300
