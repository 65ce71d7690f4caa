// attention_tc.cuh -- what the tensor-core attention kernels share: MMAs with an operand in TMEM,
// tiles of [T, heads, dim] operands in shared memory, and how a tile finds its sequence.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace boost_gb300 {

constexpr int kTile = 128;               // rows of a tile: lanes of TMEM

// D[tmem] (+)= A[tmem] * B[smem], kind::f16: A holds two bf16 values a column, 128 rows.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same over a CTA pair: 256 rows, 128 of them in each CTA's TMEM, and B split along N.
__device__ __forceinline__ void tc_mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem,
                                                    uint64_t b_desc, uint32_t idesc,
                                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on a barrier of a CTA of the cluster (its cluster address): what this thread has written
// is seen by a thread of that CTA that has waited with mbar_try_wait_cluster.
__device__ __forceinline__ void mbar_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrive there and expect bytes of copies (which carry their own order: as a release, the arrival
// would wait about 1100 cycles for this thread's earlier ones).
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Each thread of the warp writes 32 consecutive columns of its TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Each thread of the warp writes 8 consecutive columns of its TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Each thread of the warp writes 16 consecutive columns of its TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values an instruction (each rounded as alone).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// A wait of the whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait_all(uint64_t* bar, uint32_t parity, DeviceError* err,
                                              uint32_t where, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, err, where, limit_ns));
}

// A tile lies in shared memory as boxes of 64 values a row: rows of 128 bytes, 128-byte swizzle,
// 16 KB a box. As K-major operand (the values are contracted) a step of 16 values is 32 bytes
// within a box; as MN-major operand (the rows are contracted) a step of 16 rows is 2048 bytes, and
// the next 64 values are the next box.
constexpr int kBoxBytes = kTile * 128;

//
// The products' issuers are converged warps that form the descriptors, an elected lane issues:
// with constant steps behind a base in uniform registers an MMA costs a few instructions. (With
// the steps' addresses formed in the elected lane's own loop, an MMA of 64 cycles took about 125.)
__device__ __forceinline__ uint64_t desc_k_major(uint32_t base) {
  return desc_hi_sw128(16u, 1024u) | ((base >> 4) & 0x3FFFu);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t base) {
  return desc_hi_sw128(kBoxBytes, 1024u) | ((base >> 4) & 0x3FFFu);
}

// D = X Y^T over `steps` steps of 16 values (MAX at most), both K-major, Y's boxes YBOX bytes apart.
template <int CG, int MAX, int YBOX = kBoxBytes>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc,
                                             int steps) {
#pragma unroll
  for (int kk = 0; kk < MAX; ++kk) {
    const uint64_t xk = x + (kk >> 2) * (kBoxBytes >> 4) + (kk & 3) * 2;
    const uint64_t yk = y + (kk >> 2) * (YBOX >> 4) + (kk & 3) * 2;
    if (kk < steps) {
      if constexpr (CG == 2) tc_mma_bf16_pair(d, xk, yk, idesc, kk > 0);
      else tc_mma_bf16(d, xk, yk, idesc, kk > 0);
    }
  }
}

// D (+)= A Y over the tile's 128 rows, or over every STEP-th 16 of them from the FROM-th up to the
// TO-th, A in TMEM as parts of `COLS` values that lie COLS columns apart, Y MN-major.
template <int CG, int COLS, int FROM = 0, int STEP = 1, int TO = kTile / 16>
__device__ __forceinline__ void issue_sums(uint32_t d, uint32_t a, uint64_t y, uint32_t idesc,
                                           bool more) {
#pragma unroll
  for (int kk = FROM; kk < TO; kk += STEP) {
    const uint32_t ak = a + 16 * kk / COLS * COLS + 16 * kk % COLS / 2;
    if constexpr (CG == 2) tc_mma_bf16_ts_pair(d, ak, y + 128 * kk, idesc, kk > FROM ? 1u : more);
    else tc_mma_bf16_ts(d, ak, y + 128 * kk, idesc, kk > FROM ? 1u : more);
  }
}

// Zero rows [from, rows) of `boxes` boxes of 64 values that a TMA load has filled, by a whole warp:
// rows of another sequence may hold NaN, which a probability of 0 would not hide.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int boxes, int rows, int from, int lane) {
  for (int b = 0; b < boxes; ++b)
    for (int i = from * 8 + lane; i < rows * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + b * rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// A sequence's bounds, and one of its tiles: `tile` of `tiles`, as the grid counts them.
struct Place {
  int32_t tile, tiles;                   // tiles < 0: none
  int32_t q0, nq, k0, nk;
};

// Where tile `index` of all sequences lies, sequence s having ceil(rows / per) tiles; by a whole
// warp, each lane with a sequence of its own at a time. `keys`: the tiles are of the keys. Up to
// 32 sequences take turns (the first tile of each, the second of each that has one, ...), so that
// with a causal mask the tiles with most work, which the kernels count first, go out first; more
// sequences follow one another.
__device__ __forceinline__ Place find_tile(const int32_t* q_starts, const int32_t* k_starts,
                                           int64_t Tq, int64_t Tk, int sequences, int32_t index,
                                           int32_t per, bool keys) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kAll = 0xffffffffu;
  Place f{0, -1, 0, 0, 0, 0};
  for (int s0 = 0; s0 < sequences; s0 += 32) {
    Place mine{0, 0, 0, 0, 0, 0};
    if (s0 + lane < sequences) {
      sequence_bounds(q_starts, Tq, s0 + lane, mine.q0, mine.nq);
      sequence_bounds(k_starts, Tk, s0 + lane, mine.k0, mine.nk);
      mine.tiles = ((keys ? mine.nk : mine.nq) + per - 1) / per;
    }
    int src = -1;
    if (sequences <= 32) {
      // the last turn that begins at or before `index`: sum min(tiles, turn) <= index
      int32_t lo = 0, hi = static_cast<int32_t>(__reduce_max_sync(kAll, mine.tiles));
      const int32_t all = static_cast<int32_t>(__reduce_add_sync(kAll, mine.tiles));
      if (index >= all) return f;
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) / 2;
        if (static_cast<int32_t>(__reduce_add_sync(kAll, min(mine.tiles, mid))) <= index) lo = mid;
        else hi = mid;
      }
      const int32_t rest = index - static_cast<int32_t>(__reduce_add_sync(kAll, min(mine.tiles, lo)));
      const uint32_t has = __ballot_sync(kAll, mine.tiles > lo);
      const uint32_t before = has & ((1u << lane) - 1u);
      src = __ffs(__ballot_sync(kAll, mine.tiles > lo && __popc(before) == rest)) - 1;
      f.tile = lo;
    } else {
      int32_t sum = mine.tiles;          // up to and with this lane's
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t below = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += below;
      }
      const uint32_t has = __ballot_sync(kAll, index < sum);
      if (has != 0) {
        src = __ffs(has) - 1;
        // (inside the sequence whatever the starts hold: sums over ones that overlap may wrap)
        f.tile = min(max(index - __shfl_sync(kAll, sum - mine.tiles, src), 0),
                     max(__shfl_sync(kAll, mine.tiles, src) - 1, 0));
      } else {
        index -= __shfl_sync(kAll, sum, 31);
      }
    }
    if (src >= 0) {
      f.tiles = __shfl_sync(kAll, mine.tiles, src);
      f.q0 = __shfl_sync(kAll, mine.q0, src);
      f.nq = __shfl_sync(kAll, mine.nq, src);
      f.k0 = __shfl_sync(kAll, mine.k0, src);
      f.nk = __shfl_sync(kAll, mine.nk, src);
      return f;
    }
  }
  return f;
}

// ----------------------------------------------------------------- work after work
// A CTA (or a pair) that is done takes the place of one that has not begun yet
// (clusterlaunchcontrol): tiles go out in the grid's order to whoever is free, and what a launch
// costs each (barriers, TMEM, the search for its sequence, the first loads) is paid once or hidden.
// One warp asks, looks the tile up and leaves it for the others, once the loading warp is near the
// end of the tile before: no CTA holds work for long that an idle one could have.

// Ask for a CTA (cluster) to cancel: 16 bytes at the same place in every CTA of the cluster, which
// complete on each one's `bar`.
template <int CG>
__device__ __forceinline__ void clc_try_cancel(void* response, uint64_t* bar) {
  if constexpr (CG == 2)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_u32(response)),
        "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".b128 [%0], [%1];" ::"r"(smem_u32(response)),
        "r"(smem_u32(bar))
        : "memory");
}

// The first CTA of the cancelled cluster (x), or -1 if there was none.
__device__ __forceinline__ int32_t clc_answer(const void* response) {
  uint32_t canceled, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(canceled), "=r"(x)
      : "r"(smem_u32(response))
      : "memory");
  return canceled != 0u ? static_cast<int32_t>(x) : -1;
}

// The grid's order: heads in equal sets of about `bytes` of the other side (what the tiles stream
// through, which stays in L2), within a set tile by tile, the set's heads side by side.
struct Order {
  int32_t heads, set, tiles;             // tiles: the most that there can be
};

inline Order grid_order(int64_t heads, int64_t tiles, double bytes_per_head, double bytes) {
  const double sets = std::min(std::floor(bytes_per_head * heads / bytes + 0.5), 1.0 * heads);
  const int64_t n = std::max<int64_t>(1, static_cast<int64_t>(sets));
  return {static_cast<int32_t>(heads), static_cast<int32_t>((heads + n - 1) / n),
          static_cast<int32_t>(tiles)};
}

struct Work {
  Place at;
  int32_t head;                          // < 0: no more
};

struct Schedule {
  uint4 response;
  uint64_t clc_bar, clc_free;            // an answer is there; both CTAs have read it (the even's)
  uint64_t want;                         // the loading warp wants more (the even's)
  uint64_t full[2], empty[2];
  Work work[2];
};

// Barriers of a schedule that `readers` warps of this CTA follow; by one thread.
template <int CG>
__device__ __forceinline__ void schedule_init(Schedule* s, int readers) {
  mbar_init(&s->clc_bar, 1);
  mbar_init(&s->clc_free, CG);
  mbar_init(&s->want, 1);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&s->full[i], 1);
    mbar_init(&s->empty[i], readers);
  }
}

// The warp that asks: work after work, `per` rows a tile.
template <int CG>
__device__ __forceinline__ void schedule(Schedule* s, const int32_t* q_starts,
                                         const int32_t* k_starts, int64_t Tq, int64_t Tk,
                                         int sequences, const Order& order, int32_t per, bool keys,
                                         int rank, DeviceError* err, uint64_t limit_ns) {
  const int lane = threadIdx.x & 31;
  int32_t cta = static_cast<int32_t>(blockIdx.x);
  for (uint32_t n = 0;; ++n) {
    const int i = n & 1;
    Work w;
    w.head = -1;
    if (cta >= 0) {
      const int32_t work = cta / CG, span = order.set * order.tiles, first = work / span * order.set;
      const int32_t set = min(order.set, order.heads - first), at = work % span;
      w.head = first + at % set;
      w.at = find_tile(q_starts, k_starts, Tq, Tk, sequences, at / set, per, keys);
    }
    if (!warp_wait_all(&s->empty[i], (n >> 1 & 1) ^ 1, err, 31, limit_ns)) return;
    if (lane == 0) {
      s->work[i] = w;
      mbar_arrive(&s->full[i]);
    }
    __syncwarp();
    if (cta < 0) return;
    // (the answer's place is free: both CTAs have read the last one)
    if (rank == 0 && n > 0 && !warp_wait_all(&s->clc_free, (n - 1) & 1, err, 32, limit_ns)) return;
    if (rank == 0 && !warp_wait_all(&s->want, n & 1, err, 35, limit_ns)) return;
    if (elect_one()) {
      mbar_arrive_expect_tx(&s->clc_bar, 16);
      if (rank == 0) clc_try_cancel<CG>(&s->response, &s->clc_bar);
    }
    __syncwarp();
    // (not given up for another wait's sake: the answer must not land behind this CTA)
    if (!warp_wait_all(&s->clc_bar, n & 1, nullptr, 0, limit_ns)) {
      record_error(err, kErrTimeout, 33);
      return;
    }
    cta = clc_answer(&s->response);
    fence_proxy_async_smem();            // (read before the next answer is written)
    __syncwarp();
    if (elect_one()) {
      if constexpr (CG == 2) mbar_arrive_release(mapa_shared(smem_u32(&s->clc_free), 0));
      else mbar_arrive(&s->clc_free);
    }
    __syncwarp();
  }
}

// The even CTA's loading warp asks for the work behind its n-th.
__device__ __forceinline__ void want_work(Schedule* s) {
  if (elect_one()) mbar_arrive(&s->want);
  __syncwarp();
}

// A reader's next work, the n-th; false after the last.
__device__ __forceinline__ bool next_work(Schedule* s, uint32_t& n, Work& w, DeviceError* err,
                                          uint64_t limit_ns) {
  const int i = n & 1;
  if (!warp_wait_all(&s->full[i], n >> 1 & 1, err, 34, limit_ns)) return false;
  w = s->work[i];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&s->empty[i]);
  ++n;
  return w.head >= 0;
}

// Most tiles that sequences of T rows in all can have.
inline int64_t most_tiles(int64_t T, int64_t per, int64_t sequences) {
  const int64_t n = T / per + (sequences < T ? sequences : T);
  return n < T ? n : T;
}

// Tensor map of a [T, heads, dim] operand with boxes of 64 values, `box_heads` heads and `rows`
// tokens; an empty operand (whose tiles are never loaded) as one row of `any`.
inline bool heads_map(CUtensorMap* m, const __nv_bfloat16* at, const void* any, int64_t T,
                      int64_t heads, int64_t dim, int64_t ts, int64_t hs, uint32_t box_heads,
                      uint32_t rows) {
  EncodeFn enc = get_encode();
  if (enc == nullptr) return false;
  const bool none = T == 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(none ? 1 : T)};
  // the stride of a single head or token says nothing: a plain one in its place
  const cuuint64_t strides[2] = {2ull * (heads > 1 ? hs : dim), 2ull * (T > 1 ? ts : heads * dim)};
  const cuuint32_t box[3] = {64, box_heads, rows}, ones[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             none ? const_cast<void*>(any) : const_cast<__nv_bfloat16*>(at), dims, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace boost_gb300
