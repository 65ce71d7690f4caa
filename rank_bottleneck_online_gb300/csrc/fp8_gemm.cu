// fp8_gemm.cu -- out[g] = act(row_scale (.) (A[g] B[g]^T)) for 8-bit operands with a
// power-of-two scale for each block of 128 along K.
//
// The tensor core applies the scales itself: tcgen05.mma kind::mxf8f6f4 multiplies K = 32
// values a step by one E8M0 scale of each row of A and of B, which it reads from TMEM. A
// block of 128 is four steps with the same byte of the scale words, and a scale tile (128
// rows x 4 blocks, 512 bytes, the layout the operands are stored in) serves sixteen: it
// travels with the operands of its first block (TMA, then tcgen05.cp to TMEM, which runs in
// order with the MMAs). So the scales cost no arithmetic, and the sums stay in fp32 in TMEM
// over the whole of K. (Scales of any value would have to be applied by the CUDA cores: each
// block's 128 x 256 partial product read from TMEM and joined by an FMA each, a half of the
// tensor cores' time at this tile.)
//
// The shape of the kernel is the bf16 engine's: a persistent grid, one CTA an SM, warp 0
// streams operand tiles (128 bytes of K) with TMA, warp 1 issues the MMAs, warps 2..9 read
// the accumulator and store it. A CTA pair (CG = 2) shares a 256 x BN tile.
//
// A few tiles with a long K: the CTAs of a cluster share a tile's K (CG = 1), and each joins a
// part of its rows from all their parts in shared memory, in a fixed order.
//
// TMEM: 512 columns hold two accumulators of 256 less the scales. The second begins at 224
// and shares 32 columns with the first; the epilogue reads those first and lets the next
// tile's MMAs start, so the two tiles still overlap but for that read.
//
// Measured (alone; back to back the power cap takes 13-18%): 8192^3 292 us, 3.76 PFLOP/s, twice
// the measured bf16 burst; 16384 x 2048 x 4096 81 us, 3.40 PFLOP/s, the tensor pipe busy 75% of
// the time (waves 6.7 of 7, the first loads, the last epilogue); 2 x 16384 x 11008 x 1024
// 233 us, 3.17 PFLOP/s, where 721 MB of stores share L2 with the operand loads. Clusters of two
// and four pairs that share operand rows by multicast, 192- and 128-column tiles, and tiles of
// 448 columns in parts of 256 and 192 were slower at these sizes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "fp8.cuh"
#include "internal.h"
#include "simple.cuh"

namespace boost_gb300 {

namespace {

constexpr int kKBytes = 128;           // K of one stage: a swizzle row, and a scale block

struct Fp8Params {
  CUtensorMap tmA, tmB;                // (K, rows, G) bytes, boxes 128 x a CTA's rows
  CUtensorMap tmSA, tmSB;              // scale tiles (128 words, tiles of K, row tiles of all G)
  CUtensorMap tmO;                     // out (N, M, G), boxes 32 x 32
  int32_t M, N, G, num_kb;
  int32_t m_tiles, n_tiles;            // of 128 CG x BN
  int32_t a_row_tiles, b_row_tiles;    // scale tiles along the rows of one matrix
  int32_t split, kb_split;             // CTAs that share a tile's K (CG = 1), blocks of each
  int32_t a_fmt, b_fmt, act;
  const float* row_scale;
  __nv_bfloat16* out;
  DeviceError* err;
  uint64_t wait_limit_ns;
};

template <int BN, int CG>
struct Fp8Cfg {
  static constexpr int kEpiW = 8;
  static constexpr int kThreads = 32 * (2 + kEpiW);
  static constexpr int kBRows = BN / CG;               // B rows staged by one CTA
  static constexpr int kABytes = kBM * kKBytes;
  static constexpr int kBBytes = kBRows * kKBytes;
  static constexpr int kSfTilesB = BN / 128;
  static constexpr int kSfBytes = kScaleTile * (1 + kSfTilesB);
  static constexpr int kStgBytes = kEpiW * 2048;
  static constexpr int kStages0 = (232448 - 2048 - kStgBytes) / (kABytes + kBBytes + kSfBytes);
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int kAcc1 = BN == 256 ? 224 : BN;   // column of the second accumulator
  static constexpr bool kOverlap = kAcc1 < BN;
  static constexpr int kSfCols = 4 * (1 + kSfTilesB);
  static constexpr int kSfCol = 512 - 32;              // two buffers of kSfCols columns
  static constexpr int kBarBytes = 8 * (2 * kStages + 2 + 2 + 1) + 16;
  static constexpr int kSfOffset = kStages * (kABytes + kBBytes);
  static constexpr int kBarOffset = kSfOffset + kStages * kSfBytes;
  static constexpr int kStgOffset = (kBarOffset + kBarBytes + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = 1024 + kStgOffset + kStgBytes;
  static constexpr int kPartPitch = BN * 4 + 16;       // bytes a row of a shared tile's part
  static constexpr int kTileM = kBM * CG;
  static_assert(BN % 128 == 0 && BN <= 256, "whole scale tiles");
  static_assert(kAcc1 + BN <= kSfCol && 2 * kSfCols <= 32, "TMEM");
  static_assert(kStages >= 4 && kSmemBytes <= 232448, "shared memory");
  static_assert(kBM * kPartPitch <= kSfOffset, "the part fits the operand ring");
};

struct Tile {
  int32_t g, m0, n0;
};

// Tiles in order: matrix, then groups of 8 rows of tiles with m fastest, so that a wave
// shares columns of B and the group's rows of A in L2.
template <int BN, int CG>
__device__ __forceinline__ Tile tile_at(const Fp8Params& p, int32_t tile) {
  constexpr int kGroup = 8;
  const int32_t per = p.m_tiles * p.n_tiles;
  const int32_t g = tile / per, rem = tile - g * per;
  const int32_t full = kGroup * p.n_tiles, band = rem / full;
  const int32_t rows = min(kGroup, p.m_tiles - band * kGroup);
  const int32_t at = rem - band * full;
  return {g, (band * kGroup + at % rows) * (kBM * CG), at / rows * BN};
}

// A wait of the whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, DeviceError* err,
                                          uint32_t where, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, err, where, limit_ns));
}

template <int BN, int CG>
__global__ void __launch_bounds__(Fp8Cfg<BN, CG>::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
  using Cfg = Fp8Cfg<BN, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + Cfg::kStages * Cfg::kABytes;
  uint8_t* sS = smem + Cfg::kSfOffset;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOffset);
  uint64_t* empty_bar = full_bar + Cfg::kStages;
  uint64_t* tfull_bar = empty_bar + Cfg::kStages;      // an accumulator is complete
  uint64_t* tfree_bar = tfull_bar + 2;                 // the next tile may overwrite it
  uint64_t* done_bar = tfree_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = CG > 1 ? crank : 0;            // CTA within its pair
  const bool leader = rank == 0;
  const int32_t num_tiles = p.G * p.m_tiles * p.n_tiles;
  // With a shared K a cluster of `split` CTAs has one tile, and this CTA blocks [kb0, kb1).
  const int32_t ctas = CG > 1 ? CG : p.split;
  const int32_t first_tile = static_cast<int32_t>(blockIdx.x) / ctas;
  const int32_t tile_stride = static_cast<int32_t>(gridDim.x) / ctas;
  const int32_t kb0 = CG > 1 ? 0 : static_cast<int32_t>(crank) * p.kb_split;
  const int32_t kb1 = min(p.num_kb, kb0 + p.kb_split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tfree_bar[a], Cfg::kEpiW * CG);
    }
    mbar_init(done_bar, 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(&p.tmSA);
    tma_prefetch_desc(&p.tmSB);
    tma_prefetch_desc(&p.tmO);
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
  if constexpr (CG > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // Everything above touches only shared memory, TMEM and the kernel parameters.
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (as the MMA issuer: the whole warp runs the loop, an elected lane issues)
    int stage = 0;
    uint32_t phase = 0, armed_mask = 0, parity_mask = 0;
    bool ok = true;
    for (int32_t tile = first_tile; tile < num_tiles && ok; tile += tile_stride) {
      const Tile t = tile_at<BN, CG>(p, tile);
      const int32_t m_own = t.m0 + static_cast<int32_t>(rank) * kBM;
      const int32_t n_own = t.n0 + static_cast<int32_t>(rank) * Cfg::kBRows;
      // scale tiles: of this CTA's rows of A and all the tile's columns of B
      const int32_t ra = t.g * p.a_row_tiles + m_own / 128;
      const int32_t rb = t.g * p.b_row_tiles + t.n0 / 128;
      for (int32_t kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty_bar[stage], phase ^ 1u, p.err, 21, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        const bool scales = (kb & 3) == 0 || kb == kb0;
        armed_mask |= 1u << stage;
        parity_mask = (parity_mask & ~(1u << stage)) | (phase << stage);
        if (elect_one()) {
          uint8_t* dA = sA + stage * Cfg::kABytes;
          uint8_t* dB = sB + stage * Cfg::kBBytes;
          uint8_t* dS = sS + stage * Cfg::kSfBytes;
          if (leader)
            mbar_arrive_expect_tx(&full_bar[stage],
                                  CG * (Cfg::kABytes + Cfg::kBBytes + (scales ? Cfg::kSfBytes : 0)));
          if constexpr (CG == 2) {
            const uint32_t bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
            tma_load_3d_pair(dA, &p.tmA, bar, kb * kKBytes, m_own, t.g);
            tma_load_3d_pair(dB, &p.tmB, bar, kb * kKBytes, n_own, t.g);
            if (scales) {
              tma_load_3d_pair(dS, &p.tmSA, bar, 0, kb >> 2, ra);
              tma_load_3d_pair(dS + kScaleTile, &p.tmSB, bar, 0, kb >> 2, rb);
            }
          } else {
            tma_load_3d(dA, &p.tmA, &full_bar[stage], kb * kKBytes, m_own, t.g);
            tma_load_3d(dB, &p.tmB, &full_bar[stage], kb * kKBytes, n_own, t.g);
            if (scales) {
              tma_load_3d(dS, &p.tmSA, &full_bar[stage], 0, kb >> 2, ra);
              tma_load_3d(dS + kScaleTile, &p.tmSB, &full_bar[stage], 0, kb >> 2, rb);
            }
          }
        }
        __syncwarp();
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // the copies started here have landed before the CTA exits (both CTAs' complete on the
    // even CTA's barriers)
    if (leader) {
      for (int s = 0; s < Cfg::kStages; ++s) {
        if (armed_mask & (1u << s)) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&full_bar[s], (parity_mask >> s) & 1u)) {
            if (globaltimer_ns() - t0 > p.wait_limit_ns) {
              record_error(p.err, kErrTimeout, 27);
              break;
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues: with the loop itself on one
    // lane, the descriptors live in ordinary registers and the issue of an MMA takes longer than
    // its 128 cycles (8192^3: 335 us, about 185 cycles an MMA, and 292 us like this).
    if (leader) {
      int stage = 0;
      uint32_t phase = 0, sf = 0;                      // sf: which scale buffer
      const uint32_t idesc = idesc_mxf8_f32(kBM * CG, BN, p.a_fmt, p.b_fmt);
      const uint64_t hi = desc_hi_sw128(16u, 1024u);
      const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB), s0 = smem_u32(sS);
      bool ok = true;
      int32_t it = 0;                                  // tiles of this CTA so far
      for (int32_t tile = first_tile; tile < num_tiles && ok; tile += tile_stride, ++it) {
        const int acc = it & 1;
        // Free: the accumulator's own tile before last has been read (parity of its use), or,
        // where the two share columns, those of the last tile, which comes after that.
        const int wait_acc = Cfg::kOverlap ? acc ^ 1 : acc;
        const uint32_t uses = static_cast<uint32_t>(Cfg::kOverlap ? (it + 1) >> 1 : it >> 1);
        if (!warp_wait(&tfree_bar[wait_acc], (uses & 1u) ^ 1u, p.err, 22, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * Cfg::kAcc1;
        uint32_t sa = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
          if (!warp_wait(&full_bar[stage], phase, p.err, 23, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool scales = (kb & 3) == 0 || kb == kb0;
          if (scales) {
            sa = tmem_base + Cfg::kSfCol + sf * 16;
            sf ^= 1u;
          }
          const uint64_t ad = hi | (((a0 + stage * Cfg::kABytes) >> 4) & 0x3FFFu);
          const uint64_t bd = hi | (((b0 + stage * Cfg::kBBytes) >> 4) & 0x3FFFu);
          const uint64_t sd = smem_desc_scales(s0 + stage * Cfg::kSfBytes);
          const uint32_t id = idesc | idesc_scale_id(kb & 3);
          if (elect_one()) {
            if (scales) {
#pragma unroll
              for (int i = 0; i <= Cfg::kSfTilesB; ++i)
                tc_cp_scales<CG>(sa + 4 * i, sd + i * (kScaleTile >> 4));
            }
#pragma unroll
            for (int kk = 0; kk < kKBytes / 32; ++kk)
              tc_mma_mxf8<CG>(d_tmem, ad + 2 * kk, bd + 2 * kk, id, sa, sa + 4,
                              kk > 0 ? 1u : (kb > kb0 ? 1u : 0u));
            if constexpr (CG == 2)
              tc_commit_pair_mc(&empty_bar[stage], static_cast<uint16_t>(3));
            else
              tc_commit(&empty_bar[stage]);
          }
          __syncwarp();
          if (++stage == Cfg::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (elect_one()) {
          if constexpr (CG == 2)
            tc_commit_pair_mc(&tfull_bar[acc], static_cast<uint16_t>(3));
          else
            tc_commit(&tfull_bar[acc]);
        }
        __syncwarp();
      }
      // every MMA issued here is complete before TMEM is released
      if (elect_one()) {
        if constexpr (CG == 2) tc_commit_pair(done_bar); else tc_commit(done_bar);
      }
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done_bar, 0)) {
        if (globaltimer_ns() - t0 > p.wait_limit_ns) {
          record_error(p.err, kErrTimeout, 28);
          break;
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- epilogue
    // Two warps a lane quarter: warp `half` takes 32-column chunks half, half + 2, ... of the
    // first accumulator in falling order and of the second in rising order, so that the
    // shared columns (the last chunk and the first) are read at once.
    const int q = warp & 3, half = (warp - 2) / 4;
    StoreRing<1, true> ring{smem + Cfg::kStgOffset + (warp - 2) * 2048, 0};
    int32_t it = 0;
    for (int32_t tile = first_tile; tile < num_tiles; tile += tile_stride, ++it) {
      const int acc = it & 1;
      const Tile t = tile_at<BN, CG>(p, tile);
      const int32_t row0 = t.m0 + static_cast<int32_t>(rank) * kBM + q * 32;
      const int32_t row = row0 + lane;
      const float scale = p.row_scale != nullptr && row < p.M ? p.row_scale[row] : 1.0f;
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * Cfg::kAcc1;
      if (!bounded_wait(&tfull_bar[acc], static_cast<uint32_t>(it >> 1) & 1u, p.err, 24,
                        p.wait_limit_ns))
        break;
      tc_fence_after();
      constexpr int kChunks = BN / 64;                 // of one warp
      if (CG == 1 && p.split > 1) {
        // this CTA's part of the tile to shared memory (the ring: its operands are used up)
        float* mine = reinterpret_cast<float*>(smem + (q * 32 + lane) * Cfg::kPartPitch);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = 2 * i + half;
          float v[32];
          tmem_ld_32x32b_x32(t_row + c * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(mine + c * 32 + j) =
                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        break;                                         // (one tile a cluster)
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = 2 * (acc == 0 ? kChunks - 1 - i : i) + half;
        float v[32];
        tmem_ld_32x32b_x32(t_row + c * 32, v);
        tmem_ld_wait();
        if (i == (Cfg::kOverlap ? 0 : kChunks - 1)) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 2)
              mbar_arrive_cluster(mapa_shared(smem_u32(&tfree_bar[acc]), 0));
            else
              mbar_arrive(&tfree_bar[acc]);
          }
        }
        const int32_t col0 = t.n0 + c * 32;
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          pk[j] = pack_bf16x2(act_fwd(v[2 * j] * scale, p.act), act_fwd(v[2 * j + 1] * scale, p.act));
        if (col0 < p.N && row0 < p.M)
          store_chunk_bf16(ring, lane, pk, &p.tmO, true, col0, row0, t.g,
                           static_cast<__nv_bfloat16*>(nullptr), 0, 0, 0);
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  if (CG == 1 && p.split > 1) {
    // The parts are summed in the CTAs' order; each CTA takes every split-th row.
    cluster_sync();
    constexpr int kVec = BN / 4;
    const Tile t = tile_at<BN, CG>(p, first_tile);
    const int32_t rows = (min(kBM, p.M - t.m0) - static_cast<int32_t>(crank) + p.split - 1) / p.split;
    for (int32_t i = threadIdx.x; i < rows * kVec; i += Cfg::kThreads) {
      const int32_t r = i / kVec * p.split + static_cast<int32_t>(crank), c = i % kVec * 4;
      if (t.n0 + c >= p.N) continue;
      const uint32_t at = smem_u32(smem) + r * Cfg::kPartPitch + c * 4;
      float4 v = ld_cluster_f4(mapa_shared(at, 0));
      for (int32_t k = 1; k < p.split; ++k) {
        const float4 w = ld_cluster_f4(mapa_shared(at, k));
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
      }
      const int32_t row = t.m0 + r;
      const float f = p.row_scale != nullptr ? p.row_scale[row] : 1.0f;
      *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t.g) * p.M + row) * p.N + t.n0 + c) =
          make_uint2(pack_bf16x2(act_fwd(v.x * f, p.act), act_fwd(v.y * f, p.act)),
                     pack_bf16x2(act_fwd(v.z * f, p.act), act_fwd(v.w * f, p.act)));
    }
  }
  // (a CTA whose shared memory others read stays until they have)
  tc_fence_before();
  if (CG > 1 || p.split > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

// ----------------------------------------------------------------------- host
bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t d0, uint64_t d1,
              uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1, uint32_t b2,
              CUtensorMapSwizzle swizzle) {
  EncodeFn enc = get_encode();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
  const cuuint32_t box[3] = {b0, b1, b2}, ones[3] = {1, 1, 1};
  return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `split` CTAs of a cluster share a tile's K (CG = 1).
template <int BN, int CG>
cudaError_t launch_shape(const Fp8GemmParams& g, int split, cudaStream_t stream) {
  using Cfg = Fp8Cfg<BN, CG>;
  const auto kern = fp8_gemm_kernel<BN, CG>;
  const boost_fp8_matmul_desc& d = g.d;
  Fp8Params p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t M = d.M, N = d.N, K = d.K, G = d.G;
  const uint64_t kt = scale_tiles_k(d.K), ra = (M + 127) / 128, rb = (N + 127) / 128;
  if (!make_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a, K, M, G, d.a_pitch, M * d.a_pitch,
                kKBytes, kBM, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.b, K, N, G, d.b_pitch, N * d.b_pitch,
                kKBytes, Cfg::kBRows, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.tmSA, CU_TENSOR_MAP_DATA_TYPE_INT32, g.a_sf, 128, kt, ra * G, kScaleTile,
                kt * kScaleTile, 128, 1, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&p.tmSB, CU_TENSOR_MAP_DATA_TYPE_INT32, g.b_sf, 128, kt, rb * G, kScaleTile,
                kt * kScaleTile, 128, 1, Cfg::kSfTilesB, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&p.tmO, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.out, N, M, G, 2 * N, 2 * M * N, 32, 32,
                1, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.G = static_cast<int32_t>(G);
  p.num_kb = static_cast<int32_t>((K + kKBytes - 1) / kKBytes);
  p.m_tiles = static_cast<int32_t>((M + Cfg::kTileM - 1) / Cfg::kTileM);
  p.n_tiles = static_cast<int32_t>((N + BN - 1) / BN);
  p.a_row_tiles = static_cast<int32_t>(ra);
  p.b_row_tiles = static_cast<int32_t>(rb);
  // every CTA of a cluster has a block at least
  p.kb_split = (p.num_kb + split - 1) / split;
  p.split = (p.num_kb + p.kb_split - 1) / p.kb_split;
  p.a_fmt = d.a_fmt;
  p.b_fmt = d.b_fmt;
  p.act = d.act;
  p.row_scale = g.row_scale;
  p.out = static_cast<__nv_bfloat16*>(g.out);
  p.err = static_cast<DeviceError*>(g.ws);
  p.wait_limit_ns = wait_limit_ns();

  // per-device state, filled once (host threads may do so concurrently with the same values)
  static std::atomic<int> resident[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
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
  cfg.numAttrs = 1;
  int groups = dev < 64 ? resident[dev].load(std::memory_order_acquire) : 0;
  if (groups == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    if (e != cudaSuccess) return e;
    groups = current_num_sms() / CG;
    if (CG > 1) {
      int n = 0;
      cfg.gridDim = dim3(static_cast<unsigned>(groups * CG), 1, 1);
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0)
        groups = std::min(groups, n);
      else
        cudaGetLastError();
    }
    if (dev < 64) resident[dev].store(groups, std::memory_order_release);
  }
  const int64_t tiles = static_cast<int64_t>(p.G) * p.m_tiles * p.n_tiles;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, groups) * CG), 1, 1);
  if (CG == 1 && p.split > 1) {
    attr[0].val.clusterDim.x = p.split;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split), 1, 1);
  }
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

size_t fp8_gemm_workspace(const boost_fp8_matmul_desc&) { return 256; }

// Launch shape by a model of its time in microseconds, fitted to 44 sizes (M from 1 to 1024,
// N x K from 1536 x 2048 to 11008 x 1024; most are within 15%):
//   CTA pairs, 256 x 256:  7 + waves (0.7 + 0.265 blocks of K)
//   single CTAs, 128 x 128:  6 + waves (0.4 + 0.225 blocks): a CTA's operands arrive at the
//     SM's 64 bytes a cycle from L2, so the smaller tile's block is hardly quicker and only
//     wins by using more SMs (M = 512, 4096 x 4096: 14.5 against 16.6 us)
//   the same with K shared by a cluster:  7.5 + 0.225 of its blocks + 2.2 to join 128 rows,
//     all of that once more for every further wave of clusters (M = 1, 1024 x 11008: 25.4 us
//     on 8 CTAs, 9.7 us on 64)
cudaError_t launch_fp8_gemm(const Fp8GemmParams& g, cudaStream_t stream) {
  const boost_fp8_matmul_desc& d = g.d;
  const int sms = current_num_sms();
  const double blocks = static_cast<double>((d.K + kKBytes - 1) / kKBytes);
  auto waves = [&](int64_t m, int64_t n, int64_t slots) {
    const int64_t tiles = d.G * ((d.M + m - 1) / m) * ((d.N + n - 1) / n);
    return static_cast<double>((tiles + slots - 1) / std::max<int64_t>(slots, 1));
  };
  double best = 7.0 + waves(256, 256, sms / 2) * (0.7 + 0.265 * blocks);
  int split = 0;                         // 0: CTA pairs
  const double single = 6.0 + waves(128, 128, sms) * (0.4 + 0.225 * blocks);
  if (single < best) {
    best = single;
    split = 1;
  }
  for (int c = 2; c <= 8 && c <= blocks; ++c) {
    // (clusters sit inside one of eight GPCs of 18 to 20 SMs; 15 of eight CTAs fit)
    const int slots = (sms / 8 - 1) / c * 8 - (c == 8);
    const double join = 2.2 * std::min<int64_t>(d.M, 128) / 128.0;
    const double t = waves(128, 128, slots) * (7.5 + 0.225 * std::ceil(blocks / c) + join);
    if (t < best) {
      best = t;
      split = c;
    }
  }
  if (split == 0) return launch_shape<256, 2>(g, 1, stream);
  return launch_shape<128, 1>(g, split, stream);
}

}  // namespace boost_gb300
