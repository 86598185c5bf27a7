// Gradients of the gated MLP's two projections as tcgen05 products on CTA
// pairs (cta_group::2, 256 x 256 output tiles, fp32 accumulators in TMEM).
//
// Forward (fused_large_m_pair.cu): G = A W1, U = A W2, Y = SiLU(G) * U, and
// Out = Y W3 + R. With s = 1 / (1 + e^-G) the gradients are
//   dU = dY * G s,   dG = dY * U * s (1 + G (1 - s))          (kGrad)
//   dA = dG W1^T + dU W2^T          or   dY = dOut W3^T       (input gradient)
//   dW1 = A^T dG, dW2 = A^T dU      or   dW3 = Y^T dOut       (weight gradient)
// G and U are not kept by the forward; kGrad recomputes them in the forward's
// own pipeline and its epilogue turns the fp32 accumulators and dY into dG and
// dU, each rounded once to bf16: they are operands of tensor-core products, and
// an operand held in 32 bits would run at half the rate (tf32) or three times
// the products (split bf16). The rounding is independent from element to
// element, so the relative error of a gradient grows by sqrt(2) over rounding
// its exact value to bf16, whatever the length of the sum.
//
// One kernel body, three operand shapes. Every load is a TMA box of 128-byte
// rows under the 128-byte swizzle; what differs is which tensor dimension is
// contiguous and so which "major" the MMA descriptors state:
//   kGrad    rows [m][k] x packed weight [n][k]: both contiguous along the sum
//   input    rows [m][n] contiguous along the sum; the packed weight's tiles
//            [n][64 k] hold the sum along their rows (MN-major), so the same
//            packed weight serves the forward and this product, no transpose
//   weight   both operands are row-major with the sum (tokens) down the rows:
//            MN-major twice, no transposed copy of anything is written
// An MN-major operand of 128 columns x 128 of the sum comes as two boxes of 64
// columns x 128 rows, one in each of two consecutive stages (8-row groups 1024
// bytes apart, the other 64 columns one stage further), so the input and weight
// gradients use their stages in pairs, 128 of the sum at a time. Boxes of 64
// rows, two to a stage, hold the same bytes but load slower: the 7B weight
// gradient of the down-projection took 365 us against 310 (one 3-D box for
// both) and 415 (two 2-D boxes); the loads, not the MN-major MMAs, were what
// it waited for (K-major descriptors on the same bytes: 365 us too).
//
// Roles as in the forward pair kernel: warp 0 TMA producer, warp 1 MMA issuer
// (even CTA), then 8 epilogue warps, two for each 32 rows (with 4, short sums
// waited for them: 16 tokens on the 7B weights 215 against 201 us); 6 stages of
// 32 KB per CTA; two accumulators of 256 columns, so a tile's epilogue runs
// under the next tile's MMAs; every wait is bounded (ptx.cuh).
//
// kGrad has tiles of 128 gate and the matching 128 up columns. Where the tiles of
// its last round would leave half of the pairs idle, they are cut into halves of
// 64 columns (half-width MMAs read the left operand twice as often, so whole
// rounds of halves would be slower: 2280 against 1820 us for the 7B backward).
//
// The input and the weight gradients do not depend on one another, so one
// launch computes both: its units are the input gradient's tiles, then the
// weight gradient's, and unit_at() deals them to the pairs so that pairs with
// one input tile fewer take as many weight tiles more. A launch of its own for
// each left a part-filled last round twice, and on short sums (0.5B, 128
// tokens) its start-up cost as much as its work.
//
// Few output tiles: with `splits` > 1 each tile's sum is cut into that many
// parts, each part's fp32 accumulator goes to the workspace and
// reduce_parts_kernel adds the parts in order (results do not depend on
// timing) and rounds once.
//
// With Gate and Up kept by the forward (checkpoint.cu makes dG and dU) only the second
// launch runs. kScaled: dG and dU hold a factor for each token that is not dA's, so the
// epilogue divides dA's rows by it (a template argument: as a branch at run time it cost the
// other launches of this kernel 4 % at the 0.5B shape).
//
// Measured, 7B block, 4096 tokens, one call at a time: dG and dU 567-573 us (1.95
// PFLOP/s), both gradients 1114-1125 us (1.98), tensor pipe 92 % busy in each; back
// to back at the power cap 1974 us in all (1.69 PFLOP/s). 16 tokens on the same
// weights: 174 us for 272 MB read twice and 272 MB written (writes alone run at 4.0
// TB/s here). 0.5B block, 128 tokens: 27.7 us, three launches that each wait for one
// another (9, 15 and 4 us alone).
#include <type_traits>

#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kOperandBytes = 128 * kBlockK * 2;       // 16 KB: 128 rows (or columns) x 64 of the sum
constexpr int kStageBytes = 2 * kOperandBytes;         // per CTA
constexpr int kStages = 6;
constexpr int kAccCols = 256;
constexpr int kStgBytes = 32 * 128;                    // 32 rows x 128 B store staging
constexpr int kEpiWarps = 8;                           // 2 per tensor-memory lane quarter
constexpr int kNumStg = kEpiWarps;                     // 1 per epilogue warp
constexpr int kBackThreads = 64 + 32 * kEpiWarps;
constexpr int kBarBytes = 256;
constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes + size_t(kNumStg) * kStgBytes + kBarBytes;
static_assert(kStages % 2 == 0, "stages are used in pairs");
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes, "barrier slots");

__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int group_m, int& mb,
                                            int& nb) {
  const int per_group = group_m * tiles_n;
  const int g = t / per_group;
  const int first_m = g * group_m;
  const int gm = min(tiles_m - first_m, group_m);
  const int r = t - g * per_group;
  mb = first_m + r % gm;
  nb = r / gm;
}

// The `step`-th unit of a pair: an input-gradient unit, then weight-gradient
// units; -1 past the last. Of `in_units` = q pairs + r, pairs r.. have one unit
// fewer (when r > 0) and first take `early_rounds` rounds of weight units among
// themselves; all pairs share the rest round by round.
__device__ __forceinline__ int unit_at(const BackwardParams& p, int pair, int pairs, int step,
                                       bool& weight) {
  const int r = p.in_units % pairs;
  const int mine = p.in_units / pairs + (pair < r ? 1 : 0);
  weight = step >= mine;
  if (!weight) return pair + step * pairs;
  int k = step - mine, first = 0;
  if (r > 0) {
    if (pair >= r) {
      if (k < p.early_rounds) return pair - r + k * (pairs - r);
      k -= p.early_rounds;
    }
    first = p.early_rounds * (pairs - r);
  }
  const int64_t u = first + pair + int64_t(k) * pairs;
  return u < p.w_units ? static_cast<int>(u) : -1;
}

// First stage of a part of the sum; whole pairs of stages except for kGrad.
template <bool kGrad>
__device__ __forceinline__ int part_begin(const BackwardProduct& g, int part) {
  constexpr int kUnit = kGrad ? 1 : 2;
  return static_cast<int>(int64_t(part) * (g.slices / kUnit) / g.splits) * kUnit;
}

// A kGrad unit: a whole tile, or from unit full_units on a half of one.
__device__ __forceinline__ void grad_unit(const BackwardParams& p, int u, int& tile, int& bn, int& off) {
  const int h = u - p.full_units;
  tile = h < 0 ? u : p.full_units + (h >> 1);
  bn = h < 0 ? kPackBlockN : kPackBlockN / 2;
  off = h < 0 ? 0 : (h & 1) * (kPackBlockN / 2);
}

template <bool kGrad, bool kScaled>
__global__ void __launch_bounds__(kBackThreads, 1)
    backward_pair_kernel(const __grid_constant__ BackwardParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_addr(smem);
  const uint32_t sB = sA + kStages * kOperandBytes;
  const uint32_t sStg = sB + kStages * kOperandBytes;
  uint8_t* bar_ptr = smem + size_t(kStages) * kStageBytes + kNumStg * kStgBytes;
  const uint32_t bar0 = smem_addr(bar_ptr);
  // barrier slots: full[S] | empty[S] | tmem_full[2] | tmem_empty[2] | drain
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * kStages;
  const uint32_t tfull0 = bar0 + 16u * kStages, tempty0 = tfull0 + 16u;
  const uint32_t drain_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * (2 * kStages + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());
  const int pairs = static_cast<int>(cluster_count_x());
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  const uint32_t full0_lead = mapa_shared(full0, 0);
  const uint32_t tempty0_lead = mapa_shared(tempty0, 0);

  if (threadIdx.x == 0) {
    const BackwardProduct& g = p.in_units > 0 ? p.in : p.w;  // the other one's maps may be unset
    prefetch_tmap(&g.tmap_a0);
    prefetch_tmap(&g.tmap_b0);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8u * s, 1);   // rank 0's producer arrives (with both CTAs' bytes)
      mbar_init(empty0 + 8u * s, 1);  // rank 0's MMA commit, multicast to both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);   // multicast MMA commit
      mbar_init(tempty0 + 8u * b, 2 * kEpiWarps);  // epilogue warps x 2 CTAs (used on rank 0)
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  cluster_arrive();  // both CTAs run, their barriers initialised
  cluster_wait();
  pdl_wait();
  if (warp == 1) tmem_alloc_pair(smem_addr(tmem_slot), 2 * kAccCols);
  tc_fence_before();
  cluster_arrive();  // tensor memory allocated; the producer need not wait for that
  if (warp != 0) cluster_wait();
  tc_fence_after();
  if (warp == 1) tmem_relinquish_pair();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    // (the whole warp waits and counts, one lane issues, as below)
    {
      const bool one = elect_one();
      int s = 0;
      uint32_t ph = 0;
      uint32_t filled = 0, fill_ph = 0;
      bool skip_once = p.inject_stall != 0;
      bool ok = true;
      bool weight;
      for (int step = 0, u; ok && (u = unit_at(p, pair, pairs, step, weight)) >= 0; ++step) {
        const BackwardProduct& g = weight ? p.w : p.in;
        int tile = u / g.splits, part = u - tile * g.splits, bn = kPackBlockN, off = 0;
        if constexpr (kGrad) grad_unit(p, u, tile, bn, off);
        int mb, nb;
        tile_coords(tile, g.tiles_m, g.tiles_n, g.group_m, mb, nb);
        const int r0 = mb * 2 * kTileM + static_cast<int>(rank) * kTileM;  // output row of this CTA
        const int begin = part_begin<kGrad>(g, part), end = part_begin<kGrad>(g, part + 1);
        // Few tokens: boxes end with the last 8 (16) of them, and a CTA whose rows all
        // lie past the output loads none. What the MMA then reads past them only
        // reaches rows that are not stored, or is left out of the sum.
        const bool rows_here = weight || r0 < g.rows;
        const bool rows_peer = weight || mb * 2 * kTileM + kTileM < g.rows;  // the odd CTA's
        const CUtensorMap* map_b = bn == kPackBlockN ? &g.tmap_b0 : &g.tmap_b1;  // kGrad
        const uint32_t bytes = g.a_bytes * (rows_peer ? 2 : 1) + 2 * (weight ? g.a_bytes : bn * kBlockK * 2);
        for (int i = begin; i < end; ++i) {
          if (!mbar_wait_warp(empty0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          if (skip_once) {
            skip_once = false;  // testing hook: both CTAs leave this stage unfilled
          } else {
            if (one) {
              if (leader) mbar_arrive_expect_tx(full0 + 8u * s, bytes);
              const uint32_t fb = full0_lead + 8u * s;
              const uint32_t da = sA + s * kOperandBytes, db = sB + s * kOperandBytes;
              if constexpr (kGrad) {
                // A rows [r0, +128); bn gate (rank 0) or up (rank 1) rows of tile (nb, i)
                if (rows_here) tma_load_2d_pair(da, &g.tmap_a0, fb, i * kBlockK, r0);
                tma_load_3d_pair(db, map_b, fb, 0,
                                 static_cast<int>(rank) * kPackBlockN + off, nb * g.slices + i);
              } else if (!weight) {
                // stages 2 d, 2 d + 1: rows [128 h, +128) of packed tile row j (a gate/up
                // tile holds 128 gate then 128 up columns of the sum, a down tile 256);
                // left operand: 64 of those columns of the sum a stage; right operand:
                // all 128, for 64 of this CTA's 128 output columns a stage (a block past
                // the last one reads another tile or zeros; its columns lie outside the
                // output and are not stored)
                const int j = i >> 2, h = (i >> 1) & 1, e = i & 1;
                const int col = (g.two ? j * kPackBlockN : j * 2 * kPackBlockN + h * kPackBlockN) + e * kBlockK;
                if (rows_here) tma_load_2d_pair(da, g.two && h ? &g.tmap_a1 : &g.tmap_a0, fb, col, r0);
                tma_load_3d_pair(db, &g.tmap_b0, fb, 0, h * kPackBlockN,
                                 j * g.col_slices + nb * 4 + static_cast<int>(rank) * 2 + e);
              } else {
                // stages 2 d, 2 d + 1: tokens [128 d, +128), 64 of this CTA's 128 output
                // rows and 64 of its 128 output columns a stage
                const int m = (i >> 1) * 2 * kBlockK, e = (i & 1) * kBlockK;
                const int c0 =
                    g.two ? nb * kTileM : nb * 2 * kTileM + static_cast<int>(rank) * kTileM;
                tma_load_2d_pair(da, &g.tmap_a0, fb, r0 + e, m);
                tma_load_2d_pair(db, g.two && rank ? &g.tmap_b1 : &g.tmap_b0, fb, c0 + e, m);
              }
            }
            filled |= 1u << s;
            fill_ph = (fill_ph & ~(1u << s)) | (ph << s);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (one) pdl_launch_dependents();
      // Rank 0's full barriers count both CTAs' bytes: once they complete, every
      // copy issued by the pair for those stages has landed.
      if (leader && one)
        for (int i = 0; i < kStages; ++i)
          if (filled & (1u << i)) mbar_wait_drain(full0 + 8u * i, (fill_ph >> i) & 1u, wc);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (rank 0)
    // The whole warp waits and counts, one lane issues: with one lane in the loop from
    // the start the descriptors are not warp-uniform to the compiler, and the issue
    // itself held the tensor pipe up. Here and in the producer, 7B block, 4096 tokens:
    // dG and dU 1.11 -> 0.99 M cycles, both gradients 2.11 -> 1.98.
    if (leader) {
      const bool one = elect_one();
      int s = 0;
      uint32_t ph = 0;
      int buf = 0;
      uint32_t acc_ph = 0;
      bool ok = true, weight;
      for (int step = 0, u; ok && (u = unit_at(p, pair, pairs, step, weight)) >= 0; ++step) {
        const BackwardProduct& g = weight ? p.w : p.in;
        const int part = u % g.splits;
        const int begin = part_begin<kGrad>(g, part), end = part_begin<kGrad>(g, part + 1);
        if (!mbar_wait_warp(tempty0 + 8u * buf, acc_ph ^ 1u, wc, kSiteMmaTmemEmpty)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * kAccCols;
        if constexpr (kGrad) {
          // the instruction descriptors as constants: 3 % of this kernel on the 7B shape
          const auto issue = [&](auto columns) {
            constexpr uint32_t kIdesc = idesc_bf16_f32(2 * kTileM, decltype(columns)::value);
            for (int i = begin; i < end; ++i) {
              if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteMmaFull)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t adesc = smem_desc_sw128(sA + s * kOperandBytes);
              const uint64_t bdesc = smem_desc_sw128(sB + s * kOperandBytes);
              if (one) {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                  mma_bf16_pair(d, adesc + 2u * k, bdesc + 2u * k, kIdesc, (i != begin || k != 0) ? 1u : 0u);
                mma_commit_pair_multicast(empty0 + 8u * s, 0x3);  // frees the stage in both CTAs
              }
              __syncwarp();
              if (++s == kStages) {
                s = 0;
                ph ^= 1u;
              }
            }
          };
          if (u < p.full_units)
            issue(std::integral_constant<int, 2 * kPackBlockN>{});
          else
            issue(std::integral_constant<int, kPackBlockN>{});
        } else {
          // Bits 15 (left) and 16 (right) of the descriptor mark MN-major operands.
          // 16 of the sum are 16 rows of 128 bytes of an MN-major operand, 32 bytes
          // along a K-major row (four in each of the two stages).
          const auto issue = [&](auto of_weight) {
            constexpr bool kWeight = decltype(of_weight)::value;
            constexpr uint32_t kIdesc =
                idesc_bf16_f32(2 * kTileM, kAccCols) | (kWeight ? 1u << 15 : 0u) | (1u << 16);
            for (int i = begin; i < end; i += 2) {  // s is even: every unit has whole pairs of stages
              if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteMmaFull) ||
                  !mbar_wait_warp(full0 + 8u * (s + 1), ph, wc, kSiteMmaFull)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t pa = sA + s * kOperandBytes;
              const uint64_t adesc = kWeight ? smem_desc_sw128_mn(pa, kOperandBytes) : smem_desc_sw128(pa);
              const uint64_t bdesc = smem_desc_sw128_mn(sB + s * kOperandBytes, kOperandBytes);
              // weight gradient: no MMA for 16 tokens that do not exist (capped before it is
              // rounded up, as up to 2^31 - 1 tokens are left)
              const int ksteps = kWeight ? (min(g.sum - (i >> 1) * 2 * kBlockK, 2 * kBlockK) + 15) / 16 : 8;
              if (one) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const uint64_t da = adesc + (kWeight ? (2048u >> 4) * k
                                                      : 2u * (k & 3) + (k >> 2) * (kOperandBytes >> 4));
                  if (k < ksteps)
                    mma_bf16_pair(d, da, bdesc + (2048u >> 4) * k, kIdesc, (i != begin || k != 0) ? 1u : 0u);
                }
                mma_commit_pair_multicast(empty0 + 8u * s, 0x3);  // frees the stages in both CTAs
                mma_commit_pair_multicast(empty0 + 8u * (s + 1), 0x3);
              }
              __syncwarp();
              s += 2;
              if (s == kStages) {
                s = 0;
                ph ^= 1u;
              }
            }
          };
          if (weight)
            issue(std::true_type{});
          else
            issue(std::false_type{});
        }
        if (!ok) break;
        if (one) mma_commit_pair_multicast(tfull0 + 8u * buf, 0x3);  // both halves of the accumulator ready
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1u;
      }
      if (one) {
        mma_commit_pair_multicast(drain_bar, 0x1);
        mbar_wait_drain(drain_bar, 0, wc);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const int ew = warp - 2;
    const int half = ew >> 2;  // this warp's half of the tile's columns
    const uint32_t stg = sStg + ew * kStgBytes;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    int buf = 0;
    uint32_t acc_ph = 0;
    bool weight;
    for (int step = 0, unit; (unit = unit_at(p, pair, pairs, step, weight)) >= 0; ++step) {
      const BackwardProduct& pr = weight ? p.w : p.in;
      int tile = unit / pr.splits, part = unit - tile * pr.splits, bn = kPackBlockN, off = 0;
      if constexpr (kGrad) grad_unit(p, unit, tile, bn, off);
      int mb, nb;
      tile_coords(tile, pr.tiles_m, pr.tiles_n, pr.group_m, mb, nb);
      const int row0 = mb * 2 * kTileM + static_cast<int>(rank) * kTileM + q * 32;
      uint4 dyv[4];
      const __nv_bfloat16* dy_row = nullptr;
      const int col0 = nb * kPackBlockN + off + half * (bn / 2);
      const auto load_dy = [&](int c) {  // this thread's row of dY, columns of chunk c
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = col0 + 32 * c + 8 * e;
          dyv[e] = row0 + lane < pr.rows && col < pr.cols
                       ? *reinterpret_cast<const uint4*>(dy_row + col)
                       : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if constexpr (kGrad) {
        dy_row = static_cast<const __nv_bfloat16*>(p.dy) + static_cast<size_t>(row0 + lane) * pr.cols;
        load_dy(0);
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait(tfull0 + 8u * buf, acc_ph, wc, kSiteEpiTmemFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_off + buf * kAccCols;
      if constexpr (kGrad) {
        // the width as a constant: 3 % of this kernel on the 7B shape
        const auto chunk_loop = [&](auto width) {
          constexpr int kBN = decltype(width)::value, kChunks = kBN / 64;  // 32 columns of this warp
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            uint32_t g[32], u[32];
            tmem_ld_x32(tacc + half * (kBN / 2) + c * 32, g);
            tmem_ld_x32(tacc + kBN + half * (kBN / 2) + c * 32, u);
            uint4 dyc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) dyc[e] = dyv[e];
            if (c + 1 < kChunks) load_dy(c + 1);
            tmem_wait_ld();
            reg_fence(g);
            reg_fence(u);
            if (c == kChunks - 1) {  // this warp's part of the accumulator is read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(tempty0_lead + 8u * buf);
            }
            if (lane == 0) bulk_wait_read<0>();  // the previous store has read the staging
            __syncwarp();
            const uint32_t row_addr = stg + lane * 64;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t wg[4], wu[4];
              const uint32_t dw[4] = {dyc[j].x, dyc[j].y, dyc[j].z, dyc[j].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i0 = 8 * j + 2 * e;
                const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&dw[e]);
                float dg0, du0, dg1, du1;
                gate_grads(__uint_as_float(g[i0]), __uint_as_float(u[i0]), __low2float(h), dg0, du0);
                gate_grads(__uint_as_float(g[i0 + 1]), __uint_as_float(u[i0 + 1]), __high2float(h),
                           dg1, du1);
                wg[e] = pack_bf16x2(dg0, dg1);
                wu[e] = pack_bf16x2(du0, du1);
              }
              const uint32_t off = (j ^ ((lane >> 1) & 3)) << 4;
              st_shared_v4(row_addr + off, wg[0], wg[1], wg[2], wg[3]);
              st_shared_v4(row_addr + 2048 + off, wu[0], wu[1], wu[2], wu[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int ncol = col0 + c * 32;
              if (ncol < pr.cols && row0 < pr.rows) {
                tma_store_2d(&pr.tmap_o0, stg, ncol, row0);
                tma_store_2d(&pr.tmap_o1, stg + 2048, ncol, row0);
              }
              bulk_commit();
            }
          }
        };
        if (bn == kPackBlockN)
          chunk_loop(std::integral_constant<int, kPackBlockN>{});
        else
          chunk_loop(std::integral_constant<int, kPackBlockN / 2>{});
      } else {
        // this warp's 128 columns, 64 at a time: fp32 parts (32 columns, 128-byte
        // rows, a store) to the workspace, or 64 bf16 columns to the output
        const bool parts = pr.splits > 1;
        // kScaled: the rows of dG and dU came with a factor of their token's (checkpoint.cu)
        float by = 1.0f;
        if (kScaled && !weight && row0 + lane < pr.rows)
          by = 1.0f / split_scale(pr.row_scale[row0 + lane]).factor;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t x[32], y[32];
          tmem_ld_x32(tacc + half * 128 + c * 64, x);
          tmem_ld_x32(tacc + half * 128 + c * 64 + 32, y);
          tmem_wait_ld();
          reg_fence(x);
          reg_fence(y);
          if constexpr (kScaled) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = __float_as_uint(__uint_as_float(x[i]) * by);
              y[i] = __float_as_uint(__uint_as_float(y[i]) * by);
            }
          }
          if (c == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0_lead + 8u * buf);
          }
          const bool two = weight && pr.two;  // the halves are two outputs
          const CUtensorMap* mapo = two && half ? &pr.tmap_o1 : &pr.tmap_o0;
          const int ncol = (two ? nb * kTileM : nb * 2 * kTileM + half * kTileM) + c * 64;
          if (parts) {
            // part-major rows: the store maps see splits * padded rows
            const int prow = part * pr.part_rows + row0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (lane == 0) bulk_wait_read<0>();
              __syncwarp();
              const uint32_t row_addr = stg + lane * 128;
              const uint32_t* v = h ? y : x;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                st_shared_v4(row_addr + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1],
                             v[4 * j + 2], v[4 * j + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (ncol + 32 * h < pr.cols && row0 < pr.rows)
                  tma_store_2d(mapo, stg, ncol + 32 * h, prow);
                bulk_commit();
              }
            }
          } else {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            const uint32_t row_addr = stg + lane * 128;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t* v = j < 4 ? x + 8 * j : y + 8 * (j - 4);
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
              st_shared_v4(row_addr + ((j ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (ncol < pr.cols && row0 < pr.rows) tma_store_2d(mapo, stg, ncol, row0);
              bulk_commit();
            }
          }
        }
      }
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1u;
    }
    tc_fence_before();
    cluster_arrive_release();  // the accumulators have been read; the last stores go on
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  // Neither CTA leaves while the pair's MMAs may still read its shared memory
  // or the peer may still arrive on its barriers.
  if (warp == 0) cluster_wait();
  if (warp < 2) {
    tc_fence_before();
    cluster_arrive_release();
  }
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kAccCols);
  }
  cluster_arrive();  // nor while the peer gives its tensor memory back
  cluster_wait();
}

// out[r][c] = bf16(sum over parts, in order, of parts[part][r][c]) for each
// output cut into parts: one pass over fp32 values that are mostly still in L2,
// 8 columns a thread.
__global__ void __launch_bounds__(256) reduce_parts_kernel(const __grid_constant__ ReduceParams p) {
  pdl_launch_dependents();
  pdl_wait();
  for (int o = 0; o < p.count; ++o) {
    const ReduceOutput& r = p.out[o];
    const size_t items = static_cast<size_t>(r.rows) * (r.cols / 8);
    const size_t part_stride = static_cast<size_t>(r.part_rows) * r.cols;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < items;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
      const float* src = r.parts + i * 8;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 8
      for (int s = 0; s < r.splits; ++s) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + s * part_stride));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src + s * part_stride + 4));
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
      }
      uint4 v;
      v.x = pack_bf16x2(a.x, a.y);
      v.y = pack_bf16x2(a.z, a.w);
      v.z = pack_bf16x2(b.x, b.y);
      v.w = pack_bf16x2(b.z, b.w);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.out) + i * 8) = v;
    }
  }
}

cudaLaunchConfig_t backward_config(int grid, cudaStream_t stream, cudaLaunchAttribute* attr,
                                   bool with_pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kBackThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = with_pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

bool valid(const BackwardProduct& g, int units) {
  return units == 0 ||
         (g.splits >= 1 && g.slices >= g.splits && g.group_m >= 1 &&
          int64_t(g.tiles_m) * g.tiles_n * g.splits == units &&
          (g.splits == 1 || (g.part_rows >= g.rows && (g.part_rows % 32) == 0)));
}

bool valid_grad(const BackwardParams& p) {
  const int halves = p.in_units - p.full_units;
  return p.w_units == 0 && p.in.splits == 1 && p.full_units >= 0 && halves >= 0 && (halves % 2) == 0 &&
         valid(p.in, p.full_units + halves / 2);
}

template <bool kGrad, bool kScaled>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(backward_pair_kernel<kGrad, kScaled>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
}

}  // namespace

cudaError_t configure_backward_pair(int* max_pairs) {
  cudaError_t e = set_smem<true, false>();
  if (e == cudaSuccess) e = set_smem<false, false>();
  if (e == cudaSuccess) e = set_smem<false, true>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = backward_config(2, nullptr, attr, false);
  return cudaOccupancyMaxActiveClusters(max_pairs, backward_pair_kernel<true, false>, &cfg);
}

cudaError_t launch_backward_pair(const BackwardParams& p, bool grad, int pairs, cudaStream_t stream) {
  const int r = pairs > 0 ? p.in_units % pairs : 0;
  if (pairs < 1 || p.in_units + int64_t(p.w_units) < pairs || !valid(p.w, p.w_units) ||
      !(grad ? valid_grad(p) : valid(p.in, p.in_units)) || p.early_rounds < 0 ||
      int64_t(p.early_rounds) * (pairs - r) > p.w_units)
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = backward_config(2 * pairs, stream, attr, pdl_enabled());
  const cudaError_t e = grad             ? cudaLaunchKernelEx(&cfg, backward_pair_kernel<true, false>, p)
                        : p.in.row_scale ? cudaLaunchKernelEx(&cfg, backward_pair_kernel<false, true>, p)
                                         : cudaLaunchKernelEx(&cfg, backward_pair_kernel<false, false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_reduce_parts(const ReduceParams& p, cudaStream_t stream) {
  size_t items = 1;
  for (int o = 0; o < p.count; ++o) {
    const size_t n = static_cast<size_t>(p.out[o].rows) * (p.out[o].cols / 8);
    items = n > items ? n : items;
  }
  const size_t blocks = (items + 255) / 256;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 1216 ? blocks : 1216));  // 8 blocks per SM
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, reduce_parts_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
