// Large-M fused SwiGLU kernel on CTA pairs: Y = SiLU(A W1) * (A W2) for
// 256-token tiles computed by two SMs with tcgen05.mma.cta_group::2.
//
// Same method as fused_large_m.cu (one packed weight stream, gate and up
// columns side by side in one fp32 TMEM accumulator, SiLU * mul epilogue
// overlapped with the next tile's MMAs; "Tile-Level Activation Overlap for
// Efficient LLM Inference", gist.science, section "Methodology"), with the
// operand traffic of each SM cut by a third:
//
//  * a cluster of two CTAs owns a 256 x 128 output tile; CTA rank r loads A
//    rows [128 r, 128 r + 128) of the tile and packed-weight rows
//    [128 r, 128 r + 128) of the (column block, K slice) tile, i.e. rank 0
//    the 128 gate columns and rank 1 the 128 matching up columns;
//  * rank 0 issues one MMA of M=256, N=256, K=16 per step over both CTAs'
//    shared memory; each CTA's TMEM receives its 128 rows x (128 gate | 128 up)
//    columns, so each CTA's epilogue is the single-CTA one;
//  * per 64-deep K step each CTA pulls 32 KB (16 KB A + 16 KB W) instead of
//    48 KB, and the ring holds 6 stages;
//  * both CTAs' loads complete on rank 0's "full" barrier; rank 0's MMA
//    completions arrive on both CTAs' "empty" and "accumulator full"
//    barriers (multicast commit); both epilogues arrive on rank 0's
//    "accumulator empty" barrier; every wait is bounded (ptx.cuh).
//
// Tile rounds are kept loosely in step across the pairs: pair p takes tiles
// p, p + pairs, p + 2 pairs, ... (round 0, 1, 2, ...), and the tiles of one
// round share A rows and weight columns through L2 only while the pairs are
// near each other. Left alone, pairs drift apart by whole rounds over a long
// run (the 72B prefill read its operands 7-11 times over from DRAM), so the
// even CTA's producer, before the loads of its round r tile, waits until every
// pair has issued all loads of its round r - 2 tile (a per-round counter in
// global memory, tagged with a launch number the CTAs draw on the device, so
// graph replays count apart: every launch takes one block of kPaceBlock
// numbers from a global ticket, pair 0 all but pairs - 1 of them, so blocks
// stay aligned whatever the grid sizes of earlier launches). Every such wait
// is bounded and, if it runs out, only turns pacing off for the rest of the
// launch; results never depend on it. Paced are bf16 gate/up launches with
// K >= 8192 (long tiles; the 72B prefill): DRAM reads 11.0-13.4 -> 7.9-8.8 GB
// per launch at the same time (lag 1: much slower; lag 4: more reads).
// Shorter tiles lose time when paced, since the slowest pair of each round
// then sets everyone's pace. Consecutive rounds share their A rows (a row
// group's tiles run down the columns), so on the paced shapes odd rounds
// walk K backwards and start on the A slices the previous round loaded last,
// while L2 still holds them: the 72B prefill read 8.0 -> 6.3 GB and ran 2 %
// faster. Unpaced launches keep one direction: their pairs drift apart by
// whole rounds, so the tiles in flight would mix both directions (before the
// pacing, alternating directions raised the reads of both 72B forms).
//
// With kDown the same pipeline computes the MLP's down-projection
// Out = Y x W3 + R: a tile is 256 consecutive output columns (rank r loads
// packed rows [128 r, 128 r + 128) of W3's tile), and the epilogue stores
// accumulator + residual for all 256 columns.
//
// With kMx (block-scaled E4M3: one power-of-two scale per 32 K values) each
// CTA also loads, per stage, the scale block of its 128 A rows and both of the
// packed tile's weight-scale blocks (gate, up: the MMA's 256 B columns). A
// warp of the even CTA of its own copies them, as soon as a stage has landed,
// into that stage's slot of both CTAs' tensor memory (tcgen05.cp.cta_group::2,
// each CTA from its own shared memory) and signals their completion on a
// per-stage barrier; the MMA issuer waits for it and issues kind::mxf8f6f4
// MMAs, so the copies never sit in the MMA issuer's own stream of tensor
// instructions (copies issued there, just before the MMAs that read them,
// left the tensor pipe idle for a while at every stage; issuing them one stage
// early there was slower still). The scale slots take the second half of
// tensor memory, so the accumulator is single-buffered: the next tile's MMAs
// wait for the epilogue to have read the previous one. To keep that wait short the
// block-scaled form runs 8 epilogue warps (two per tensor-memory lane
// quarter, 64 output columns each) that load their whole share of the
// accumulator into registers, release it at once, and only then apply
// SiLU(g) * u and store, each through one store-staging buffer of its own
// (the wait on its previous store overlaps the next tile's MMAs).
//
// With kLora (bf16) each token also has a low-rank adapter a = index[m]: after
// a tile's K slices come, for every adapter present in its 256 tokens
// (lora_shrink.cu lists them and makes V), slices whose left operand is V with
// the rows of other adapters zero and whose right operand is Lb[a]: one with
// gate V (MMA N = 128, into the gate columns) and one with up V (up columns),
// or a single one over all 256 columns of the down-projection. Up to 64 ranks
// fill one 128-byte row, so an adapter costs a tile one or two short slices
// (rank / 16 MMAs each) of its K / 64, and Gate, Up and their deltas meet in
// the fp32 accumulator before SiLU. Lb comes by TMA into the stage's weight
// half; four warps write the masked V rows into its A half (thread = row) and
// signal a barrier of their own, which the MMA issuer waits for beside the
// stage's. (Alternating adapter and K slices instead: 660 against 640 us on the
// 7B shape, 4096 tokens of rank 64.) Measured there: 585 us against 541 without
// adapters; the adapter slices' MMAs are 2 % of the tensor pipe's work, the waits
// around them the rest. Non-finite entries of an Lb stay with the tokens of that
// adapter (lora_lb.cuh); each CTA's warps look through the rows that its own copy
// brought, so an Lb copy signals its own CTA, and those warps the even one. (They write
// the V of the next slice first: 631 us with the look as without it; 640 where they
// looked through each slice before the next V.)
#include "kernels.h"
#include "lora_lb.cuh"
#include "ptx.cuh"

namespace swg {
namespace {

template <bool kMx, bool kLora = false>
struct PairCfg {
  static constexpr int kBN = 128;                        // output columns per tile
  static constexpr int kABytes = 128 * kBlockK * 2;      // 16 KB: this CTA's 128 A rows
  static constexpr int kBBytes = 128 * kBlockK * 2;      // 16 KB: this CTA's 128 weight rows
  static constexpr int kStageBytes = kABytes + kBBytes;  // 32 KB per CTA, 64 KB per pair
  static constexpr int kStages = 6;
  static constexpr int kEpiWarps = kMx ? 8 : 4;          // 2 per lane quarter when block-scaled
  // TMA producer and MMA issuer warps, the epilogue warps, and (block-scaled)
  // a warp that copies each stage's scales into tensor memory, or (adapters)
  // four that write masked V rows
  static constexpr int kThreadsT = 64 + 32 * kEpiWarps + (kMx ? 32 : kLora ? 128 : 0);
  static constexpr int kAccCols = 2 * kBN;               // 256 fp32 columns: gate | up
  static constexpr int kTmemCols = 2 * kAccCols;         // double buffered (bf16, per-tensor FP8)
  static constexpr int kStgBytes = 32 * 32 * 2;          // 32 rows x 64 B store staging
  static constexpr int kNumStg = 8;                      // 2 per warp, or 1 per warp with 8 warps
  static constexpr int kTaints = 16;  // adapters: tile rounds that keep a mark
  static constexpr int kBarBytes = kLora ? 512 : 256;
  // block-scaled FP8: 1.5 KB of scales per stage (A block, gate and up weight blocks)
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes +
                                  size_t(kNumStg) * kStgBytes +
                                  (kMx ? size_t(kStages) * kSfStageBytes : 0) + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory budget");
  static constexpr int kBars = (kLora ? 5 : 3) * kStages + 6;
  static_assert(8 * kBars + 8 + (kLora ? 4 * kTaints : 0) <= kBarBytes, "barrier slots");
  static constexpr int kSfCol = kAccCols;  // scale slots after the single accumulator
  static_assert(!kMx || kSfCol + kStages * kSfTmemCols <= kTmemCols, "tensor memory budget");
};

__device__ __forceinline__ void pair_tile_coords(int t, int tiles_m, int tiles_n, int group_m,
                                                 int& mb, int& nb) {
  const int per_group = group_m * tiles_n;
  const int g = t / per_group;
  const int first_m = g * group_m;
  const int gm = min(tiles_m - first_m, group_m);
  const int r = t - g * per_group;
  mb = first_m + r % gm;
  nb = r / gm;
}

// Round pacing state (see the head of this file): the even CTA of every pair
// draws from g_pace_ticket, launch number = ticket / kPaceBlock + 1 (32 bits);
// g_pace_round[r] holds (launch number << 32) | pairs that issued all loads of
// their round r tile; g_pace_run_out counts waits that ran out (testing).
constexpr int kPaceLag = 2;
constexpr int kPaceRounds = 1024;               // rounds beyond this are not paced
constexpr uint64_t kPaceWaitNs = 200000;        // one wait's limit: then pacing stops
constexpr int kPaceMinSlices = 128;             // paced only with K >= 128 slices of 64
constexpr unsigned long long kPaceBlock = 1024;  // tickets per launch (>= pairs)
__device__ unsigned long long g_pace_ticket;
__device__ unsigned long long g_pace_round[kPaceRounds];
__device__ unsigned long long g_pace_run_out;

// Waits (bounded) until `need` pairs of launch `epoch` counted themselves in
// round r; false if the wait ran out or a later launch owns the counter.
__device__ __forceinline__ bool pace_wait(int r, unsigned long long epoch, unsigned need) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    const unsigned long long v = *reinterpret_cast<volatile unsigned long long*>(&g_pace_round[r]);
    if ((v >> 32) == epoch && static_cast<unsigned>(v & 0xffffffffull) >= need) return true;
    if ((v >> 32) > epoch) return false;
    if (globaltimer_ns() - t0 > kPaceWaitNs) {
      atomicAdd(&g_pace_run_out, 1ull);
      return false;
    }
  }
}

// Counts this pair in for round r of launch `epoch` (a counter left by
// another launch restarts at 1).
__device__ __forceinline__ void pace_count(int r, unsigned long long epoch) {
  unsigned long long* c = &g_pace_round[r];
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(c), assumed;
  do {
    assumed = old;
    const unsigned long long next = (assumed >> 32) == epoch ? assumed + 1ull : (epoch << 32) | 1ull;
    old = atomicCAS(c, assumed, next);
  } while (old != assumed);
}

template <bool kFp8, bool kDown, bool kMx, bool kLora>
__global__ void __launch_bounds__(PairCfg<kMx, kLora>::kThreadsT, 1)
    fused_large_m_pair_kernel(const __grid_constant__ LargeMParams p) {
  using C = PairCfg<kMx, kLora>;
  static_assert(!kLora || !kFp8, "adapters go with bf16");
  static_assert(!kMx || (kFp8 && !kDown), "block scales go with E4M3 gate/up inputs");
  constexpr int kAccBufs = kMx ? 1 : 2;  // accumulator buffers in tensor memory
  // K values per stage: 64 bf16 or 128 E4M3, a 128-byte row either way
  constexpr int kBK = kFp8 ? kBlockK8 : kBlockK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_addr(smem);
  const uint32_t sB = sA + C::kStages * C::kABytes;
  const uint32_t sStg = sB + C::kStages * C::kBBytes;
  const uint32_t sSf = sStg + C::kNumStg * C::kStgBytes;  // scales (kMx): kStages x 1.5 KB
  uint8_t* bar_ptr = smem + size_t(C::kStages) * C::kStageBytes + C::kNumStg * C::kStgBytes +
                     (kMx ? size_t(C::kStages) * kSfStageBytes : 0);
  const uint32_t bar0 = smem_addr(bar_ptr);
  // barrier slots: full[S] | empty[S] | tmem_full[2] | tmem_empty[2] | drain |
  // scales_ready[S] (adapters: V rows ready) | scale-copy drain | adapters: V slot free[S] |
  // this CTA's Lb rows landed[S]
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * C::kStages;
  const uint32_t tfull0 = bar0 + 16u * C::kStages, tempty0 = tfull0 + 16u;
  const uint32_t drain_bar = tempty0 + 16u;
  const uint32_t sready0 = drain_bar + 8u, sdrain_bar = sready0 + 8u * C::kStages;
  const uint32_t vfree0 = sdrain_bar + 8u, lbfull0 = vfree0 + 8u * C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [round % kTaints] = round + 1: some Lb row of that round's tile was not finite.
  // (The V warps are at most two accumulators and six stages ahead of the epilogue.)
  volatile int* taint = abort_flag + 1;
  static_assert(C::kTaints > 2 + C::kStages, "marks outlive the rounds in flight");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());
  const int pairs = static_cast<int>(cluster_count_x());
  const int num_tiles = p.tiles_m * p.tiles_n;
  const int num_kb = (p.K + kBK - 1) / kBK;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  constexpr int kHalves = kDown ? 1 : 2;  // adapter slices: gate and up, or one
  const auto lora_slices = [&](int t) {
    int mb, nb;
    pair_tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, mb, nb);
    return p.lora_lists[static_cast<size_t>(mb) * kLoraListInts] * kHalves;
  };
  // rank 0's full and tmem_empty barriers, as seen from either CTA of the pair
  const uint32_t full0_lead = mapa_shared(full0, 0);
  const uint32_t tempty0_lead = mapa_shared(tempty0, 0);

  if (threadIdx.x == 0) {
    prefetch_tmap(&p.tmap_a);
    prefetch_tmap(&p.tmap_w);
    prefetch_tmap(&p.tmap_y);
    if constexpr (kMx) {
      prefetch_tmap(&p.tmap_sw);
      prefetch_tmap(&p.tmap_sa);
    }
    if constexpr (kLora) prefetch_tmap(&p.tmap_lb);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8u * s, 1);   // rank 0's producer arrives (with both CTAs' bytes)
      mbar_init(empty0 + 8u * s, 1);  // rank 0's MMA commit, multicast to both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);   // multicast MMA commit
      mbar_init(tempty0 + 8u * b, 2 * C::kEpiWarps);  // epilogue warps x 2 CTAs (used on rank 0)
    }
    mbar_init(drain_bar, 1);
    // scale-copy commit, or (adapters) 4 warps x 2 CTAs (used on rank 0)
    for (int s = 0; s < C::kStages; ++s) mbar_init(sready0 + 8u * s, kLora ? 8 : 1);
    mbar_init(sdrain_bar, 1);
    if constexpr (kLora) {
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(vfree0 + 8u * s, 1);  // this CTA's producer
        mbar_init(lbfull0 + 8u * s, 1);
      }
      for (int i = 0; i < C::kTaints; ++i) taint[i] = 0;
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  // With adapters the kernel before this one makes V and the lists, and lets this grid
  // start when it has itself waited for all before it: the first K slices (by TMA, from
  // L2) need no wait, what reads V and lists or writes outputs has its own.
  if (!kLora || !p.lora_early) pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    // (the whole warp waits and counts, one lane issues, as below)
    {
      const bool one = elect_one();
      if (kLora) fence_proxy_async();
      int s = 0;
      uint32_t ph = 0;
      uint32_t filled = 0, fill_ph = 0;
      uint32_t lb_filled = 0, lb_ph = 0;  // adapters: phase of each stage's Lb barrier
      bool skip_once = p.inject_stall != 0;
      bool ok = true;
      // round pacing on the even CTA (the odd one follows through the empty
      // barriers); the launch number is drawn when the previous launch of this
      // kernel in the stream has finished: after the grid-dependency wait, or (adapters
      // with lora_early) because the kernel that makes V had its wait behind it when it
      // let this one start. The launch's draws add up to kPaceBlock, so the next
      // launch starts a fresh block.
      const bool can_pace = pairs <= static_cast<int>(kPaceBlock);
      unsigned long long epoch = 0;  // of the issuing lane
      if (leader && can_pace && one) {
        const unsigned long long take = pair == 0 ? kPaceBlock - static_cast<unsigned long long>(pairs - 1) : 1ull;
        epoch = ((atomicAdd(&g_pace_ticket, take) / kPaceBlock) + 1ull) & 0xffffffffull;
      }
      // only long bf16 gate/up tiles (K >= 8192, the 72B shape): with shorter
      // tiles the slowest pair of each round sets everyone's pace (7B prefill
      // +30 %, FP8 72B +13 %, block-scaled 7B +73 % when paced)
      const bool long_tiles = !kFp8 && !kDown && num_kb >= kPaceMinSlices;  // same in both CTAs
      const bool paced = leader && can_pace && long_tiles;
      bool pacing = paced;  // off for the rest of the launch once a wait runs out
      int round = 0;
      for (int t = pair; ok && t < num_tiles; t += pairs, ++round) {
        if (pacing && round >= kPaceLag && round - kPaceLag < kPaceRounds) {
          const int r = round - kPaceLag;
          const bool in_time =
              !one || pace_wait(r, epoch, static_cast<unsigned>(min(pairs, num_tiles - r * pairs)));
          pacing = __all_sync(0xffffffffu, in_time);
        }
        int mb, nb;
        pair_tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, mb, nb);
        const int m0 = mb * 2 * kTileM + static_cast<int>(rank) * kTileM;
        const int wtile = nb * num_kb;                        // (column block nb, K slice 0)
        const int wrow = static_cast<int>(rank) * kPackBlockN;  // gate rows (0) / up rows (1)
        // adapters present in this tile, read well before they are needed (but in the first)
        const int* list = nullptr;
        int extra = 0;
        if constexpr (kLora) {
          list = p.lora_lists + static_cast<size_t>(mb) * kLoraListInts;
          if (round > 0) extra = list[0] * kHalves;
        }
        // paced shapes: odd rounds walk K backwards and start on the A slices
        // the previous round (same row tiles) read last, while L2 holds them
        const bool backwards = long_tiles && (round & 1) != 0;
        for (int i = 0; i < num_kb; ++i) {
          const int kb = backwards ? num_kb - 1 - i : i;
          if (!mbar_wait_warp(empty0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          if (skip_once) {
            skip_once = false;  // testing hook: both CTAs leave this stage unfilled
          } else {
            if (one) {
              if (leader)
                mbar_arrive_expect_tx(full0 + 8u * s, 2 * (C::kStageBytes + (kMx ? kSfStageBytes : 0)));
              const uint32_t fb = full0_lead + 8u * s;
              tma_load_2d_pair(sA + s * C::kABytes, &p.tmap_a, fb, kb * kBK, m0);
              tma_load_3d_pair(sB + s * C::kBBytes, &p.tmap_w, fb, 0, wrow, wtile + kb);
              if constexpr (kMx) {
                // this CTA's A rows: block (m0 / 128, kb), 2 rows of 256 bytes; both
                // weight-scale blocks of the tile (gate, up), 4 rows
                const uint32_t sf = sSf + s * kSfStageBytes;
                tma_load_2d_pair(sf, &p.tmap_sa, fb, 0, 2 * ((m0 / kTileM) * num_kb + kb));
                tma_load_2d_pair(sf + kSfBlockBytes, &p.tmap_sw, fb, 0, 4 * (wtile + kb));
              }
            }
            filled |= 1u << s;
            fill_ph = (fill_ph & ~(1u << s)) | (ph << s);
          }
          __syncwarp();
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if constexpr (kLora) {
          if (round == 0) {
            pdl_wait();
            extra = list[0] * kHalves;
          }
          // Lb rows of every adapter present in this tile, to the weight half
          for (int i = 0; ok && i < extra; ++i) {
            if (!mbar_wait_warp(empty0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
              ok = false;
              break;
            }
            if (one) {
              mbar_arrive(vfree0 + 8u * s);  // the stage's A half is free for V rows
              // this CTA's half of the MMA's N rows: 64 gate (up) columns, or 128 output columns
              if (leader) mbar_arrive(full0 + 8u * s);  // nothing to wait for: the V warps do
              mbar_arrive_expect_tx(lbfull0 + 8u * s, C::kBBytes / kHalves);
              const int a = list[1 + i / kHalves];
              const int n0 = kDown ? nb * 2 * C::kBN + static_cast<int>(rank) * C::kBN
                                   : nb * C::kBN + static_cast<int>(rank) * (C::kBN / 2);
              tma_load_3d(sB + s * C::kBBytes, &p.tmap_lb, lbfull0 + 8u * s, 0, n0,
                          a * kHalves + i % kHalves);
            }
            __syncwarp();
            filled |= 1u << s;
            fill_ph = (fill_ph & ~(1u << s)) | (ph << s);
            lb_filled |= 1u << s;
            lb_ph ^= 1u << s;
            if (++s == C::kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        if (paced && ok && one && round < kPaceRounds) pace_count(round, epoch);
      }
      if (one) pdl_launch_dependents();
      // Rank 0's full barriers count both CTAs' bytes: once they complete, every
      // copy issued by the pair for those stages has landed.
      if (leader && one)
        for (int i = 0; i < C::kStages; ++i)
          if (filled & (1u << i)) mbar_wait_drain(full0 + 8u * i, (fill_ph >> i) & 1u, wc);
      for (int i = 0; kLora && one && i < C::kStages; ++i)  // lb_ph has been flipped past the last use
        if (lb_filled & (1u << i)) mbar_wait_drain(lbfull0 + 8u * i, ((lb_ph >> i) & 1u) ^ 1u, wc);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (rank 0)
    // The whole warp waits and counts, one lane issues: with one lane in the loop from the
    // start the descriptors are not warp-uniform to the compiler, and the issue itself held
    // the tensor pipe up. In this role, the producer's and the scale copies', at 7B prefill
    // 566 -> 548 us, E4M3 313 -> 294, block-scaled 375 -> 325; 72B, at the power cap,
    // 4.37 -> 4.24 ms, E4M3 2.10 -> 2.03, block-scaled 2.40 -> 2.13; 4096 tokens of rank 64
    // 640 -> 596 us.
    if (leader) {
      const bool one = elect_one();
      constexpr uint32_t kIdesc = kFp8 ? idesc_e4m3_f32(2 * kTileM, 2 * C::kBN)
                                       : idesc_bf16_f32(2 * kTileM, 2 * C::kBN);
      constexpr uint32_t kIdescMx = idesc_mx_e4m3(2 * kTileM, 2 * C::kBN, 0);
      int s = 0;
      uint32_t ph = 0;
      int buf = 0;
      uint32_t acc_ph = 0;
      uint32_t vph = 0;  // adapters: phase of each stage's V barrier
      int next_extra = -1;  // adapter slices of the next tile; the first one's are read late
      bool ok = true;
      for (int t = pair; ok && t < num_tiles; t += pairs) {
        // adapter slices of this tile; the next tile's count is on its way
        int extra = kLora ? next_extra : 0;
        if (kLora && extra >= 0) next_extra = t + pairs < num_tiles ? lora_slices(t + pairs) : 0;
        if (!mbar_wait_warp(tempty0 + 8u * buf, acc_ph ^ 1u, wc, kSiteMmaTmemEmpty)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * C::kAccCols;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          // block-scaled: the scale-copy warp has put this stage's scales in
          // its tensor-memory slot
          if (kMx && !mbar_wait_warp(sready0 + 8u * s, ph, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = smem_desc_sw128(sA + s * C::kABytes);
          const uint64_t bdesc = smem_desc_sw128(sB + s * C::kBBytes);
          // scale slot of this stage: A rows [0, 4), B columns 0..127 [4, 8), 128..255 [8, 12)
          const uint32_t tsf = tmem_base + C::kSfCol + uint32_t(s) * kSfTmemCols;
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // four 32-byte K steps per 128-byte row
              if constexpr (kMx)  // K step k consumes scale group k of the slice (IDs at bits 4, 29)
                mma_mx_pair(d, adesc + 2u * k, bdesc + 2u * k,
                            kIdescMx | (uint32_t(k) << 4) | (uint32_t(k) << 29), tsf, tsf + 4,
                            (kb | k) != 0 ? 1u : 0u);
              else if constexpr (kFp8)
                mma_e4m3_pair(d, adesc + 2u * k, bdesc + 2u * k, kIdesc, (kb | k) != 0 ? 1u : 0u);
              else
                mma_bf16_pair(d, adesc + 2u * k, bdesc + 2u * k, kIdesc, (kb | k) != 0 ? 1u : 0u);
            }
            mma_commit_pair_multicast(empty0 + 8u * s, 0x3);  // frees the stage in both CTAs
          }
          __syncwarp();
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if constexpr (kLora) {
          if (extra < 0) {
            pdl_wait();
            extra = lora_slices(t);
            next_extra = t + pairs < num_tiles ? lora_slices(t + pairs) : 0;
          }
          constexpr uint32_t kIdescV = idesc_bf16_f32(2 * kTileM, 2 * C::kBN / kHalves);
          const int ksteps = (p.lora_rank + 15) / 16;
          for (int i = 0; ok && i < extra; ++i) {
            if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteMmaFull) ||
                !mbar_wait_warp(sready0 + 8u * s, (vph >> s) & 1u, wc, kSiteLora)) {
              ok = false;
              break;
            }
            vph ^= 1u << s;
            tc_fence_after();
            const uint64_t vdesc = smem_desc_sw128(sA + s * C::kABytes);
            const uint64_t bdesc = smem_desc_sw128(sB + s * C::kBBytes);
            const uint32_t dv = d + (i % kHalves) * C::kBN;
            if (one) {
              for (int k = 0; k < ksteps; ++k)
                mma_bf16_pair(dv, vdesc + 2u * k, bdesc + 2u * k, kIdescV, 1u);
              mma_commit_pair_multicast(empty0 + 8u * s, 0x3);
            }
            __syncwarp();
            if (++s == C::kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        if (!ok) break;
        if (one) mma_commit_pair_multicast(tfull0 + 8u * buf, 0x3);  // both halves of the accumulator ready
        if (++buf == kAccBufs) {
          buf = 0;
          acc_ph ^= 1u;
        }
      }
      if (one) {
        mma_commit_pair_multicast(drain_bar, 0x1);
        mbar_wait_drain(drain_bar, 0, wc);
      }
    }
    __syncwarp();
  } else if (kMx && warp == 2 + C::kEpiWarps) {
    // ------------------------------------------------ scale copies (rank 0)
    // Each stage's scales go from shared to tensor memory (both CTAs, each
    // from its own shared memory) as soon as the stage has landed, in a
    // stream of tcgen05 operations of their own, and the MMA issuer waits
    // for their completion. A slot is refilled only after its stage was
    // refilled, i.e. after the MMAs that read its previous contents completed.
    if (leader) {
      const bool one = elect_one();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = pair; ok && t < num_tiles; t += pairs) {
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteScaleCopy)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tsf = tmem_base + C::kSfCol + uint32_t(s) * kSfTmemCols;
          const uint32_t sf = sSf + s * kSfStageBytes;
          if (one) {
            tmem_cp_sf_pair(tsf, smem_desc_sf(sf));
            tmem_cp_sf_pair(tsf + 4, smem_desc_sf(sf + kSfBlockBytes));
            tmem_cp_sf_pair(tsf + 8, smem_desc_sf(sf + 2 * kSfBlockBytes));
            mma_commit_pair_multicast(sready0 + 8u * s, 0x1);
          }
          __syncwarp();
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (one) {
        mma_commit_pair_multicast(sdrain_bar, 0x1);
        mbar_wait_drain(sdrain_bar, 0, wc);
      }
    }
    __syncwarp();
  } else if (kLora && warp >= 2 + C::kEpiWarps) {
    // ------------------------------------------------ masked V rows (both CTAs)
    // Thread = row of this CTA's 128; the row's own adapter's slices get its V,
    // every other slice zeros, in the swizzled layout a TMA load would write.
    pdl_wait();
    const int row = threadIdx.x - (64 + 32 * C::kEpiWarps);
    const uint32_t sready0_lead = mapa_shared(sready0, 0);
    const int chunks = p.lora_rank / 8, padded = (p.lora_rank + 15) / 16 * 2;
    // this thread's Lb row of a slice: all of one of 128, or half of one of 64
    const int lb_row = kDown ? row : row & 63, lb_begin = kDown ? 0 : row >> 6 << 2;
    const int lb_end = kDown ? chunks : min(chunks, lb_begin + 4);
    int s = 0;        // stage, in step with the producer
    uint32_t vph = 0, ph = 0;  // phases of each stage's V-slot-free and Lb barriers
    int round = 0;
    bool ok = true;
    for (int t = pair; ok && t < num_tiles; t += pairs, ++round) {
      int mb, nb;
      pair_tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, mb, nb);
      const int* list = p.lora_lists + static_cast<size_t>(mb) * kLoraListInts;
      const int extra = list[0] * kHalves;
      const int64_t m = int64_t(mb) * 2 * kTileM + static_cast<int>(rank) * kTileM + row;
      const int own = m < p.M ? p.lora_index[m] : -1;
      const uint4* v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.lora_v) +
                                                      static_cast<size_t>(m) * p.lora_rank * kHalves);
      // the row's V and the first adapters of the list, loaded while the tile's K
      // slices go by (loaded per slice, their latency left the tensor pipe idle at
      // every adapter slice: 679 against 668 us on the 7B shape, 4096 tokens, rank 64)
      constexpr int kChunks = kLoraMaxRank / 8;
      uint4 x[kHalves][kChunks];
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          x[h][c] = own >= 0 && own < p.lora_count && c < chunks ? v[h * chunks + c]
                                                                 : make_uint4(0u, 0u, 0u, 0u);
      const int ahead = list[1 + min(lane, max(extra / kHalves - 1, 0))];
      s = (s + num_kb) % C::kStages;
      // V of slice i is written before the Lb rows of slice i - 1 are looked through: the
      // stage after this one is free by then (more than two stages)
      for (int i = 0; i <= extra; ++i) {
        if (i < extra) {
          const int at = i / kHalves, sv = (s + min(i, 1)) % C::kStages;
          const int a = at < 32 ? __shfl_sync(0xffffffffu, ahead, at) : list[1 + at];
          ok = __all_sync(0xffffffffu, mbar_wait(vfree0 + 8u * sv, (vph >> sv) & 1u, wc, kSiteLora));
          if (!ok) break;
          vph ^= 1u << sv;
          const uint32_t dst = sA + sv * C::kABytes + row * 128;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < padded) {
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (a == own) w = kHalves == 2 && (i & 1) ? x[kHalves - 1][c] : x[0][c];
              st_shared_v4(dst + ((c ^ (row & 7)) << 4), w.x, w.y, w.z, w.w);
            }
          fence_proxy_async_smem();
        }
        if (i == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(lbfull0 + 8u * s, (ph >> s) & 1u, wc, kSiteLora));
        if (!ok) break;
        ph ^= 1u << s;
        if (clean_lb_row<kDown ? kChunks : kChunks / 2>(sB + s * C::kBBytes, lb_row, lb_begin, lb_end)) {
          // both CTAs' epilogues read columns made from this row
          const uint32_t mark = smem_addr(const_cast<int*>(taint)) + 4u * (round % C::kTaints);
          st_shared_cluster(mapa_shared(mark, 0), round + 1);
          st_shared_cluster(mapa_shared(mark, 1), round + 1);
          fence_proxy_async_smem();
          __threadfence();
        }
        __syncwarp();
        // Every writer has made its rows visible to the tensor core's reads of this
        // CTA's own shared memory; the arrival only lets the even CTA issue the MMA.
        // (Releasing at cluster scope here took 1250 cycles a slice.)
        if (lane == 0) mbar_arrive_remote(sready0_lead + 8u * s);
        if (++s == C::kStages) s = 0;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const int ew = warp - 2;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const float sg = kFp8 ? p.scale_gate : 1.0f, su = kFp8 ? p.scale_up : 1.0f;
    if (kLora) pdl_wait();
    int buf = 0;
    uint32_t acc_ph = 0;
    int sbuf = 0;
    int round = 0;
    for (int t = pair; t < num_tiles; t += pairs, ++round) {
      int mb, nb;
      pair_tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, mb, nb);
      const int row0 = mb * 2 * kTileM + static_cast<int>(rank) * kTileM + q * 32;
      const int col0 = nb * (kDown ? 2 * C::kBN : C::kBN);
      int ok = 1;
      if (lane == 0) ok = mbar_wait(tfull0 + 8u * buf, acc_ph, wc, kSiteEpiTmemFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_off + buf * C::kAccCols;
      // adapters: what this row's own Lb lost (lora_lb.cuh), in a marked tile
      int own = -1;
      if (kLora && taint[round % C::kTaints] == round + 1 && row0 + lane < p.M)
        own = p.lora_index[row0 + lane];
      const bool restore = own >= 0 && own < p.lora_count;
      const size_t own_lb = static_cast<size_t>(own) * kHalves * p.N;
      const size_t own_v = (static_cast<size_t>(row0) + lane) * kHalves;
      if constexpr (kMx) {
        // this warp's 64 output columns [64 h, 64 h + 64): gate and up, all loaded
        // before the accumulator is released to the next tile's MMAs
        const int h = ew >> 2;
        uint32_t g0[32], g1[32], u0[32], u1[32];
        tmem_ld_x32(tacc + 64 * h, g0);
        tmem_ld_x32(tacc + 64 * h + 32, g1);
        tmem_ld_x32(tacc + C::kBN + 64 * h, u0);
        tmem_ld_x32(tacc + C::kBN + 64 * h + 32, u1);
        tmem_wait_ld();
        reg_fence(g0);
        reg_fence(g1);
        reg_fence(u0);
        reg_fence(u1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0_lead + 8u * buf);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t* g = c ? g1 : g0;
          const uint32_t* u = c ? u1 : u0;
          if (lane == 0) bulk_wait_read<0>();  // this warp's one staging buffer is free again
          __syncwarp();
          const uint32_t stg = sStg + ew * C::kStgBytes;
          const uint32_t row_addr = stg + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i0 = 8 * j + 2 * e;
              w[e] = pack_bf16x2(silu_mul(__uint_as_float(g[i0]), __uint_as_float(u[i0])),
                                 silu_mul(__uint_as_float(g[i0 + 1]), __uint_as_float(u[i0 + 1])));
            }
            st_shared_v4(row_addr + ((j ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int ncol = col0 + 64 * h + 32 * c;
            if (ncol < p.N && row0 < p.M) tma_store_2d(&p.tmap_y, stg, ncol, row0);
            bulk_commit();
          }
        }
      } else if constexpr (kDown) {
        // 256 output columns: accumulator + residual, 32 columns per store
        const __nv_bfloat16* res = reinterpret_cast<const __nv_bfloat16*>(p.residual);
        const int row = row0 + lane;
#pragma unroll 1
        for (int c = 0; c < C::kAccCols / 32; ++c) {
          uint32_t a[32];
          tmem_ld_x32(tacc + c * 32, a);
          tmem_wait_ld();
          reg_fence(a);
          if (c == C::kAccCols / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0_lead + 8u * buf);
          }
          const int ncol = col0 + c * 32;
          if (kLora && restore) {
#pragma unroll 1
            for (int j = 0; j < 32 && ncol + j < p.N; ++j) {
              const float d = nonfinite_delta(p.lora_lb, own_lb + ncol + j, p.lora_v, own_v, p.lora_rank);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e == j) a[e] = __float_as_uint(__uint_as_float(a[e]) + d);
            }
          }
          float add[32];
#pragma unroll
          for (int gq = 0; gq < 4; ++gq) {  // 8 columns (16 bytes) at a time; N % 8 == 0
            const int col = ncol + gq * 8;
            uint4 rv = make_uint4(0u, 0u, 0u, 0u);
            if (res && row < p.M && col < p.N)
              rv = *reinterpret_cast<const uint4*>(res + static_cast<size_t>(row) * p.N + col);
            const uint32_t w4[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w4[e]);
              add[gq * 8 + 2 * e] = __low2float(h);
              add[gq * 8 + 2 * e + 1] = __high2float(h);
            }
          }
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          const uint32_t stg = sStg + (ew * 2 + sbuf) * C::kStgBytes;
          const uint32_t row_addr = stg + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i0 = 8 * j + 2 * e;
              w[e] = pack_bf16x2(__uint_as_float(a[i0]) + add[i0],
                                 __uint_as_float(a[i0 + 1]) + add[i0 + 1]);
            }
            st_shared_v4(row_addr + ((j ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (ncol < p.N && row0 < p.M) tma_store_2d(&p.tmap_y, stg, ncol, row0);
            bulk_commit();
          }
          sbuf ^= 1;
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < C::kBN / 32; ++c) {
          uint32_t g[32], u[32];
          tmem_ld_x32(tacc + c * 32, g);
          tmem_ld_x32(tacc + C::kBN + c * 32, u);
          tmem_wait_ld();
          reg_fence(g);
          reg_fence(u);
          if (c == C::kBN / 32 - 1) {  // this CTA's half of the accumulator is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0_lead + 8u * buf);
          }
          if (kLora && restore) {
            const int ncol = col0 + c * 32;
#pragma unroll 1
            for (int j = 0; j < 32 && ncol + j < p.N; ++j) {
              const size_t lb_row = own_lb + ncol + j;
              const float dg = nonfinite_delta(p.lora_lb, lb_row, p.lora_v, own_v, p.lora_rank);
              const float du = nonfinite_delta(p.lora_lb, lb_row + p.N, p.lora_v, own_v + 1, p.lora_rank);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e == j) {
                  g[e] = __float_as_uint(__uint_as_float(g[e]) + dg);
                  u[e] = __float_as_uint(__uint_as_float(u[e]) + du);
                }
            }
          }
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          const uint32_t stg = sStg + (ew * 2 + sbuf) * C::kStgBytes;
          const uint32_t row_addr = stg + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i0 = 8 * j + 2 * e;
              w[e] = pack_bf16x2(
                  silu_mul(sg * __uint_as_float(g[i0]), su * __uint_as_float(u[i0])),
                  silu_mul(sg * __uint_as_float(g[i0 + 1]), su * __uint_as_float(u[i0 + 1])));
            }
            st_shared_v4(row_addr + ((j ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int ncol = col0 + c * 32;
            if (ncol < p.N && row0 < p.M) tma_store_2d(&p.tmap_y, stg, ncol, row0);
            bulk_commit();
          }
          sbuf ^= 1;
        }
      }
      if (++buf == kAccBufs) {
        buf = 0;
        acc_ph ^= 1u;
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  // Neither CTA leaves while the pair's MMAs may still read its shared memory
  // or the peer may still arrive on its barriers.
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::kTmemCols);
  }
}

cudaLaunchConfig_t pair_config(int grid, cudaStream_t stream, cudaLaunchAttribute* attr,
                               bool with_pdl, bool mx = false, bool lora = false) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(mx     ? PairCfg<true>::kThreadsT
                      : lora ? PairCfg<false, true>::kThreadsT
                             : PairCfg<false>::kThreadsT);
  cfg.dynamicSmemBytes = mx     ? PairCfg<true>::kSmem
                         : lora ? PairCfg<false, true>::kSmem
                                : PairCfg<false>::kSmem;
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

}  // namespace

cudaError_t configure_large_m_pair(int* max_pairs) {
  cudaError_t e = cudaFuncSetAttribute(fused_large_m_pair_kernel<false, false, false, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(PairCfg<false>::kSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fused_large_m_pair_kernel<true, false, false, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(PairCfg<false>::kSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fused_large_m_pair_kernel<false, true, false, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(PairCfg<false>::kSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fused_large_m_pair_kernel<true, false, true, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(PairCfg<true>::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config(2, nullptr, attr, false);
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, fused_large_m_pair_kernel<false, false, false, false>, &cfg);
  if (e != cudaSuccess) return e;
  *max_pairs = clusters;
  return cudaSuccess;
}

cudaError_t configure_large_m_pair_lora() {
  const cudaError_t e = cudaFuncSetAttribute(fused_large_m_pair_kernel<false, false, false, true>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(PairCfg<false, true>::kSmem));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(fused_large_m_pair_kernel<false, true, false, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(PairCfg<false, true>::kSmem));
}

size_t large_m_pair_smem_bytes() { return PairCfg<false>::kSmem; }
int large_m_pair_stages(bool mx) { return mx ? PairCfg<true>::kStages : PairCfg<false>::kStages; }

cudaError_t large_m_pair_pace_run_out(unsigned long long* count) {
  return cudaMemcpyFromSymbol(count, g_pace_run_out, sizeof(*count));
}

cudaError_t launch_large_m_pair(const LargeMParams& p, cudaStream_t stream) {
  if (p.grid < 2 || (p.grid % 2) != 0 || p.bn != PairCfg<false>::kBN) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config(p.grid, stream, attr, pdl_enabled(), p.mx != 0, p.lora != 0);
  if (p.fp8 && p.down) return cudaErrorInvalidValue;  // no FP8 down-projection
  if (p.mx && !p.fp8) return cudaErrorInvalidValue;   // block scales go with E4M3 values
  if (p.lora && (p.fp8 || p.lora_rank < 8 || p.lora_rank > kLoraMaxRank || (p.lora_rank % 8) != 0 ||
                 !p.lora_v || !p.lora_index || !p.lora_lists))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      p.lora && p.down ? cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<false, true, false, true>, p)
      : p.lora ? cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<false, false, false, true>, p)
      : p.down  ? cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<false, true, false, false>, p)
      : p.mx  ? cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<true, false, true, false>, p)
      : p.fp8 ? cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<true, false, false, false>, p)
              : cudaLaunchKernelEx(&cfg, fused_large_m_pair_kernel<false, false, false, false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
