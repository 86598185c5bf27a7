// The gated MLP's projections in 8-bit integers: codes A8 [M, K] with a scale per
// token, weight codes with a scale per output column,
//   G = (A8 W1_8) sa[m] s1[n],  U = (A8 W2_8) sa[m] s2[n],  Y = SiLU(G) U
//   Out = (Y8 W3_8) sy[m] s3[n] + R                               (kDown)
//
// The tensor cores of sm_103a have no 8-bit integer kind (ptxas refuses
// tcgen05.mma kind::i8 for it), so the products run in kind::f16: every code is an
// fp16 exactly, a product of two is an integer below 2^14, and the fp32 sums are
// exact while below 2^24. What 8 bits save is memory and its traffic: the weights
// stay 8 bits in HBM, L2 and shared memory, and become fp16 on the way into tensor
// memory, which holds the MMA's left operand. So the weight rows are the MMA's M
// side (128 lanes of tensor memory a CTA) and the tokens its N side, for one token
// as for many. Packed rows alternate 16 gate and the 16 matching up columns, so
// that a warp of the epilogue has both (32 lanes) and exchanges them by shuffles.
//
//   warp 0      TMA producer: per stage 128 of K: 128 weight rows of 128 codes, and
//               the tokens' codes (or fp16 values)
//   warp 1      MMA issuer
//   warps 2-9   thread = weight row: 64 codes from shared memory (16-byte pieces of
//               a 128-byte swizzled row, free of bank conflicts), each byte b = q + 128
//               set into the fp16 1024 + b and 1152 taken away (2 instructions for 2
//               codes), then one tcgen05.st of 32 columns; four warps do the first 64 of K
//               of a stage, four the rest (16 warps in two sets: slower, the polls of more
//               waiting warps cost more than the work: 7B, 16 tokens 24.7 -> 27.5 us).
//               A slot of tensor memory holds a stage; a ring of them runs ahead of the MMAs.
//   warps 10-17 epilogue, under the next unit's MMAs (two accumulators)
//
// Few tokens (kPair false): a unit is 128 weight rows and up to 64 tokens on one CTA. The epilogue's
// warps first turn the tokens' codes of every stage into fp16 in shared memory (the
// MMA's right operand), so that one token needs no kernel but this. With few units for the SMs,
// K is split over a cluster of `splits` CTAs whose fp32 partial sums meet in shared
// memory (summed in rank order, so results do not depend on timing).
// More tokens (kPair): a unit is 256 weight rows and up to 192 tokens on a CTA pair
// (cta_group::2: each CTA holds 128 weight rows in its tensor memory and half of the
// tokens in its shared memory); a kernel before this one turns the tokens' codes into
// fp16 once for all column blocks, which leaves the epilogue to run under the next unit's
// MMAs (widened by the epilogue's warps here too: 333 tokens, K 1424, N 5000 19.5 us, so 15.6).
#include <cuda_fp16.h>

#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kConvWarps = 8, kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (2 + kConvWarps + kEpiWarps8);
constexpr int kMaxStages8 = 10;
constexpr int kMaxSplits8 = 8;
constexpr int kTmem8 = 512;
constexpr int kBarBytes8 = 768;
constexpr size_t kSmemLimit8 = 232448;
constexpr int kSubK = 64;    // K values of a 128-byte row of fp16
constexpr int kRows8 = 128;  // packed weight rows of a CTA's unit

// Four codes, biased to bytes 0..255, as two words of fp16 pairs: byte b under 0x64 is 1024 + b.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  lo = __byte_perm(w, 0x64646464u, 0x4140);
  hi = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), bias);
  const __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), bias);
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread: A in 128 lanes, two consecutive
// fp16 values of K a 32-bit column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// kind::f16, D fp32, A and B fp16 (formats 0), both K-major.
__device__ __forceinline__ uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// `bytes` (a multiple of 16) of consecutive global memory to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

struct Unit {
  int block, group;
};

// Units in groups of `group_m` token groups: a group's tokens go by before the next columns.
__device__ __forceinline__ Unit unit_of(const Int8Params& p, int u) {
  const int per = p.group_m * p.blocks;
  const int g = u / per, first = g * p.group_m;
  const int gm = min(p.mgroups - first, p.group_m);
  const int r = u - g * per;
  return Unit{r / gm, first + r % gm};
}

// Four columns of one token from the fp32 sums of the 128 rows of weight block `ub`: item i of 32
// (down-projection), or of 16 (gate and up).
template <bool kDown, typename Sum>
__device__ __forceinline__ void finish4(const Int8Params& p, int64_t m, int ub, int i, float sa, Sum sum) {
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + static_cast<size_t>(m) * p.N;
  if constexpr (kDown) {
    const int n = ub * kRows8 + i * 4;  // N % 8 == 0: n < N implies n + 3 < N
    if (n >= p.N) return;
    const float4 v = sum(i * 4), s = *reinterpret_cast<const float4*>(p.scale0 + n);
    float o[4] = {v.x * sa * s.x, v.y * sa * s.y, v.z * sa * s.z, v.w * sa * s.w};
    if (p.residual) {
      const uint2 rr = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.residual) +
                                                       static_cast<size_t>(m) * p.N + n);
      o[0] += __uint_as_float(rr.x << 16);
      o[1] += __uint_as_float(rr.x & 0xffff0000u);
      o[2] += __uint_as_float(rr.y << 16);
      o[3] += __uint_as_float(rr.y & 0xffff0000u);
    }
    *reinterpret_cast<uint2*>(y + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  } else {
    const int n = ub * (kRows8 / 2) + i * 4, r = (i >> 2) * 32 + (i & 3) * 4;
    if (n >= p.N) return;
    const float4 g = sum(r), u = sum(r + 16);
    const float4 s = *reinterpret_cast<const float4*>(p.scale0 + n);
    const float4 t = *reinterpret_cast<const float4*>(p.scale1 + n);
    *reinterpret_cast<uint2*>(y + n) =
        make_uint2(pack_bf16x2(silu_mul(g.x * sa * s.x, u.x * sa * t.x), silu_mul(g.y * sa * s.y, u.y * sa * t.y)),
                   pack_bf16x2(silu_mul(g.z * sa * s.z, u.z * sa * t.z), silu_mul(g.w * sa * s.w, u.w * sa * t.w)));
  }
}

template <bool kDown, bool kPair>
__global__ void __launch_bounds__(kThreads8, 1) int8_gemm_kernel(const __grid_constant__ Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr uint32_t kWBytes = kRows8 * 128;
  const int mt = p.mt, stages = p.stages, slots = p.slots;
  const int mine = kPair ? mt / 2 : mt;  // tokens whose values this CTA holds
  const uint32_t x_bytes = static_cast<uint32_t>(mine) * 256, raw_bytes = kPair ? 0u : static_cast<uint32_t>(mine) * 128;
  const uint32_t stage_bytes = kWBytes + x_bytes + raw_bytes;  // a multiple of 1024
  const uint32_t s0 = smem_addr(smem);
  uint8_t* bar_ptr = smem + size_t(stages) * stage_bytes;
  const uint32_t bar0 = smem_addr(bar_ptr);
  // barrier slots: full[10] | ready[10] | done[10] | sums[2] | sums read[2] | drain, of a stage:
  // full: weights (and codes of tokens) landed, in this CTA; ready: both operands are in fp16, in the
  // CTA that issues; done: its MMAs are, which frees its shared memory and its slot. One commit
  // and one wait of the issuing warp a stage: with a ready and a free barrier for each 64 of K
  // beside the tokens' that warp was what the decode kernel waited for.
  const uint32_t full0 = bar0, ready0 = full0 + 8u * kMaxStages8, done0 = ready0 + 8u * kMaxStages8;
  const uint32_t tfull0 = done0 + 8u * kMaxStages8, tempty0 = tfull0 + 16u, drain = tempty0 + 16u;
  constexpr int kBars = 3 * kMaxStages8 + 5;
  static_assert(8 * kBars + 8 <= kBarBytes8, "barrier slots");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_kb = (p.K + kBlockK8 - 1) / kBlockK8;
  const int splits = kPair ? 1 : p.splits;
  const uint32_t rank = kPair || splits > 1 ? cluster_ctarank() : 0;
  const bool leader = !kPair || rank == 0;
  const int part = kPair ? 0 : static_cast<int>(rank);
  const int per = kPair ? 2 : splits;  // CTAs a unit takes
  const int first = blockIdx.x / per, step = gridDim.x / per;
  const int units = p.blocks * p.mgroups;
  const int kb_begin = part * num_kb / splits, kb_end = (part + 1) * num_kb / splits;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  // weight block of 128 packed rows: the upper or lower half of a packed tile
  const auto block_of = [&](const Unit& u) { return kPair ? 2 * u.block + static_cast<int>(rank) : u.block; };
  const auto weights = [&](int ub, int kb) {
    return static_cast<const uint8_t*>(p.w) + (static_cast<size_t>(ub >> 1) * num_kb + kb) * (2 * kWBytes) +
           (ub & 1) * kWBytes;
  };
  // warps that widen tokens: 16 codes a lane and stage
  const int tok_warps = min(kEpiWarps8, mt / 4);
  // the even CTA's barriers, as seen from either CTA of a pair
  const uint32_t ready0_lead = kPair ? mapa_shared(ready0, 0) : ready0;
  const uint32_t tempty0_lead = kPair ? mapa_shared(tempty0, 0) : tempty0;

  if (threadIdx.x == 0) {
    prefetch_tmap(&p.tmap_x);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      // the converting warps (of both CTAs), and the ones that widen tokens, or the even producer
      mbar_init(ready0 + 8u * s, kPair ? 2 * kConvWarps + 1 : kConvWarps + tok_warps);
      mbar_init(done0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, kPair ? 2 * kEpiWarps8 : kEpiWarps8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (kPair) {
    cluster_arrive();  // both CTAs run, their barriers initialised
    cluster_wait();
    pdl_wait();
    if (warp == 1) tmem_alloc_pair(smem_addr(tmem_slot), kTmem8);
    tc_fence_before();
    cluster_arrive();  // tensor memory allocated; the producer need not wait for that
    if (warp != 0) cluster_wait();
    tc_fence_after();
    if (warp == 1) tmem_relinquish_pair();
  } else {
    if (warp == 1) {
      tmem_alloc(smem_addr(tmem_slot), kTmem8);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  // the slots, then the accumulators, two of mt columns
  const uint32_t acc0 = tmem_base + static_cast<uint32_t>(slots * 64);
  if (!kPair) pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const bool one = elect_one();
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    int s = 0;
    uint32_t ph = 0, filled = 0, fill_ph = 0;
    bool ok = true, skip_once = p.inject_stall != 0;
    for (int u = first; ok && u < units; u += step) {
      const Unit un = unit_of(p, u);
      const int ub = block_of(un);
      const int m0 = un.group * mt + (kPair ? static_cast<int>(rank) * mine : 0);
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(done0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        if (skip_once) {
          skip_once = false;  // testing hook: leave this stage unfilled
        } else {
          if (one) {
            const uint32_t fb = full0 + 8u * s, sw = s0 + s * stage_bytes, sx = sw + kWBytes;
            mbar_arrive_expect_tx(fb, kWBytes + raw_bytes);
            if (p.mgroups > 1)  // other CTAs read the same weights
              bulk_load(sw, weights(ub, kb), kWBytes, fb);
            else
              bulk_load_hint(sw, weights(ub, kb), kWBytes, fb, pol_w);
            if constexpr (kPair) {
              if (leader) mbar_arrive_expect_tx(ready0 + 8u * s, 2 * x_bytes);
              tma_load_2d_pair(sx, &p.tmap_x, ready0_lead + 8u * s, kb * kBlockK8, m0);
              tma_load_2d_pair(sx + x_bytes / 2, &p.tmap_x, ready0_lead + 8u * s, kb * kBlockK8 + kSubK, m0);
            } else {
              tma_load_2d_hint(sx + x_bytes, &p.tmap_x, fb, kb * kBlockK8, m0, pol_x);
            }
          }
          filled |= 1u << s;
          fill_ph = (fill_ph & ~(1u << s)) | (ph << s);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (one) pdl_launch_dependents();
    // copies in flight: a pair's token copies are counted on the even CTA
    for (int i = 0; one && i < stages; ++i)
      if (filled & (1u << i)) {
        mbar_wait_drain(full0 + 8u * i, (fill_ph >> i) & 1u, wc);
        if (kPair && leader) mbar_wait_drain(ready0 + 8u * i, (fill_ph >> i) & 1u, wc);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (the even CTA of a pair)
    if (leader) {
      const bool one = elect_one();
      const uint32_t idesc = idesc_f16_f32(kPair ? 256 : 128, mt);
      int s = 0, t = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        if (!mbar_wait_warp(tempty0 + 8u * buf, acc_ph ^ 1u, wc, kSiteMmaTmemEmpty)) break;
        tc_fence_after();
        const uint32_t d = acc0 + static_cast<uint32_t>(buf * mt);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_warp(ready0 + 8u * s, ph, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t xdesc = smem_desc_sw128(s0 + s * stage_bytes + kWBytes);
          const uint64_t next = x_bytes / 2 >> 4;  // the tokens' second 64 of K
          const uint32_t a = tmem_base + static_cast<uint32_t>(t) * 64;
          if (one) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // 16 of K: 8 columns of the slot, 32 bytes of a token's row
              const uint32_t acc = (kb != kb_begin || k != 0) ? 1u : 0u;
              const uint64_t x = xdesc + 2u * (k & 3) + (k >> 2) * next;
              if constexpr (kPair)
                mma_f16_ts_pair(d, a + 8 * k, x, idesc, acc);
              else
                mma_f16_ts(d, a + 8 * k, x, idesc, acc);
            }
            if constexpr (kPair)
              mma_commit_pair_multicast(done0 + 8u * s, 0x3);
            else
              mma_commit(done0 + 8u * s);
          }
          __syncwarp();
          if (++t == slots) t = 0;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (one) {
          if constexpr (kPair)
            mma_commit_pair_multicast(tfull0 + 8u * buf, 0x3);
          else
            mma_commit(tfull0 + 8u * buf);
        }
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1u;
      }
      if (one) {
        if constexpr (kPair)
          mma_commit_pair_multicast(drain, 0x1);
        else
          mma_commit(drain);
        mbar_wait_drain(drain, 0, wc);
      }
    }
    __syncwarp();
  } else if (warp < 2 + kConvWarps) {
    // ------------------------------------------------ weights to fp16 in tensor memory
    const int sub = (warp - 2) >> 2, q = warp & 3;  // this warp's half of a stage, its lanes
    const int row = q * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    // The slot of this stage was last that of the stage `slots` before; where the ring of stages is
    // no longer than that of slots, this stage's copies already waited for that one.
    const bool behind = slots < stages;
    int s = 0, t = 0, old = stages - slots;  // old: the ring index of the stage `slots` before
    uint32_t ph = 0, old_ph = 1;               // a first use waits for nothing
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteConvert)) {
          ok = false;
          break;
        }
        const uint32_t src = s0 + s * stage_bytes + row * 128;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = ld_shared_v4(src + (((sub * 4 + j) ^ (row & 7)) << 4));
        if (behind && !mbar_wait_warp(done0 + 8u * old, old_ph, wc, kSiteConvert)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          widen4(v[j].x, r[8 * j], r[8 * j + 1]);
          widen4(v[j].y, r[8 * j + 2], r[8 * j + 3]);
          widen4(v[j].z, r[8 * j + 4], r[8 * j + 5]);
          widen4(v[j].w, r[8 * j + 6], r[8 * j + 7]);
        }
        tmem_st_x32(tmem_base + static_cast<uint32_t>(t) * 64 + sub * 32 + lane_off, r);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        // (the slot is this CTA's own tensor memory: the even CTA only learns that it may issue,
        // so the arrival needs no release at cluster scope, which took 1000 cycles)
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_remote(ready0_lead + 8u * s);
          else
            mbar_arrive(ready0 + 8u * s);
        }
        if (++t == slots) t = 0;
        if (++old == stages) {
          old = 0;
          old_ph ^= 1u;
        }
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ tokens to fp16, epilogue
    const int ew = warp - 2 - kConvWarps, q = warp & 3;
    const int tid = ew * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    int s = 0, buf = 0;
    uint32_t ph = 0, acc_ph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      const Unit un = unit_of(p, u);
      if constexpr (!kPair) {
        for (int kb = kb_begin; ew < tok_warps && kb < kb_end; ++kb) {
          if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteConvert)) {
            ok = false;
            break;
          }
          const uint32_t sx = s0 + s * stage_bytes + kWBytes, raw = sx + x_bytes;
          for (int i = tid; i < mt * 8; i += 32 * tok_warps) {
            const int r = i >> 3, c = i & 7;  // 16 codes of token r
            const uint4 v = ld_shared_v4(raw + r * 128 + ((c ^ (r & 7)) << 4));
            uint32_t w[8];
            widen4(v.x ^ 0x80808080u, w[0], w[1]);
            widen4(v.y ^ 0x80808080u, w[2], w[3]);
            widen4(v.z ^ 0x80808080u, w[4], w[5]);
            widen4(v.w ^ 0x80808080u, w[6], w[7]);
            const uint32_t dst = sx + (c >> 2) * (x_bytes / 2) + r * 128;
            const int cc = (c & 3) * 2;
            st_shared_v4(dst + ((cc ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
            st_shared_v4(dst + (((cc + 1) ^ (r & 7)) << 4), w[4], w[5], w[6], w[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready0 + 8u * s);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (!mbar_wait_warp(tfull0 + 8u * buf, acc_ph, wc, kSiteEpiTmemFull)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tacc = acc0 + static_cast<uint32_t>(buf * mt) + lane_off;
      const int m0 = un.group * mt, mcount = min(mt, p.M - m0);
      // two warps share a quarter of the rows: chunks of 16 tokens in turn
      const int chunks = mt / 16, mine_from = ew >> 2;
      if (splits > 1) {
        // fp32 sums of this K part to shared memory: [token][128]
#pragma unroll 1
        for (int c = mine_from; c < chunks; c += 2) {
          uint32_t a[16];
          tmem_ld_x16(tacc + c * 16, a);
          tmem_wait_ld();
          reg_fence(a);
          float* dst = reinterpret_cast<float*>(smem) + size_t(c * 16) * kRows8 + q * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[i * kRows8] = __uint_as_float(a[i]);
        }
      } else {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
        const int ub = block_of(un);
        // gate and up: 16 lanes have gate columns, 16 the up columns beside them
        const bool lower = lane < 16;
        const int n = kDown ? ub * kRows8 + q * 32 + lane : ub * (kRows8 / 2) + q * 16 + (lane & 15);
        const bool there = n < p.N;
        const float t0 = there ? p.scale0[n] : 0.0f;
        const float t1 = !kDown && there ? p.scale1[n] : 0.0f;
        const __nv_bfloat16* res = kDown ? static_cast<const __nv_bfloat16*>(p.residual) : nullptr;
#pragma unroll 1
        for (int c = mine_from; c < chunks; c += 2) {
          const int base = c * 16;
          uint32_t a[16];
          tmem_ld_x16(tacc + base, a);
          tmem_wait_ld();
          reg_fence(a);
          if (c + 2 >= chunks) {  // this warp's part of the sums is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (kPair)
                mbar_arrive_cluster(tempty0_lead + 8u * buf);
              else
                mbar_arrive(tempty0 + 8u * buf);
            }
          }
          // a token's scale in lane (token % 16); columns n and n + 1 meet in one of two lanes, each
          // with half of the tokens, and go out together. No branch before the stores, so that the
          // chunk's loads, exchanges and exponentials overlap (one by one: 3000 cycles a chunk).
          const float scales = p.scale_x[m0 + min(base + (lane & 15), mcount - 1)];
          const bool odd = lane & 1;
          __nv_bfloat16* out = y + static_cast<size_t>(m0 + base) * p.N + (n & ~1);
          if constexpr (kDown) {
            float o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __uint_as_float(a[i]) * __shfl_sync(0xffffffffu, scales, i) * t0;
            const int at = odd ? 8 : 0;  // even lanes take the first 8 tokens
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              r[i] = res && there && base + at + i < mcount
                         ? *reinterpret_cast<const uint32_t*>(res + static_cast<size_t>(m0 + base + at + i) * p.N +
                                                              (n & ~1))
                         : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float got = __shfl_xor_sync(0xffffffffu, odd ? o[i] : o[i + 8], 1);
              const float lo = odd ? got : o[i], hi = odd ? o[i + 8] : got;
              if (there && base + at + i < mcount)
                *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(at + i) * p.N) =
                    pack_bf16x2(lo + __uint_as_float(r[i] << 16), hi + __uint_as_float(r[i] & 0xffff0000u));
            }
          } else {
            // of two tokens the lower lanes finish the first, the upper ones the second
            const int half = lower ? 0 : 1;
            uint32_t w[4];  // tokens 4 j + half and 4 j + 2 + half
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float o[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int i = 4 * j + 2 * e;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, lower ? a[i + 1] : a[i], 16);
                const float g = __uint_as_float(lower ? a[i] : got), v = __uint_as_float(lower ? got : a[i + 1]);
                const float sa = __shfl_sync(0xffffffffu, scales, i + half);
                o[e] = silu_mul(g * sa * t0, v * sa * t1);
              }
              w[j] = pack_bf16x2(o[0], o[1]);
            }
            const int at = (odd ? 8 : 0) + half;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t own = odd ? w[j + 2] : w[j];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[j] : w[j + 2], 1);
              const uint32_t first_of = odd ? got : own, second_of = odd ? own : got;  // columns n & ~1 and n | 1
              if (there && base + at + 4 * j < mcount)
                *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(at + 4 * j) * p.N) =
                    __byte_perm(first_of, second_of, 0x5410);
              if (there && base + at + 4 * j + 2 < mcount)
                *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(at + 4 * j + 2) * p.N) =
                    __byte_perm(first_of, second_of, 0x7632);
            }
          }
        }
        if (chunks == 1 && mine_from == 1 && lane == 0) mbar_arrive(tempty0 + 8u * buf);  // had no chunk (never a pair)
      }
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1u;
    }
    __syncwarp();
  }

  if (!kPair && splits > 1) {
    // every CTA of the cluster gets here, whatever its waits returned
    cluster_sync();
    const Unit un = unit_of(p, first);
    const int m0 = un.group * mt, mcount = min(mt, p.M - m0);
    const uint32_t local = smem_addr(smem);
    constexpr int kItems = kDown ? 32 : 16;
    for (int i = part * kThreads8 + threadIdx.x; i < mcount * kItems; i += splits * kThreads8) {
      const int m = i / kItems;
      finish4<kDown>(p, m0 + m, un.block, i % kItems, p.scale_x[m0 + m], [&](int r) {
        // all parts' loads before their sum, in rank order
        float4 a[kMaxSplits8];
#pragma unroll
        for (int k = 0; k < kMaxSplits8; ++k)
          if (k < splits)
            a[k] = ld_shared_cluster_v4(mapa_shared(local, static_cast<uint32_t>(k)) +
                                        4u * static_cast<uint32_t>(m * kRows8 + r));
        float4 v = a[0];
#pragma unroll
        for (int k = 1; k < kMaxSplits8; ++k)
          if (k < splits) {
            v.x += a[k].x; v.y += a[k].y; v.z += a[k].z; v.w += a[k].w;
          }
        return v;
      });
    }
    // No CTA leaves while a peer may still read its sums. Every value that a thread read there has gone
    // into a store of its own by now, so its reads are over when it arrives (a release, ahead of the
    // stores, would say so to the memory model too: 0.5B down, 128 tokens 9.1 -> 9.7 us, 1 token 6.7 -> 6.9).
    cluster_arrive();
    cluster_wait();
  }
  // Neither CTA of a pair leaves while the pair's MMAs may still read its memory or the peer
  // may still arrive on its barriers.
  if (kPair && warp == 0) cluster_wait();
  tc_fence_before();
  if constexpr (kPair) {
    cluster_arrive_release();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem_base, kTmem8);
    else
      tmem_dealloc(tmem_base, kTmem8);
  }
  if constexpr (kPair) {  // nor while the peer gives its tensor memory back
    cluster_arrive();
    cluster_wait();
  }
}

// Codes as fp16 values, 16 a thread and step.
__global__ void __launch_bounds__(256) widen_kernel(const uint4* codes, uint4* out, size_t items, int tail) {
  pdl_launch_dependents();
  pdl_wait();
  if (tail && blockIdx.x == 0 && threadIdx.x == 0) {  // the last 8
    const uint2 v = *reinterpret_cast<const uint2*>(codes + items);
    uint32_t w[4];
    widen4(v.x ^ 0x80808080u, w[0], w[1]);
    widen4(v.y ^ 0x80808080u, w[2], w[3]);
    out[2 * items] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  for (size_t i = blockIdx.x * size_t(256) + threadIdx.x; i < items; i += size_t(gridDim.x) * 256) {
    const uint4 v = ld_global_v4(codes + i);
    uint32_t w[8];
    widen4(v.x ^ 0x80808080u, w[0], w[1]);
    widen4(v.y ^ 0x80808080u, w[2], w[3]);
    widen4(v.z ^ 0x80808080u, w[4], w[5]);
    widen4(v.w ^ 0x80808080u, w[6], w[7]);
    out[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    out[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Weight codes [rows of the sum, columns] to packed tiles [256][128], biased to q + 128 (128
// where there is none): 256 columns of one matrix, or 128 of two, 16 of each in turn. A unit's
// 128 rows are one contiguous copy of 16 KB: as a tiled TMA load (128 rows of 128 bytes, about 4
// cycles a row) it was what the decode kernel waited for.
__global__ void __launch_bounds__(256)
    pack_int8_kernel(const uint8_t* w1, const uint8_t* w2, uint32_t* wp, int K, int N, int k_slices, int down) {
  __shared__ uint8_t tile[kBlockK8][2 * kRows8 + 4];  // [k][packed row]
  const int b = blockIdx.x, j = blockIdx.y;
  const int k0 = b * kBlockK8;
  for (int idx = threadIdx.x; idx < kBlockK8 * 2 * kRows8; idx += 256) {
    const int t = idx / (2 * kRows8), c = idx % (2 * kRows8);  // column c of the tile's 256, or c % 128 of two
    const int k = k0 + t, cc = c % kRows8;
    const int n = down ? j * 2 * kRows8 + c : j * kRows8 + cc;
    const int row = down ? c : (cc / 16) * 32 + (c / kRows8) * 16 + cc % 16;
    const uint8_t* src = down || c < kRows8 ? w1 : w2;
    tile[t][row] = 0x80u ^ (k < K && n < N ? src[static_cast<size_t>(k) * N + n] : uint8_t(0));
  }
  __syncthreads();
  // 16-byte pieces of a row in the order c ^ (row % 8), as the converting warps read them
  uint32_t* out = wp + (static_cast<size_t>(j) * k_slices + b) * (2 * kRows8 * kBlockK8 / 4);
  for (int idx = threadIdx.x; idx < 2 * kRows8 * kBlockK8 / 4; idx += 256) {
    const int i = idx / (kBlockK8 / 4), t = (idx % (kBlockK8 / 4) * 4) ^ ((i & 7) << 4);
    out[idx] = tile[t][i] | uint32_t(tile[t + 1][i]) << 8 | uint32_t(tile[t + 2][i]) << 16 | uint32_t(tile[t + 3][i]) << 24;
  }
}

size_t stage_bytes8(int mt, bool pair) {
  return size_t(kRows8) * 128 + (pair ? size_t(mt) / 2 * 256 : size_t(mt) * 384);
}

template <bool kDown, bool kPair>
cudaError_t configure_t(int* clusters) {
  cudaError_t e = cudaFuncSetAttribute(int8_gemm_kernel<kDown, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemLimit8));
  for (int s = kPair ? 2 : 1; e == cudaSuccess && s <= (kPair ? 2 : kMaxSplits8); ++s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(kThreads8);
    cfg.dynamicSmemBytes = kSmemLimit8;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters[s], int8_gemm_kernel<kDown, kPair>, &cfg);
  }
  return e;
}

}  // namespace

cudaError_t configure_int8(int (&clusters)[9], int* pairs) {
  int other[9];
  cudaError_t e = configure_t<false, false>(clusters);
  if (e == cudaSuccess) e = configure_t<true, false>(other);
  if (e == cudaSuccess) e = configure_t<false, true>(other);
  if (e == cudaSuccess) e = configure_t<true, true>(other);
  if (e == cudaSuccess) *pairs = other[2];
  return e;
}

int int8_stages(int mt, bool pair) {
  const size_t n = (kSmemLimit8 - 1024 - kBarBytes8) / stage_bytes8(mt, pair);
  return static_cast<int>(n > kMaxStages8 ? kMaxStages8 : n);
}

cudaError_t launch_int8_gemm(const Int8Params& p, bool down, cudaStream_t stream) {
  const int num_kb = (p.K + kBlockK8 - 1) / kBlockK8;
  const int64_t units = int64_t(p.blocks) * p.mgroups;
  const bool pair = p.pair != 0;
  const int per = pair ? 2 : p.splits;
  if (p.mt < 16 || p.mt > (pair ? kInt8PairTokens : kInt8Tokens) || (p.mt % 16) != 0 || p.stages < 2 ||
      p.stages > int8_stages(p.mt, pair) || p.group_m < 1 || p.splits < 1 || p.splits > kMaxSplits8 || p.splits > num_kb ||
      p.grid < per || (p.grid % per) != 0 || p.grid / per > units ||
      (!pair && p.splits > 1 && (p.grid / per != units || size_t(p.mt) * kRows8 * 4 > p.stages * stage_bytes8(p.mt, pair))))
    return cudaErrorInvalidValue;
  Int8Params q = p;
  q.slots = (kTmem8 - 2 * p.mt) / 64;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = 1024 + kBarBytes8 + p.stages * stage_bytes8(p.mt, pair);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = per;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 2 : 1;
  const cudaError_t e = pair ? (down ? cudaLaunchKernelEx(&cfg, int8_gemm_kernel<true, true>, q)
                                     : cudaLaunchKernelEx(&cfg, int8_gemm_kernel<false, true>, q))
                             : (down ? cudaLaunchKernelEx(&cfg, int8_gemm_kernel<true, false>, q)
                                     : cudaLaunchKernelEx(&cfg, int8_gemm_kernel<false, false>, q));
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_widen(const void* codes, void* out, size_t values, cudaStream_t stream) {
  const size_t items = values / 16, blocks = items > 0 ? (items + 255) / 256 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, widen_kernel, static_cast<const uint4*>(codes),
                                           static_cast<uint4*>(out), items, static_cast<int>(values % 16 / 8));
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pack_int8(const void* w1, const void* w2, void* wp, int K, int N, bool down, cudaStream_t stream) {
  const int per = down ? 2 * kRows8 : kRows8;
  const int k_slices = (K + kBlockK8 - 1) / kBlockK8;
  pack_int8_kernel<<<dim3(k_slices, (N + per - 1) / per), 256, 0, stream>>>(
      static_cast<const uint8_t*>(w1), static_cast<const uint8_t*>(w2), static_cast<uint32_t*>(wp), K, N, k_slices,
      down ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace swg
