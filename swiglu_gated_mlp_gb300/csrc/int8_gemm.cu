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
// side (128 lanes) and the tokens its N side, for one token as for many:
//
//   warp 0      TMA producer: per stage one packed weight tile (rows of 128 codes,
//               gate rows then up rows) and the tokens' 128 codes (or fp16 values)
//   warp 1      MMA issuer
//   warps 2-9   thread = weight row: 64 codes from shared memory (16-byte pieces of
//               a 128-byte swizzled row, free of bank conflicts), each byte b = q + 128
//               set into the fp16 1024 + b and 1152 taken away (2 instructions for 2
//               codes), then one tcgen05.st of 32 columns. A slot of tensor memory
//               holds 64 of K for all rows of the tile; a ring of them runs ahead of
//               the MMAs.
//   warps 10-17 epilogue; with few tokens they first turn the tokens' codes of every
//               stage into fp16 in shared memory (the MMA's right operand). With more
//               tokens a kernel before this one does that once for all column blocks.
//
// A CTA owns `kHalves` x 128 weight rows (gate and up of 128 columns; 128 or 256
// columns of the down-projection) and mt <= 128 tokens. With few such units for the
// SMs, K is split over a cluster of `splits` CTAs whose fp32 partial sums meet in
// shared memory (summed in rank order, so results do not depend on timing). Units
// beyond the resident CTAs are taken in rounds.
#include <cuda_fp16.h>

#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kConvWarps = 8, kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (2 + kConvWarps + kEpiWarps8);
constexpr int kMaxStages8 = 8;
constexpr int kMaxSlots = 16;
constexpr int kTmem8 = 512;
constexpr int kBarBytes8 = 512;
constexpr size_t kSmemLimit8 = 232448;
constexpr int kSubK = 64;  // K values of a slot

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

// Outputs of 4 consecutive columns of one token from its fp32 sums.
template <bool kDown, int kHalves>
__device__ __forceinline__ void finish4(const Int8Params& p, int64_t m, int block, int r, float sa, float4 g,
                                        float4 u) {
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + static_cast<size_t>(m) * p.N;
  if constexpr (kDown) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int n = (block * kHalves + h) * kPackBlockN + r;
      if (n >= p.N) continue;  // N % 8 == 0: n < N implies n + 3 < N
      const float4 v = h ? u : g;
      const float4 s = *reinterpret_cast<const float4*>(p.scale0 + n);
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
    }
  } else {
    const int n = block * kPackBlockN + r;
    if (n >= p.N) return;
    const float4 s = *reinterpret_cast<const float4*>(p.scale0 + n);
    const float4 t = *reinterpret_cast<const float4*>(p.scale1 + n);
    *reinterpret_cast<uint2*>(y + n) =
        make_uint2(pack_bf16x2(silu_mul(g.x * sa * s.x, u.x * sa * t.x), silu_mul(g.y * sa * s.y, u.y * sa * t.y)),
                   pack_bf16x2(silu_mul(g.z * sa * s.z, u.z * sa * t.z), silu_mul(g.w * sa * s.w, u.w * sa * t.w)));
  }
}

template <bool kDown, int kHalves>
__global__ void __launch_bounds__(kThreads8, 1) int8_gemm_kernel(const __grid_constant__ Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr uint32_t kWBytes = kHalves * kPackBlockN * 128;
  const int mt = p.mt, stages = p.stages, slots = p.slots;
  const bool wide = p.wide != 0;  // tokens come as fp16
  const uint32_t x_bytes = static_cast<uint32_t>(mt) * 256, raw_bytes = wide ? 0u : static_cast<uint32_t>(mt) * 128;
  const uint32_t stage_bytes = kWBytes + x_bytes + raw_bytes;  // a multiple of 1024
  const uint32_t s0 = smem_addr(smem);
  uint8_t* bar_ptr = smem + size_t(stages) * stage_bytes;
  const uint32_t bar0 = smem_addr(bar_ptr);
  // barrier slots: full[8] | empty[8] | tokens ready[8] | slot ready[16] | slot free[16] | sums | sums read | drain
  const uint32_t full0 = bar0, empty0 = full0 + 8u * kMaxStages8, tok0 = empty0 + 8u * kMaxStages8;
  const uint32_t ready0 = tok0 + 8u * kMaxStages8, free0 = ready0 + 8u * kMaxSlots;
  const uint32_t tfull = free0 + 8u * kMaxSlots, tempty = tfull + 8u, drain = tempty + 8u;
  constexpr int kBars = 3 * kMaxStages8 + 2 * kMaxSlots + 3;
  static_assert(8 * kBars + 8 <= kBarBytes8, "barrier slots");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_kb = (p.K + kBlockK8 - 1) / kBlockK8;
  const int splits = p.splits;
  const int part = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / splits, step = gridDim.x / splits;  // units of this CTA (cluster)
  const int units = p.blocks * p.mgroups;
  const int kb_begin = part * num_kb / splits, kb_end = (part + 1) * num_kb / splits;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  // a packed tile holds 256 rows; with one half a block is its upper or lower 128
  const auto wtile = [&](int block) { return (kHalves == 2 ? block : block >> 1) * num_kb; };
  const auto wrow = [&](int block) { return kHalves == 2 ? 0 : (block & 1) * kPackBlockN; };

  if (threadIdx.x == 0) {
    prefetch_tmap(&p.tmap_x);
    prefetch_tmap(&p.tmap_w);
    // weights are no product of the kernel before this one: its first tiles on their way to L2
    // meanwhile (L2 is coherent: safe even if they were)
    const int npre = min(p.l2_prefetch, kb_end - kb_begin);
    const uint64_t pol = policy_evict_first();
    const Unit u = unit_of(p, first);
    for (int i = 0; i < npre; ++i)
      tma_prefetch_l2_3d_hint(&p.tmap_w, 0, wrow(u.block), wtile(u.block) + kb_begin + i, pol);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
      mbar_init(tok0 + 8u * s, kEpiWarps8);
    }
    for (int t = 0; t < slots; ++t) {
      mbar_init(ready0 + 8u * t, 4 * kHalves);  // the warps that write a slot
      mbar_init(free0 + 8u * t, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, kEpiWarps8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmem8);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  // the slots, then the accumulators, mt columns of each half
  const uint32_t slot_base = tmem_base;
  const uint32_t acc0 = tmem_base + static_cast<uint32_t>(slots * 32 * kHalves);
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const bool one = elect_one();
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    int s = 0;
    uint32_t ph = 0, filled = 0, fill_ph = 0;
    bool ok = true, skip_once = p.inject_stall != 0;
    for (int u = first; ok && u < units; u += step) {
      const Unit un = unit_of(p, u);
      const int tile = wtile(un.block), row = wrow(un.block), m0 = un.group * mt;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(empty0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        if (skip_once) {
          skip_once = false;  // testing hook: leave this stage unfilled
        } else {
          if (one) {
            const uint32_t fb = full0 + 8u * s, sw = s0 + s * stage_bytes, sx = sw + kWBytes;
            mbar_arrive_expect_tx(fb, kWBytes + (wide ? x_bytes : raw_bytes));
            if (p.mgroups > 1)  // other CTAs read the same weights
              tma_load_3d(sw, &p.tmap_w, fb, 0, row, tile + kb);
            else
              tma_load_3d_hint(sw, &p.tmap_w, fb, 0, row, tile + kb, pol_w);
            if (wide) {
              tma_load_2d_hint(sx, &p.tmap_x, fb, kb * kBlockK8, m0, pol_x);
              tma_load_2d_hint(sx + x_bytes / 2, &p.tmap_x, fb, kb * kBlockK8 + kSubK, m0, pol_x);
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
    for (int i = 0; one && i < stages; ++i)
      if (filled & (1u << i)) mbar_wait_drain(full0 + 8u * i, (fill_ph >> i) & 1u, wc);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    const bool one = elect_one();
    const uint32_t idesc = idesc_f16_f32(128, mt);
    int s = 0, t = 0;
    uint32_t ph = 0, tph = 0, acc_ph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      if (!mbar_wait_warp(tempty, acc_ph ^ 1u, wc, kSiteMmaTmemEmpty)) break;
      tc_fence_after();
      for (int kb = kb_begin; ok && kb < kb_end; ++kb) {
        if (!mbar_wait_warp(wide ? full0 + 8u * s : tok0 + 8u * s, ph, wc, kSiteMmaFull)) {
          ok = false;
          break;
        }
        const uint32_t sx = s0 + s * stage_bytes + kWBytes;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          if (!mbar_wait_warp(ready0 + 8u * t, tph, wc, kSiteConvert)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t xdesc = smem_desc_sw128(sx + sub * (x_bytes / 2));
          const uint32_t a = slot_base + static_cast<uint32_t>(t) * (32 * kHalves);
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 16 of K: 8 columns of the slot, 32 bytes of a token's row
              const uint32_t acc = (kb != kb_begin || sub != 0 || k != 0) ? 1u : 0u;
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                mma_f16_ts(acc0 + h * mt, a + 32 * h + 8 * k, xdesc + 2u * k, idesc, acc);
            }
            mma_commit(free0 + 8u * t);
            if (sub == 1) mma_commit(empty0 + 8u * s);
          }
          __syncwarp();
          if (++t == slots) {
            t = 0;
            tph ^= 1u;
          }
        }
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (one) mma_commit(tfull);
      acc_ph ^= 1u;
    }
    if (one) {
      mma_commit(drain);
      mbar_wait_drain(drain, 0, wc);
    }
    __syncwarp();
  } else if (warp < 2 + kConvWarps) {
    // ------------------------------------------------ weights to fp16 in tensor memory
    const int cw = warp - 2, q = warp & 3;
    const int row = (kHalves == 2 ? (cw >> 2) * kPackBlockN : 0) + q * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t col = kHalves == 2 ? static_cast<uint32_t>(cw >> 2) * 32 : 0;
    int s = 0, t = 0;
    uint32_t ph = 0, tph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      for (int kb = kb_begin; ok && kb < kb_end; ++kb) {
        if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteConvert)) {
          ok = false;
          break;
        }
        const uint32_t src = s0 + s * stage_bytes + row * 128;
#pragma unroll 1
        for (int sub = 0; sub < 2; ++sub) {
          // with one half, four of the eight warps take each slot
          if (kHalves == 2 || sub == (cw >> 2)) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ld_shared_v4(src + (((sub * 4 + j) ^ (row & 7)) << 4));
            if (!mbar_wait_warp(free0 + 8u * t, tph ^ 1u, wc, kSiteConvert)) {
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
            tmem_st_x32(slot_base + static_cast<uint32_t>(t) * (32 * kHalves) + col + lane_off, r);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready0 + 8u * t);
          }
          if (++t == slots) {
            t = 0;
            tph ^= 1u;
          }
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
    const int n_row = q * 32 + lane;  // this thread's weight row
    int s = 0;
    uint32_t ph = 0, acc_ph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      const Unit un = unit_of(p, u);
      if (!wide) {
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteConvert)) {
            ok = false;
            break;
          }
          const uint32_t sx = s0 + s * stage_bytes + kWBytes, raw = sx + x_bytes;
          for (int i = tid; i < mt * 8; i += 32 * kEpiWarps8) {
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
          if (lane == 0) mbar_arrive(tok0 + 8u * s);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (!mbar_wait_warp(tfull, acc_ph, wc, kSiteEpiTmemFull)) {
        ok = false;
        break;
      }
      acc_ph ^= 1u;
      tc_fence_after();
      const int m0 = un.group * mt, mcount = min(mt, p.M - m0);
      // two warps share a quarter of the rows: chunks of 16 tokens in turn
      const int chunks = mt / 16;
      if (splits > 1) {
        // fp32 sums of this K part to shared memory: [h][token][128]
#pragma unroll 1
        for (int c = ew >> 2; c < chunks; c += 2) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t a[16];
            tmem_ld_x16(acc0 + lane_off + h * mt + c * 16, a);
            tmem_wait_ld();
            reg_fence(a);
            float* dst = reinterpret_cast<float*>(smem) + (size_t(h) * mt + c * 16) * kPackBlockN + n_row;
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i * kPackBlockN] = __uint_as_float(a[i]);
          }
        }
      } else {
        const int n0 = un.block * (kDown ? kHalves : 1) * kPackBlockN + n_row;  // gate column, or the first half's
        const int n1 = kDown ? n0 + kPackBlockN : n0;
        const float t0 = n0 < p.N ? p.scale0[n0] : 0.0f;
        const float t1 = kHalves == 2 && n1 < p.N ? (kDown ? p.scale0 : p.scale1)[n1] : 0.0f;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
        const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(p.residual);
#pragma unroll 1
        for (int c = ew >> 2; c < chunks; c += 2) {
          uint32_t g[16], v[16];
          tmem_ld_x16(acc0 + lane_off + c * 16, g);
          if constexpr (kHalves == 2) tmem_ld_x16(acc0 + lane_off + mt + c * 16, v);
          tmem_wait_ld();
          reg_fence(g);
          if constexpr (kHalves == 2) reg_fence(v);
          if (c + 2 >= chunks) {  // this warp's part of the sums is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int m = c * 16 + i;
            if (m >= mcount) break;
            const float sa = p.scale_x[m0 + m];
            const size_t at = static_cast<size_t>(m0 + m) * p.N;
            if constexpr (kDown) {
              if (n0 < p.N) {
                float o = __uint_as_float(g[i]) * sa * t0;
                if (res) o += __bfloat162float(res[at + n0]);
                y[at + n0] = __float2bfloat16(o);
              }
              if (kHalves == 2 && n1 < p.N) {
                float o = __uint_as_float(v[i]) * sa * t1;
                if (res) o += __bfloat162float(res[at + n1]);
                y[at + n1] = __float2bfloat16(o);
              }
            } else if (n0 < p.N) {
              y[at + n0] = __float2bfloat16(silu_mul(__uint_as_float(g[i]) * sa * t0, __uint_as_float(v[i]) * sa * t1));
            }
          }
        }
        if (chunks == 1 && (ew >> 2) == 1 && lane == 0) mbar_arrive(tempty);  // had no chunk
      }
    }
    __syncwarp();
  }

  if (splits > 1) {
    // every CTA of the cluster gets here, whatever its waits returned
    cluster_sync();
    const Unit un = unit_of(p, first);
    const int m0 = un.group * mt, mcount = min(mt, p.M - m0);
    const uint32_t local = smem_addr(smem);
    for (int i = part * kThreads8 + threadIdx.x; i < mcount * 32; i += splits * kThreads8) {
      const int m = i >> 5, r = (i & 31) * 4;
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), v = g;
      for (int k = 0; k < splits; ++k) {
        const uint32_t base = mapa_shared(local, static_cast<uint32_t>(k));
        const float4 a = ld_shared_cluster_v4(base + 4u * static_cast<uint32_t>(m * kPackBlockN + r));
        g.x += a.x; g.y += a.y; g.z += a.z; g.w += a.w;
        if constexpr (kHalves == 2) {
          const float4 b = ld_shared_cluster_v4(base + 4u * static_cast<uint32_t>((mt + m) * kPackBlockN + r));
          v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
        }
      }
      finish4<kDown, kHalves>(p, m0 + m, un.block, r, p.scale_x[m0 + m], g, v);
    }
    cluster_sync();  // no CTA leaves while a peer may still read its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmem8);
  }
}

// Codes as fp16 values, 16 a thread and step.
__global__ void __launch_bounds__(256) widen_kernel(const uint4* codes, uint4* out, size_t items) {
  pdl_launch_dependents();
  pdl_wait();
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
// where there is none): gate rows then up rows of 128 columns, or 256 columns of one matrix.
__global__ void __launch_bounds__(256)
    pack_int8_kernel(const uint8_t* w1, const uint8_t* w2, uint32_t* wp, int K, int N, int k_slices, int down) {
  __shared__ uint8_t tile[kBlockK8][2 * kPackBlockN + 4];
  const int b = blockIdx.x, j = blockIdx.y;
  const int k0 = b * kBlockK8;
  for (int idx = threadIdx.x; idx < kBlockK8 * 2 * kPackBlockN; idx += 256) {
    const int t = idx / (2 * kPackBlockN), i = idx % (2 * kPackBlockN);
    const int k = k0 + t, n = down ? j * 2 * kPackBlockN + i : j * kPackBlockN + i % kPackBlockN;
    const uint8_t* src = down || i < kPackBlockN ? w1 : w2;
    tile[t][i] = 0x80u ^ (k < K && n < N ? src[static_cast<size_t>(k) * N + n] : uint8_t(0));
  }
  __syncthreads();
  uint32_t* out = wp + (static_cast<size_t>(j) * k_slices + b) * (2 * kPackBlockN * kBlockK8 / 4);
  for (int idx = threadIdx.x; idx < 2 * kPackBlockN * kBlockK8 / 4; idx += 256) {
    const int i = idx / (kBlockK8 / 4), t = idx % (kBlockK8 / 4) * 4;
    out[idx] = tile[t][i] | uint32_t(tile[t + 1][i]) << 8 | uint32_t(tile[t + 2][i]) << 16 | uint32_t(tile[t + 3][i]) << 24;
  }
}

template <bool kDown, int kHalves>
cudaError_t configure_t(int* clusters) {
  cudaError_t e = cudaFuncSetAttribute(int8_gemm_kernel<kDown, kHalves>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemLimit8));
  if (e != cudaSuccess) return e;
  for (int s = 1; s <= 8; ++s) {
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
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, int8_gemm_kernel<kDown, kHalves>, &cfg);
    if (e != cudaSuccess) return e;
    clusters[s] = n;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t configure_int8(int (&clusters)[9]) {
  int other[9];
  cudaError_t e = configure_t<false, 2>(clusters);
  if (e == cudaSuccess) e = configure_t<true, 2>(other);
  if (e == cudaSuccess) e = configure_t<true, 1>(other);
  return e;
}

// Stages of a ring for `halves` x 128 weight rows and mt tokens.
int int8_stages(int halves, int mt, bool wide) {
  const size_t stage = size_t(halves) * kPackBlockN * 128 + size_t(mt) * (wide ? 256 : 384);
  const size_t n = (kSmemLimit8 - 1024 - kBarBytes8) / stage;
  return static_cast<int>(n > kMaxStages8 ? kMaxStages8 : n);
}

size_t int8_smem_bytes(int halves, int mt, bool wide, int stages) {
  return 1024 + kBarBytes8 + size_t(stages) * (size_t(halves) * kPackBlockN * 128 + size_t(mt) * (wide ? 256 : 384));
}

cudaError_t launch_int8_gemm(const Int8Params& p, bool down, cudaStream_t stream) {
  const int num_kb = (p.K + kBlockK8 - 1) / kBlockK8;
  const int64_t units = int64_t(p.blocks) * p.mgroups;
  if ((p.halves != 1 && p.halves != 2) || (p.halves == 1 && !down) || p.mt < 16 || p.mt > 128 || (p.mt % 16) != 0 ||
      p.stages < 2 || p.stages > int8_stages(p.halves, p.mt, p.wide != 0) || p.group_m < 1 || p.splits < 1 ||
      p.splits > 8 || p.splits > num_kb || p.grid < p.splits || (p.grid % p.splits) != 0 ||
      (p.splits > 1 && (p.grid / p.splits != units ||
                        size_t(p.halves) * p.mt * kPackBlockN * 4 >
                            size_t(p.stages) * (size_t(p.halves) * kPackBlockN * 128 + size_t(p.mt) * (p.wide ? 256 : 384)))))
    return cudaErrorInvalidValue;
  Int8Params q = p;
  const int slots = (kTmem8 - p.halves * p.mt) / (32 * p.halves);
  q.slots = slots > kMaxSlots ? kMaxSlots : slots;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = int8_smem_bytes(p.halves, p.mt, p.wide != 0, p.stages);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  const cudaError_t e = !down           ? cudaLaunchKernelEx(&cfg, int8_gemm_kernel<false, 2>, q)
                        : p.halves == 2 ? cudaLaunchKernelEx(&cfg, int8_gemm_kernel<true, 2>, q)
                                        : cudaLaunchKernelEx(&cfg, int8_gemm_kernel<true, 1>, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_widen(const void* codes, void* out, size_t values, cudaStream_t stream) {
  const size_t items = values / 16, blocks = (items + 255) / 256;
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
                                           static_cast<uint4*>(out), items);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pack_int8(const void* w1, const void* w2, void* wp, int K, int N, bool down, cudaStream_t stream) {
  const int per = down ? 2 * kPackBlockN : kPackBlockN;
  const int k_slices = (K + kBlockK8 - 1) / kBlockK8;
  pack_int8_kernel<<<dim3(k_slices, (N + per - 1) / per), 256, 0, stream>>>(
      static_cast<const uint8_t*>(w1), static_cast<const uint8_t*>(w2), static_cast<uint32_t*>(wp), K, N, k_slices,
      down ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace swg
