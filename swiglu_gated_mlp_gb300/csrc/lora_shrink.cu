// First half of the low-rank adapters: each token's V = scale_a * x La[a]^T
// with a = index[token], for the kernels that add V Lb[a]^T to the shared
// projection (fused_small_m.cu and fused_large_m_pair.cu, kLora).
//
// La [L, hr, K] holds the rows that one adapter shrinks to: gate then up rows
// of a gate/up adapter (hr = 2 rank), or the rank rows of a down adapter. Per
// token the product is hr x K, far below the projection's, so what counts is
// that it reads x once and each adapter present once, and ends early.
//
// V is rounded to bf16, the operand type of the expanding product: the delta it
// enters is a fraction of the projection, which is itself rounded to bf16.
//
// One or a few tokens of a small rank need no kernel here: the decode kernel's
// CTAs make V (own_v() in lora_api.cu).
//
// Few tokens: lora_shrink_dot_kernel, plain dot products in fp32. One CTA takes
// a token and 4 rows; its 8 warps (32 for a long K) split K, so that few loads
// follow one another: 3.6 us for 16 tokens, 32 rows, K 3584; 4.9 us for 16 rows,
// K 18944. Each token reads its adapter's rows again from L2, so 128 tokens of 128
// rows take about 20 us; tensor-core tiles there were slower with more than two
// adapters (88 against 71 us for the call with 8).
//
// Either kernel lets the projection's start as soon as it has itself waited for the
// grids before it. The decode kernel's weight stream runs beside it, and V only has to be
// there for the adapter slices at its end; CTA pairs load their first K slices beside it and
// allocate tensor memory when it has ended (lora_api.cu). 333 tokens, K 1416,
// N 5000 30.5 -> 24.4 us, 200 tokens, down, N 18944 79 -> 45, 128 tokens, down, N 4864
// 18.0 -> 16.4, 16 tokens, K 3584, N 18944 49.8 -> 48.3. (Before, the projection's
// kernel started with this one, did its set-up and staged weight tiles in L2, then
// waited for all of V; for 16 tokens, down, N 18944 that was as fast, 28.9 / 29.2.)
//
// Many tokens: lora_shrink_tile_kernel, tcgen05 with 128 tokens as the MMA's
// M side and the rows of the adapters present in the tile as its N side. The
// tile's tokens are multiplied by every adapter present (a tile of one prompt
// has one), and each token keeps its own adapter's columns: a value of another
// adapter, finite or not, never reaches it. K is split over a cluster of up to
// 8 CTAs, whose fp32 sums are added in order through distributed shared memory.
// A stage holds 64 of K for the tokens and for as many adapters as the tile has
// (up to per_pass), and the ring as many stages as fit, so that with one adapter
// most of what is in flight are tokens. The first tokens are on their way before
// the adapters are known (a hash table in shared memory finds them; comparing
// every token with all before it took 2.6 us of 26). The kernel also lists, per
// 256 tokens (a CTA pair's tile), the adapters present in the order of their
// first token, so that no sum's order depends on timing. 4096 tokens, rank 64:
// 26 us at K 3584 (30 MB; 10 us of it the start, the lists and the cluster's sums)
// and 46 us at K 18944 (138 MB; tiles with one adapter stream at 5.5 TB/s, those
// with several wait for their own stages).
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

// ------------------------------------------------------------- few tokens ---

constexpr int kDotRows = 4;
constexpr int kDotThreads = 1024;  // at most

__global__ void __launch_bounds__(kDotThreads)
    lora_shrink_dot_kernel(const __grid_constant__ LoraShrinkParams p) {
  __shared__ float sums[kDotThreads / 32][kDotRows];
  // The decode kernel starts its weight stream when this grid has seen all before it
  // complete, and waits for this grid where it reads V; this grid takes little room.
  pdl_wait();
  pdl_launch_dependents();
  const int threads = blockDim.x;
  const int row_blocks = (p.hr + kDotRows - 1) / kDotRows;
  const int m = blockIdx.x / row_blocks;
  const int r0 = (blockIdx.x % row_blocks) * kDotRows;
  const int a = p.index[m];
  if (a < 0 || a >= p.count) return;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) +
                                                  static_cast<size_t>(m) * p.K);
  const uint4* la = reinterpret_cast<const uint4*>(
      static_cast<const __nv_bfloat16*>(p.la) + (static_cast<size_t>(a) * p.hr + r0) * p.K);
  const int chunks = p.K / 8;
  float acc[kDotRows] = {};
#pragma unroll 4
  for (int i = threadIdx.x; i < chunks; i += threads) {
    const uint4 xv = x[i];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)  // hr is a multiple of 8: every row exists
      acc[r] = dot8(xv, la[static_cast<size_t>(r) * chunks + i], acc[r]);
  }
#pragma unroll
  for (int r = 0; r < kDotRows; ++r)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) sums[threadIdx.x >> 5][r] = acc[r];
  __syncthreads();
  if (threadIdx.x < kDotRows) {
    float v = 0.0f;
    for (int w = 0; w < threads / 32; ++w) v += sums[w][threadIdx.x];
    static_cast<__nv_bfloat16*>(p.v)[static_cast<size_t>(m) * p.hr + r0 + threadIdx.x] =
        __float2bfloat16_rn(v * p.scale[a]);
  }
}

// ------------------------------------------------------------ many tokens ---

constexpr int kTileThreads = 256;
constexpr int kTileCols = 256;                                     // accumulator columns
constexpr int kXBytes = 128 * kBlockK * 2;                         // 16 KB of tokens
constexpr int kTileStages = 8;                                     // at most
constexpr int kPartPad = 4;                                        // floats, against bank conflicts
constexpr int kTileBar = 256;
constexpr int kEarlyLoads = 3;                                     // the ring has at least as many stages
constexpr int kHashSlots = 512;                                    // for up to 256 adapters
constexpr size_t kTileSmem = 223232;  // with 7.8 KB of static shared memory
// What the ring may take. With one pass over the tile's adapters the sums lie
// where the ring was; with more, the rest of it holds the sums of `rb` columns.
__host__ __device__ constexpr int tile_ring(int rb, bool one_pass) {
  return static_cast<int>((kTileSmem - 1024 - kTileBar -
                           (one_pass ? 0 : size_t(128) * (rb + kPartPad) * 4)) / 1024 * 1024);
}
static_assert(tile_ring(2 * kLoraMaxRank, false) >= kEarlyLoads * (kXBytes + kTileCols * kBlockK * 2), "stages");
static_assert(8 * (2 * kTileStages + 3) + 8 <= kTileBar, "barrier slots");

// The slot of `a` in a table of adapters (empty slots hold -1).
__device__ __forceinline__ int slot_of(int* table, int a) {
  uint32_t h = (static_cast<uint32_t>(a) * 2654435761u) >> 23;  // 9 bits: kHashSlots
  for (;;) {  // at most 256 of the 512 slots are taken: an empty one comes
    const int old = atomicCAS(table + h, -1, a);
    if (old == -1 || old == a) return static_cast<int>(h);
    h = (h + 1) & (kHashSlots - 1);
  }
}

__global__ void __launch_bounds__(kTileThreads, 1)
    lora_shrink_tile_kernel(const __grid_constant__ LoraShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ int ids[2 * kTileM];                // adapters of the 256 tokens (-1: none)
  __shared__ int seen[kHashSlots];               // hash table of the 256 tokens' adapters
  __shared__ int first[2][kHashSlots];           // their first token among the 256, and in this tile
  __shared__ int mine[kTileM];                   // adapters present among this tile's 128 tokens
  __shared__ int counts[2][kTileThreads / 32];
  const int rb = p.rb;                           // accumulator columns of one adapter
  const int part_stride = rb + kPartPad;
  const uint32_t s0 = smem_addr(smem);
  uint8_t* bar_ptr = smem + kTileSmem - 1024 - kTileBar;
  const uint32_t bar0 = smem_addr(bar_ptr);
  // barrier slots: full[8] | empty[8] | tmem_full | tmem_empty | drain
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * kTileStages;
  const uint32_t tfull = bar0 + 16u * kTileStages, tempty = tfull + 8u, drain_bar = tfull + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * (2 * kTileStages + 3));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = p.splits;
  const int kpart = blockIdx.x % splits, tile = blockIdx.x / splits;  // kpart: rank in the cluster
  const int m0 = tile * kTileM;
  const int half = tile & 1;            // which 128 of the 256 tokens
  const int begin = kpart * p.slices / splits, end = (kpart + 1) * p.slices / splits;

  if (tid == 0) {
    prefetch_tmap(&p.tmap_x);
    prefetch_tmap(&p.tmap_la);
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 4);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTileCols);
    tmem_relinquish();
  }
  for (int i = tid; i < kHashSlots; i += kTileThreads) {
    seen[i] = -1;
    first[0][i] = first[1][i] = kTileThreads;
  }
  pdl_wait();
  pdl_launch_dependents();  // as above
  // The producer's first token loads do not need the adapters.
  const int early = min(kEarlyLoads, end - begin);
  if (tid == 0 && !p.inject_stall) {
    for (int s = 0; s < early; ++s) {
      mbar_expect_tx(full0 + 8u * s, kXBytes);
      tma_load_2d(s0 + s * kXBytes, &p.tmap_x, full0 + 8u * s, (begin + s) * kBlockK, m0);
    }
  }
  int own;
  {
    const int64_t m = int64_t(m0) - half * kTileM + tid;
    const int a = m < p.M ? p.index[m] : -1;
    own = a >= 0 && a < p.count ? a : -1;
    ids[tid] = own;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  // The adapters of the 256 tokens (for the pair kernel) and of this tile's 128.
  const bool in_tile = tid / kTileM == half;
  const int slot = own >= 0 ? slot_of(seen, own) : 0;
  if (own >= 0) {
    atomicMin(&first[0][slot], tid);
    if (in_tile) atomicMin(&first[1][slot], tid);
  }
  __syncthreads();
  const bool first256 = own >= 0 && first[0][slot] == tid;
  const bool first128 = own >= 0 && in_tile && first[1][slot] == tid;
  const uint32_t b256 = __ballot_sync(0xffffffffu, first256), b128 = __ballot_sync(0xffffffffu, first128);
  if (lane == 0) {
    counts[0][warp] = __popc(b256);
    counts[1][warp] = __popc(b128);
  }
  __syncthreads();
  int n256 = 0, n128 = 0, at256 = 0, at128 = 0;
#pragma unroll
  for (int w = 0; w < kTileThreads / 32; ++w) {
    if (w < warp) {
      at256 += counts[0][w];
      at128 += counts[1][w];
    }
    n256 += counts[0][w];
    n128 += counts[1][w];
  }
  const uint32_t below = (1u << lane) - 1u;
  if (first128) mine[at128 + __popc(b128 & below)] = own;
  if (half == 0 && kpart == 0) {
    int* list = p.lists + static_cast<size_t>(tile >> 1) * kLoraListInts;
    if (first256) list[1 + at256 + __popc(b256 & below)] = own;
    if (tid == 0) list[0] = n256;
  }
  __syncthreads();

  const int per_pass = p.per_pass;  // adapters side by side in the accumulator
  const int passes = (n128 + per_pass - 1) / per_pass;
  const uint32_t la_bytes = static_cast<uint32_t>(rb) * 128u;
  // ring: tokens of every stage, then adapter rows of every stage
  const uint32_t la_stage = max(min(per_pass, n128), 1) * la_bytes;
  const int ring = tile_ring(rb, passes <= 1);
  const int stages = min(static_cast<int>(ring / (kXBytes + la_stage)), kTileStages);
  float* part = reinterpret_cast<float*>(passes <= 1 ? smem : smem + ring);
  const uint32_t sla = s0 + stages * kXBytes;
  if (warp == 0) {
    {
      const bool one = elect_one();
      int s = 0;
      uint32_t ph = 0, filled = 0, fill_ph = 0;
      bool skip_once = p.inject_stall != 0, ok = true;
      for (int pass = 0; ok && pass < passes; ++pass) {
        const int g0 = pass * per_pass, gn = min(per_pass, n128 - g0);
        for (int i = begin; i < end; ++i) {
          if (!mbar_wait_warp(empty0 + 8u * s, ph ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          if (skip_once) {
            skip_once = false;  // testing hook: leave this stage unfilled
          } else {
            const uint32_t fb = full0 + 8u * s;
            const bool loaded = pass == 0 && i - begin < early && !p.inject_stall;
            if (one) {
              mbar_arrive_expect_tx(fb, (loaded ? 0 : kXBytes) + gn * la_bytes);
              if (!loaded) tma_load_2d(s0 + s * kXBytes, &p.tmap_x, fb, i * kBlockK, m0);
              for (int g = 0; g < gn; ++g)
                tma_load_2d(sla + s * la_stage + g * la_bytes, &p.tmap_la, fb, i * kBlockK,
                            mine[g0 + g] * p.hr);
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
      if (one && passes == 0 && !p.inject_stall)  // no adapter: let the early loads land
        for (int s2 = 0; s2 < early; ++s2) {
          mbar_arrive(full0 + 8u * s2);
          mbar_wait_drain(full0 + 8u * s2, 0, wc);
        }
      for (int i = 0; one && i < stages; ++i)
        if (filled & (1u << i)) mbar_wait_drain(full0 + 8u * i, (fill_ph >> i) & 1u, wc);
    }
    __syncwarp();
  } else if (warp == 1) {
    {
      const bool one = elect_one();  // waits and counts by the whole warp: see the pair kernel
      const uint32_t idesc = idesc_bf16_f32(kTileM, rb);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int pass = 0; ok && pass < passes; ++pass) {
        const int gn = min(per_pass, n128 - pass * per_pass);
        if (pass > 0 && !mbar_wait_warp(tempty, (pass - 1) & 1, wc, kSiteMmaTmemEmpty)) break;
        tc_fence_after();
        for (int i = begin; i < end; ++i) {
          if (!mbar_wait_warp(full0 + 8u * s, ph, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t xdesc = smem_desc_sw128(s0 + s * kXBytes);
          if (one) {
            for (int g = 0; g < gn; ++g) {
              const uint64_t ldesc = smem_desc_sw128(sla + s * la_stage + g * la_bytes);
#pragma unroll
              for (uint32_t k = 0; k < 4; ++k)
                mma_bf16(tmem_base + g * rb, xdesc + 2u * k, ldesc + 2u * k, idesc,
                         (i != begin || k != 0) ? 1u : 0u);
            }
            mma_commit(empty0 + 8u * s);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok && one) mma_commit(tfull);
      }
      if (one) {
        mma_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0, wc);
      }
    }
    __syncwarp();
  } else if (warp < 6) {
    // each thread keeps its token's own adapter's columns
    const int q = warp & 3, row = q * 32 + lane;
    const int my = ids[half * kTileM + row];
    float* dst = part + row * part_stride;
    for (int pass = 0; pass < passes; ++pass) {
      int ok = 1;
      if (lane == 0) ok = mbar_wait(tfull, pass & 1, wc, kSiteEpiTmemFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const int g0 = pass * per_pass, gn = min(per_pass, n128 - g0);
      for (int g = 0; g < gn; ++g) {
        const bool keep = mine[g0 + g] == my;
        if (!__any_sync(0xffffffffu, keep)) continue;
        for (int c = 0; c < rb; c += 16) {
          uint32_t v[16];
          tmem_ld_x16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + g * rb + c, v);
          tmem_wait_ld();
          reg_fence(v);
          if (keep)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<uint4*>(dst + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
    }
    __syncwarp();
  }
  // Every part's sums are in its CTA's shared memory: each CTA adds its share
  // of the rows over the parts in order, scales, rounds and stores.
  tc_fence_before();
  cluster_sync();
  const int rows = kTileM / splits, chunks = p.hr / 8;
  // a peer with another number of passes cannot be: the cluster shares the tokens
  const uint32_t local = smem_addr(part);
  for (int i = tid; i < rows * chunks; i += kTileThreads) {
    const int row = kpart * rows + i / chunks, c = (i % chunks) * 8;
    const int a = ids[half * kTileM + row];
    if (a < 0) continue;  // no adapter (or no token): V is not read
    const float f = p.scale[a];
    float4 u[8], w[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)  // every part's loads before the sums
      if (s < splits) {
        const uint32_t src = mapa_shared(local, s) + 4u * (row * part_stride + c);
        u[s] = ld_shared_cluster_v4(src);
        w[s] = ld_shared_cluster_v4(src + 16u);
      }
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < splits) {
        x.x += u[s].x; x.y += u[s].y; x.z += u[s].z; x.w += u[s].w;
        y.x += w[s].x; y.y += w[s].y; y.z += w[s].z; y.w += w[s].w;
      }
    uint4 o;
    o.x = pack_bf16x2(x.x * f, x.y * f);
    o.y = pack_bf16x2(x.z * f, x.w * f);
    o.z = pack_bf16x2(y.x * f, y.y * f);
    o.w = pack_bf16x2(y.z * f, y.w * f);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v) +
                              (static_cast<size_t>(m0) + row) * p.hr + c) = o;
  }
  cluster_sync();  // no CTA leaves while a peer may still read its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTileCols);
  }
}

}  // namespace

cudaError_t configure_lora_shrink() {
  cudaError_t e = cudaFuncSetAttribute(lora_shrink_tile_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kTileSmem));
  // The same split of the L1/shared array as the decode kernel's, so that its
  // CTAs can join an SM that still runs this kernel.
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(lora_shrink_dot_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             100);
  return e;
}

cudaError_t launch_lora_shrink(const LoraShrinkParams& p, cudaStream_t stream) {
  if (p.M < 1 || p.hr < 8 || (p.hr % 8) != 0 || p.hr > 2 * kLoraMaxRank) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cudaError_t e;
  if (p.tiles == 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(p.M) * ((p.hr + kDotRows - 1) / kDotRows));
    cfg.blockDim = dim3(p.K >= 8192 ? kDotThreads : 256);
    e = cudaLaunchKernelEx(&cfg, lora_shrink_dot_kernel, p);
  } else {
    if (p.splits < 1 || p.splits > 8 || (kTileM % p.splits) != 0 || p.slices < p.splits ||
        (p.rb % 16) != 0 || p.rb < p.hr || p.rb > 2 * kLoraMaxRank || p.per_pass < 1 ||
        p.per_pass * p.rb > kTileCols)
      return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(p.tiles) * p.splits);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = kTileSmem;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, lora_shrink_tile_kernel, p);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
