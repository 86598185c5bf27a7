// What the backward pass does with Gate and Up kept in 8 bits (int8.cuh): codes
// [M, N] of each and scales [2, blocks, M] (block b: columns 128 b .. 128 b + 127;
// a warp of the forward's epilogue, thread = token, writes 32 of them in one line).
//   checkpoint_output  Y = SiLU(g) u, for the down-projection's weight gradient
//   checkpoint_grads   dG and dU from dY, in bf16 for the tensor-core products that
//                      follow (backward_pair.cu says why). Where the input was kept
//                      as codes q and a scale s per token too, its values q s would be
//                      rounded to bf16 as an operand of the weight gradients; with
//                      s = p f (split_scale()) q p is exact, so that is the operand, and
//                      the other one is f dG (f dU), rounded once as dG itself would be.
//                      The input gradient divides its rows by f again, in fp32.
// Both stream: a thread takes 8 columns of every gridDim.y-th row, and holds the
// loads of two rows at a time. Measured, N 18944: Y of 4096 tokens 52-65 us (310 MB, 4.8-6.0
// TB/s; the larger with cold caches); dG and dU of 2048 tokens 51 us cold, 287 MB, DRAM 71 % and 2.65
// instructions a cycle: the arithmetic is the next bound. Most of dG and dU stays in L2 for the products.
#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kThreadsC = 128;
constexpr int kRows = 2;  // rows whose loads are under way together

__device__ __forceinline__ uint2 ld_codes(const void* p, size_t at) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(static_cast<const uint8_t*>(p) + at));
  return v;
}

__device__ __forceinline__ float ld_scale(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void values_of(const uint2& codes, float scale, float (&v)[8]) {
  float a[4], b[4];
  unpack_codes(codes.x, a);
  unpack_codes(codes.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i] * scale;
    v[4 + i] = b[i] * scale;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

template <bool kGrads>
__global__ void __launch_bounds__(kThreadsC)
    checkpoint_kernel(const __grid_constant__ CheckpointParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int rows_step = gridDim.y;
  if (kGrads && static_cast<int>(blockIdx.x) >= p.col_blocks) {  // the input's values
    const int col = ((blockIdx.x - p.col_blocks) * kThreadsC + threadIdx.x) * 8;
    if (col >= p.K) return;
    for (int64_t m = blockIdx.y; m < p.M; m += rows_step) {
      const size_t at = static_cast<size_t>(m) * p.K + col;
      float v[8];
      values_of(ld_codes(p.a_codes, at), split_scale(ld_scale(p.a_scale + m)).power, v);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a_out) + at) = pack8(v);
    }
    return;
  }
  const int col = (blockIdx.x * kThreadsC + threadIdx.x) * 8;
  if (col >= p.N) return;
  const int block = col / kKeepBlock, blocks = (p.N + kKeepBlock - 1) / kKeepBlock;
  const float* gate_scale = p.scale + static_cast<size_t>(block) * p.M;
  const float* up_scale = p.scale + static_cast<size_t>(blocks + block) * p.M;
  for (int64_t m0 = blockIdx.y; m0 < p.M; m0 += int64_t(kRows) * rows_step) {
    uint2 gc[kRows], uc[kRows];
    uint4 dy[kRows];
    float gs[kRows], us[kRows], as[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t m = min(m0 + int64_t(r) * rows_step, int64_t(p.M) - 1);
      const size_t at = static_cast<size_t>(m) * p.N + col;
      gc[r] = ld_codes(p.gate, at);
      uc[r] = ld_codes(p.up, at);
      if constexpr (kGrads)
        dy[r] = ld_global_v4(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dy) + at));
      gs[r] = ld_scale(gate_scale + m);
      us[r] = ld_scale(up_scale + m);
      as[r] = kGrads && p.a_scale ? ld_scale(p.a_scale + m) : 1.0f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t m = m0 + int64_t(r) * rows_step;
      if (m >= p.M) break;
      const size_t at = static_cast<size_t>(m) * p.N + col;
      float g[8], u[8];
      values_of(gc[r], gs[r], g);
      values_of(uc[r], us[r], u);
      if constexpr (kGrads) {
        const uint32_t w[4] = {dy[r].x, dy[r].y, dy[r].z, dy[r].w};
        const float f = split_scale(as[r]).factor;  // dG and dU are linear in dY
        float dg[8], du[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gate_grads(g[2 * i], u[2 * i], f * __uint_as_float(w[i] << 16), dg[2 * i], du[2 * i]);
          gate_grads(g[2 * i + 1], u[2 * i + 1], f * __uint_as_float(w[i] & 0xffff0000u), dg[2 * i + 1],
                     du[2 * i + 1]);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out0) + at) = pack8(dg);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out1) + at) = pack8(du);
      } else {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = silu_mul(g[i], u[i]);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out0) + at) = pack8(y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_checkpoint(const CheckpointParams& p, bool grads, cudaStream_t stream) {
  const auto blocks_of = [](int cols) { return (cols / 8 + kThreadsC - 1) / kThreadsC; };
  CheckpointParams q = p;
  q.col_blocks = blocks_of(p.N);
  const int x = q.col_blocks + (grads && p.a_codes ? blocks_of(p.K) : 0);
  // about 64 blocks an SM (four rounds of those that fit; at 4096 tokens, N 18944 Y takes 58 us with
  // one round, 52 with four; the whole backward pass 1256 and 1240)
  const int64_t want = (152 * 64 + x - 1) / x, rows = (int64_t(p.M) + kRows - 1) / kRows;
  const int64_t y = want < rows ? want : rows;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(x, static_cast<unsigned>(y));
  cfg.blockDim = dim3(kThreadsC);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = grads ? cudaLaunchKernelEx(&cfg, checkpoint_kernel<true>, q)
                              : cudaLaunchKernelEx(&cfg, checkpoint_kernel<false>, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
