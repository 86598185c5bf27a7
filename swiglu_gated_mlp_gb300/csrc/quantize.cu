// Tokens in 8-bit integers: x [M, K] bf16 -> codes [M, K] and a scale per token
// (int8.cuh). One block a row, one read: the row stays in registers (rows too
// long for that are read again, from L2) between its largest magnitude and its
// codes. bf16 magnitudes compare as integers, two to a word, NaN above infinity
// above every number. Rows of bf16 values often lie exactly halfway between two
// codes (the largest a multiple of 127 of some unit), where x * (127 / m) in fp32
// would round either way; those near a half are decided by comparing 254 |x| with
// (2 q + 1) m, both exact in fp32.
#include <algorithm>

#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kHeld = 8;  // 16-byte pieces of a row that a thread keeps

__device__ __forceinline__ uint32_t max_bits(uint32_t acc, const uint4& v) {
  acc = __vmaxu2(acc, v.x & 0x7fff7fffu);
  acc = __vmaxu2(acc, v.y & 0x7fff7fffu);
  acc = __vmaxu2(acc, v.z & 0x7fff7fffu);
  return __vmaxu2(acc, v.w & 0x7fff7fffu);
}

// 127 x / m rounded, where x * (127 / m) is too near to halfway between two codes.
__device__ __noinline__ float code_near_half(float x, float m, float q, float off) {
  const float a = fabsf(x), top = fabsf(q);
  const float below = (x < 0.0f ? -off : off) > 0.0f ? top : top - 1.0f;
  // scaled by 2^-9, so that neither product overflows
  const float side = 0.49609375f * a - (2.0f * below + 1.0f) * (m * 0.001953125f);
  const float half_even = (static_cast<int>(below) & 1) ? below + 1.0f : below;
  const float r = side > 0.0f ? below + 1.0f : side < 0.0f ? below : half_even;
  return x < 0.0f ? -r : r;
}

__device__ __forceinline__ uint32_t code_of(float x, float m, float inverse) {
  const float t = fmaf(x, inverse, kRoundMagic);
  const float q = t - kRoundMagic;
  const float off = fmaf(x, inverse, -q);
  if (fabsf(off) > 0.4999f) return __float_as_uint(code_near_half(x, m, q, off) + kRoundMagic);
  return __float_as_uint(t);
}

__device__ __forceinline__ uint2 codes_of(const uint4& v, float m, float inverse) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_of(__uint_as_float(w[i] << 16), m, inverse);
    c[2 * i + 1] = code_of(__uint_as_float(w[i] & 0xffff0000u), m, inverse);
  }
  return make_uint2(pack_low_bytes(c[0], c[1], c[2], c[3]), pack_low_bytes(c[4], c[5], c[6], c[7]));
}

__global__ void __launch_bounds__(1024)
    quantize_rows_kernel(const uint4* x, uint2* codes, float* scale, int chunks) {
  __shared__ uint32_t part[32];
  pdl_launch_dependents();
  pdl_wait();
  const size_t row = blockIdx.x;
  const uint4* src = x + row * chunks;
  const int threads = blockDim.x;
  uint4 v[kHeld];
  uint32_t acc = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = threadIdx.x + j * threads;
    v[j] = c < chunks ? ld_global_v4(src + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int j = 0; j < kHeld; ++j) acc = max_bits(acc, v[j]);
  for (int c = threadIdx.x + kHeld * threads; c < chunks; c += threads) acc = max_bits(acc, ld_global_v4(src + c));
  acc = max(acc & 0xffffu, acc >> 16);
  acc = __reduce_max_sync(0xffffffffu, acc);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  acc = part[min(threadIdx.x & 31, (threads >> 5) - 1)];
  acc = __reduce_max_sync(0xffffffffu, acc);
  const float largest = __uint_as_float(acc << 16);
  const QuantScale q = quant_scale(largest);
  const float m = fmaxf(largest, 7.888609052210118e-31f);
  if (threadIdx.x == 0) scale[row] = q.scale;
  uint2* dst = codes + row * chunks;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = threadIdx.x + j * threads;
    if (c < chunks) dst[c] = codes_of(v[j], m, q.inverse);
  }
  for (int c = threadIdx.x + kHeld * threads; c < chunks; c += threads)
    dst[c] = codes_of(ld_global_v4(src + c), m, q.inverse);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, void* codes, float* scale, int M, int K, cudaStream_t stream) {
  const int chunks = K / 8;
  // many rows: up to 8 pieces a thread, so that several blocks of an SM load while others reduce;
  // few rows: one or two, for the time of a row
  const int pieces = M > 304 ? kHeld : 2;
  const int threads = std::min(1024, (chunks + 32 * pieces - 1) / (32 * pieces) * 32);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(M));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, quantize_rows_kernel, static_cast<const uint4*>(x),
                                           static_cast<uint2*>(codes), scale, chunks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
