// Tokens in 8-bit integers: x [M, K] bf16 -> codes [M, K] and a scale per token
// (int8.cuh). A block a row: its largest magnitude (bf16 magnitudes compare as
// integers, two to a word, NaN above infinity above every number), then its codes,
// from registers or, of many long rows, read again from L1. Rows of bf16 values often
// lie exactly halfway between two codes, where x * (127 / m) in fp32 would round
// either way (code_of()). Measured: 1 token of 896 1.4 us, 16 of 18944 2.2, 4096 of
// 3584 9.7 (L2), 4096 of 18944 42 (5.6 TB/s; held in registers 65: fewer blocks an SM).
#include <algorithm>

#include "int8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace swg {
namespace {

constexpr int kHeld = 4;  // 16-byte pieces of a row that a thread keeps, or loads at once

__device__ __forceinline__ uint32_t max_bits(uint32_t acc, const uint4& v) {
  acc = __vmaxu2(acc, v.x & 0x7fff7fffu);
  acc = __vmaxu2(acc, v.y & 0x7fff7fffu);
  acc = __vmaxu2(acc, v.z & 0x7fff7fffu);
  return __vmaxu2(acc, v.w & 0x7fff7fffu);
}

// 127 x / m of bf16 x and m, rounded half to even: it is a half of an odd number exactly, or (a
// ratio of integers below 2^15 and 2^8, up to a power of two) at least 2^-16 of itself away from one,
// and x * (127 / m) is within 2^-22 of it. So that product, rounded to 17 bits, lies on the right
// side of every half and on it where the quotient does.
__device__ __forceinline__ uint32_t code_of(float x, float inverse) {
  const uint32_t y = (__float_as_uint(x * inverse) + 32u) & ~63u;
  return __float_as_uint(__uint_as_float(y) + kRoundMagic);
}

__device__ __forceinline__ uint2 codes_of(const uint4& v, float inverse) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_of(__uint_as_float(w[i] << 16), inverse);
    c[2 * i + 1] = code_of(__uint_as_float(w[i] & 0xffff0000u), inverse);
  }
  return make_uint2(pack_low_bytes(c[0], c[1], c[2], c[3]), pack_low_bytes(c[4], c[5], c[6], c[7]));
}

// kTwice false: a row's pieces stay in registers, up to kHeld a thread. kTwice: they are read
// again, from L1, with four loads under way: fewer registers, twice the blocks an SM.
template <bool kTwice>
__global__ void __launch_bounds__(kTwice ? 512 : 1024, kTwice ? 3 : 1)
    quantize_rows_kernel(const uint4* x, uint2* codes, float* scale, int chunks) {
  __shared__ uint32_t part[32];
  pdl_launch_dependents();
  pdl_wait();
  const int threads = blockDim.x;
  const size_t row = blockIdx.x;
  const uint4* src = x + row * chunks;
  uint4 v[kHeld];
  uint32_t acc = 0;
  for (int c0 = threadIdx.x; c0 < chunks; c0 += kHeld * threads) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int c = c0 + j * threads;
      v[j] = c < chunks ? ld_global_v4(src + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) acc = max_bits(acc, v[j]);
  }
  acc = max(acc & 0xffffu, acc >> 16);
  acc = __reduce_max_sync(0xffffffffu, acc);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  acc = part[min(threadIdx.x & 31, (threads >> 5) - 1)];
  acc = __reduce_max_sync(0xffffffffu, acc);
  const float largest = __uint_as_float(acc << 16);
  const QuantScale q = quant_scale(largest);
  if (threadIdx.x == 0) scale[row] = q.scale;
  uint2* dst = codes + row * chunks;
  if (!kTwice && chunks <= kHeld * threads) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int c = threadIdx.x + j * threads;
      if (c < chunks) dst[c] = codes_of(v[j], q.inverse);
    }
  } else {
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += threads) dst[c] = codes_of(ld_global_v4(src + c), q.inverse);
  }
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, void* codes, float* scale, int M, int K, cudaStream_t stream) {
  const int chunks = K / 8;
  // four pieces a thread; long rows of many: eight, read twice
  const bool twice = chunks > 1024 && M > 4 * 152;
  const int per_warp = 32 * (twice ? 2 * kHeld : kHeld);
  const int threads = std::min(twice ? 512 : 1024, (chunks + per_warp - 1) / per_warp * 32);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(M));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      twice ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<true>, static_cast<const uint4*>(x),
                                 static_cast<uint2*>(codes), scale, chunks)
            : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<false>, static_cast<const uint4*>(x),
                                 static_cast<uint2*>(codes), scale, chunks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swg
