// Non-finite values of an adapter's Lb, kept from other adapters' tokens.
//
// An adapter slice multiplies V, whose rows of other adapters' tokens are zero,
// with Lb, and 0 * inf = NaN. So the warps that write V also look through the Lb
// rows that landed beside it; a row that holds an infinity or NaN (a fault of one
// tenant's adapter) loses those entries before the MMA, and the CTA is marked. A
// marked CTA's epilogue adds what was taken out to the tokens that own it,
// sum_r V[m][r] * Lb[a][n][r] over the non-finite entries, in fp32 from the
// tables: they get the infinity or NaN that the formula gives them, all others
// keep their bits. Adding it once per K part changes nothing: inf + inf = inf.
// What every call pays is the look: an integer test on 16 bytes at a time.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace swg {

// Bits 15 and 31 are set where a bf16 half has all exponent bits set (0x7f80
// plus 0x80 is 0x8000, and no smaller exponent carries into bit 15).
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  const uint32_t b = nonfinite_bits(w);
  return (b & 0x8000u ? 0u : w & 0xffffu) | (b & 0x80000000u ? 0u : w & 0xffff0000u);
}

// Zeroes the non-finite entries of 16-byte chunks [begin, end) of a 128-byte
// swizzled shared-memory row (end - begin <= kMax); whether there were any.
template <int kMax>
__device__ __forceinline__ bool clean_lb_row(uint32_t base, int row, int begin, int end) {
  const uint32_t addr = base + row * 128;
  uint32_t seen = 0;
#pragma unroll
  for (int c = 0; c < kMax; ++c) {
    if (begin + c >= end) break;
    const uint4 w = ld_shared_v4(addr + (((begin + c) ^ (row & 7)) << 4));
    seen |= nonfinite_bits(w.x) | nonfinite_bits(w.y) | nonfinite_bits(w.z) | nonfinite_bits(w.w);
  }
  if (!(seen & 0x80008000u)) return false;
#pragma unroll 1
  for (int c = begin; c < end; ++c) {
    const uint32_t at = addr + ((c ^ (row & 7)) << 4);
    const uint4 w = ld_shared_v4(at);
    st_shared_v4(at, finite_or_zero(w.x), finite_or_zero(w.y), finite_or_zero(w.z), finite_or_zero(w.w));
  }
  return true;
}

// What clean_lb_row() took from one token's output: its V row times the
// non-finite entries of the output's Lb row.
static __device__ __noinline__ float nonfinite_delta(const void* lb, size_t lb_row, const void* v, size_t v_row,
                                                     int rank) {
  const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(lb) + lb_row * rank;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(v) + v_row * rank;
  float sum = 0.0f;
  for (int r = 0; r < rank; ++r) {
    const float y = __bfloat162float(b[r]);
    if (!isfinite(y)) sum += __bfloat162float(x[r]) * y;
  }
  return sum;
}

}  // namespace swg
