// Host-side helpers that the C entry points share (defined in swiglu_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "swiglu.h"

namespace swg {
namespace api {

constexpr int kMaxDevices = 64;

struct DeviceView {  // what a launch needs of the current device's state
  int index;
  int sm_count;
  int max_pairs;        // CTA pairs of the forward pair kernel resident at once (0: none)
  uint32_t* status;     // device status record
  uint64_t timeout_ns;  // limit of one pipeline wait
  int inject_stall;     // testing hook
};

// The current device's state, set up on first use.
swiglu_status_t device_view(DeviceView* out);
// Sizes: M < 0, K or N <= 0: INVALID_ARG; not multiples of 8, beyond the limits: UNSUPPORTED.
swiglu_status_t check_shape(int64_t M, int64_t K, int64_t N);
bool aligned16(const void* p);
bool overlaps(const void* a, size_t an, const void* b, size_t bn);
int64_t padded_n(int64_t n);
int64_t k_slices(int64_t k);
int64_t padded_h(int64_t h);
// Row tiles (of 256 rows) per group of the CTA-pair kernels' tile order.
int64_t pair_group_rows(int64_t row_tiles);

// Decode-kernel work split for `blocks` weight blocks on the current device, in
// token groups of at most 128.
swiglu_status_t decode_plan(int64_t M, int64_t blocks, int64_t kslices, int* mt, int* mgroups,
                            int* stages, int* splits);

// Tensor maps through the per-thread cache.
bool encode_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle,
               CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
bool encode_3d(CUtensorMap* map, const void* base, const uint64_t dims[3],
               const uint64_t strides[2], const uint32_t box[3], CUtensorMapSwizzle swizzle);
// The packed gate/up weight or down-projection weight in boxes of {64, rows, 1}.
bool encode_packed_w(CUtensorMap* map, const void* base, int64_t K, int64_t N, uint32_t rows);
bool encode_packed_down(CUtensorMap* map, const void* base, int64_t N, int64_t H, uint32_t rows);

}  // namespace api
}  // namespace swg
