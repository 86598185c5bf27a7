// C entry points of the 8-bit format: tokens quantised, the forward that keeps
// Gate and Up, and Y restored from them. Contracts are in include/swiglu.h, the
// format in int8.cuh, the kernels in quantize.cu, checkpoint.cu and
// fused_large_m_pair.cu; the backward pass is in backward_api.cu.
#include "swiglu.h"

#include <algorithm>
#include <atomic>
#include <mutex>

#include "api_shared.h"
#include "int8.cuh"
#include "kernels.h"

namespace {

using namespace swg;
using namespace swg::api;

struct KeepState {
  std::atomic<bool> ready{false};
  swiglu_status_t status = SWIGLU_OK;
};
KeepState g_keep[kMaxDevices];
std::mutex g_keep_mu;

swiglu_status_t keep_device(DeviceView* d) {
  const swiglu_status_t st = device_view(d);
  if (st != SWIGLU_OK) return st;
  if (d->max_pairs < 1) return SWIGLU_ERR_UNSUPPORTED;
  KeepState& k = g_keep[d->index];
  if (!k.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_keep_mu);
    if (!k.ready.load(std::memory_order_relaxed)) {
      if (configure_large_m_pair_keep() != cudaSuccess) {
        cudaGetLastError();
        k.status = SWIGLU_ERR_CUDA;
      }
      k.ready.store(true, std::memory_order_release);
    }
  }
  return k.status;
}

}  // namespace

extern "C" {

swiglu_status_t swiglu_quantize_int8(const void* X, void* Q, float* scale, int64_t M, int64_t K,
                                     swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, K, 8);
  if (st != SWIGLU_OK || M == 0) return st;
  if (!X || !Q || !scale) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Q) || !aligned4(scale)) return SWIGLU_ERR_INVALID_ARG;
  const Span in[1] = {{X, size_t(M) * size_t(K) * 2}};
  const Span out[2] = {{Q, size_t(M) * size_t(K)}, {scale, size_t(M) * 4}};
  if (any_overlap(out, 2, in, 1)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  st = device_view(&d);
  if (st != SWIGLU_OK) return st;
  return launched(launch_quantize_rows(X, Q, scale, static_cast<int>(M), static_cast<int>(K),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

swiglu_status_t swiglu_forward_checkpoint(const void* A, const void* Wpacked, void* Y, void* gate, void* up,
                                          float* scale, int64_t M, int64_t K, int64_t N,
                                          swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK || M == 0) return st;
  if (!A || !Wpacked || !Y || !gate || !up || !scale) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(Wpacked) || !aligned16(Y) || !aligned16(gate) || !aligned16(up) ||
      !aligned4(scale))
    return SWIGLU_ERR_INVALID_ARG;
  const size_t codes = size_t(M) * size_t(N);
  const Span in[2] = {{A, size_t(M) * size_t(K) * 2}, {Wpacked, swiglu_packed_weight_bytes(K, N)}};
  const Span out[4] = {{Y, codes * 2}, {gate, codes}, {up, codes}, {scale, checkpoint_scales(M, N) * 4}};
  if (any_overlap(out, 4, in, 2)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  st = keep_device(&d);
  if (st != SWIGLU_OK) return st;
  // 256-token tiles on CTA pairs, whatever M: training batches fill them
  const int64_t tiles_m = (M + 2 * kTileM - 1) / (2 * kTileM), tiles_n = padded_n(N) / kPackBlockN;
  if (tiles_m * tiles_n > 2147483647) return SWIGLU_ERR_UNSUPPORTED;
  LargeMParams p{};
  const uint32_t box_rows = static_cast<uint32_t>(std::min<int64_t>(kTileM, (M + 15) / 16 * 16));
  p.keep_a_bytes = static_cast<int>(box_rows) * kBlockK * 2;
  if (!encode_2d(&p.tmap_a, A, K, M, K * 2, kBlockK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_packed_w(&p.tmap_w, Wpacked, K, N, kPackBlockN) ||
      !encode_2d(&p.tmap_y, Y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return SWIGLU_ERR_CUDA;
  p.y = Y;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.tiles_m = static_cast<int>(tiles_m);
  p.tiles_n = static_cast<int>(tiles_n);
  p.group_m = static_cast<int>(pair_group_rows(tiles_m));
  p.bn = kPackBlockN;
  p.grid = 2 * static_cast<int>(std::min<int64_t>(tiles_m * tiles_n, d.max_pairs));
  p.keep = 1;
  p.keep_gate = gate;
  p.keep_up = up;
  p.keep_scale = scale;
  p.status = d.status;
  p.timeout_ns = d.timeout_ns;
  p.inject_stall = d.inject_stall;
  return launched(launch_large_m_pair(p, reinterpret_cast<cudaStream_t>(stream)));
}

swiglu_status_t swiglu_checkpoint_output(const void* gate, const void* up, const float* scale, void* Y,
                                         int64_t M, int64_t N, swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, 8, N);
  if (st != SWIGLU_OK || M == 0) return st;
  if (!gate || !up || !scale || !Y) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(gate) || !aligned16(up) || !aligned4(scale) || !aligned16(Y)) return SWIGLU_ERR_INVALID_ARG;
  const size_t codes = size_t(M) * size_t(N);
  const Span in[3] = {{gate, codes}, {up, codes}, {scale, checkpoint_scales(M, N) * 4}};
  const Span out[1] = {{Y, codes * 2}};
  if (any_overlap(out, 1, in, 3)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  st = device_view(&d);
  if (st != SWIGLU_OK) return st;
  CheckpointParams p{};
  p.gate = gate;
  p.up = up;
  p.scale = scale;
  p.out0 = Y;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  return launched(launch_checkpoint(p, false, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
