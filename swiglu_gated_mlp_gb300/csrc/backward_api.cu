// C entry points of the gated MLP's gradients: argument checks, workspace
// layout, tile plans and launches. Contracts are in include/swiglu.h, the
// mathematics and the kernel in backward_pair.cu.
#include "swiglu.h"

#include <algorithm>
#include <atomic>
#include <mutex>

#include "api_shared.h"
#include "kernels.h"

namespace {

using namespace swg;
using namespace swg::api;

struct BackwardState {
  std::atomic<bool> ready{false};
  swiglu_status_t status = SWIGLU_OK;
  int max_pairs = 0;
};
BackwardState g_backward[kMaxDevices];
std::mutex g_backward_mu;

// The current device's view and how many CTA pairs of the kernel fit on it.
swiglu_status_t backward_device(DeviceView* d, int* pairs) {
  const swiglu_status_t st = device_view(d);
  if (st != SWIGLU_OK) return st;
  BackwardState& b = g_backward[d->index];
  if (!b.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_backward_mu);
    if (!b.ready.load(std::memory_order_relaxed)) {
      if (configure_backward_pair(&b.max_pairs) != cudaSuccess) {
        cudaGetLastError();
        b.status = SWIGLU_ERR_CUDA;
      } else if (b.max_pairs < 1) {
        b.status = SWIGLU_ERR_UNSUPPORTED;
      }
      b.ready.store(true, std::memory_order_release);
    }
  }
  *pairs = b.max_pairs;
  return b.status;
}

constexpr int64_t kTile = 2 * kTileM;       // rows and columns of an output tile
constexpr int64_t kMaxUnits = 1 << 30;      // tiles x parts of one launch

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// One product's tiles and the parts its sum is cut into.
struct ProductPlan {
  int64_t tiles_m = 0, tiles_n = 0, slices = 0, splits = 1, part_rows = 0;
  size_t part_bytes = 0;  // fp32 parts of one output
};

// `cols`: columns of one output; `outputs` of them side by side in the tiles.
ProductPlan plan_product(int64_t rows, int64_t cols, int outputs, int64_t slices, int pairs) {
  ProductPlan pl;
  pl.tiles_m = div_up(rows, kTile);
  pl.tiles_n = outputs == 2 ? div_up(cols, kTileM) : div_up(cols, kTile);
  pl.slices = slices;
  const int64_t tiles = pl.tiles_m * pl.tiles_n;
  // at least 4 slices a part: fewer do not pay for writing and adding the part
  pl.splits = std::max<int64_t>(1, std::min<int64_t>(pairs / std::max<int64_t>(tiles, 1), slices / 4));
  pl.part_rows = div_up(rows, 32) * 32;
  if (pl.splits > 1) pl.part_bytes = size_t(pl.splits) * size_t(pl.part_rows) * size_t(cols) * 4;
  return pl;
}

ProductPlan plan_input(int64_t M, int64_t K, int64_t sum, int pairs) {  // sum: padded, in 64s
  return plan_product(M, K, 1, sum, pairs);
}

ProductPlan plan_weight(int64_t rows, int64_t cols, int outputs, int64_t M, int pairs) {
  return plan_product(rows, cols, outputs, std::max<int64_t>(k_slices(M), 1), pairs);
}

bool too_many(const ProductPlan& pl) { return pl.tiles_m * pl.tiles_n * pl.splits > kMaxUnits; }

int grid_of(const ProductPlan& pl, int pairs) {
  return 2 * static_cast<int>(std::min<int64_t>(pl.tiles_m * pl.tiles_n * pl.splits, pairs));
}

void fill(BackwardParams* p, const ProductPlan& pl, const DeviceView& d, int64_t rows, int64_t cols) {
  p->rows = static_cast<int>(rows);
  p->cols = static_cast<int>(cols);
  p->slices = static_cast<int>(pl.slices);
  p->tiles_m = static_cast<int>(pl.tiles_m);
  p->tiles_n = static_cast<int>(pl.tiles_n);
  p->group_m = static_cast<int>(pair_group_rows(pl.tiles_m));
  p->splits = static_cast<int>(pl.splits);
  p->part_rows = static_cast<int>(pl.part_rows);
  p->status = d.status;
  p->timeout_ns = d.timeout_ns;
  p->inject_stall = d.inject_stall;
}

// The store map of one output (64 bf16 columns), or of its fp32 parts (32 columns).
bool encode_output(CUtensorMap* map, void* out, float* parts, const ProductPlan& pl, int64_t rows,
                   int64_t cols) {
  if (pl.splits > 1)
    return encode_2d(map, parts, cols, pl.splits * pl.part_rows, cols * 4, 32, 32,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
  return encode_2d(map, out, cols, rows, cols * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Launches one product and, if its sum is in parts, adds them.
swiglu_status_t run_product(const BackwardParams& p, int mode, const ProductPlan& pl, int pairs,
                            void* out0, void* out1, float* parts, cudaStream_t stream) {
  cudaError_t e = launch_backward_pair(p, mode, grid_of(pl, pairs), stream);
  for (int i = 0; e == cudaSuccess && pl.splits > 1 && i < (out1 ? 2 : 1); ++i)
    e = launch_reduce_parts(parts + i * (pl.part_bytes / 4), i ? out1 : out0, p.rows, p.cols,
                            p.part_rows, p.splits, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SWIGLU_ERR_CUDA;
  }
  return SWIGLU_OK;
}

swiglu_status_t zero(void* p, size_t bytes, cudaStream_t stream) {
  if (cudaMemsetAsync(p, 0, bytes, stream) == cudaSuccess) return SWIGLU_OK;
  cudaGetLastError();
  return SWIGLU_ERR_CUDA;
}

struct Span {
  const void* p;
  size_t bytes;
};

// Whether a written span overlaps any other written or read span (null: absent).
bool any_overlap(const Span* out, int outs, const Span* in, int ins) {
  for (int i = 0; i < outs; ++i) {
    if (!out[i].p) continue;
    for (int j = 0; j < ins; ++j)
      if (in[j].p && overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (out[j].p && overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

struct BackwardPlan {
  ProductPlan grad, input, weight;
  size_t grad_bytes = 0;   // dG (and dU) in the workspace
  size_t parts_bytes = 0;  // then the parts of one product at a time
  size_t bytes() const { return 2 * grad_bytes + parts_bytes; }
};

BackwardPlan plan_backward(int64_t M, int64_t K, int64_t N, int pairs) {
  BackwardPlan pl;
  pl.grad.tiles_m = div_up(M, kTile);
  pl.grad.tiles_n = div_up(N, kTileM);
  pl.grad.slices = k_slices(K);
  pl.input = plan_input(M, K, 4 * div_up(N, kTileM), pairs);
  pl.weight = plan_weight(K, N, 2, M, pairs);
  pl.grad_bytes = align256(size_t(M) * size_t(N) * 2);
  pl.parts_bytes = align256(std::max(pl.input.part_bytes, 2 * pl.weight.part_bytes));
  return pl;
}

struct DownBackwardPlan {
  ProductPlan input, weight;
  size_t bytes() const { return align256(std::max(input.part_bytes, weight.part_bytes)); }
};

DownBackwardPlan plan_down_backward(int64_t M, int64_t N, int64_t H, int pairs) {
  DownBackwardPlan pl;
  pl.input = plan_input(M, N, 4 * div_up(H, kTile), pairs);
  pl.weight = plan_weight(N, H, 1, M, pairs);
  return pl;
}

}  // namespace

extern "C" {

size_t swiglu_backward_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (swg::api::check_shape(M, K, N) != SWIGLU_OK || M == 0) return 0;
  DeviceView d;
  int pairs = 0;
  if (backward_device(&d, &pairs) != SWIGLU_OK) return 0;
  return plan_backward(M, K, N, pairs).bytes();
}

swiglu_status_t swiglu_backward(const void* A, const void* Wpacked, const void* dY, void* dA,
                                void* dW1, void* dW2, int64_t M, int64_t K, int64_t N,
                                void* workspace, size_t workspace_bytes, swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK) return st;
  if ((dW1 == nullptr) != (dW2 == nullptr)) return SWIGLU_ERR_INVALID_ARG;
  if (!dA && !dW1) return SWIGLU_OK;
  if ((dA && !aligned16(dA)) || (dW1 && (!aligned16(dW1) || !aligned16(dW2))))
    return SWIGLU_ERR_INVALID_ARG;
  const size_t w_bytes = size_t(K) * size_t(N) * 2;
  const size_t a_bytes = size_t(M) * size_t(K) * 2, y_bytes = size_t(M) * size_t(N) * 2;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // a sum over no tokens
    if (!dW1) return SWIGLU_OK;
    if (overlaps(dW1, w_bytes, dW2, w_bytes)) return SWIGLU_ERR_INVALID_ARG;
    DeviceView d;
    st = device_view(&d);
    if (st == SWIGLU_OK) st = zero(dW1, w_bytes, cs);
    return st == SWIGLU_OK ? zero(dW2, w_bytes, cs) : st;
  }
  if (!A || !Wpacked || !dY || !workspace) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(Wpacked) || !aligned16(dY) || !aligned16(workspace))
    return SWIGLU_ERR_INVALID_ARG;
  const Span in[3] = {{A, a_bytes}, {Wpacked, swiglu_packed_weight_bytes(K, N)}, {dY, y_bytes}};
  const Span out[4] = {{dA, a_bytes}, {dW1, w_bytes}, {dW2, w_bytes}, {workspace, workspace_bytes}};
  if (any_overlap(out, 4, in, 3)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  int pairs = 0;
  st = backward_device(&d, &pairs);
  if (st != SWIGLU_OK) return st;
  const BackwardPlan pl = plan_backward(M, K, N, pairs);
  if (workspace_bytes < pl.bytes()) return SWIGLU_ERR_INVALID_ARG;
  if (too_many(pl.grad) || too_many(pl.input) || too_many(pl.weight)) return SWIGLU_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* dG = ws;
  void* dU = ws + pl.grad_bytes;
  float* parts = reinterpret_cast<float*>(ws + 2 * pl.grad_bytes);
  {
    BackwardParams p{};
    fill(&p, pl.grad, d, M, N);
    p.dy = dY;
    if (!encode_2d(&p.tmap_a0, A, K, M, K * 2, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_packed_w(&p.tmap_b0, Wpacked, K, N, kPackBlockN) ||
        !encode_2d(&p.tmap_o0, dG, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_2d(&p.tmap_o1, dU, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return SWIGLU_ERR_CUDA;
    st = run_product(p, kBackwardGrad, pl.grad, pairs, nullptr, nullptr, nullptr, cs);
    if (st != SWIGLU_OK) return st;
  }
  if (dA) {
    BackwardParams p{};
    fill(&p, pl.input, d, M, K);
    p.two = 1;
    p.col_slices = static_cast<int>(k_slices(K));
    if (!encode_2d(&p.tmap_a0, dG, N, M, N * 2, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&p.tmap_a1, dU, N, M, N * 2, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_packed_w(&p.tmap_b0, Wpacked, K, N, kBlockK) ||
        !encode_output(&p.tmap_o0, dA, parts, pl.input, M, K))
      return SWIGLU_ERR_CUDA;
    st = run_product(p, kBackwardInput, pl.input, pairs, dA, nullptr, parts, cs);
    if (st != SWIGLU_OK) return st;
  }
  if (dW1) {
    BackwardParams p{};
    fill(&p, pl.weight, d, K, N);
    p.two_out = 1;
    if (!encode_2d(&p.tmap_a0, A, K, M, K * 2, kBlockK, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&p.tmap_b0, dG, N, M, N * 2, kBlockK, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&p.tmap_b1, dU, N, M, N * 2, kBlockK, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_output(&p.tmap_o0, dW1, parts, pl.weight, K, N) ||
        !encode_output(&p.tmap_o1, dW2, parts + pl.weight.part_bytes / 4, pl.weight, K, N))
      return SWIGLU_ERR_CUDA;
    st = run_product(p, kBackwardWeight, pl.weight, pairs, dW1, dW2, parts, cs);
  }
  return st;
}

size_t swiglu_down_backward_workspace_bytes(int64_t M, int64_t N, int64_t H) {
  if (swg::api::check_shape(M, N, H) != SWIGLU_OK || M == 0) return 0;
  DeviceView d;
  int pairs = 0;
  if (backward_device(&d, &pairs) != SWIGLU_OK) return 0;
  return plan_down_backward(M, N, H, pairs).bytes();
}

swiglu_status_t swiglu_down_backward(const void* dOut, const void* W3packed, const void* Y, void* dY,
                                     void* dW3, int64_t M, int64_t N, int64_t H, void* workspace,
                                     size_t workspace_bytes, swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, N, H);
  if (st != SWIGLU_OK) return st;
  if (!dY && !dW3) return SWIGLU_OK;
  if ((dY && !aligned16(dY)) || (dW3 && !aligned16(dW3))) return SWIGLU_ERR_INVALID_ARG;
  const size_t w_bytes = size_t(N) * size_t(H) * 2;
  const size_t y_bytes = size_t(M) * size_t(N) * 2, o_bytes = size_t(M) * size_t(H) * 2;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  DeviceView d;
  if (M == 0) {  // a sum over no tokens
    if (!dW3) return SWIGLU_OK;
    st = device_view(&d);
    return st == SWIGLU_OK ? zero(dW3, w_bytes, cs) : st;
  }
  // dOut always; the packed weight for dY, Y for dW3
  if (!dOut || !aligned16(dOut) || (dY && (!W3packed || !aligned16(W3packed))) ||
      (dW3 && (!Y || !aligned16(Y))) || (workspace && !aligned16(workspace)))
    return SWIGLU_ERR_INVALID_ARG;
  const Span in[3] = {{dOut, o_bytes},
                      {dY ? W3packed : nullptr, swiglu_down_packed_bytes(N, H)},
                      {dW3 ? Y : nullptr, y_bytes}};
  const Span out[3] = {{dY, y_bytes}, {dW3, w_bytes}, {workspace, workspace_bytes}};
  if (any_overlap(out, 3, in, 3)) return SWIGLU_ERR_INVALID_ARG;
  int pairs = 0;
  st = backward_device(&d, &pairs);
  if (st != SWIGLU_OK) return st;
  const DownBackwardPlan pl = plan_down_backward(M, N, H, pairs);
  if (pl.bytes() > 0 && (!workspace || workspace_bytes < pl.bytes())) return SWIGLU_ERR_INVALID_ARG;
  if (too_many(pl.input) || too_many(pl.weight)) return SWIGLU_ERR_UNSUPPORTED;
  float* parts = static_cast<float*>(workspace);
  if (dY) {
    BackwardParams p{};
    fill(&p, pl.input, d, M, N);
    p.col_slices = static_cast<int>(k_slices(N));
    if (!encode_2d(&p.tmap_a0, dOut, H, M, H * 2, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_packed_down(&p.tmap_b0, W3packed, N, H, kBlockK) ||
        !encode_output(&p.tmap_o0, dY, parts, pl.input, M, N))
      return SWIGLU_ERR_CUDA;
    st = run_product(p, kBackwardInput, pl.input, pairs, dY, nullptr, parts, cs);
    if (st != SWIGLU_OK) return st;
  }
  if (dW3) {
    BackwardParams p{};
    fill(&p, pl.weight, d, N, H);
    if (!encode_2d(&p.tmap_a0, Y, N, M, N * 2, kBlockK, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&p.tmap_b0, dOut, H, M, H * 2, kBlockK, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_output(&p.tmap_o0, dW3, parts, pl.weight, N, H))
      return SWIGLU_ERR_CUDA;
    st = run_product(p, kBackwardWeight, pl.weight, pairs, dW3, nullptr, parts, cs);
  }
  return st;
}

}  // extern "C"
