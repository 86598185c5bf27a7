// C entry points of the gated MLP's gradients: argument checks, workspace
// layout, tile plans and launches. Contracts are in include/swiglu.h, the
// mathematics and the kernel in backward_pair.cu.
#include "swiglu.h"

#include <algorithm>
#include <atomic>
#include <cstdio>
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
constexpr int64_t kMaxUnits = 1 << 30;      // tiles x parts of one product

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// One product's tiles and the parts its sum is cut into.
struct ProductPlan {
  int64_t tiles_m = 0, tiles_n = 0, slices = 0, splits = 1, part_rows = 0;
  size_t part_bytes = 0;  // fp32 parts of one output
  int64_t tiles() const { return tiles_m * tiles_n; }
  int64_t units() const { return tiles() * splits; }
  // time of an unsplit tile in slices: a tile's epilogue takes about as long as
  // the MMAs of 5 slices
  int64_t cost() const { return std::max<int64_t>(slices / splits, 5); }
};

// `cols`: columns of one output; `outputs` of them side by side in the tiles.
ProductPlan plan_product(int64_t rows, int64_t cols, int outputs, int64_t slices) {
  ProductPlan pl;
  pl.tiles_m = div_up(rows, kTile);
  pl.tiles_n = outputs == 2 ? div_up(cols, kTileM) : div_up(cols, kTile);
  pl.slices = slices;
  pl.part_rows = div_up(rows, 32) * 32;
  return pl;
}

// Cuts a product's sum so that no unit is longer than all units spread evenly
// over the pairs, in parts of at least 8 slices, and only where that saves more
// than the launch that adds the parts takes (about 24 slices).
void split(ProductPlan* pl, int64_t cols, int64_t even) {
  if (pl->slices > even + 24)
    pl->splits = std::max<int64_t>(
        1, std::min<int64_t>(div_up(pl->slices, std::max<int64_t>(even, 1)), pl->slices / 8));
  if (pl->splits > 1) pl->part_bytes = align256(size_t(pl->splits) * size_t(pl->part_rows) * size_t(cols) * 4);
}

// The input gradient [M, in_cols] and the weight gradient(s) [w_rows, w_cols]
// of one launch.
struct GradientPlan {
  ProductPlan in, w;
  int pairs = 0, early_rounds = 0;
  int w_outputs = 1;
  size_t parts_bytes() const { return in.part_bytes + w_outputs * w.part_bytes; }
  bool too_many() const { return in.units() > kMaxUnits || w.units() > kMaxUnits; }
};

GradientPlan plan_gradients(int64_t M, int64_t in_cols, int64_t in_slices, int64_t w_rows,
                            int64_t w_cols, int w_outputs, int max_pairs) {
  GradientPlan pl;
  pl.in = plan_product(M, in_cols, 1, in_slices);
  pl.w = plan_product(w_rows, w_cols, w_outputs, 2 * div_up(M, 2 * kBlockK));
  pl.w_outputs = w_outputs;
  const int64_t work = pl.in.tiles() * pl.in.cost() + pl.w.tiles() * pl.w.cost();
  const int64_t even = div_up(work, max_pairs);
  split(&pl.in, in_cols, even);
  split(&pl.w, w_cols, even);
  return pl;
}

// The pairs of a launch of the products asked for, and how many rounds of
// weight units the pairs with one input unit fewer take first.
void deal_units(GradientPlan* pl, bool in, bool w, int max_pairs, BackwardParams* p) {
  p->in_units = in ? static_cast<int>(pl->in.units()) : 0;
  p->w_units = w ? static_cast<int>(pl->w.units()) : 0;
  pl->pairs = static_cast<int>(std::min<int64_t>(int64_t(p->in_units) + p->w_units, max_pairs));
  const int early = pl->pairs - p->in_units % pl->pairs;  // pairs with one input unit fewer
  if (early == pl->pairs) return;
  const int64_t rounds = p->w_units <= early ? 1 : pl->in.cost() / pl->w.cost();
  p->early_rounds = static_cast<int>(std::min<int64_t>(rounds, p->w_units / early));
}

// Rows of a box whose rows are tokens: 128, or up to the last 16 of fewer (rows
// past the last token are zero).
uint32_t token_rows(int64_t M) {
  return static_cast<uint32_t>(std::min<int64_t>(kTileM, div_up(M, 16) * 16));
}

void fill(BackwardProduct* p, const ProductPlan& pl, int64_t rows, int64_t cols, int64_t M) {
  p->a_bytes = static_cast<int>(token_rows(M)) * kBlockK * 2;
  p->rows = static_cast<int>(rows);
  p->cols = static_cast<int>(cols);
  p->slices = static_cast<int>(pl.slices);
  p->tiles_m = static_cast<int>(pl.tiles_m);
  p->tiles_n = static_cast<int>(pl.tiles_n);
  p->group_m = static_cast<int>(pair_group_rows(pl.tiles_m));
  p->splits = static_cast<int>(pl.splits);
  p->part_rows = static_cast<int>(pl.part_rows);
}

void fill_status(BackwardParams* p, const DeviceView& d) {
  p->status = d.status;
  p->timeout_ns = d.timeout_ns;
  p->inject_stall = d.inject_stall;
}

// The store map of one output (64 bf16 columns), or of its fp32 parts (32
// columns), which are then added up after the launch.
bool encode_output(CUtensorMap* map, void* out, uint8_t* parts, const ProductPlan& pl, int64_t rows,
                   int64_t cols, ReduceParams* sums) {
  if (pl.splits == 1)
    return encode_2d(map, out, cols, rows, cols * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  sums->out[sums->count++] =
      ReduceOutput{reinterpret_cast<const float*>(parts), out, static_cast<int>(rows),
                   static_cast<int>(cols), static_cast<int>(pl.part_rows), static_cast<int>(pl.splits)};
  return encode_2d(map, parts, cols, pl.splits * pl.part_rows, cols * 4, 32, 32,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
}

// A row-major [tokens, cols] operand, 64 columns x up to 128 tokens a box.
bool encode_operand(CUtensorMap* map, const void* base, int64_t rows, int64_t cols) {
  return encode_2d(map, base, cols, rows, cols * 2, kBlockK, token_rows(rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

swiglu_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return SWIGLU_OK;
  cudaGetLastError();
  return SWIGLU_ERR_CUDA;
}

// Launches the input and weight gradients and adds what is in parts.
swiglu_status_t run_gradients(const BackwardParams& p, const GradientPlan& pl, const ReduceParams& sums,
                              cudaStream_t stream) {
  cudaError_t e = launch_backward_pair(p, false, pl.pairs, stream);
  if (e == cudaSuccess && sums.count > 0) e = launch_reduce_parts(sums, stream);
  return launched(e);
}

swiglu_status_t zero(void* p, size_t bytes, cudaStream_t stream) {
  return launched(cudaMemsetAsync(p, 0, bytes, stream));
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
  ProductPlan grad;
  int64_t grad_full = 0;  // whole tiles; the others are taken in halves
  GradientPlan gradients;
  size_t grad_bytes = 0;  // dG (and dU) in the workspace, then the parts
  size_t bytes() const { return 2 * grad_bytes + gradients.parts_bytes(); }
};

// Tiles of dG and dU that are taken whole: all of them, or those of whole rounds
// where the last round's halves still fit one round.
int64_t grad_full_tiles(int64_t tiles, int pairs) {
  const int64_t rest = tiles % pairs;
  return 2 * rest <= pairs ? tiles - rest : tiles;
}

BackwardPlan plan_backward(int64_t M, int64_t K, int64_t N, int pairs) {
  BackwardPlan pl;
  pl.grad = plan_product(M, N, 2, k_slices(K));
  pl.grad_full = grad_full_tiles(pl.grad.tiles(), pairs);
  pl.gradients = plan_gradients(M, K, 4 * div_up(N, kTileM), K, N, 2, pairs);
  pl.grad_bytes = align256(size_t(M) * size_t(N) * 2);
  return pl;
}

// Tiles and parts of the two gradient products, as deal_units() takes them, as text.
int format_gradients(GradientPlan g, int max_pairs, char* buf, size_t buflen) {
  BackwardParams p{};
  deal_units(&g, true, true, max_pairs, &p);
  return std::snprintf(buf, buflen, "input tiles=%lld parts=%lld weight tiles=%lld parts=%lld early=%d pairs=%d",
                       static_cast<long long>(g.in.tiles()), static_cast<long long>(g.in.splits),
                       static_cast<long long>(g.w.tiles()), static_cast<long long>(g.w.splits),
                       p.early_rounds, g.pairs);
}

GradientPlan plan_down_backward(int64_t M, int64_t N, int64_t H, int pairs) {
  return plan_gradients(M, N, 4 * div_up(H, kTile), N, H, 1, pairs);
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
  if (pl.grad.units() > kMaxUnits || pl.gradients.too_many()) return SWIGLU_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* dG = ws;
  void* dU = ws + pl.grad_bytes;
  uint8_t* parts = ws + 2 * pl.grad_bytes;
  {
    BackwardParams p{};
    fill(&p.in, pl.grad, M, N, M);
    fill_status(&p, d);
    p.full_units = static_cast<int>(pl.grad_full);
    p.in_units = static_cast<int>(2 * pl.grad.tiles() - pl.grad_full);
    p.dy = dY;
    if (!encode_operand(&p.in.tmap_a0, A, M, K) ||
        !encode_packed_w(&p.in.tmap_b0, Wpacked, K, N, kPackBlockN) ||
        !encode_packed_w(&p.in.tmap_b1, Wpacked, K, N, kPackBlockN / 2) ||
        !encode_2d(&p.in.tmap_o0, dG, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_2d(&p.in.tmap_o1, dU, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return SWIGLU_ERR_CUDA;
    st = launched(launch_backward_pair(p, true, std::min(p.in_units, pairs), cs));
    if (st != SWIGLU_OK) return st;
  }
  GradientPlan g = pl.gradients;
  BackwardParams p{};
  ReduceParams sums{};
  deal_units(&g, dA != nullptr, dW1 != nullptr, pairs, &p);
  fill_status(&p, d);
  if (dA) {
    fill(&p.in, g.in, M, K, M);
    p.in.two = 1;
    p.in.col_slices = static_cast<int>(k_slices(K));
    if (!encode_operand(&p.in.tmap_a0, dG, M, N) ||
        !encode_operand(&p.in.tmap_a1, dU, M, N) ||
        !encode_packed_w(&p.in.tmap_b0, Wpacked, K, N, kPackBlockN) ||
        !encode_output(&p.in.tmap_o0, dA, parts, g.in, M, K, &sums))
      return SWIGLU_ERR_CUDA;
  }
  if (dW1) {
    uint8_t* w_parts = parts + g.in.part_bytes;
    fill(&p.w, g.w, K, N, M);
    p.w.sum = static_cast<int>(M);
    p.w.two = 1;
    if (!encode_operand(&p.w.tmap_a0, A, M, K) ||
        !encode_operand(&p.w.tmap_b0, dG, M, N) ||
        !encode_operand(&p.w.tmap_b1, dU, M, N) ||
        !encode_output(&p.w.tmap_o0, dW1, w_parts, g.w, K, N, &sums) ||
        !encode_output(&p.w.tmap_o1, dW2, w_parts + g.w.part_bytes, g.w, K, N, &sums))
      return SWIGLU_ERR_CUDA;
  }
  return run_gradients(p, g, sums, cs);
}

swiglu_status_t swiglu_backward_plan_string(int64_t M, int64_t K, int64_t N, char* buf, size_t buflen) {
  if (!buf || buflen == 0) return SWIGLU_ERR_INVALID_ARG;
  buf[0] = '\0';
  swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK) return st;
  DeviceView d;
  int pairs = 0;
  st = backward_device(&d, &pairs);
  if (st != SWIGLU_OK) return st;
  const BackwardPlan pl = plan_backward(std::max<int64_t>(M, 1), K, N, pairs);
  char rest[160];
  format_gradients(pl.gradients, pairs, rest, sizeof(rest));
  std::snprintf(buf, buflen, "backward grad whole=%lld halves=%lld %s",
                static_cast<long long>(pl.grad_full),
                static_cast<long long>(2 * (pl.grad.tiles() - pl.grad_full)), rest);
  return SWIGLU_OK;
}

swiglu_status_t swiglu_down_backward_plan_string(int64_t M, int64_t N, int64_t H, char* buf,
                                                 size_t buflen) {
  if (!buf || buflen == 0) return SWIGLU_ERR_INVALID_ARG;
  buf[0] = '\0';
  swiglu_status_t st = swg::api::check_shape(M, N, H);
  if (st != SWIGLU_OK) return st;
  DeviceView d;
  int pairs = 0;
  st = backward_device(&d, &pairs);
  if (st != SWIGLU_OK) return st;
  char rest[160];
  format_gradients(plan_down_backward(std::max<int64_t>(M, 1), N, H, pairs), pairs, rest, sizeof(rest));
  std::snprintf(buf, buflen, "down_backward %s", rest);
  return SWIGLU_OK;
}

size_t swiglu_down_backward_workspace_bytes(int64_t M, int64_t N, int64_t H) {
  if (swg::api::check_shape(M, N, H) != SWIGLU_OK || M == 0) return 0;
  DeviceView d;
  int pairs = 0;
  if (backward_device(&d, &pairs) != SWIGLU_OK) return 0;
  return plan_down_backward(M, N, H, pairs).parts_bytes();
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
  GradientPlan g = plan_down_backward(M, N, H, pairs);
  if (g.parts_bytes() > 0 && (!workspace || workspace_bytes < g.parts_bytes()))
    return SWIGLU_ERR_INVALID_ARG;
  if (g.too_many()) return SWIGLU_ERR_UNSUPPORTED;
  uint8_t* parts = static_cast<uint8_t*>(workspace);
  BackwardParams p{};
  ReduceParams sums{};
  deal_units(&g, dY != nullptr, dW3 != nullptr, pairs, &p);
  fill_status(&p, d);
  if (dY) {
    fill(&p.in, g.in, M, N, M);
    p.in.col_slices = static_cast<int>(k_slices(N));
    if (!encode_operand(&p.in.tmap_a0, dOut, M, H) ||
        !encode_packed_down(&p.in.tmap_b0, W3packed, N, H, kPackBlockN) ||
        !encode_output(&p.in.tmap_o0, dY, parts, g.in, M, N, &sums))
      return SWIGLU_ERR_CUDA;
  }
  if (dW3) {
    fill(&p.w, g.w, N, H, M);
    p.w.sum = static_cast<int>(M);
    if (!encode_operand(&p.w.tmap_a0, Y, M, N) ||
        !encode_operand(&p.w.tmap_b0, dOut, M, H) ||
        !encode_output(&p.w.tmap_o0, dW3, parts + g.in.part_bytes, g.w, N, H, &sums))
      return SWIGLU_ERR_CUDA;
  }
  return run_gradients(p, g, sums, cs);
}

}  // extern "C"
