// C entry points of the projections with low-rank adapters: argument checks,
// workspace layout, launches. Contracts are in include/swiglu.h; the kernels
// are lora_shrink.cu (V), fused_small_m.cu and fused_large_m_pair.cu (kLora).
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

// Tokens of a decode CTA: one of its threads writes each token's V.
constexpr int64_t kGroupTokens = 128;

// Whether the decode kernel runs, with its work split. It takes one group of
// tokens, and more groups where 256-row pair tiles would leave the SMs idle or
// take a nearly empty round. A pair's slice takes about 0.3 us, a decode CTA's
// of 128 tokens 0.5 us (each group streams the weight; 0.6 with many groups), a K
// split 1 us. Measured, decode against pairs (in both the kernel that makes V is out
// of the way): 333 tokens of 10 adapters, K 1416 N 5000, 30.6 / 43.7 us; 200 tokens of
// 4, K 2048 N 4000 (K over 2 CTAs) 18.6 / 20.4, 500 of 3 (4 groups, K whole) 36.3 /
// 28.5; down, N 18944 H 3584, 500 tokens of 3 (K over 2) 78.9 / 92.6, 800 of 2 (7
// groups, K whole) 252 / 108; down, N 4864 H 896, 800 of 2 (7 groups, K over 4) 25.2 /
// 31.7. Where the two meet the rule is off by up to a tenth, with 8 slices and many
// adapters by a fifth (333 tokens of 10, K 512 N 2000: pairs, 24.1 / 19.2).
swiglu_status_t plan_decode(int64_t M, int64_t blocks, int64_t slices, const DeviceView& d,
                            SmallMParams* p, bool* decode) {
  const int64_t groups = (M + kGroupTokens - 1) / kGroupTokens;
  *decode = groups == 1;
  if (groups > 1 && blocks * groups > d.sm_count) return SWIGLU_OK;
  const swiglu_status_t st = decode_plan(M, blocks, slices, &p->mt, &p->mgroups, &p->stages, &p->splits);
  if (st != SWIGLU_OK || *decode || d.max_pairs < 1) return st;
  const int64_t tiles = (M + 2 * kTileM - 1) / (2 * kTileM) * blocks;
  const int64_t rounds = (tiles + d.max_pairs - 1) / d.max_pairs;
  *decode = (groups <= 4 ? 17 : 21) * slices / p->splits + (p->splits > 1 ? 40 : 0) <= 10 * rounds * slices;
  return SWIGLU_OK;
}

struct LoraState {
  std::atomic<bool> ready{false};
  swiglu_status_t status = SWIGLU_OK;
};
LoraState g_lora[kMaxDevices];
std::mutex g_lora_mu;

swiglu_status_t lora_device(DeviceView* d) {
  const swiglu_status_t st = device_view(d);
  if (st != SWIGLU_OK) return st;
  LoraState& l = g_lora[d->index];
  if (!l.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_lora_mu);
    if (!l.ready.load(std::memory_order_relaxed)) {
      if (configure_lora_shrink() != cudaSuccess || configure_small_m_lora() != cudaSuccess ||
          configure_large_m_pair_lora() != cudaSuccess) {
        cudaGetLastError();
        l.status = SWIGLU_ERR_CUDA;
      }
      l.ready.store(true, std::memory_order_release);
    }
  }
  return l.status;
}

// K parts of the tile kernel of V: as many as keep every CTA resident at once.
int shrink_splits(int64_t tiles, int64_t slices, int sm_count) {
  for (int s : {8, 4, 2})
    if (s <= slices && tiles * s <= sm_count) return s;
  return 1;
}

// Whether every decode CTA makes V itself (make_own_v()), in place of a kernel
// before it. A step there, 2 rows of V for each of 8 warps over 1024 of K, takes
// 1.5 us, a slice of weight that streams meanwhile 0.7; with more than 8000
// multiply-adds for each of those the kernel beside the stream wins. Measured, made
// inside against outside: K 896 N 4864, 7 slices a CTA, 1 token of rank 8 / 16 / 32
// (1, 2, 4 steps) 7.3 / 8.8, 8.6 / 9.1, 11.8 / 9.2 us; K 3584 N 18944, 56 slices, 1
// token of rank 8 / 32, 2 of 32 (4, 16, 32 steps) 41.0 / 43.9, 43.3 / 44.1, 44.8 / 44.7;
// down N 4864 H 896, 10 slices, 1 / 2 tokens of rank 16 (5, 10 steps) 9.3 / 9.7,
// 12.5 / 9.9; down N 18944 H 3584, 37 slices, 1 token of rank 8 / 16 (19 steps; 4100
// and 8200 multiply-adds a slice) 23.8 / 25.0, 25.9 / 24.8.
bool own_v(bool decode, int64_t M, int64_t hr, int64_t in, int splits) {
  if (!decode || M > 16 || M * hr > kLoraOwnValues) return false;
  const int64_t steps = ((M * hr + 15) / 16) * ((in + 1023) / 1024);
  const int64_t slices = (k_slices(in) + splits - 1) / splits;
  return steps <= 2 || (9 * steps <= 5 * slices && M * hr * in <= 8000 * slices);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// V, then (many tokens) the lists of adapters present.
size_t v_bytes(int64_t M, int64_t hr) { return align256(size_t(M) * size_t(hr) * 2); }

size_t workspace_bytes_for(int64_t M, int64_t hr) {
  size_t n = v_bytes(M, hr);
  if (M > kGroupTokens) n += size_t(div_up(M, 2 * kTileM)) * kLoraListInts * sizeof(int);
  return n;
}

swiglu_status_t check_rank(int64_t rank) {
  if (rank <= 0) return SWIGLU_ERR_INVALID_ARG;
  return rank % 8 == 0 && rank <= kLoraMaxRank ? SWIGLU_OK : SWIGLU_ERR_UNSUPPORTED;
}

int64_t weight_blocks(bool down, int64_t outs) {
  return down ? padded_h(outs) / 256 : padded_n(outs) / kPackBlockN;
}

// One projection with adapters: x [M, in] -> out [M, outs], `halves` = 2 for
// gate and up, 1 for the down-projection (with the residual).
struct Call {
  const void* x;
  const void* wp;
  const void* residual;
  void* out;
  int64_t M, in, outs;
  const void* la;
  const void* lb;
  const int32_t* index;
  const float* scale;
  int64_t count, rank;
  void* ws;
  size_t ws_bytes;
  int halves;
};

swiglu_status_t check_call(const Call& c) {
  swiglu_status_t st = api::check_shape(c.M, c.in, c.outs);
  if (st != SWIGLU_OK) return st;
  st = check_rank(c.rank);
  if (st != SWIGLU_OK) return st;
  if (c.count < 0) return SWIGLU_ERR_INVALID_ARG;
  // adapter rows are tensor-map coordinates
  if (c.count > 2147483647 || c.count * c.rank * c.halves > 2147483647) return SWIGLU_ERR_UNSUPPORTED;
  if (c.M == 0) return SWIGLU_OK;
  if (!c.x || !c.wp || !c.out || !aligned16(c.x) || !aligned16(c.wp) || !aligned16(c.out) ||
      (c.residual && !aligned16(c.residual)))
    return SWIGLU_ERR_INVALID_ARG;
  const size_t x_bytes = size_t(c.M) * size_t(c.in) * 2, o_bytes = size_t(c.M) * size_t(c.outs) * 2;
  const size_t w_bytes = c.halves == 2 ? swiglu_packed_weight_bytes(c.in, c.outs)
                                       : swiglu_down_packed_bytes(c.in, c.outs);
  // the residual may be the output itself (in place); nothing else overlaps it
  if (overlaps(c.out, o_bytes, c.x, x_bytes) || overlaps(c.out, o_bytes, c.wp, w_bytes) ||
      (c.residual && c.residual != c.out && overlaps(c.out, o_bytes, c.residual, o_bytes)))
    return SWIGLU_ERR_INVALID_ARG;
  if (c.count == 0) return SWIGLU_OK;
  if (!c.la || !c.lb || !c.index || !c.scale || !c.ws || !aligned16(c.la) || !aligned16(c.lb) ||
      !aligned16(c.ws) || (reinterpret_cast<uintptr_t>(c.index) & 3u) ||
      (reinterpret_cast<uintptr_t>(c.scale) & 3u) ||
      c.ws_bytes < workspace_bytes_for(c.M, c.rank * c.halves))
    return SWIGLU_ERR_INVALID_ARG;
  const size_t rows = size_t(c.count) * size_t(c.rank) * size_t(c.halves) * 2;
  const struct { const void* p; size_t n; } in[] = {
      {c.la, rows * size_t(c.in)}, {c.lb, rows * size_t(c.outs)}, {c.index, size_t(c.M) * 4},
      {c.scale, size_t(c.count) * 4}, {c.x, x_bytes}, {c.wp, w_bytes}, {c.residual, o_bytes}};
  for (int i = 0; i < 7; ++i) {
    if (!in[i].p) continue;
    if (overlaps(c.ws, c.ws_bytes, in[i].p, in[i].n)) return SWIGLU_ERR_INVALID_ARG;
    if (i < 4 && overlaps(c.out, o_bytes, in[i].p, in[i].n)) return SWIGLU_ERR_INVALID_ARG;
  }
  return overlaps(c.ws, c.ws_bytes, c.out, o_bytes) ? SWIGLU_ERR_INVALID_ARG : SWIGLU_OK;
}

swiglu_status_t run_call(const Call& c, cudaStream_t stream) {
  DeviceView d;
  swiglu_status_t st = lora_device(&d);
  if (st != SWIGLU_OK) return st;
  const bool down = c.halves == 1;
  const int64_t blocks = weight_blocks(down, c.outs);
  const int hr = static_cast<int>(c.rank * c.halves);
  const int64_t slices = k_slices(c.in);
  SmallMParams dp{};
  bool decode = false;
  st = plan_decode(c.M, blocks, slices, d, &dp, &decode);
  if (st != SWIGLU_OK) return st;
  int* lists = reinterpret_cast<int*>(static_cast<uint8_t*>(c.ws) + v_bytes(c.M, hr));

  LoraShrinkParams sp{};  // for V, unless the decode CTAs make it
  sp.x = c.x;
  sp.la = c.la;
  sp.index = c.index;
  sp.scale = c.scale;
  sp.count = static_cast<int>(c.count);
  sp.M = static_cast<int>(c.M);
  sp.K = static_cast<int>(c.in);
  sp.hr = hr;
  sp.v = c.ws;
  sp.status = d.status;
  sp.timeout_ns = d.timeout_ns;
  sp.inject_stall = d.inject_stall;
  if (c.M > kGroupTokens) {
    sp.lists = lists;
    sp.tiles = static_cast<int>(div_up(c.M, kTileM));
    sp.slices = static_cast<int>(slices);
    sp.rb = (hr + 15) / 16 * 16;
    sp.per_pass = 256 / sp.rb;
    sp.splits = shrink_splits(sp.tiles, slices, d.sm_count);
    if (!encode_2d(&sp.tmap_x, c.x, c.in, c.M, c.in * 2, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&sp.tmap_la, c.la, c.in, uint64_t(c.count) * hr, c.in * 2, kBlockK, sp.rb,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return SWIGLU_ERR_CUDA;
  }
  // Lb rows of one half of one adapter: the decode kernel takes 128 of them at a
  // time, each CTA of a pair 64 gate or up rows or 128 output columns
  const uint64_t lb_dims[3] = {uint64_t(c.rank), uint64_t(c.outs), uint64_t(c.count * c.halves)};
  const uint64_t lb_strides[2] = {uint64_t(c.rank) * 2, uint64_t(c.rank) * uint64_t(c.outs) * 2};
  const uint32_t lb_box[3] = {kBlockK, decode || down ? 128u : 64u, 1u};
  CUtensorMap tmap_lb;
  if (!encode_3d(&tmap_lb, c.lb, lb_dims, lb_strides, lb_box, CU_TENSOR_MAP_SWIZZLE_128B))
    return SWIGLU_ERR_CUDA;
  cudaError_t e;
  if (decode) {
    SmallMParams& p = dp;
    if (!encode_2d(&p.tmap_x, c.x, c.in, c.M, c.in * 2, kBlockK, p.mt, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !(down ? encode_packed_down(&p.tmap_w, c.wp, c.in, c.outs, 256)
               : encode_packed_w(&p.tmap_w, c.wp, c.in, c.outs, 2 * kPackBlockN)))
      return SWIGLU_ERR_CUDA;
    p.y = c.out;
    p.residual = c.residual;
    p.down = down;
    p.M = static_cast<int>(c.M);
    p.K = static_cast<int>(c.in);
    p.N = static_cast<int>(c.outs);
    p.grid = static_cast<int>(blocks * p.mgroups * p.splits);
    p.lora = 1;
    p.lora_rank = static_cast<int>(c.rank);
    p.lora_count = static_cast<int>(c.count);
    p.lora_v = c.ws;
    p.lora_lb = c.lb;
    p.lora_index = c.index;
    p.tmap_lb = tmap_lb;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    p.inject_stall = d.inject_stall;
    p.lora_own_v = own_v(decode, c.M, hr, c.in, p.splits);
    p.lora_x = c.x;
    p.lora_la = c.la;
    p.lora_scale = c.scale;
    e = p.lora_own_v ? cudaSuccess : launch_lora_shrink(sp, stream);
    if (e == cudaSuccess) e = launch_small_m(p, stream);
  } else {
    LargeMParams p{};
    const int64_t tiles_m = div_up(c.M, 2 * kTileM);
    const int64_t tiles_n = blocks;
    if (d.max_pairs < 1 || tiles_m * tiles_n > 2147483647) return SWIGLU_ERR_UNSUPPORTED;
    if (!(down ? encode_packed_down(&p.tmap_w, c.wp, c.in, c.outs, kPackBlockN)
               : encode_packed_w(&p.tmap_w, c.wp, c.in, c.outs, kPackBlockN)) ||
        !encode_2d(&p.tmap_y, c.out, c.outs, c.M, c.outs * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return SWIGLU_ERR_CUDA;
    p.tmap_lb = tmap_lb;
    p.tmap_a = sp.tmap_x;
    p.M = static_cast<int>(c.M);
    p.K = static_cast<int>(c.in);
    p.N = static_cast<int>(c.outs);
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles_n = static_cast<int>(tiles_n);
    p.group_m = static_cast<int>(pair_group_rows(tiles_m));
    p.bn = kPackBlockN;
    p.grid = 2 * static_cast<int>(std::min<int64_t>(tiles_m * tiles_n, d.max_pairs));
    p.down = down;
    p.residual = c.residual;
    p.lora = 1;
    p.lora_rank = static_cast<int>(c.rank);
    p.lora_count = static_cast<int>(c.count);
    p.lora_v = c.ws;
    p.lora_lb = c.lb;
    p.lora_index = c.index;
    p.lora_lists = lists;
    // Where both grids fit on the SMs together V takes no time of its own (down, 333
    // tokens of 10 adapters, N 18944, H 3584: 174 -> 98 us). Where they do not, some pairs
    // start before others: 4096 tokens, K 3584 645 -> 630 us, but with long tiles, which
    // then share less of L2, 350 -> 358 us (down, N 18944).
    p.lora_early = sp.tiles * sp.splits + p.grid <= d.sm_count || slices < 128;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    p.inject_stall = d.inject_stall;
    e = launch_lora_shrink(sp, stream);
    if (e == cudaSuccess) e = launch_large_m_pair(p, stream);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SWIGLU_ERR_CUDA;
  }
  return SWIGLU_OK;
}

swiglu_status_t lora_plan(int64_t M, int64_t in, int64_t outs, int64_t rank, bool down, char* buf,
                          size_t buflen) {
  if (!buf || buflen == 0) return SWIGLU_ERR_INVALID_ARG;
  buf[0] = '\0';
  swiglu_status_t st = api::check_shape(M, in, outs);
  if (st == SWIGLU_OK) st = check_rank(rank);
  if (st != SWIGLU_OK) return st;
  DeviceView d;
  st = lora_device(&d);
  if (st != SWIGLU_OK) return st;
  M = std::max<int64_t>(M, 1);
  const int64_t blocks = weight_blocks(down, outs), slices = k_slices(in);
  SmallMParams p{};
  bool decode = false;
  st = plan_decode(M, blocks, slices, d, &p, &decode);
  if (st != SWIGLU_OK) return st;
  const int64_t tiles = div_up(M, kTileM), hr = down ? rank : 2 * rank;
  char shrink[64];
  if (own_v(decode, M, hr, in, p.splits))
    std::snprintf(shrink, sizeof(shrink), "inside");
  else if (M <= kGroupTokens)
    std::snprintf(shrink, sizeof(shrink), "dots=%lld", static_cast<long long>(M * div_up(hr, 4)));
  else
    std::snprintf(shrink, sizeof(shrink), "tiles=%lld parts=%d", static_cast<long long>(tiles),
                  shrink_splits(tiles, slices, d.sm_count));
  if (decode)
    std::snprintf(buf, buflen, "%slora shrink %s small_m mt=%d stages=%d blocks=%lld groups=%d splits=%d",
                  down ? "down " : "", shrink, p.mt, p.stages, static_cast<long long>(blocks), p.mgroups,
                  p.splits);
  else
    std::snprintf(buf, buflen, "%slora shrink %s large_m_pair tiles=%lld max_pairs=%d", down ? "down " : "",
                  shrink, static_cast<long long>(div_up(M, 2 * kTileM) * blocks), d.max_pairs);
  return SWIGLU_OK;
}

size_t lora_workspace(int64_t M, int64_t in, int64_t outs, int64_t hr, int64_t rank) {
  if (api::check_shape(M, in, outs) != SWIGLU_OK || check_rank(rank) != SWIGLU_OK) return 0;
  return workspace_bytes_for(M, hr);
}

}  // namespace

extern "C" {

size_t swiglu_lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t rank) {
  return lora_workspace(M, K, N, 2 * rank, rank);
}

swiglu_status_t swiglu_forward_lora(const void* A, const void* Wpacked, void* Y, int64_t M, int64_t K,
                                    int64_t N, const void* La, const void* Lb, const int32_t* index,
                                    const float* scale, int64_t adapters, int64_t rank,
                                    void* workspace, size_t workspace_bytes, swiglu_stream_t stream) {
  const Call c{A,  Wpacked, nullptr, Y, M, K, N, La, Lb, index, scale, adapters, rank,
               workspace, workspace_bytes, 2};
  const swiglu_status_t st = check_call(c);
  if (st != SWIGLU_OK || M == 0) return st;
  if (adapters == 0) return swiglu_forward(A, Wpacked, Y, M, K, N, stream);
  return run_call(c, reinterpret_cast<cudaStream_t>(stream));
}

swiglu_status_t swiglu_lora_plan_string(int64_t M, int64_t K, int64_t N, int64_t rank, char* buf,
                                        size_t buflen) {
  return lora_plan(M, K, N, rank, false, buf, buflen);
}

swiglu_status_t swiglu_down_lora_plan_string(int64_t M, int64_t N, int64_t H, int64_t rank, char* buf,
                                             size_t buflen) {
  return lora_plan(M, N, H, rank, true, buf, buflen);
}

size_t swiglu_down_lora_workspace_bytes(int64_t M, int64_t N, int64_t H, int64_t rank) {
  return lora_workspace(M, N, H, rank, rank);
}

swiglu_status_t swiglu_down_forward_lora(const void* Y, const void* W3packed, const void* R, void* Out,
                                         int64_t M, int64_t N, int64_t H, const void* La,
                                         const void* Lb, const int32_t* index, const float* scale,
                                         int64_t adapters, int64_t rank, void* workspace,
                                         size_t workspace_bytes, swiglu_stream_t stream) {
  const Call c{Y, W3packed, R, Out, M, N, H, La, Lb, index, scale, adapters, rank,
               workspace, workspace_bytes, 1};
  const swiglu_status_t st = check_call(c);
  if (st != SWIGLU_OK || M == 0) return st;
  if (adapters == 0) return swiglu_down_forward(Y, W3packed, R, Out, M, N, H, stream);
  return run_call(c, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
