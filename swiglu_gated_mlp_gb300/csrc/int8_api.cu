// C entry points of the projections in 8-bit integers: argument checks, plans and
// launches. Contracts are in include/swiglu.h, the mathematics and the kernel in
// int8_gemm.cu.
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

struct Int8State {
  std::atomic<bool> ready{false};
  swiglu_status_t status = SWIGLU_OK;
  int clusters[9] = {};
  int pairs = 0;
};
Int8State g_int8[kMaxDevices];
std::mutex g_int8_mu;

swiglu_status_t int8_device(DeviceView* d, const Int8State** out) {
  const swiglu_status_t st = device_view(d);
  if (st != SWIGLU_OK) return st;
  Int8State& s = g_int8[d->index];
  if (!s.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_int8_mu);
    if (!s.ready.load(std::memory_order_relaxed)) {
      if (configure_int8(s.clusters, &s.pairs) != cudaSuccess) {
        cudaGetLastError();
        s.status = SWIGLU_ERR_CUDA;
      }
      s.ready.store(true, std::memory_order_release);
    }
  }
  *out = &s;
  return s.status;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxUnits = 1 << 30;
struct Int8Plan {
  bool pair = false;  // units on CTA pairs, tokens widened by a kernel before
  int mt = 16, splits = 1, stages = 0, grid = 0;
  int64_t blocks = 0, mgroups = 1, group_m = 1;
  size_t workspace(int64_t M, int64_t K) const { return pair ? size_t(M) * size_t(K) * 2 : 0; }
};

// What launches take, in units of 2 ns, from measurements at 16 to 4096 tokens: a stage (128 of
// K) of a unit, and all that comes before and after the stages (on pairs the kernel that widens
// the tokens too). Stages are bound by the MMAs from about 140 tokens, else by their hand-overs.
int64_t cta_stage(int64_t mt) { return 160 + mt * 4 / 3; }
int64_t pair_stage(int64_t mt) { return std::max<int64_t>(172, mt + 32); }
constexpr int64_t kCtaOnce = 2400, kPairOnce = 3600;

// One CTA a unit: groups of at most 64 tokens, K over clusters, as many CTAs as the SMs hold at once.
Int8Plan cta_plan(int64_t M, int64_t slices, int64_t halves, int sms, const Int8State& s, int64_t* cost) {
  Int8Plan pl;
  pl.blocks = halves;
  pl.mgroups = div_up(M, kInt8Tokens);
  pl.mt = static_cast<int>(div_up(div_up(M, pl.mgroups), 16) * 16);
  pl.group_m = std::min<int64_t>(pl.mgroups, 32);
  pl.stages = int8_stages(pl.mt, false);
  const int64_t units = pl.blocks * pl.mgroups;
  for (int c = 2; c <= 8; ++c)
    if (units * c <= sms && c <= slices && s.clusters[c] >= units) pl.splits = c;
  pl.grid = static_cast<int>(pl.splits > 1 ? units * pl.splits : std::min<int64_t>(units, sms));
  *cost = div_up(units, sms) * div_up(slices, pl.splits) * cta_stage(pl.mt) + kCtaOnce;
  return pl;
}

// CTA pairs: the tokens of a unit that make the rounds of all units shortest.
Int8Plan pair_plan(int64_t M, int64_t K, int64_t slices, int64_t halves, const Int8State& s, int64_t* cost) {
  Int8Plan pl;
  pl.pair = true;
  pl.blocks = div_up(halves, 2);
  *cost = INT64_MAX;
  for (int64_t mt = 32; mt <= kInt8PairTokens; mt += 16) {
    const int64_t c = div_up(pl.blocks * div_up(M, mt), s.pairs) * slices * pair_stage(mt) + kPairOnce;
    if (c > *cost) continue;
    *cost = c;
    pl.mgroups = div_up(M, mt);
  }
  pl.mt = static_cast<int>(std::max<int64_t>(32, div_up(div_up(M, pl.mgroups), 16) * 16));
  // token groups whose values stay in L2 (half of it) while the columns go by; at 4096 tokens: K
  // 18944 all 26 groups at once 335 us, 9 of them 327; K 3584 6 groups 552, 11 540, all 22 532
  pl.group_m = std::clamp<int64_t>((int64_t(64) << 20) / (pl.mt * K * 2), 1, std::min<int64_t>(pl.mgroups, 32));
  pl.stages = int8_stages(pl.mt, true);
  pl.grid = 2 * static_cast<int>(std::min<int64_t>(pl.blocks * pl.mgroups, s.pairs));
  return pl;
}

// M tokens, sums over K, N outputs. Measured, CTAs / pairs (us): K 896 N 4864, 128 tokens 7.1 / 8.2,
// 256 11.9 / 10.3; K 3584 N 18944, 80 tokens 56 / 27; down, N 18944 H 3584, 128 tokens 38 / 53, 256
// 71 / 56; N 4864 H 896, 512 tokens 13.4 / 20.3, 1000 21.2 / 21.8.
Int8Plan make_plan(int64_t M, int64_t K, int64_t N, bool down, int sms, const Int8State& s) {
  const int64_t slices = div_up(K, kBlockK8);
  const int64_t halves = div_up(N, down ? 128 : 64);  // packed blocks of 128 rows
  int64_t cta_cost = 0, pair_cost = 0;
  const Int8Plan on_ctas = cta_plan(M, slices, halves, sms, s, &cta_cost);
  if (s.pairs < 1) return on_ctas;
  // rows of codes that do not start on 16 bytes cannot be loaded as such: widened first, they do
  const bool by_rows = K % 16 == 0;
  const Int8Plan on_pairs = pair_plan(M, K, slices, halves, s, &pair_cost);
  return !by_rows || pair_cost < cta_cost ? on_pairs : on_ctas;
}

size_t packed_bytes(int64_t K, int64_t N, bool down) {
  const int64_t blocks = down ? div_up(N, 256) : div_up(N, 128);
  return size_t(blocks) * size_t(div_up(K, kBlockK8)) * 32768;
}

swiglu_status_t pack(const void* w1, const void* w2, void* wp, int64_t K, int64_t N, bool down,
                     swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(0, K, N);
  if (st != SWIGLU_OK) return st;
  if (!w1 || !w2 || !wp) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(w1) || !aligned16(w2) || !aligned16(wp)) return SWIGLU_ERR_INVALID_ARG;
  const size_t w_bytes = size_t(K) * size_t(N);
  const Span in[2] = {{w1, w_bytes}, {w2, w_bytes}}, out[1] = {{wp, packed_bytes(K, N, down)}};
  if (any_overlap(out, 1, in, 2)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  st = device_view(&d);
  if (st != SWIGLU_OK) return st;
  return launched(launch_pack_int8(w1, w2, wp, static_cast<int>(K), static_cast<int>(N), down,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

// Whether calls of M tokens or fewer take pairs. Their rounds, and the tokens of a CTA's unit, are
// whole numbers, so a batch may go back to single CTAs where a smaller one took pairs (down, K 464, N
// 9808: pairs at 97 tokens, CTAs at some more). What CTAs take is constant up to the next change of a unit's
// tokens, what pairs take never falls with M: the first M of each such range decides it. More than
// kManyTokens count as pairs without a look.
constexpr int64_t kManyTokens = 4096;
bool pairs_up_to(int64_t M, int64_t K, int64_t N, bool down, int sms, const Int8State& s) {
  if (M > kManyTokens) return s.pairs >= 1;
  for (int64_t m = 1; m <= M;) {
    const Int8Plan pl = make_plan(m, K, N, down, sms, s);
    if (pl.pair) return true;
    m = std::min(kInt8Tokens * pl.mgroups, pl.mt * pl.mgroups) + 1;
  }
  return false;
}

// What calls of up to M tokens need, so that one workspace serves every smaller batch.
size_t workspace_for(int64_t M, int64_t K, int64_t N, bool down) {
  if (swg::api::check_shape(M, K, N) != SWIGLU_OK || M == 0) return 0;
  DeviceView d;
  const Int8State* s = nullptr;
  if (int8_device(&d, &s) != SWIGLU_OK) return 0;
  return pairs_up_to(M, K, N, down, d.sm_count, *s) ? size_t(M) * size_t(K) * 2 : 0;
}

// One projection: x [M, K] codes -> y [M, N].
swiglu_status_t project(const void* x, const float* scale_x, const void* wp, const float* scale0,
                        const float* scale1, const void* residual, void* y, int64_t M, int64_t K, int64_t N,
                        bool down, void* workspace, size_t workspace_bytes, swiglu_stream_t stream) {
  swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK || M == 0) return st;
  if (!x || !scale_x || !wp || !scale0 || !scale1 || !y) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned4(scale_x) || !aligned16(wp) || !aligned16(scale0) || !aligned16(scale1) ||
      !aligned16(y) || (residual && !aligned16(residual)) || (workspace && !aligned16(workspace)))
    return SWIGLU_ERR_INVALID_ARG;
  const size_t y_bytes = size_t(M) * size_t(N) * 2;
  const Span in[6] = {{x, size_t(M) * size_t(K)},
                      {scale_x, size_t(M) * 4},
                      {wp, packed_bytes(K, N, down)},
                      {scale0, size_t(N) * 4},
                      {scale1, size_t(N) * 4},
                      {residual == y ? nullptr : residual, y_bytes}};  // in place is allowed
  const Span out[2] = {{y, y_bytes}, {workspace, workspace_bytes}};
  if (any_overlap(out, 2, in, 6)) return SWIGLU_ERR_INVALID_ARG;
  DeviceView d;
  const Int8State* s = nullptr;
  st = int8_device(&d, &s);
  if (st != SWIGLU_OK) return st;
  const Int8Plan pl = make_plan(M, K, N, down, d.sm_count, *s);
  if (pl.blocks * pl.mgroups > kMaxUnits || (!pl.pair && K % 16 != 0)) return SWIGLU_ERR_UNSUPPORTED;
  const size_t need = pl.workspace(M, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_INVALID_ARG;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  Int8Params p{};
  p.w = wp;
  const uint32_t box = static_cast<uint32_t>(pl.pair ? pl.mt / 2 : pl.mt);
  if (pl.pair) {
    if (!encode_2d(&p.tmap_x, workspace, K, M, K * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B)) return SWIGLU_ERR_CUDA;
    st = launched(launch_widen(x, workspace, size_t(M) * size_t(K), cs));
    if (st != SWIGLU_OK) return st;
  } else if (!encode_2d(&p.tmap_x, x, K, M, K, 128, box, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_DATA_TYPE_UINT8)) {
    return SWIGLU_ERR_CUDA;
  }
  p.y = y;
  p.residual = residual;
  p.scale_x = scale_x;
  p.scale0 = scale0;
  p.scale1 = scale1;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.pair = pl.pair ? 1 : 0;
  p.blocks = static_cast<int>(pl.blocks);
  p.mt = pl.mt;
  p.mgroups = static_cast<int>(pl.mgroups);
  p.group_m = static_cast<int>(pl.group_m);
  p.splits = pl.splits;
  p.stages = pl.stages;
  p.grid = pl.grid;
  p.status = d.status;
  p.timeout_ns = d.timeout_ns;
  p.inject_stall = d.inject_stall;
  return launched(launch_int8_gemm(p, down, cs));
}

swiglu_status_t plan_string(const char* what, int64_t M, int64_t K, int64_t N, bool down, char* buf, size_t buflen) {
  if (!buf || buflen == 0) return SWIGLU_ERR_INVALID_ARG;
  buf[0] = '\0';
  swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK) return st;
  DeviceView d;
  const Int8State* s = nullptr;
  st = int8_device(&d, &s);
  if (st != SWIGLU_OK) return st;
  const Int8Plan pl = make_plan(std::max<int64_t>(M, 1), K, N, down, d.sm_count, *s);
  std::snprintf(buf, buflen, "%s %s mt=%d groups=%lld blocks=%lld splits=%d stages=%d grid=%d", what,
                pl.pair ? "pairs" : "ctas", pl.mt, static_cast<long long>(pl.mgroups),
                static_cast<long long>(pl.blocks), pl.splits, pl.stages, pl.grid);
  return SWIGLU_OK;
}

}  // namespace

extern "C" {

size_t swiglu_packed_weight_bytes_int8(int64_t K, int64_t N) {
  return swg::api::check_shape(0, K, N) == SWIGLU_OK ? packed_bytes(K, N, false) : 0;
}

swiglu_status_t swiglu_pack_weights_int8(const void* W1, const void* W2, void* Wpacked, int64_t K, int64_t N,
                                         swiglu_stream_t stream) {
  return pack(W1, W2, Wpacked, K, N, false, stream);
}

size_t swiglu_int8_workspace_bytes(int64_t M, int64_t K, int64_t N) { return workspace_for(M, K, N, false); }

swiglu_status_t swiglu_forward_int8(const void* A, const float* scale_a, const void* Wpacked, const float* scale_w1,
                                    const float* scale_w2, void* Y, int64_t M, int64_t K, int64_t N,
                                    void* workspace, size_t workspace_bytes, swiglu_stream_t stream) {
  return project(A, scale_a, Wpacked, scale_w1, scale_w2, nullptr, Y, M, K, N, false, workspace, workspace_bytes,
                 stream);
}

swiglu_status_t swiglu_plan_string_int8(int64_t M, int64_t K, int64_t N, char* buf, size_t buflen) {
  return plan_string("int8", M, K, N, false, buf, buflen);
}

size_t swiglu_down_packed_bytes_int8(int64_t N, int64_t H) {
  return swg::api::check_shape(0, N, H) == SWIGLU_OK ? packed_bytes(N, H, true) : 0;
}

swiglu_status_t swiglu_pack_down_weights_int8(const void* W3, void* W3packed, int64_t N, int64_t H,
                                              swiglu_stream_t stream) {
  return pack(W3, W3, W3packed, N, H, true, stream);
}

size_t swiglu_down_int8_workspace_bytes(int64_t M, int64_t N, int64_t H) { return workspace_for(M, N, H, true); }

swiglu_status_t swiglu_down_forward_int8(const void* Y, const float* scale_y, const void* W3packed,
                                         const float* scale_w3, const void* R, void* Out, int64_t M, int64_t N,
                                         int64_t H, void* workspace, size_t workspace_bytes,
                                         swiglu_stream_t stream) {
  return project(Y, scale_y, W3packed, scale_w3, scale_w3, R, Out, M, N, H, true, workspace, workspace_bytes, stream);
}

swiglu_status_t swiglu_down_plan_string_int8(int64_t M, int64_t N, int64_t H, char* buf, size_t buflen) {
  return plan_string("down_int8", M, N, H, true, buf, buflen);
}

}  // extern "C"
