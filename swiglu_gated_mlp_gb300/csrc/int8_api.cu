// C entry points of the projections in 8-bit integers: argument checks, plans and
// launches. Contracts are in include/swiglu.h, the mathematics and the kernel in
// int8_gemm.cu.
#include "swiglu.h"

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstdlib>
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
const int kKeepAhead = std::getenv("SWIGLU_I8_KEEP") ? 1 : 0;
const int kL2Ahead = std::getenv("SWIGLU_I8_AHEAD") ? std::atoi(std::getenv("SWIGLU_I8_AHEAD")) : 16;

struct Int8Plan {
  bool pair = false;  // units on CTA pairs, tokens widened by a kernel before
  int mt = 16, splits = 1, stages = 0, grid = 0;
  int64_t blocks = 0, mgroups = 1;
  size_t workspace(int64_t M, int64_t K) const { return pair ? size_t(M) * size_t(K) * 2 : 0; }
};

// M tokens, sums over K, N outputs.
Int8Plan make_plan(int64_t M, int64_t K, int64_t N, bool down, int sms, const Int8State& s) {
  Int8Plan pl;
  const int64_t slices = div_up(K, kBlockK8);
  const int64_t halves = div_up(N, down ? 128 : 64);  // packed blocks of 128 rows
  pl.pair = s.pairs > 0 && M > 4 * kInt8Tokens;
  const int64_t most = pl.pair ? kInt8PairTokens : kInt8Tokens, unit = pl.pair ? 32 : 16;
  pl.blocks = pl.pair ? div_up(halves, 2) : halves;
  pl.mgroups = div_up(M, most);
  pl.mt = static_cast<int>(div_up(div_up(M, pl.mgroups), unit) * unit);
  pl.stages = int8_stages(pl.mt, pl.pair);
  if (std::getenv("SWIGLU_I8_STAGES")) pl.stages = std::min(pl.stages, std::atoi(std::getenv("SWIGLU_I8_STAGES")));
  const int64_t units = pl.blocks * pl.mgroups;
  if (pl.pair) {
    pl.grid = 2 * static_cast<int>(std::min<int64_t>(units, s.pairs));
    return pl;
  }
  // K over clusters, as many CTAs as the SMs hold at once
  for (int c = 2; c <= 8; ++c)
    if (units * c <= sms && c <= slices && s.clusters[c] >= units) pl.splits = c;
  pl.grid = static_cast<int>(pl.splits > 1 ? units * pl.splits : std::min<int64_t>(units, sms));
  return pl;
}

swiglu_status_t check(int64_t M, int64_t K, int64_t N) {
  const swiglu_status_t st = swg::api::check_shape(M, K, N);
  if (st != SWIGLU_OK) return st;
  return K % 16 == 0 ? SWIGLU_OK : SWIGLU_ERR_UNSUPPORTED;  // 16-byte rows of codes
}

size_t packed_bytes(int64_t K, int64_t N, bool down) {
  const int64_t blocks = down ? div_up(N, 256) : div_up(N, 128);
  return size_t(blocks) * size_t(div_up(K, kBlockK8)) * 32768;
}

swiglu_status_t pack(const void* w1, const void* w2, void* wp, int64_t K, int64_t N, bool down,
                     swiglu_stream_t stream) {
  swiglu_status_t st = check(0, K, N);
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

size_t workspace_for(int64_t M, int64_t K, int64_t N, bool down) {
  if (check(M, K, N) != SWIGLU_OK || M == 0) return 0;
  DeviceView d;
  const Int8State* s = nullptr;
  if (int8_device(&d, &s) != SWIGLU_OK) return 0;
  return make_plan(M, K, N, down, d.sm_count, *s).workspace(M, K);
}

// One projection: x [M, K] codes -> y [M, N].
swiglu_status_t project(const void* x, const float* scale_x, const void* wp, const float* scale0,
                        const float* scale1, const void* residual, void* y, int64_t M, int64_t K, int64_t N,
                        bool down, void* workspace, size_t workspace_bytes, swiglu_stream_t stream) {
  swiglu_status_t st = check(M, K, N);
  if (st != SWIGLU_OK || M == 0) return st;
  if (!x || !scale_x || !wp || !scale0 || !scale1 || !y) return SWIGLU_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(scale_x) || !aligned16(wp) || !aligned16(scale0) || !aligned16(scale1) ||
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
  if (pl.blocks * pl.mgroups > kMaxUnits) return SWIGLU_ERR_UNSUPPORTED;
  const size_t need = pl.workspace(M, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_INVALID_ARG;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  Int8Params p{};
  p.w = wp;
  if (pl.pair) {
    if (!encode_2d(&p.tmap_x, workspace, K, M, K * 2, 64, pl.mt / 2, CU_TENSOR_MAP_SWIZZLE_128B)) return SWIGLU_ERR_CUDA;
    st = launched(launch_widen(x, workspace, size_t(M) * size_t(K), cs));
    if (st != SWIGLU_OK) return st;
  } else if (!encode_2d(&p.tmap_x, x, K, M, K, 128, pl.mt, CU_TENSOR_MAP_SWIZZLE_128B,
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
  p.group_m = static_cast<int>(std::min<int64_t>(pl.mgroups, 32));
  p.splits = pl.splits;
  p.stages = pl.stages;
  p.grid = pl.grid;
  p.l2_prefetch = pl.pair ? 2 : kL2Ahead;
  p.keep_ahead = kKeepAhead;
  p.status = d.status;
  p.timeout_ns = d.timeout_ns;
  p.inject_stall = d.inject_stall;
  return launched(launch_int8_gemm(p, down, cs));
}

swiglu_status_t plan_string(const char* what, int64_t M, int64_t K, int64_t N, bool down, char* buf, size_t buflen) {
  if (!buf || buflen == 0) return SWIGLU_ERR_INVALID_ARG;
  buf[0] = '\0';
  swiglu_status_t st = check(M, K, N);
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
  return check(0, K, N) == SWIGLU_OK ? packed_bytes(K, N, false) : 0;
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
  return check(0, N, H) == SWIGLU_OK ? packed_bytes(N, H, true) : 0;
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
