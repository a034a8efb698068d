// The C ABI of include/moe.h: host-side argument checks, workspace carving
// and the launch sequence of the layer on the caller's stream.  Nothing here
// allocates device memory or synchronises, except moe_device_status.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe.h"
#include "common.cuh"
#include "host_guard.cuh"
#include "kernels.cuh"

namespace moe {

int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

int device_smem_per_block() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 227 * 1024;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess || n <= 0)
    return 227 * 1024;
  return n;
}

// Router kernel choice: with many experts the router is a real GEMM
// (2*T*d*E flops: 30 GFLOP for T=8192, d=7168, E=256) and runs on the tensor
// cores with the top-k fused into the epilogue; with few experts (or fp32,
// which must not use TF32) W_r fits in shared memory and a warp per token on
// the CUDA cores is cheaper than a 128-token tensor tile; a decode-sized batch
// (at most 64 tokens) gets a block per token on the CUDA cores either way.
cudaError_t launch_router_topk(const RouterArgs& a, cudaStream_t stream) {
  if (router_uses_tc(a.bf16, a.E, a.T)) return launch_router_topk_tc(a, stream);
  return launch_router_topk_simt(a, stream);
}

moe_status check_config(const moe_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->d_model <= 0 || c->d_ff <= 0 || c->n_experts <= 0 || c->top_k <= 0) return MOE_ERR_INVALID_ARG;
  if (c->d_model % 8 != 0 || c->d_ff % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (c->top_k > c->n_experts) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->gating < MOE_SOFTMAX_ALL_RENORM || c->gating > MOE_SOFTMAX_ALL_NO_RENORM) return MOE_ERR_INVALID_ARG;
  if (c->expert_act != MOE_ACT_SWIGLU && c->expert_act != MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
  if (!(c->capacity_factor >= 0.0f) || std::isinf(c->capacity_factor)) return MOE_ERR_INVALID_ARG;
  if (c->bias_select_only != 0 && c->bias_select_only != 1) return MOE_ERR_INVALID_ARG;
  if (c->wait_limit_ns < 0) return MOE_ERR_INVALID_ARG;
  if (c->weight_format != MOE_W_NATIVE && c->weight_format != MOE_W_E4M3) return MOE_ERR_INVALID_ARG;
  // 8-bit experts: bf16 activations; rows of 8-bit codes must be whole 16-byte lines
  if (c->weight_format == MOE_W_E4M3 &&
      (c->dtype != MOE_BF16 || c->d_model % 16 != 0 || c->d_ff % 16 != 0 ||
       (c->n_shared > 0 && c->d_ff_shared % 16 != 0)))
    return MOE_ERR_UNSUPPORTED;
  if (c->n_shared < 0) return MOE_ERR_INVALID_ARG;
  if (c->n_shared > 0 && (c->d_ff_shared <= 0 || c->d_ff_shared % 8 != 0)) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > kMaxExperts || c->top_k > kMaxTopK || c->n_shared > 1) return MOE_ERR_UNSUPPORTED;
  if (c->T * (int64_t)c->top_k >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  // tensor-map row coordinates are 32-bit
  if ((int64_t)c->n_experts * 2 * c->d_ff >= (int64_t(1) << 31) ||
      (int64_t)c->n_experts * c->d_model >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

namespace {

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t elem_bytes(const moe_config* c) { return c->dtype == MOE_BF16 ? 2 : 4; }

// Rows each expert keeps: ceil(T*k/E * capacity_factor) in double, at most T
// (no expert is chosen twice by one token); T*k when dropless.
int64_t capacity_rows(const moe_config* c) {
  if (c->capacity_factor == 0.0f) return c->T * c->top_k;
  const double cap = std::ceil((double)(c->T * c->top_k) / (double)c->n_experts * (double)c->capacity_factor);
  return cap >= (double)c->T ? c->T : (int64_t)cap;
}

struct Carve {
  int* status;
  int32_t *ids, *counts, *offsets, *perm, *row_of, *chunk_counts;
  float* w;
  void *x_perm, *h, *y_perm, *h_s, *y_s;
  float* partial;           // decode split-K partial tiles (bf16 decode regime only)
  int64_t partial_slots;
  int* counters;
  int64_t counter_cap;
  float* aux_part;          // router penalty partial sums [kAuxMaxBlocks][E + 1]
  // 8-bit experts: E4M3 codes and per-row scales of x_perm, h and the shared
  // expert's x and h
  uint8_t *xq, *hq, *xq_s, *hq_s;
  float *sx, *sh, *sx_s, *sh_s;
  size_t total;
};

// Does this config run its routed / shared experts on the decode kernel?
bool decode_routed(const moe_config* c) {
  return c->dtype == MOE_BF16 && use_decode_ffn(c->T * c->top_k, c->n_experts, true);
}
bool decode_shared(const moe_config* c) {
  return c->dtype == MOE_BF16 && c->n_shared > 0 && use_decode_ffn(c->T, 1, false);
}

// Lay out the workspace; with base == nullptr only sizes are computed.
Carve carve(const moe_config* c, void* base) {
  Carve k{};
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    void* p = b ? b + off : nullptr;
    off += up(bytes);
    return p;
  };
  const int64_t n = c->T * c->top_k;
  const size_t eb = elem_bytes(c);
  k.status = static_cast<int*>(take(16));
  k.ids = static_cast<int32_t*>(take(sizeof(int32_t) * n));
  k.w = static_cast<float*>(take(sizeof(float) * n));
  k.counts = static_cast<int32_t*>(take(sizeof(int32_t) * c->n_experts));
  k.offsets = static_cast<int32_t*>(take(sizeof(int32_t) * (c->n_experts + 1)));
  k.perm = static_cast<int32_t*>(take(sizeof(int32_t) * n));
  k.row_of = static_cast<int32_t*>(take(sizeof(int32_t) * n));
  k.chunk_counts = static_cast<int32_t*>(take(sizeof(int32_t) * (size_t)c->n_experts * permute_n_chunks(n)));
  // with 8-bit experts moe_forward gathers E4M3 codes (xq) and no bf16 copy
  k.x_perm = take(c->weight_format == MOE_W_E4M3 ? 0 : eb * n * c->d_model);
  k.h = take(eb * n * c->d_ff);
  k.y_perm = take(eb * n * c->d_model);
  if (c->n_shared > 0) {
    k.h_s = take(eb * c->T * c->d_ff_shared);
    k.y_s = take(eb * c->T * c->d_model);
  }
  k.aux_part = static_cast<float*>(take(sizeof(float) * (size_t)kAuxMaxBlocks * (c->n_experts + 1)));
  if (c->weight_format == MOE_W_E4M3) {
    k.xq = static_cast<uint8_t*>(take((size_t)n * c->d_model));
    k.sx = static_cast<float*>(take(sizeof(float) * n));
    k.hq = static_cast<uint8_t*>(take((size_t)n * c->d_ff));
    k.sh = static_cast<float*>(take(sizeof(float) * n));
    if (c->n_shared > 0) {
      k.xq_s = static_cast<uint8_t*>(take((size_t)c->T * c->d_model));
      k.sx_s = static_cast<float*>(take(sizeof(float) * c->T));
      k.hq_s = static_cast<uint8_t*>(take((size_t)c->T * c->d_ff_shared));
      k.sh_s = static_cast<float*>(take(sizeof(float) * c->T));
    }
  }
  if (decode_routed(c) || decode_shared(c)) {
    k.partial_slots = decode_partial_slots();
    k.partial = static_cast<float*>(take(sizeof(float) * 128 * kDecodeTokens * (size_t)k.partial_slots));
    k.counter_cap = std::max(decode_counter_cap(n, c->n_experts, c->d_model, c->d_ff),
                             c->n_shared ? decode_counter_cap(c->T, 1, c->d_model, c->d_ff_shared) : 0);
    k.counters = static_cast<int*>(take(sizeof(int) * (size_t)k.counter_cap));
  }
  k.total = off;
  return k;
}

moe_status check_ws(const moe_config* c, const void* ws, size_t ws_bytes) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < carve(c, nullptr).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

uint64_t wait_limit(const moe_config* c) { return c->wait_limit_ns > 0 ? (uint64_t)c->wait_limit_ns : 2000000000ull; }

// After a call's host checks: the injected launch failure (host_guard.cuh),
// then the switch to the device that owns `p` and the check of the stream.
moe_status enter(DeviceGuard& g, const void* p, cudaStream_t stream) {
  if (launch_failure_injected()) return MOE_ERR_CUDA;
  const moe_status st = g.bind(p);
  return st != MOE_OK ? st : g.check_stream(stream);
}

// a_quantized: 8-bit experts whose input rows are already in xq / sx;
// chained: a layer step that cleared the decode counters ahead and chains its
// launches (pdl.cuh)
cudaError_t run_ffn(const moe_config* c, const Carve& k, const void* a, const int32_t* offsets, int G, int64_t rows,
                    int f, const void* w_gu, const void* w_d, void* h, void* y, cudaStream_t s, bool shared = false,
                    bool a_quantized = false, bool chained = false, int part = kFfnBoth) {
  GroupedFfnArgs g{a, offsets, w_gu, w_d, h, y, rows, G, c->d_model, f, c->expert_act, k.status, wait_limit(c),
                   false, nullptr, nullptr, nullptr, k.partial, k.partial_slots, k.counters, k.counter_cap,
                   chained, part};
  if (c->dtype != MOE_BF16) return launch_grouped_ffn_f32_simt(g, s);
  if (c->weight_format == MOE_W_E4M3) {
    // the expert input -> E4M3 codes and per-token scales (only the rows in use)
    uint8_t* xq = shared ? k.xq_s : k.xq;
    float* sx = shared ? k.sx_s : k.sx;
    if (!a_quantized && part != kFfnGemm2) {
      const cudaError_t e = launch_quantize_e4m3(a, rows, offsets ? offsets + G : nullptr, c->d_model, xq, sx, s);
      if (e != cudaSuccess) return e;
    }
    g.a = xq;
    g.fp8 = true;
    g.sa = sx;
    g.hq = shared ? k.hq_s : k.hq;
    g.sh = shared ? k.sh_s : k.sh;
  }
  if (k.partial != nullptr && use_decode_ffn(rows, G, offsets != nullptr)) return launch_grouped_ffn_bf16_decode(g, s);
  return launch_grouped_ffn_bf16_tc(g, s);
}

moe_status check_route_config(const moe_route_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->n_experts <= 0 || c->top_k <= 0 || c->n_groups <= 0 || c->reserved != 0)
    return MOE_ERR_INVALID_ARG;
  if (c->logits_stride != 0 && c->logits_stride < c->n_experts) return MOE_ERR_INVALID_ARG;
  if (c->n_experts % c->n_groups != 0 || c->topk_groups < 1 || c->topk_groups > c->n_groups)
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)c->top_k > (int64_t)c->topk_groups * (c->n_experts / c->n_groups)) return MOE_ERR_INVALID_ARG;
  if (c->group_top != 1 && c->group_top != 2) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->renormalise != 0 && c->renormalise != 1) return MOE_ERR_INVALID_ARG;
  if (c->logits_dtype != MOE_F32 && c->logits_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->weight_scale)) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > kMaxExperts || c->top_k > kMaxTopK || c->n_groups > 32) return MOE_ERR_UNSUPPORTED;
  const int64_t stride = c->logits_stride ? c->logits_stride : c->n_experts;
  if (c->T >= (int64_t(1) << 31) / c->top_k || stride > (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int64_t route_stride(const moe_route_config* c) { return c->logits_stride ? c->logits_stride : c->n_experts; }

RouteArgs route_args(const moe_route_config* c, const void* logits, const float* bias, int32_t* ids, float* w) {
  return RouteArgs{logits, bias, ids, w, c->T, route_stride(c), c->n_experts, c->top_k, c->n_groups, c->topk_groups,
                   c->group_top, c->score == MOE_SCORE_SIGMOID, c->renormalise != 0, c->logits_dtype == MOE_BF16,
                   c->weight_scale, false};
}

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) % kAlign) == 0; }

moe_status check_adapter_config(const moe_config* c, const moe_adapter_config* ad) {
  const moe_status st = check_config(c);
  if (st != MOE_OK) return st;
  if (ad == nullptr || ad->n_adapters <= 0 || ad->rank <= 0 || ad->rank % 8 != 0 || ad->reserved != 0 ||
      (ad->shared != 0 && ad->shared != 1))
    return MOE_ERR_INVALID_ARG;
  if (ad->shared && c->n_shared == 0) return MOE_ERR_INVALID_ARG;
  if (ad->n_adapters > 65536 || ad->rank > 128) return MOE_ERR_UNSUPPORTED;
  if (!ad->shared && (int64_t)c->n_experts * ad->n_adapters > kAdapterMaxPairs) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

AdapterShape adapter_shape(const moe_config* c, int N, int r, bool shared) {
  const int act = c->expert_act == MOE_ACT_GELU ? kEpiGELU : kEpiSwiGLU;
  return AdapterShape{c->T, shared ? c->T : c->T * c->top_k, c->d_model, shared ? c->d_ff_shared : c->d_ff,
                      shared ? 1 : c->n_experts, shared ? 1 : c->top_k, N, r, act, c->dtype == MOE_BF16};
}

moe_status adapter_apply(const moe_config* cfg, const moe_adapter_config* ad, bool gate_up, void* plan,
                         size_t plan_bytes, const void* x, const void* a, const void* b, const float* scale,
                         const void* base, void* out, cudaStream_t stream) {
  moe_status st = check_adapter_config(cfg, ad);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  const AdapterShape s = adapter_shape(cfg, ad->n_adapters, ad->rank, ad->shared != 0);
  if (!plan || !aligned256(plan)) return MOE_ERR_INVALID_ARG;
  if (plan_bytes < adapter_plan_bytes(s)) return MOE_ERR_WORKSPACE;
  if (!x || !a || !b || !scale || !base || !out || !aligned16(x) || !aligned16(a) || !aligned16(b) ||
      !aligned16(scale) || !aligned16(base) || !aligned16(out) || x == out)
    return MOE_ERR_INVALID_ARG;
  if (gate_up && base == out && cfg->expert_act != MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, plan, stream)) != MOE_OK) return st;
  if ((st = g.same_device(out)) != MOE_OK) return st;
  MOE_CUDA_TRY(launch_adapter_apply(s, AdapterApply{gate_up, x, a, b, scale, base, out, plan, static_cast<int*>(plan),
                                                   wait_limit(cfg)}, stream));
  return MOE_OK;
}

// What a layer call with adapters needs beyond moe_workspace_bytes: the
// pre-activations and the plan of the routed and of the shared experts, and
// the dispatched rows themselves where 8-bit experts keep only their codes.
struct RoutedCarve {
  void *pre, *pre_s, *plan, *plan_s, *x_perm;
  size_t total;
};
RoutedCarve carve_routed(const moe_config* c, const moe_adapters* ad, void* base) {
  RoutedCarve k{};
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = carve(c, nullptr).total;
  auto take = [&](size_t bytes) -> void* {
    void* p = b ? b + off : nullptr;
    off += up(bytes);
    return p;
  };
  const size_t eb = elem_bytes(c);
  const size_t halves = c->expert_act == MOE_ACT_GELU ? 1 : 2;
  if (ad && (ad->a_gate_up || ad->a_down)) {
    k.plan = take(adapter_plan_bytes(adapter_shape(c, ad->n_adapters, ad->rank, false)));
    if (ad->a_gate_up) {
      k.pre = take(eb * halves * (size_t)(c->T * c->top_k) * c->d_ff);
      if (c->weight_format == MOE_W_E4M3) k.x_perm = take(eb * (size_t)(c->T * c->top_k) * c->d_model);
    }
  }
  if (ad && (ad->a_gate_up_shared || ad->a_down_shared)) {
    k.plan_s = take(adapter_plan_bytes(adapter_shape(c, ad->n_adapters, ad->rank, true)));
    if (ad->a_gate_up_shared) k.pre_s = take(eb * halves * (size_t)c->T * c->d_ff_shared);
  }
  k.total = off;
  return k;
}

moe_status check_adapters(const moe_config* c, const moe_adapters* ad) {
  if (ad == nullptr) return MOE_OK;
  // the routed and the shared experts have a plan each, with limits of their own
  const bool shared = ad->a_gate_up_shared || ad->b_gate_up_shared || ad->a_down_shared || ad->b_down_shared;
  const bool routed = ad->a_gate_up || ad->b_gate_up || ad->a_down || ad->b_down || !shared;
  for (int sh = 0; sh < 2; ++sh) {
    if (!(sh ? shared : routed)) continue;
    const moe_adapter_config ac{ad->n_adapters, ad->rank, sh, 0};
    const moe_status st = check_adapter_config(c, &ac);
    if (st != MOE_OK) return st;
  }
  const void* p[] = {ad->token_adapter, ad->scale,         ad->a_gate_up,        ad->b_gate_up,     ad->a_down,
                     ad->b_down,        ad->a_gate_up_shared, ad->b_gate_up_shared, ad->a_down_shared, ad->b_down_shared};
  for (const void* q : p)
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  for (int i = 2; i < 10; i += 2)
    if ((p[i] == nullptr) != (p[i + 1] == nullptr)) return MOE_ERR_INVALID_ARG;  // a without its b
  if (c->T > 0 && (!ad->token_adapter || !ad->scale)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// One group of experts (routed or shared) with adapters: the plan, the first
// product (without its activation where it has adapters, which then add and
// activate), the second product, its adapters.  a_quantized as in run_ffn.
cudaError_t run_adapted_ffn(const moe_config* c, const Carve& k, const moe_adapters* ad, void* plan, void* pre,
                            const void* x, const int32_t* offsets, const int32_t* perm, int G, int64_t rows, int f,
                            const void* w_gu, const void* w_d, void* h, void* y, bool shared, bool a_quantized,
                            cudaStream_t s) {
  const AdapterShape sh = adapter_shape(c, ad->n_adapters, ad->rank, shared);
  const void* a1 = shared ? ad->a_gate_up_shared : ad->a_gate_up;
  const void* b1 = shared ? ad->b_gate_up_shared : ad->b_gate_up;
  const void* a2 = shared ? ad->a_down_shared : ad->a_down;
  const void* b2 = shared ? ad->b_down_shared : ad->b_down;
  cudaError_t e = launch_adapter_plan(sh, offsets, perm, ad->token_adapter, plan, k.status, wait_limit(c), s);
  if (e != cudaSuccess) return e;
  e = run_ffn(c, k, x, offsets, G, rows, f, w_gu, w_d, a1 ? pre : h, y, s, shared, a_quantized, true,
              a1 ? kFfnGemm1Plain : kFfnGemm1);
  if (e != cudaSuccess) return e;
  if (a1) {
    e = launch_adapter_apply(sh, AdapterApply{true, x, a1, b1, ad->scale, pre, h, plan, k.status, wait_limit(c)}, s);
    if (e != cudaSuccess) return e;
  }
  e = run_ffn(c, k, x, offsets, G, rows, f, w_gu, w_d, h, y, s, shared, true, true, kFfnGemm2);
  if (e != cudaSuccess || !a2) return e;
  return launch_adapter_apply(sh, AdapterApply{false, h, a2, b2, ad->scale, y, y, plan, k.status, wait_limit(c)}, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_workspace_bytes(const moe_config* cfg) {
  if (check_config(cfg) != MOE_OK) return 0;
  return carve(cfg, nullptr).total;
}

size_t moe_e4m3_weight_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return 0;
  return e4m3_codes_bytes(rows, cols) + sizeof(float) * (size_t)rows;
}

moe_status moe_quantize_e4m3(const void* src, int64_t rows, int32_t cols, void* blob, moe_stream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!src || !blob || !aligned16(src) || (reinterpret_cast<uintptr_t>(blob) % kAlign) != 0)
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  const moe_status st = enter(g, blob, stream);
  if (st != MOE_OK) return st;
  uint8_t* q = static_cast<uint8_t*>(blob);
  float* sc = reinterpret_cast<float*>(q + e4m3_codes_bytes(rows, cols));
  MOE_CUDA_TRY(launch_quantize_e4m3(src, rows, nullptr, cols, q, sc, stream));
  return MOE_OK;
}

int64_t moe_expert_capacity(const moe_config* cfg) {
  if (check_config(cfg) != MOE_OK) return -1;
  return capacity_rows(cfg);
}

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported configuration";
    case MOE_ERR_WORKSPACE: return "workspace too small";
    case MOE_ERR_CUDA: return "CUDA error";
    case MOE_ERR_TIMEOUT: return "device wait timed out";
    case MOE_ERR_BAD_EXPERT_ID: return "expert id out of range";
    case MOE_ERR_BAD_ADAPTER_ID: return "adapter id out of range";
  }
  return "unknown status";
}

moe_status moe_router_topk(const moe_config* cfg, const void* x, const void* w_router, const float* logit_bias,
                           int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_ws(cfg, ws, ws_bytes)) != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!x || !w_router || !topk_ids || !topk_w || !aligned16(x) || !aligned16(w_router) || !aligned16(topk_ids) ||
      !aligned16(topk_w) || (logit_bias && !aligned16(logit_bias)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  Carve k = carve(cfg, ws);
  RouterArgs a{x, w_router, logit_bias, topk_ids, topk_w, cfg->T, cfg->d_model, cfg->n_experts, cfg->top_k,
               cfg->gating, cfg->bias_select_only, cfg->dtype == MOE_BF16, k.status, wait_limit(cfg)};
  MOE_CUDA_TRY(launch_router_topk(a, stream));
  return MOE_OK;
}

moe_status moe_router_aux_losses(const moe_config* cfg, const void* x, const void* w_router, const int32_t* counts,
                                 float* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_ws(cfg, ws, ws_bytes)) != MOE_OK) return st;
  if (!counts || !out || !aligned16(counts) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!x || !w_router || !aligned16(x) || !aligned16(w_router))) return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  if (cfg->T == 0) {
    MOE_CUDA_TRY(cudaMemsetAsync(out, 0, 2 * sizeof(float), stream));
    return MOE_OK;
  }
  Carve k = carve(cfg, ws);
  // the selection itself is recomputed into the workspace and discarded
  RouterArgs a{x, w_router, nullptr, k.ids, k.w, cfg->T, cfg->d_model, cfg->n_experts, cfg->top_k,
               cfg->gating, cfg->bias_select_only, cfg->dtype == MOE_BF16, k.status, wait_limit(cfg), k.aux_part};
  MOE_CUDA_TRY(launch_router_aux_losses(a, counts, out, stream));
  return MOE_OK;
}

moe_status moe_permute(const moe_config* cfg, const int32_t* topk_ids, const void* x, int32_t* counts,
                       int32_t* offsets, int32_t* perm, int32_t* row_of, void* x_perm, void* ws, size_t ws_bytes,
                       moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_ws(cfg, ws, ws_bytes)) != MOE_OK) return st;
  if (!counts || !offsets || !aligned16(counts) || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!topk_ids || !perm || !row_of || !x || !x_perm || !aligned16(topk_ids) || !aligned16(perm) ||
                     !aligned16(row_of) || !aligned16(x) || !aligned16(x_perm)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  Carve k = carve(cfg, ws);
  PermuteArgs a{topk_ids, x, counts, offsets, perm, row_of, x_perm, k.chunk_counts, cfg->T * cfg->top_k,
                cfg->top_k, cfg->d_model, cfg->n_experts, (int)elem_bytes(cfg), k.status, capacity_rows(cfg)};
  MOE_CUDA_TRY(launch_permute(a, stream));
  return MOE_OK;
}

moe_status moe_grouped_ffn(const moe_config* cfg, const void* x_perm, const int32_t* offsets, const void* w_gate_up,
                           const void* w_down, void* y_perm, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_ws(cfg, ws, ws_bytes)) != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!x_perm || !offsets || !w_gate_up || !w_down || !y_perm || !aligned16(x_perm) || !aligned16(offsets) ||
      !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(y_perm))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  Carve k = carve(cfg, ws);
  MOE_CUDA_TRY(run_ffn(cfg, k, x_perm, offsets, cfg->n_experts, cfg->T * cfg->top_k, cfg->d_ff, w_gate_up, w_down,
                       k.h, y_perm, stream));
  return MOE_OK;
}

moe_status moe_combine(const moe_config* cfg, const void* y_perm, const int32_t* row_of, const float* topk_w,
                       const void* y_shared, void* y, moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!y_perm || !row_of || !topk_w || !y || !aligned16(y_perm) || !aligned16(row_of) || !aligned16(topk_w) ||
      !aligned16(y) || (y_shared && !aligned16(y_shared)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, y, stream)) != MOE_OK) return st;
  CombineArgs a{y_perm, row_of, topk_w, y_shared, y, cfg->T, cfg->top_k, cfg->d_model, cfg->dtype == MOE_BF16};
  MOE_CUDA_TRY(launch_combine(a, stream));
  return MOE_OK;
}

moe_status moe_combine_backward(const moe_config* cfg, const void* grad_y, const void* y_perm,
                                const int32_t* row_of, const float* topk_w, void* grad_y_perm, float* grad_w,
                                moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if (!grad_y_perm && !grad_w) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!grad_y || !row_of || !aligned16(grad_y) || !aligned16(row_of) || (grad_w && !y_perm) ||
      (grad_y_perm && !topk_w) || !aligned16(y_perm) || !aligned16(topk_w) || !aligned16(grad_y_perm) ||
      !aligned16(grad_w))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, grad_y, stream)) != MOE_OK) return st;
  if (grad_y_perm == grad_y) return MOE_ERR_INVALID_ARG;  // other tokens' rows would overwrite what a token reads
  CombineBackwardArgs a{grad_y, y_perm, row_of, topk_w, grad_y_perm, grad_w, cfg->T, cfg->top_k, cfg->d_model,
                        cfg->dtype == MOE_BF16};
  MOE_CUDA_TRY(launch_combine_backward(a, stream));
  return MOE_OK;
}

moe_status moe_route_topk(const moe_route_config* cfg, const void* logits, const float* select_bias,
                          int32_t* topk_ids, float* topk_w, moe_stream_t stream) {
  moe_status st = check_route_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w || !aligned16(logits) || !aligned16(topk_ids) || !aligned16(topk_w) ||
      !aligned16(select_bias))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, topk_ids, stream)) != MOE_OK) return st;
  if ((st = g.same_device(logits)) != MOE_OK) return st;
  MOE_CUDA_TRY(launch_route_topk(route_args(cfg, logits, select_bias, topk_ids, topk_w), stream));
  return MOE_OK;
}

moe_status moe_route_backward(const moe_route_config* cfg, const void* logits, const int32_t* topk_ids,
                              const float* grad_w, const int32_t* counts, float balance_coef, float z_coef,
                              void* grad_logits, moe_stream_t stream) {
  moe_status st = check_route_config(cfg);
  if (st != MOE_OK) return st;
  if (!std::isfinite(balance_coef) || !std::isfinite(z_coef)) return MOE_ERR_INVALID_ARG;
  if (balance_coef != 0.f && (!counts || !aligned16(counts))) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!logits || !grad_logits || logits == grad_logits || !aligned16(logits) || !aligned16(grad_logits) ||
      (grad_w && !topk_ids) || !aligned16(grad_w) || !aligned16(topk_ids))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, grad_logits, stream)) != MOE_OK) return st;
  if ((st = g.same_device(logits)) != MOE_OK) return st;
  RouteBackwardArgs a{logits, topk_ids, grad_w, counts, balance_coef, z_coef, grad_logits, cfg->T, route_stride(cfg),
                      cfg->n_experts, cfg->top_k, cfg->score == MOE_SCORE_SIGMOID, cfg->renormalise != 0,
                      cfg->logits_dtype == MOE_BF16, cfg->weight_scale, false};
  MOE_CUDA_TRY(launch_route_backward(a, stream));
  return MOE_OK;
}

moe_status moe_forward(const moe_config* cfg, const void* x, const void* w_router, const float* logit_bias,
                       const void* w_gate_up, const void* w_down, const void* ws_gate_up, const void* ws_down,
                       void* y, int32_t* opt_topk_ids, float* opt_topk_w, int32_t* opt_counts, void* ws,
                       size_t ws_bytes, moe_stream_t stream) {
  return moe_forward_traced(cfg, x, w_router, logit_bias, w_gate_up, w_down, ws_gate_up, ws_down, y, opt_topk_ids,
                            opt_topk_w, opt_counts, ws, ws_bytes, stream, nullptr);
}

moe_status moe_forward_traced(const moe_config* cfg, const void* x, const void* w_router, const float* logit_bias,
                              const void* w_gate_up, const void* w_down, const void* ws_gate_up,
                              const void* ws_down, void* y, int32_t* opt_topk_ids, float* opt_topk_w,
                              int32_t* opt_counts, void* ws, size_t ws_bytes, moe_stream_t stream,
                              const moe_event_t* stage_events) {
  // stage boundary i: record stage_events[i] (when given) on the stream
  auto mark = [&](int i) -> cudaError_t {
    if (stage_events == nullptr || stage_events[i] == nullptr) return cudaSuccess;
    return cudaEventRecord(stage_events[i], stream);
  };
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_ws(cfg, ws, ws_bytes)) != MOE_OK) return st;
  if (cfg->T == 0) {  // nothing to read or write: clear the status word and the optional counts
    if (opt_counts && !aligned16(opt_counts)) return MOE_ERR_INVALID_ARG;
    DeviceGuard g;
    if ((st = enter(g, ws, stream)) != MOE_OK) return st;
    MOE_CUDA_TRY(cudaMemsetAsync(ws, 0, 16, stream));
    if (opt_counts) MOE_CUDA_TRY(cudaMemsetAsync(opt_counts, 0, sizeof(int32_t) * cfg->n_experts, stream));
    return MOE_OK;
  }
  if (!x || !w_router || !w_gate_up || !w_down || !y || !aligned16(x) || !aligned16(w_router) ||
      !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(y) || (logit_bias && !aligned16(logit_bias)) ||
      (opt_topk_ids && !aligned16(opt_topk_ids)) || (opt_topk_w && !aligned16(opt_topk_w)) ||
      (opt_counts && !aligned16(opt_counts)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!ws_gate_up || !ws_down || !aligned16(ws_gate_up) || !aligned16(ws_down)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  if ((st = g.same_device(x)) != MOE_OK) return st;
  Carve k = carve(cfg, ws);
  MOE_CUDA_TRY(mark(0));
  MOE_CUDA_TRY(cudaMemsetAsync(k.status, 0, 16, stream));
  // The launches of the step are chained (pdl.cuh): each kernel after the
  // router may be scheduled while its predecessor finishes.  The decode
  // kernels' unit counters are cleared here, ahead of the chain, instead of
  // by a clearing launch in front of GEMM-1.
  if (k.counters) MOE_CUDA_TRY(cudaMemsetAsync(k.counters, 0, sizeof(int) * (size_t)k.counter_cap, stream));
  int32_t* ids = opt_topk_ids ? opt_topk_ids : k.ids;
  float* w = opt_topk_w ? opt_topk_w : k.w;
  int32_t* counts = opt_counts ? opt_counts : k.counts;
  RouterArgs ra{x, w_router, logit_bias, ids, w, cfg->T, cfg->d_model, cfg->n_experts, cfg->top_k,
                cfg->gating, cfg->bias_select_only, cfg->dtype == MOE_BF16, k.status, wait_limit(cfg)};
  MOE_CUDA_TRY(launch_router_topk(ra, stream));
  MOE_CUDA_TRY(mark(1));
  // 8-bit experts: the dispatch writes no bf16 copy; each token is quantised
  // once, straight from x, and its codes go to its rows
  const bool e4m3 = cfg->weight_format == MOE_W_E4M3;
  PermuteArgs pa{ids, x, counts, k.offsets, k.perm, k.row_of, e4m3 ? nullptr : k.x_perm, k.chunk_counts,
                 cfg->T * cfg->top_k, cfg->top_k, cfg->d_model, cfg->n_experts, (int)elem_bytes(cfg), k.status,
                 capacity_rows(cfg), true};
  MOE_CUDA_TRY(launch_permute(pa, stream));
  if (e4m3)
    MOE_CUDA_TRY(
        launch_gather_quantize_e4m3(x, k.row_of, cfg->top_k, cfg->T, cfg->d_model, k.xq, k.sx, true, stream));
  MOE_CUDA_TRY(mark(2));
  MOE_CUDA_TRY(run_ffn(cfg, k, k.x_perm, k.offsets, cfg->n_experts, cfg->T * cfg->top_k, cfg->d_ff, w_gate_up,
                       w_down, k.h, k.y_perm, stream, false, e4m3, true));
  MOE_CUDA_TRY(mark(3));
  if (cfg->n_shared > 0)
    MOE_CUDA_TRY(run_ffn(cfg, k, x, nullptr, 1, cfg->T, cfg->d_ff_shared, ws_gate_up, ws_down, k.h_s, k.y_s, stream,
                         true, false, true));
  MOE_CUDA_TRY(mark(4));
  CombineArgs ca{k.y_perm, k.row_of, w, cfg->n_shared > 0 ? k.y_s : nullptr, y, cfg->T, cfg->top_k,
                 cfg->d_model, cfg->dtype == MOE_BF16, true};
  MOE_CUDA_TRY(launch_combine(ca, stream));
  MOE_CUDA_TRY(mark(5));
  return MOE_OK;
}

size_t moe_adapter_plan_bytes(const moe_config* cfg, const moe_adapter_config* ad) {
  if (check_adapter_config(cfg, ad) != MOE_OK) return 0;
  return adapter_plan_bytes(adapter_shape(cfg, ad->n_adapters, ad->rank, ad->shared != 0));
}

moe_status moe_adapter_plan(const moe_config* cfg, const moe_adapter_config* ad, const int32_t* offsets,
                            const int32_t* perm, const int32_t* token_adapter, void* plan, size_t plan_bytes,
                            moe_stream_t stream) {
  moe_status st = check_adapter_config(cfg, ad);
  if (st != MOE_OK) return st;
  const AdapterShape s = adapter_shape(cfg, ad->n_adapters, ad->rank, ad->shared != 0);
  if (!plan || !aligned256(plan)) return MOE_ERR_INVALID_ARG;
  if (plan_bytes < adapter_plan_bytes(s)) return MOE_ERR_WORKSPACE;
  if (cfg->T > 0 && (!token_adapter || !aligned16(token_adapter) || !aligned16(offsets) || !aligned16(perm) ||
                     (ad->shared ? offsets || perm : !offsets || !perm)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, plan, stream)) != MOE_OK) return st;
  const size_t clear = adapter_plan_clear_bytes(s);
  if (clear) MOE_CUDA_TRY(cudaMemsetAsync(plan, 0, clear, stream));
  MOE_CUDA_TRY(launch_adapter_plan(s, offsets, perm, token_adapter, plan, static_cast<int*>(plan), wait_limit(cfg), stream));
  return MOE_OK;
}

moe_status moe_adapter_gate_up(const moe_config* cfg, const moe_adapter_config* ad, void* plan, size_t plan_bytes,
                               const void* x, const void* a, const void* b, const float* scale, const void* pre,
                               void* h, moe_stream_t stream) {
  return adapter_apply(cfg, ad, true, plan, plan_bytes, x, a, b, scale, pre, h, stream);
}

moe_status moe_adapter_down(const moe_config* cfg, const moe_adapter_config* ad, void* plan, size_t plan_bytes,
                            const void* h, const void* a, const void* b, const float* scale, const void* base,
                            void* y, moe_stream_t stream) {
  return adapter_apply(cfg, ad, false, plan, plan_bytes, h, a, b, scale, base, y, stream);
}

size_t moe_forward_routed_workspace_bytes(const moe_config* cfg, const moe_adapters* adapters) {
  if (check_config(cfg) != MOE_OK || check_adapters(cfg, adapters) != MOE_OK) return 0;
  return carve_routed(cfg, adapters, nullptr).total;
}

moe_status moe_forward_routed(const moe_config* cfg, const moe_route_config* route, const moe_adapters* adapters,
                              const void* x, const void* logits, const float* select_bias, const void* w_gate_up,
                              const void* w_down, const void* ws_gate_up, const void* ws_down, void* y,
                              int32_t* opt_topk_ids, float* opt_topk_w, int32_t* opt_counts, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  if ((st = check_route_config(route)) != MOE_OK) return st;
  if (route->T != cfg->T || route->n_experts != cfg->n_experts || route->top_k != cfg->top_k)
    return MOE_ERR_INVALID_ARG;
  if ((st = check_adapters(cfg, adapters)) != MOE_OK) return st;
  if (ws == nullptr || !aligned256(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < carve_routed(cfg, adapters, nullptr).total) return MOE_ERR_WORKSPACE;
  if (opt_counts && !aligned16(opt_counts)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) {  // nothing to read or write: clear the status word and the optional counts
    DeviceGuard g;
    if ((st = enter(g, ws, stream)) != MOE_OK) return st;
    MOE_CUDA_TRY(cudaMemsetAsync(ws, 0, 16, stream));
    if (opt_counts) MOE_CUDA_TRY(cudaMemsetAsync(opt_counts, 0, sizeof(int32_t) * cfg->n_experts, stream));
    return MOE_OK;
  }
  if (!x || !logits || !w_gate_up || !w_down || !y || !aligned16(x) || !aligned16(logits) || !aligned16(w_gate_up) ||
      !aligned16(w_down) || !aligned16(y) || !aligned16(select_bias) || !aligned16(opt_topk_ids) ||
      !aligned16(opt_topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!ws_gate_up || !ws_down || !aligned16(ws_gate_up) || !aligned16(ws_down)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard g;
  if ((st = enter(g, ws, stream)) != MOE_OK) return st;
  if ((st = g.same_device(x)) != MOE_OK) return st;
  if ((st = g.same_device(logits)) != MOE_OK) return st;
  const Carve k = carve(cfg, ws);
  const RoutedCarve rk = carve_routed(cfg, adapters, ws);
  // everything that has to be zero is cleared ahead of the chain of launches (pdl.cuh)
  MOE_CUDA_TRY(cudaMemsetAsync(k.status, 0, 16, stream));
  if (k.counters) MOE_CUDA_TRY(cudaMemsetAsync(k.counters, 0, sizeof(int) * (size_t)k.counter_cap, stream));
  for (int sh = 0; sh < 2; ++sh) {
    void* plan = sh ? rk.plan_s : rk.plan;
    const size_t clear =
        plan ? adapter_plan_clear_bytes(adapter_shape(cfg, adapters->n_adapters, adapters->rank, sh != 0)) : 0;
    if (clear) MOE_CUDA_TRY(cudaMemsetAsync(plan, 0, clear, stream));
  }
  int32_t* ids = opt_topk_ids ? opt_topk_ids : k.ids;
  float* w = opt_topk_w ? opt_topk_w : k.w;
  int32_t* counts = opt_counts ? opt_counts : k.counts;
  MOE_CUDA_TRY(launch_route_topk(route_args(route, logits, select_bias, ids, w), stream));
  // 8-bit experts: the dispatch writes codes straight from x (moe_forward),
  // unless adapters need the rows themselves
  const bool e4m3 = cfg->weight_format == MOE_W_E4M3;
  void* x_perm = e4m3 ? rk.x_perm : k.x_perm;
  PermuteArgs pa{ids, x, counts, k.offsets, k.perm, k.row_of, x_perm, k.chunk_counts, cfg->T * cfg->top_k,
                 cfg->top_k, cfg->d_model, cfg->n_experts, (int)elem_bytes(cfg), k.status, capacity_rows(cfg), true,
                 -1};
  MOE_CUDA_TRY(launch_permute(pa, stream));
  const bool codes = e4m3 && x_perm == nullptr;
  if (codes)
    MOE_CUDA_TRY(
        launch_gather_quantize_e4m3(x, k.row_of, cfg->top_k, cfg->T, cfg->d_model, k.xq, k.sx, true, stream));
  const int64_t rows = cfg->T * cfg->top_k;
  if (rk.plan)
    MOE_CUDA_TRY(run_adapted_ffn(cfg, k, adapters, rk.plan, rk.pre, x_perm, k.offsets, k.perm, cfg->n_experts, rows,
                                 cfg->d_ff, w_gate_up, w_down, k.h, k.y_perm, false, codes, stream));
  else
    MOE_CUDA_TRY(run_ffn(cfg, k, x_perm, k.offsets, cfg->n_experts, rows, cfg->d_ff, w_gate_up, w_down, k.h,
                         k.y_perm, stream, false, codes, true));
  if (rk.plan_s)
    MOE_CUDA_TRY(run_adapted_ffn(cfg, k, adapters, rk.plan_s, rk.pre_s, x, nullptr, nullptr, 1, cfg->T,
                                 cfg->d_ff_shared, ws_gate_up, ws_down, k.h_s, k.y_s, true, false, stream));
  else if (cfg->n_shared > 0)
    MOE_CUDA_TRY(run_ffn(cfg, k, x, nullptr, 1, cfg->T, cfg->d_ff_shared, ws_gate_up, ws_down, k.h_s, k.y_s, stream,
                         true, false, true));
  CombineArgs ca{k.y_perm, k.row_of, w, cfg->n_shared > 0 ? k.y_s : nullptr, y, cfg->T, cfg->top_k,
                 cfg->d_model, cfg->dtype == MOE_BF16, true};
  MOE_CUDA_TRY(launch_combine(ca, stream));
  return MOE_OK;
}

moe_status moe_device_status(const void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (ws == nullptr || ws_bytes < 16 || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0) return MOE_ERR_INVALID_ARG;
  MOE_CUDA_TRY(cudaStreamSynchronize(stream));
  int v = 0;
  MOE_CUDA_TRY(cudaMemcpy(&v, ws, sizeof(int), cudaMemcpyDeviceToHost));
  if (v == kDevTimeout) return MOE_ERR_TIMEOUT;
  if (v == kDevBadExpertId) return MOE_ERR_BAD_EXPERT_ID;
  if (v == kDevBadAdapterId) return MOE_ERR_BAD_ADAPTER_ID;
  return v == 0 ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
