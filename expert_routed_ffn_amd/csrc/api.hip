// api.hip -- the C ABI entry points: argument checks, workspace sizes, and
// hand-off to the kernel launchers.  A failing check enqueues nothing.
#include <cstdio>
#include <string>

#include "internal.hpp"

namespace moe {

static thread_local std::string g_last_error;

void set_error(const std::string& msg) { g_last_error = msg; }

moe_status fail(moe_status st, const std::string& msg) {
  set_error(msg);
  return st;
}

moe_status check_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

moe_status check_launch(const char* what) { return check_hip(hipGetLastError(), what); }

ProfileReq& profile_req() {
  static thread_local ProfileReq req;
  return req;
}

static int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

#ifndef MOE_STAGE_IN_GATEUP
#define MOE_STAGE_IN_GATEUP 1
#endif
constexpr bool kStageInGateup = MOE_STAGE_IN_GATEUP != 0;
#ifndef MOE_RESOLVE_IN_GATEUP
#define MOE_RESOLVE_IN_GATEUP 1
#endif
constexpr bool kResolveInGateup = MOE_RESOLVE_IN_GATEUP != 0;

BlobLayout blob_layout(int H, int I, int bits) {
  const int64_t gu_codes = (int64_t)I * H * bits / 8, gu_sm = (int64_t)I * (H / 32) * 4;
  const int64_t d_codes = (int64_t)H * I * bits / 8, d_sm = (int64_t)H * (I / 32) * 4;
  BlobLayout L;
  int64_t o = 0;
  L.gate_codes = o; o = up256(o + gu_codes);
  L.gate_sm = o;    o = up256(o + gu_sm);
  L.up_codes = o;   o = up256(o + gu_codes);
  L.up_sm = o;      o = up256(o + gu_sm);
  L.down_codes = o; o = up256(o + d_codes);
  L.down_sm = o;    o = up256(o + d_sm);
  L.bytes = o;
  return L;
}

}  // namespace moe

using namespace moe;

namespace {

std::string fmt(const char* f, long long a = 0, long long b = 0, long long c = 0) {
  char buf[256];
  snprintf(buf, sizeof buf, f, a, b, c);
  return buf;
}

moe_status check_ek(const char* fn, int E, int k) {
  if (E < 1 || E > kMaxE) return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": E=%lld outside [1, 1024]", E));
  if (k < 1 || k > kMaxK || k > E)
    return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": k=%lld outside [1, min(16, E=%lld)]", k, E));
  return MOE_OK;
}

moe_status check_shape(const char* fn, int H, int I, int bits) {
  if (bits < 2 || bits > 4) return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": bits=%lld (2, 3 or 4)", bits));
  if (H < 32 || H > 16384 || H % 32)
    return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": H=%lld (multiple of 32 in [32, 16384])", H));
  if (I < 32 || I > 8192 || I % 32)
    return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": I=%lld (multiple of 32 in [32, 8192])", I));
  return MOE_OK;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// Whether two buffers (null: none) share a byte.
bool overlap(const void* p, uint64_t n, const void* q, uint64_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + m && b < a + n;
}
struct Span {
  const void* p;
  uint64_t n;
};
// Whether a buffer that is written shares a byte with one that is read or with another that is written.
template <size_t O, size_t I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Span& s : in)
      if (overlap(out[i].p, out[i].n, s.p, s.n)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_last_error(void) { return g_last_error.c_str(); }

const char* moe_status_string(moe_status st) {
  switch (st) {
    case MOE_OK: return "MOE_OK";
    case MOE_EINVAL: return "MOE_EINVAL";
    case MOE_EUNSUPPORTED: return "MOE_EUNSUPPORTED";
    case MOE_EWORKSPACE: return "MOE_EWORKSPACE";
    case MOE_EHIP: return "MOE_EHIP";
    case MOE_ENOTPINNED: return "MOE_ENOTPINNED";
    case MOE_ECAPACITY: return "MOE_ECAPACITY";
  }
  return "unknown moe_status";
}

size_t moe_expert_bytes(int H, int I, int bits) {
  if (check_shape("moe_expert_bytes", H, I, bits) != MOE_OK) return 0;
  return (size_t)blob_layout(H, I, bits).bytes;
}

moe_status moe_route_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w, hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_route_topk: T < 0");
  if (moe_status st = check_ek("moe_route_topk", E, k)) return st;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !w) return fail(MOE_EINVAL, "moe_route_topk: null pointer");
  return launch_route_topk(logits, T, E, k, ids, w, stream);
}

moe_status moe_router_logits(const void* x, moe_dtype x_t, const void* w_r, int T, int H, int E, float* logits,
                             hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_router_logits: T < 0");
  if (x_t != MOE_F32 && x_t != MOE_BF16) return fail(MOE_EINVAL, "moe_router_logits: bad x dtype");
  if (E < 1 || E > kMaxE) return fail(MOE_EUNSUPPORTED, fmt("moe_router_logits: E = %d outside 1..%d", E, kMaxE));
  if (H < 32 || H > 16384 || H % 32 != 0)
    return fail(MOE_EUNSUPPORTED, fmt("moe_router_logits: H = %d (needs a multiple of 32 in 32..16384)", H));
  if (T == 0) return MOE_OK;
  if (!x || !w_r || !logits) return fail(MOE_EINVAL, "moe_router_logits: null pointer");
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_r)) & 15)
    return fail(MOE_EINVAL, "moe_router_logits: x and w_r must be 16-byte aligned");
  return launch_router_logits(x, x_t == MOE_F32, reinterpret_cast<const uint16_t*>(w_r), T, H, E, logits, stream);
}

moe_status moe_router_topk(const void* x, moe_dtype x_t, const void* w_r, int T, int H, int E, int k, float* logits,
                           int32_t* ids, float* w, hipStream_t stream) {
  if (moe_status st = check_ek("moe_router_topk", E, k)) return st;
  if (T > 0 && (!ids || !w)) return fail(MOE_EINVAL, "moe_router_topk: null pointer");
  if (moe_status st = moe_router_logits(x, x_t, w_r, T, H, E, logits, stream)) return st;
  if (T == 0) return MOE_OK;
  return launch_route_topk(logits, T, E, k, ids, w, stream);
}

size_t moe_dispatch_workspace_bytes(int T, int k, int E) {
  if (T < 0 || k < 1 || E < 1) return 0;
  return dispatch_ws_bytes(T * k, E);
}

moe_status moe_dispatch(const int32_t* ids, int T, int k, int E, int32_t* offsets, int32_t* sorted_assign,
                        int32_t* assign_pos, int32_t* active, int32_t* n_active, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_dispatch: T < 0");
  if (moe_status st = check_ek("moe_dispatch", E, k)) return st;
  if ((int64_t)T * k > (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "moe_dispatch: T*k above 2^24");
  if (!offsets || !n_active) return fail(MOE_EINVAL, "moe_dispatch: null pointer");
  if (T > 0 && (!ids || !sorted_assign || !assign_pos || !active))
    return fail(MOE_EINVAL, "moe_dispatch: null pointer");
  const size_t need = dispatch_ws_bytes(T * k, E);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_dispatch: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  return launch_dispatch(ids, T * k, E, offsets, sorted_assign, assign_pos, active, n_active, ws, stream);
}

// AUTO: GEMV up to 128 routed rows, MFMA above.  On the 512-expert, top-10,
// 2048 x 512 layer the two paths cross between T = 12 (GEMV 61 us, MFMA
// 64 us per layer step) and T = 16 (77 us, 67 us).
constexpr int64_t kAutoGemvMaxRows = 128;
static moe_ffn_path resolve_path(moe_ffn_path p, int T, int k) {
  if (p == MOE_PATH_AUTO) return (int64_t)T * k <= kAutoGemvMaxRows ? MOE_PATH_GEMV : MOE_PATH_MFMA;
  return p;
}

size_t moe_expert_ffn_workspace_bytes(const moe_qlayer* q, int T, int k, moe_ffn_path path) {
  if (!q || T < 0 || k < 1) return 0;
  if (resolve_path(path, T, k) == MOE_PATH_GEMV) return ffn_gemv_ws_bytes(T, k, q->E, q->H, q->I);
  return ffn_mfma_ws_bytes(T, k, q->E, q->H, q->I);
}

moe_status moe_expert_ffn_q(const moe_qlayer* q, const void* x, moe_dtype x_t, int T, int k, const int32_t* offsets,
                            const int32_t* sorted_assign, const int32_t* active, const int32_t* n_active, void* y,
                            moe_dtype y_t, moe_ffn_path path, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "moe_expert_ffn_q";
  if (!q) return fail(MOE_EINVAL, "moe_expert_ffn_q: null moe_qlayer");
  if (T < 0) return fail(MOE_EINVAL, "moe_expert_ffn_q: T < 0");
  if (moe_status st = check_ek(fn, q->E, k)) return st;
  if (moe_status st = check_shape(fn, q->H, q->I, q->bits)) return st;
  if (x_t != MOE_F32 && x_t != MOE_BF16) return fail(MOE_EINVAL, "moe_expert_ffn_q: x dtype");
  if (y_t != MOE_F32 && y_t != MOE_BF16) return fail(MOE_EINVAL, "moe_expert_ffn_q: y dtype");
  if (path != MOE_PATH_AUTO && path != MOE_PATH_GEMV && path != MOE_PATH_MFMA)
    return fail(MOE_EINVAL, "moe_expert_ffn_q: path");
  if ((int64_t)T * k > (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "moe_expert_ffn_q: T*k above 2^24");
  if (T == 0) return MOE_OK;
  if (!q->base || !x || !offsets || !sorted_assign || !active || !n_active || !y)
    return fail(MOE_EINVAL, "moe_expert_ffn_q: null pointer");
  const int64_t eb = blob_layout(q->H, q->I, q->bits).bytes;
  if (q->stride < eb || q->stride % 256)
    return fail(MOE_EINVAL, fmt("moe_expert_ffn_q: stride %lld (needs >= %lld and a multiple of 256)", q->stride, eb));
  if (!aligned(q->base, 256)) return fail(MOE_EINVAL, "moe_expert_ffn_q: base not 256-byte aligned");
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 256))
    return fail(MOE_EINVAL, "moe_expert_ffn_q: x or y not 16-byte aligned, or ws not 256-byte aligned");
  const moe_ffn_path p = resolve_path(path, T, k);
  const size_t need = moe_expert_ffn_workspace_bytes(q, T, k, p);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_expert_ffn_q: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  if (p == MOE_PATH_GEMV)
    return launch_ffn_gemv(*q, x, x_t, T, k, offsets, sorted_assign, active, n_active, y, y_t, ws, stream);
  return launch_ffn_mfma(*q, x, x_t, T, k, offsets, sorted_assign, active, n_active, y, y_t, ws, stream);
}

size_t moe_layer_decode_workspace_bytes(const moe_qlayer* q, int T, int k) {
  if (!q || T < 0 || k < 1 || q->E < 1) return 0;
  return decode_ws(nullptr, T, k, q->E, q->H, q->I).bytes;
}

moe_status moe_layer_decode(const moe_qlayer* q, const float* logits, const void* x, moe_dtype x_t, int T, int k,
                            const void* residual, moe_dtype r_t, int32_t* ids, float* w, int32_t* offsets,
                            int32_t* sorted_assign, int32_t* assign_pos, int32_t* active, int32_t* n_active, void* y,
                            moe_dtype y_t, float* out, uint16_t* out_bf16, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  const char* fn = "moe_layer_decode";
  if (!q) return fail(MOE_EINVAL, "moe_layer_decode: null moe_qlayer");
  if (T < 0) return fail(MOE_EINVAL, "moe_layer_decode: T < 0");
  if (T > kDescT) return fail(MOE_EUNSUPPORTED, fmt("moe_layer_decode: T=%lld above 12", T));
  if (moe_status st = check_ek(fn, q->E, k)) return st;
  if (moe_status st = check_shape(fn, q->H, q->I, q->bits)) return st;
  if (x_t != MOE_F32 && x_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode: x dtype");
  if (y_t != MOE_F32 && y_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode: y dtype");
  if (residual && r_t != MOE_F32 && r_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode: residual dtype");
  if (T == 0) return MOE_OK;
  if (!q->base || !logits || !x || !ids || !w || !offsets || !sorted_assign || !assign_pos || !active || !n_active ||
      !y || !out)
    return fail(MOE_EINVAL, "moe_layer_decode: null pointer");
  const int64_t eb = blob_layout(q->H, q->I, q->bits).bytes;
  if (q->stride < eb || q->stride % 256)
    return fail(MOE_EINVAL, fmt("moe_layer_decode: stride %lld (needs >= %lld and a multiple of 256)", q->stride, eb));
  if (!aligned(q->base, 256)) return fail(MOE_EINVAL, "moe_layer_decode: base not 256-byte aligned");
  const uintptr_t r_align = r_t == MOE_F32 ? 16 : 8;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(ws, 256) ||
      (residual && !aligned(residual, r_align)) || (out_bf16 && !aligned(out_bf16, 8)))
    return fail(MOE_EINVAL, "moe_layer_decode: misaligned buffer");
  const DecodeWs W = decode_ws(ws, T, k, q->E, q->H, q->I);
  if (ws_bytes < W.bytes)
    return fail(MOE_EWORKSPACE, fmt("moe_layer_decode: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)W.bytes));
  FoldedCombine fc;
  const bool fold = gemv_folds_combine(q->H, q->I);
  if (fold) {
    fc.w = w;
    fc.residual = residual;
    fc.r_t = r_t;
    fc.out = out;
    fc.out_bf16 = out_bf16;
  }
  if (fold && decode_routes_in_gateup(q->H, q->I, T, k))
    return launch_decode_routed(*q, logits, x, x_t, T, k, ids, w, offsets, sorted_assign, assign_pos, active,
                                n_active, W, y, y_t, fc, stream);
  if (moe_status st = launch_route_dispatch_decode(logits, T, q->E, k, ids, w, offsets, sorted_assign, assign_pos,
                                                   active, n_active, W, stream))
    return st;
  if (moe_status st = launch_ffn_gemv_steps(*q, x, x_t, T, k, sorted_assign, n_active, W, y, y_t, fc, stream))
    return st;
  return fold ? MOE_OK : launch_combine(y, y_t, w, T, k, q->H, residual, r_t, out, out_bf16, stream);
}

moe_status moe_layer_decode_slots(const moe_qlayer* q, moe_slot_table* t, int layer, const float* logits,
                                  const void* x, moe_dtype x_t, int T, int k, const void* residual, moe_dtype r_t,
                                  int32_t* ids, float* w, int32_t* offsets, int32_t* sorted_assign,
                                  int32_t* assign_pos, int32_t* active, int32_t* n_active, void* y, moe_dtype y_t,
                                  float* out, uint16_t* out_bf16, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "moe_layer_decode_slots";
  if (!q) return fail(MOE_EINVAL, "moe_layer_decode_slots: null moe_qlayer");
  if (!slot_table_device_mode(t)) return fail(MOE_EINVAL, "moe_layer_decode_slots: the table is not in device mode");
  const SlotTableView v = slot_table_view(t);
  if (layer < 0 || layer >= v.L) return fail(MOE_EINVAL, "moe_layer_decode_slots: layer out of range");
  if (q->E != v.E || q->base != v.slots || (size_t)q->stride != v.expert_bytes || q->slot_map != v.map + (size_t)layer * v.E)
    return fail(MOE_EINVAL, "moe_layer_decode_slots: q must be the table's view of `layer` (base = slots, stride = "
                            "expert_bytes, slot_map = map + layer * E)");
  if (T < 0) return fail(MOE_EINVAL, "moe_layer_decode_slots: T < 0");
  if (T > kDescT) return fail(MOE_EUNSUPPORTED, fmt("moe_layer_decode_slots: T=%lld above 12", T));
  if (moe_status st = check_ek(fn, q->E, k)) return st;
  if (moe_status st = check_shape(fn, q->H, q->I, q->bits)) return st;
  if ((int64_t)std::min(q->E, T * k) > v.n_slots)
    return fail(MOE_ECAPACITY, "moe_layer_decode_slots: more routed experts possible than slots");
  if (x_t != MOE_F32 && x_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode_slots: x dtype");
  if (y_t != MOE_F32 && y_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode_slots: y dtype");
  if (residual && r_t != MOE_F32 && r_t != MOE_BF16) return fail(MOE_EINVAL, "moe_layer_decode_slots: residual dtype");
  if (T == 0) return MOE_OK;
  if (!logits || !x || !ids || !w || !offsets || !sorted_assign || !assign_pos || !active || !n_active || !y || !out)
    return fail(MOE_EINVAL, "moe_layer_decode_slots: null pointer");
  const uintptr_t r_align = r_t == MOE_F32 ? 16 : 8;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(ws, 256) ||
      (residual && !aligned(residual, r_align)) || (out_bf16 && !aligned(out_bf16, 8)))
    return fail(MOE_EINVAL, "moe_layer_decode_slots: misaligned buffer");
  const DecodeWs W = decode_ws(ws, T, k, q->E, q->H, q->I);
  if (ws_bytes < W.bytes)
    return fail(MOE_EWORKSPACE, fmt("moe_layer_decode_slots: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)W.bytes));
  if (kResolveInGateup && gemv_stages_misses(q->H, q->I) && decode_routes_in_gateup(q->H, q->I, T, k)) {
    FoldedCombine fc;
    fc.w = w;
    fc.residual = residual;
    fc.r_t = r_t;
    fc.out = out;
    fc.out_bf16 = out_bf16;
    return launch_decode_routed_slots(*q, t, layer, logits, x, x_t, T, k, ids, w, offsets, sorted_assign, assign_pos,
                                      active, n_active, W, y, y_t, fc, stream);
  }
  if (moe_status st = launch_route_dispatch_resolve(logits, T, q->E, k, ids, w, offsets, sorted_assign, assign_pos,
                                                    active, n_active, W, t, layer, stream))
    return st;
  // Wide shapes stage the misses inside the gate/up launch, overlapping their
  // transfer with the resident experts' rows; other shapes copy them first.
  const bool stage = kStageInGateup && gemv_stages_misses(q->H, q->I);
  if (!stage)
    if (moe_status st = launch_slot_copy(t, stream)) return st;
  const MissStage ms{v.copies, v.ncopies, v.host_dev};
  FoldedCombine fc;
  const bool fold = gemv_folds_combine(q->H, q->I);
  if (fold) {
    fc.w = w;
    fc.residual = residual;
    fc.r_t = r_t;
    fc.out = out;
    fc.out_bf16 = out_bf16;
  }
  if (moe_status st = launch_ffn_gemv_steps(*q, x, x_t, T, k, sorted_assign, n_active, W, y, y_t, fc, stream,
                                            stage ? &ms : nullptr))
    return st;
  return fold ? MOE_OK : launch_combine(y, y_t, w, T, k, q->H, residual, r_t, out, out_bf16, stream);
}

moe_status moe_combine(const void* y, moe_dtype y_t, const float* w, int T, int k, int H, const void* residual,
                       moe_dtype r_t, float* out, uint16_t* out_bf16, hipStream_t stream) {
  if (T < 0 || H < 1) return fail(MOE_EINVAL, "moe_combine: T < 0 or H < 1");
  if (k < 1 || k > kMaxK) return fail(MOE_EUNSUPPORTED, "moe_combine: k outside [1, 16]");
  if (H % 4) return fail(MOE_EUNSUPPORTED, "moe_combine: H must be a multiple of 4");
  if (y_t != MOE_F32 && y_t != MOE_BF16) return fail(MOE_EINVAL, "moe_combine: y dtype");
  if (residual && r_t != MOE_F32 && r_t != MOE_BF16) return fail(MOE_EINVAL, "moe_combine: residual dtype");
  if (T == 0) return MOE_OK;
  if (!y || !w || !out) return fail(MOE_EINVAL, "moe_combine: null pointer");
  const uintptr_t r_align = r_t == MOE_F32 ? 16 : 8;
  if (!aligned(y, 16) || !aligned(out, 16) || (residual && !aligned(residual, r_align)) ||
      (out_bf16 && !aligned(out_bf16, 8)))
    return fail(MOE_EINVAL, "moe_combine: misaligned buffer");
  return launch_combine(y, y_t, w, T, k, H, residual, r_t, out, out_bf16, stream);
}

// ---- the trainable parts ----

size_t moe_balance_loss_workspace_bytes(int T, int E) {
  if (T < 0 || E < 1 || E > kMaxE) return 0;
  return balance_loss_ws_bytes(T, E);
}

moe_status moe_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int k,
                            float* loss, int32_t* counts, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_balance_loss: T < 0");
  if (moe_status st = check_ek("moe_balance_loss", E, k)) return st;
  if ((int64_t)T * k > (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "moe_balance_loss: T*k above 2^24");
  if (!loss || !counts) return fail(MOE_EINVAL, "moe_balance_loss: null pointer");
  if (T > 0 && (!logits || !ids || !lse)) return fail(MOE_EINVAL, "moe_balance_loss: null pointer");
  if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(lse, 4) ||
      !aligned(ws, 16))
    return fail(MOE_EINVAL, "moe_balance_loss: misaligned buffer");
  const size_t need = balance_loss_ws_bytes(T, E);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_balance_loss: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  const uint64_t n_t = (uint64_t)T * 4;
  const Span out[] = {{loss, 8}, {counts, (uint64_t)E * 4 + 4}, {lse, n_t}, {ws, need}};
  const Span in[] = {{logits, n_t * E}, {ids, n_t * k}, {mask, (uint64_t)T}};
  if (any_overlap(out, in)) return fail(MOE_EINVAL, "moe_balance_loss: an output or ws overlaps another buffer");
  return launch_balance_loss(logits, ids, mask, T, E, k, loss, counts, lse, ws, stream);
}

moe_status moe_route_backward(const float* logits, const int32_t* ids, const float* w, const float* dw,
                              const float* lse, const int32_t* counts, const float* dloss, int T, int E, int k,
                              float* dlogits, hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_route_backward: T < 0");
  if (moe_status st = check_ek("moe_route_backward", E, k)) return st;
  if ((int64_t)T * k > (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "moe_route_backward: T*k above 2^24");
  if (T == 0) return MOE_OK;
  if (!dlogits) return fail(MOE_EINVAL, "moe_route_backward: null pointer");
  if ((w == nullptr) != (dw == nullptr)) return fail(MOE_EINVAL, "moe_route_backward: w and dw go together");
  if ((lse == nullptr) != (counts == nullptr) || (lse == nullptr) != (dloss == nullptr))
    return fail(MOE_EINVAL, "moe_route_backward: lse, counts and dloss go together");
  if (!w && !lse) return fail(MOE_EINVAL, "moe_route_backward: neither gate weights nor losses");
  if ((w && !ids) || (lse && !logits)) return fail(MOE_EINVAL, "moe_route_backward: null pointer");
  if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(w, 4) || !aligned(dw, 4) || !aligned(lse, 4) ||
      !aligned(counts, 4) || !aligned(dloss, 4) || !aligned(dlogits, 4))
    return fail(MOE_EINVAL, "moe_route_backward: misaligned buffer");
  const uint64_t te = (uint64_t)T * E * 4, tk = (uint64_t)T * k * 4;
  if (overlap(dlogits, te, lse ? logits : nullptr, te) || overlap(dlogits, te, w, tk) || overlap(dlogits, te, dw, tk) ||
      overlap(dlogits, te, w ? ids : nullptr, tk) || overlap(dlogits, te, lse, (uint64_t)T * 4) ||
      overlap(dlogits, te, counts, (uint64_t)E * 4 + 4) || overlap(dlogits, te, dloss, 8))
    return fail(MOE_EINVAL, "moe_route_backward: dlogits overlaps an input");
  return launch_route_backward(logits, ids, w, dw, lse, counts, dloss, T, E, k, dlogits, stream);
}

moe_status moe_combine_backward(const void* y, moe_dtype y_t, const float* w, const void* dout, moe_dtype dout_t,
                                int T, int k, int H, float* dw, void* dy, hipStream_t stream) {
  if (T < 0 || H < 1) return fail(MOE_EINVAL, "moe_combine_backward: T < 0 or H < 1");
  if (k < 1 || k > kMaxK) return fail(MOE_EUNSUPPORTED, "moe_combine_backward: k outside [1, 16]");
  if (H % 4) return fail(MOE_EUNSUPPORTED, "moe_combine_backward: H must be a multiple of 4");
  if ((int64_t)T * k > (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "moe_combine_backward: T*k above 2^24");
  if (y_t != MOE_F32 && y_t != MOE_BF16) return fail(MOE_EINVAL, "moe_combine_backward: y dtype");
  if (dout_t != MOE_F32 && dout_t != MOE_BF16) return fail(MOE_EINVAL, "moe_combine_backward: dout dtype");
  if (T == 0) return MOE_OK;  // (pointers to no elements may be null)
  if (!dw && !dy) return fail(MOE_EINVAL, "moe_combine_backward: neither dw nor dy");
  if (!dout || (dw && !y) || (dy && !w)) return fail(MOE_EINVAL, "moe_combine_backward: null pointer");
  if (!aligned(y, 16) || !aligned(dy, 16) || !aligned(dout, 16) || !aligned(w, 4) || !aligned(dw, 4))
    return fail(MOE_EINVAL, "moe_combine_backward: misaligned buffer");
  const uint64_t ny = (uint64_t)T * k * H * (y_t == MOE_F32 ? 4 : 2), nd = (uint64_t)T * H * (dout_t == MOE_F32 ? 4 : 2),
                 nw = (uint64_t)T * k * 4;
  if (overlap(dy, ny, dw ? y : nullptr, ny) || overlap(dy, ny, dout, nd) || overlap(dy, ny, w, nw) ||
      overlap(dw, nw, y, ny) || overlap(dw, nw, dout, nd) || overlap(dw, nw, dy ? w : nullptr, nw) ||
      overlap(dw, nw, dy, ny))
    return fail(MOE_EINVAL, "moe_combine_backward: an output overlaps another buffer");
  return launch_combine_backward(y, y_t, w, dout, dout_t, T, k, H, dw, dy, stream);
}

}  // extern "C"

namespace {

constexpr int kLinearMaxT = 1 << 20, kLinearMaxK = 16384, kLinearMaxN = 16384;

bool is_act(moe_act a) {
  return a == MOE_ACT_NONE || a == MOE_ACT_GELU || a == MOE_ACT_SILU || a == MOE_ACT_SWIGLU;
}
bool linear_k(int K) { return K >= 32 && K <= kLinearMaxK && K % 32 == 0; }
bool linear_n(int N) { return N >= 1 && N <= kLinearMaxN; }

moe_status check_linear(const char* fn, int T, int K, int N, moe_act act) {
  if (T < 0) return fail(MOE_EINVAL, std::string(fn) + ": T < 0");
  if (!is_act(act)) return fail(MOE_EINVAL, std::string(fn) + ": activation");
  if (T > kLinearMaxT) return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": T=%lld above 2^20", T));
  if (!linear_k(K)) return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": K=%lld (multiple of 32 in [32, 16384])", K));
  if (!linear_n(N)) return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": N=%lld outside [1, 16384]", N));
  return MOE_OK;
}

// What a workspace is asked for: other calls, which are refused or have no rows, need none.
bool linear_has_work(int T, int K, int N, moe_act act) {
  return T >= 1 && T <= kLinearMaxT && linear_k(K) && linear_n(N) && is_act(act);
}
bool is_dtype(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }
uintptr_t elem(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }

constexpr int kNewtonMaxSide = 16384, kNewtonMaxSteps = 16;
constexpr float kNewtonCoef[3] = {3.4445f, -4.7750f, 2.0315f};

bool newton_size(int B, int R, int K) {  // of work there is
  if (B < 1 || R < 1 || K < 1 || R > kNewtonMaxSide || K > kNewtonMaxSide) return false;
  const int64_t per = ceil_div(R, 64) * ceil_div(K, 64) * 4096;
  return B <= ((int64_t)1 << 33) / per;
}
moe_status check_newton(const char* fn, int B, int R, int K) {
  if (B < 0) return fail(MOE_EINVAL, std::string(fn) + ": B < 0");
  if (!newton_size(B < 1 ? 1 : B, R, K))
    return fail(MOE_EUNSUPPORTED, std::string(fn) + fmt(": B=%lld, R=%lld, K=%lld (R and K in [1, 16384], padded values up to 2^33)",
                                                        B, R, K));
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int T, int K, int N, moe_act act, moe_dtype x_t, moe_dtype y_t) {
  if (!linear_has_work(T, K, N, act) || !is_dtype(x_t) || !is_dtype(y_t)) return 0;
  return linear_ws_bytes(T, K, N, act, x_t, y_t);
}

moe_status moe_linear(const void* x, moe_dtype x_t, const void* w, const float* bias, moe_act act,
                      const void* residual, moe_dtype r_t, int T, int K, int N, void* y, moe_dtype y_t, void* pre,
                      void* ws, size_t ws_bytes, hipStream_t stream) {
  if (moe_status st = check_linear("moe_linear", T, K, N, act)) return st;
  if (!is_dtype(x_t)) return fail(MOE_EINVAL, "moe_linear: x dtype");
  if (!is_dtype(y_t)) return fail(MOE_EINVAL, "moe_linear: y dtype");
  if (residual && !is_dtype(r_t)) return fail(MOE_EINVAL, "moe_linear: residual dtype");
  if (T == 0) return MOE_OK;
  if (!x || !w || !y) return fail(MOE_EINVAL, "moe_linear: null pointer");
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(ws, 256) || !aligned(bias, 4) || !aligned(y, elem(y_t)) ||
      !aligned(pre, elem(y_t)) || (residual && !aligned(residual, elem(r_t))))
    return fail(MOE_EINVAL, "moe_linear: misaligned buffer (x and w need 16 bytes, ws 256)");
  const size_t need = linear_ws_bytes(T, K, N, act, x_t, y_t);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_linear: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  const uint64_t R = act == MOE_ACT_SWIGLU ? 2 * (uint64_t)N : N;
  const uint64_t nx = (uint64_t)T * K * elem(x_t), nw = R * K * 2, ny = (uint64_t)T * N * elem(y_t),
                 np = (uint64_t)T * R * elem(y_t), nr = (uint64_t)T * N * elem(r_t);
  // y may be the residual itself, which nothing else may touch
  const bool in_place = residual == y && r_t == y_t;
  const Span out[] = {{y, ny}, {pre, np}, {ws, need}};
  const Span in[] = {{x, nx}, {w, nw}, {bias, R * 4}, {in_place ? nullptr : residual, nr}};
  if (any_overlap(out, in))
    return fail(MOE_EINVAL, "moe_linear: an output or ws overlaps another buffer (y may only be the residual itself)");
  return launch_linear(x, x_t, reinterpret_cast<const uint16_t*>(w), bias, act, residual, r_t, T, K, N, y, y_t, pre, ws,
                       stream);
}

size_t moe_linear_backward_workspace_bytes(int T, int K, int N, moe_act act, moe_dtype dy_t, moe_dtype x_t,
                                           moe_dtype dx_t, moe_dtype dw_t, int need) {
  if (!linear_has_work(T, K, N, act) || !is_dtype(dy_t) || !is_dtype(x_t) || !is_dtype(dx_t) || !is_dtype(dw_t)) return 0;
  return linear_backward_ws_bytes(T, K, N, act, dy_t, x_t, dx_t, dw_t, need);
}

moe_status moe_linear_backward(const void* dy, moe_dtype dy_t, const void* pre, const void* x, moe_dtype x_t,
                               const void* w, moe_act act, int T, int K, int N, void* dx, moe_dtype dx_t, void* dw,
                               moe_dtype dw_t, float* db, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (moe_status st = check_linear("moe_linear_backward", T, K, N, act)) return st;
  if (!is_dtype(dy_t)) return fail(MOE_EINVAL, "moe_linear_backward: dy dtype");
  if (!is_dtype(x_t)) return fail(MOE_EINVAL, "moe_linear_backward: x dtype");
  if (!is_dtype(dx_t) || !is_dtype(dw_t)) return fail(MOE_EINVAL, "moe_linear_backward: dx or dw dtype");
  if (T > 0 && !dx && !dw && !db) return fail(MOE_EINVAL, "moe_linear_backward: no output wanted");
  if (T > 0 && (!dy || (dw && !x) || (dx && !w) || (act != MOE_ACT_NONE && !pre)))
    return fail(MOE_EINVAL, "moe_linear_backward: null pointer");
  if ((dw && !aligned(x, 16)) || (dx && !aligned(w, 16)) || !aligned(ws, 256) || !aligned(dx, 16) || !aligned(dw, 16) ||
      !aligned(db, 4) || !aligned(dy, elem(dy_t)) || (act != MOE_ACT_NONE && !aligned(pre, elem(dy_t))))
    return fail(MOE_EINVAL, "moe_linear_backward: misaligned buffer (x, w, dx and dw need 16 bytes, ws 256)");
  const int bits = (dx ? MOE_NEED_DX : 0) | (dw ? MOE_NEED_DW : 0) | (db ? MOE_NEED_DB : 0);
  const size_t need = T > 0 ? linear_backward_ws_bytes(T, K, N, act, dy_t, x_t, dx_t, dw_t, bits) : 0;
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_linear_backward: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  const uint64_t R = act == MOE_ACT_SWIGLU ? 2 * (uint64_t)N : N;
  const Span out[] = {{dx, (uint64_t)T * K * elem(dx_t)}, {dw, R * K * elem(dw_t)}, {db, R * 4}, {ws, need}};
  const Span in[] = {{dy, (uint64_t)T * N * elem(dy_t)},
                     {act == MOE_ACT_NONE ? nullptr : pre, (uint64_t)T * R * elem(dy_t)},
                     {dw ? x : nullptr, (uint64_t)T * K * elem(x_t)},
                     {dx ? w : nullptr, R * K * 2}};
  if (any_overlap(out, in)) return fail(MOE_EINVAL, "moe_linear_backward: an output or ws overlaps another buffer");
  return launch_linear_backward(dy, dy_t, pre, x, x_t, reinterpret_cast<const uint16_t*>(w), act, T, K, N, dx, dx_t, dw,
                                dw_t, db, ws, stream);
}

moe_status moe_linear_form(int T, int K, int N, moe_act act, moe_dtype x_t, moe_dtype y_t, int32_t form[4]) {
  if (moe_status st = check_linear("moe_linear_form", T, K, N, act)) return st;
  if (T == 0 || !form) return fail(MOE_EINVAL, "moe_linear_form: no rows, or a null pointer");
  if (!is_dtype(x_t) || !is_dtype(y_t)) return fail(MOE_EINVAL, "moe_linear_form: dtype");
  linear_form(T, K, N, act, x_t, y_t, form);
  return MOE_OK;
}

moe_status moe_linear_backward_form(int T, int K, int N, moe_act act, moe_dtype dy_t, moe_dtype x_t, moe_dtype dx_t,
                                    moe_dtype dw_t, int need, int32_t form[4]) {
  if (moe_status st = check_linear("moe_linear_backward_form", T, K, N, act)) return st;
  if (T == 0 || !form) return fail(MOE_EINVAL, "moe_linear_backward_form: no rows, or a null pointer");
  if (!is_dtype(dy_t) || !is_dtype(x_t) || !is_dtype(dx_t) || !is_dtype(dw_t))
    return fail(MOE_EINVAL, "moe_linear_backward_form: dtype");
  linear_backward_form(T, K, N, act, dy_t, x_t, dx_t, dw_t, need, form);
  return MOE_OK;
}

size_t moe_orthogonalize_workspace_bytes(int B, int R, int K, moe_dtype o_t) {
  if (!newton_size(B, R, K) || !is_dtype(o_t)) return 0;
  return orthogonalize_ws_bytes(B, R, K, o_t);
}

moe_status moe_orthogonalize(const void* g, moe_dtype g_t, float* momentum, double beta, int nesterov, int B, int R, int K,
                             int steps, const float* coef, double eps, void* o, moe_dtype o_t, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  if (moe_status st = check_newton("moe_orthogonalize", B, R, K)) return st;
  if (!is_dtype(g_t) || !is_dtype(o_t)) return fail(MOE_EINVAL, "moe_orthogonalize: g or o dtype");
  if (!(beta >= 0.0 && beta < 1.0)) return fail(MOE_EINVAL, "moe_orthogonalize: beta outside [0, 1)");
  if (!(eps >= 0.0 && eps < __builtin_huge_val())) return fail(MOE_EINVAL, "moe_orthogonalize: eps");
  if (steps < 1 || steps > kNewtonMaxSteps) return fail(MOE_EUNSUPPORTED, fmt("moe_orthogonalize: steps=%lld outside [1, 16]", steps));
  float every[3 * kNewtonMaxSteps];
  for (int i = 0; i < 3 * steps; ++i) {
    every[i] = coef ? coef[i] : kNewtonCoef[i % 3];
    if (!__builtin_isfinite(every[i])) return fail(MOE_EINVAL, "moe_orthogonalize: a coefficient is not finite");
  }
  if (B == 0) return MOE_OK;
  if (!g || !o) return fail(MOE_EINVAL, "moe_orthogonalize: null pointer");
  if (!aligned(g, elem(g_t)) || !aligned(o, elem(o_t)) || !aligned(momentum, 4) || !aligned(ws, 256))
    return fail(MOE_EINVAL, "moe_orthogonalize: misaligned buffer (ws needs 256 bytes)");
  const size_t need = orthogonalize_ws_bytes(B, R, K, o_t);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, fmt("moe_orthogonalize: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  const uint64_t n = (uint64_t)B * R * K;
  const Span out[] = {{momentum, n * 4}, {o, n * elem(o_t)}, {ws, need}};
  const Span in[] = {{g, n * elem(g_t)}};
  if (any_overlap(out, in)) return fail(MOE_EINVAL, "moe_orthogonalize: an output or ws overlaps another buffer");
  return launch_orthogonalize(g, g_t, momentum, beta, nesterov, B, R, K, steps, every, eps, o, o_t, ws, stream);
}

moe_status moe_orthogonalize_form(int B, int R, int K, moe_dtype o_t, int32_t form[4]) {
  if (moe_status st = check_newton("moe_orthogonalize_form", B, R, K)) return st;
  if (B == 0 || !form) return fail(MOE_EINVAL, "moe_orthogonalize_form: no matrices, or a null pointer");
  if (!is_dtype(o_t)) return fail(MOE_EINVAL, "moe_orthogonalize_form: dtype");
  orthogonalize_form(B, R, K, o_t, form);
  return MOE_OK;
}

moe_status moe_quantize_rows(const void* x, moe_dtype x_t, int T, int K, int8_t* q, float* scale, hipStream_t stream) {
  if (T < 0) return fail(MOE_EINVAL, "moe_quantize_rows: T < 0");
  if (T > kLinearMaxT) return fail(MOE_EUNSUPPORTED, fmt("moe_quantize_rows: T=%lld above 2^20", T));
  if (!linear_k(K)) return fail(MOE_EUNSUPPORTED, fmt("moe_quantize_rows: K=%lld (multiple of 32 in [32, 16384])", K));
  if (!is_dtype(x_t)) return fail(MOE_EINVAL, "moe_quantize_rows: x dtype");
  if (T == 0) return MOE_OK;
  if (!x || !q || !scale) return fail(MOE_EINVAL, "moe_quantize_rows: null pointer");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4))
    return fail(MOE_EINVAL, "moe_quantize_rows: misaligned buffer (x and q need 16 bytes)");
  const uint64_t n = (uint64_t)T * K;
  const Span out[] = {{q, n}, {scale, (uint64_t)T * 4}};
  const Span in[] = {{x, n * elem(x_t)}};
  if (any_overlap(out, in)) return fail(MOE_EINVAL, "moe_quantize_rows: an output overlaps another buffer");
  return launch_quantize_rows(x, x_t, T, K, q, scale, stream);
}

size_t moe_linear_q8_workspace_bytes(int T, int K, int N, moe_act act, moe_dtype x_t) {
  if (!linear_has_work(T, K, N, act) || !(is_dtype(x_t) || x_t == MOE_I8)) return 0;
  return linear_q8_ws_bytes(T, K, N, act, x_t);
}

moe_status moe_linear_q8(const void* x, moe_dtype x_t, const float* x_scale, const int8_t* w, const float* w_scale,
                         const float* bias, moe_act act, const void* residual, moe_dtype r_t, int T, int K, int N,
                         void* y, moe_dtype y_t, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (moe_status st = check_linear("moe_linear_q8", T, K, N, act)) return st;
  if (!is_dtype(x_t) && x_t != MOE_I8) return fail(MOE_EINVAL, "moe_linear_q8: x dtype");
  if (!is_dtype(y_t)) return fail(MOE_EINVAL, "moe_linear_q8: y dtype");
  if (residual && !is_dtype(r_t)) return fail(MOE_EINVAL, "moe_linear_q8: residual dtype");
  if (x_t != MOE_I8 && x_scale) return fail(MOE_EINVAL, "moe_linear_q8: x_scale goes with 8-bit x");
  if (T == 0) return MOE_OK;
  if (!x || !w || !w_scale || !y || (x_t == MOE_I8 && !x_scale)) return fail(MOE_EINVAL, "moe_linear_q8: null pointer");
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(ws, 256) || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(bias, 4) || !aligned(y, elem(y_t)) || (residual && !aligned(residual, elem(r_t))))
    return fail(MOE_EINVAL, "moe_linear_q8: misaligned buffer (x and w need 16 bytes, ws 256)");
  const size_t need = linear_q8_ws_bytes(T, K, N, act, x_t);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, fmt("moe_linear_q8: workspace %lld bytes, needs %lld", (long long)ws_bytes,
                                    (long long)need));
  const uint64_t R = act == MOE_ACT_SWIGLU ? 2 * (uint64_t)N : N;
  // y may be the residual itself, which nothing else may touch
  const bool in_place = residual == y && r_t == y_t;
  const Span out[] = {{y, (uint64_t)T * N * elem(y_t)}, {ws, need}};
  const Span in[] = {{x, (uint64_t)T * K * (x_t == MOE_I8 ? 1 : elem(x_t))}, {x_scale, (uint64_t)T * 4}, {w, R * K},
                     {w_scale, R * 4}, {bias, R * 4},
                     {in_place ? nullptr : residual, residual ? (uint64_t)T * N * elem(r_t) : 0}};
  if (any_overlap(out, in))
    return fail(MOE_EINVAL, "moe_linear_q8: an output or ws overlaps another buffer (y may only be the residual itself)");
  return launch_linear_q8(x, x_t, x_scale, w, w_scale, bias, act, residual, r_t, T, K, N, y, y_t, ws, stream);
}

moe_status moe_linear_q8_form(int T, int K, int N, moe_act act, moe_dtype x_t, int32_t form[3]) {
  if (moe_status st = check_linear("moe_linear_q8_form", T, K, N, act)) return st;
  if (T == 0 || !form) return fail(MOE_EINVAL, "moe_linear_q8_form: no rows, or a null pointer");
  if (!is_dtype(x_t) && x_t != MOE_I8) return fail(MOE_EINVAL, "moe_linear_q8_form: dtype");
  linear_q8_form(T, K, N, act, x_t, form);
  return MOE_OK;
}

moe_status moe_profile_next_launch(moe_kernel kernel, hipEvent_t start, hipEvent_t stop) {
  if ((int)kernel < 0 || (int)kernel > (int)MOE_KERNEL_ORTHOGONALIZE) return fail(MOE_EINVAL, "moe_profile_next_launch: kernel");
  if (!start || !stop) return fail(MOE_EINVAL, "moe_profile_next_launch: null event");
  ProfileReq& p = profile_req();
  p.kernel = (int)kernel;
  p.start = start;
  p.stop = stop;
  return MOE_OK;
}

}  // extern "C"
