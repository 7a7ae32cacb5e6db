// api.hip -- host side of the C ABI declared in include/moe_decode.h:
// argument validation, workspace layout and kernel launches.  All checks are
// host-only and run before anything is enqueued.
#include "moe_decode.h"

#include <mutex>
#include <new>

#include "device_common.h"
#include "embed.h"
#include "lm_loss.h"
#include "lora.h"
#include "products.h"
#include "token_rows.h"
#include "wide.h"

namespace moe {
hipError_t launch_router(const uint16_t* x, const Weights& w, const Ws& ws, const Dims& d,
                         hipStream_t stream);
hipError_t launch_route(int rfmt, const Weights& w, const Ws& ws, const Dims& d,
                        hipStream_t stream);
bool fused_route(const Dims& d);
hipError_t launch_upgate(int rfmt, int max_groups, const Weights& w, const Ws& ws,
                         const Dims& d, hipStream_t stream);
hipError_t launch_down(int rfmt, int max_groups, const Weights& w, const Ws& ws, const Dims& d,
                       hipStream_t stream);
hipError_t launch_combine(const Ws& ws, const Dims& d, uint16_t* out, hipStream_t stream);
int upgate_k_parts(int hidden, int routed_fmt);
hipError_t launch_lowbit_q1(const uint8_t* blocks, const uint16_t* x, uint16_t* y, int rows,
                            int n, int k, const LoraArgs* lora, hipStream_t stream);
hipError_t launch_gemv_fp8(const uint8_t* codes, const float* scales, const uint16_t* x,
                           uint16_t* y, int rows, int n, int k, const LoraArgs* lora,
                           hipStream_t stream);
hipError_t launch_gemv_bf16(const uint16_t* w, const uint16_t* x, uint16_t* y, int rows, int n,
                            int k, const LoraArgs* lora, hipStream_t stream);

__global__ void moe_fill_u32_kernel(uint32_t* p, size_t n, uint32_t v) {
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x)
    p[i] = v;
}
}  // namespace moe

using namespace moe;

// Device scratch of moe_decode_step_noalloc: the workspace of a step that
// brings none.  One copy per GPU the library runs on, held until the process
// ends.  In host code `scratch` names a host-side stand-in, not the device
// array: the device address comes from hipGetSymbolAddress, once per device
// (scratch_on_device below), and only that address is handed to kernels.
constexpr size_t kScratchBytes = MOE_DECODE_NOALLOC_MAX_WORKSPACE;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

namespace {

constexpr uint32_t kKnownFlags = MOE_F_NO_DEDUP;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Plan {
  int H, I, E, Is, R, imax, groups, ks;
  size_t off_logits, off_rstd, off_ids, off_gates, off_ngroups, off_gexpert,
      off_gowner, off_gmask, off_gslot, off_grows, off_gnrows, off_actq, off_actqp, off_acts, off_mid,
      off_midq, off_midqs, off_ypart, off_actu, off_blkrec, off_waitto, total;
};

bool is_mult(int v, int m) { return v > 0 && v % m == 0; }

moe_status plan_config(const moe_decode_config* c, Plan* p) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->top_k != 8) return MOE_ERR_UNSUPPORTED;
  if (!is_mult(c->hidden, 128) || c->hidden > 16384) return MOE_ERR_UNSUPPORTED;
  if (!is_mult(c->inter, 128) || c->inter > 16384) return MOE_ERR_UNSUPPORTED;
  // the shared expert, when present, has the routed experts' intermediate size
  if (c->shared_inter != 0 && c->shared_inter != c->inter) return MOE_ERR_UNSUPPORTED;
  if (!is_mult(c->n_experts, 16) || c->n_experts > 1024) return MOE_ERR_UNSUPPORTED;
  if (c->max_rows < 1 || c->max_rows > 8) return MOE_ERR_INVALID_ARG;
  if (c->routed_fmt != MOE_FMT_FP8_E4M3_B128 && c->routed_fmt != MOE_FMT_MXFP4 &&
      c->routed_fmt != MOE_FMT_Q1_G128)
    return MOE_ERR_UNSUPPORTED;
  // 1-bit routed experts: up/gate items of 4 groups (hidden % 512), down rows
  // of whole 36-byte chunks loaded at once (inter % 256, at most 4096), FP8
  // activations (their MFMA is FP8 x FP8)
  if (c->routed_fmt == MOE_FMT_Q1_G128 &&
      (c->hidden % 512 || c->inter % 256 || c->inter > 4096 || c->act_fmt != MOE_ACT_FP8_B128))
    return MOE_ERR_UNSUPPORTED;
  // MXFP4 up/gate items are two K blocks wide; the down GEMV keeps its
  // columns' mid split into bf16 hi + lo in LDS (4 bytes an element, up to 8
  // columns): I <= 4096
  if (c->routed_fmt == MOE_FMT_MXFP4 && (c->hidden % 256 || c->inter > 4096))
    return MOE_ERR_UNSUPPORTED;
  if (c->shared_inter > 0 && c->shared_fmt != MOE_FMT_FP8_E4M3_B128) return MOE_ERR_UNSUPPORTED;
  if (c->flags & ~kKnownFlags) return MOE_ERR_UNSUPPORTED;
  if (c->act_fmt != MOE_ACT_FP8_B128 && c->act_fmt != MOE_ACT_BF16) return MOE_ERR_UNSUPPORTED;
  // bf16 activations: the up/gate's bf16 MFMA takes FP8 weights only
  if (c->act_fmt == MOE_ACT_BF16 && c->routed_fmt != MOE_FMT_FP8_E4M3_B128)
    return MOE_ERR_UNSUPPORTED;
  if (!(c->rms_eps >= 0.0f) || c->rms_eps > 1.0f) return MOE_ERR_INVALID_ARG;

  p->H = c->hidden;
  p->I = c->inter;
  p->E = c->n_experts;
  p->Is = c->shared_inter;
  p->R = c->max_rows;
  p->imax = p->I > p->Is ? p->I : p->Is;
  const int picks = 8 * p->R;
  p->groups = (c->flags & MOE_F_NO_DEDUP) ? picks : (picks < p->E ? picks : p->E);
  p->ks = upgate_k_parts(p->H, c->routed_fmt);

  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  const size_t R = p->R, E = p->E, H = p->H, G = p->groups, IM = p->imax;
  p->off_logits = take(R * E * 4);
  p->off_rstd = take(R * 4);
  p->off_ids = take(R * 8 * 4);
  p->off_gates = take(R * 8 * 4);
  p->off_ngroups = take(4);
  p->off_gexpert = take(G * 4);
  p->off_gowner = take(G * 2);
  p->off_gmask = take(G);
  p->off_gslot = take(G * 8);
  p->off_grows = take(G * 8);
  p->off_gnrows = take(G);
  p->off_actq = take(R * H);
  p->off_actqp = take(c->routed_fmt == MOE_FMT_Q1_G128 ? R * H : 0);  // 1-bit operand order
  p->off_acts = take(R * (H / 128) * 4);
  const size_t U = R * 9;  // (row, pick) pairs, pick 8 = the shared expert
  p->off_mid = take(U * IM * 4);
  p->off_midq = take(U * IM);
  p->off_midqs = take(U * (IM / 128) * 4);
  p->off_ypart = take(U * H * 4);
  p->off_actu = take(R * H * 2);
  // one record per up/gate block of the routing launch: at most Is/16 + G*I/16
  p->off_blkrec = take((p->Is / 16 + G * (p->I / 16)) * 8);
  p->off_waitto = take(4);
  p->total = o;
  return MOE_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// The kernels' view of a workspace laid out by `p` from base address `b`.
Ws make_view(char* b, const Plan& p) {
  Ws v;
  v.logits = reinterpret_cast<float*>(b + p.off_logits);
  v.rstd = reinterpret_cast<float*>(b + p.off_rstd);
  v.ids = reinterpret_cast<int32_t*>(b + p.off_ids);
  v.gates = reinterpret_cast<float*>(b + p.off_gates);
  v.n_groups = reinterpret_cast<int32_t*>(b + p.off_ngroups);
  v.grp_expert = reinterpret_cast<int32_t*>(b + p.off_gexpert);
  v.grp_owner = reinterpret_cast<uint8_t*>(b + p.off_gowner);
  v.grp_mask = reinterpret_cast<uint8_t*>(b + p.off_gmask);
  v.grp_slot = reinterpret_cast<uint8_t*>(b + p.off_gslot);
  v.grp_rows = reinterpret_cast<uint8_t*>(b + p.off_grows);
  v.grp_nrows = reinterpret_cast<uint8_t*>(b + p.off_gnrows);
  v.act_q = reinterpret_cast<uint8_t*>(b + p.off_actq);
  v.act_qp = reinterpret_cast<uint8_t*>(b + p.off_actqp);
  v.act_s = reinterpret_cast<float*>(b + p.off_acts);
  v.mid = reinterpret_cast<float*>(b + p.off_mid);
  v.midq = reinterpret_cast<uint8_t*>(b + p.off_midq);
  v.midqs = reinterpret_cast<float*>(b + p.off_midqs);
  v.ypart = reinterpret_cast<float*>(b + p.off_ypart);
  v.act_u = reinterpret_cast<uint16_t*>(b + p.off_actu);
  v.blk_rec = reinterpret_cast<uint64_t*>(b + p.off_blkrec);
  v.wait_timeouts = reinterpret_cast<uint32_t*>(b + p.off_waitto);
  return v;
}

}  // namespace

struct moe_decode_ctx {
  moe_decode_config cfg;
  Plan plan;
  char* ws;
  Ws view;
  hipEvent_t events[MOE_DECODE_N_KERNELS + 1];
  bool timing;
  int last_rows;  // rows of the last step enqueued, 0 before the first
  uint32_t wait_ticks;  // cap of the routing launch's waits
  int withhold;         // 1: the routing block publishes no records
};

// Default cap of a routed up/gate block's wait for its record: 10 ms of the
// 100 MHz real-time counter, far beyond the routing's few microseconds.
constexpr uint32_t kDefaultWaitTicks = 1000000u;

extern "C" {

size_t moe_decode_workspace_size(const moe_decode_config* cfg) {
  Plan p;
  if (plan_config(cfg, &p) != MOE_OK) return 0;
  return p.total;
}

moe_status moe_decode_init(const moe_decode_config* cfg, void* workspace, size_t ws_bytes,
                           hipStream_t stream, moe_decode_ctx** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  Plan p;
  moe_status st = plan_config(cfg, &p);
  if (st != MOE_OK) return st;
  if (!workspace || ((uintptr_t)workspace & 255u)) return MOE_ERR_WORKSPACE;
  if (ws_bytes < p.total) return MOE_ERR_WORKSPACE;
  moe_decode_ctx* c = new (std::nothrow) moe_decode_ctx();
  if (!c) return MOE_ERR_DEVICE;
  c->cfg = *cfg;
  c->plan = p;
  c->ws = static_cast<char*>(workspace);
  c->timing = false;
  c->last_rows = 0;
  c->wait_ticks = kDefaultWaitTicks;
  c->withhold = 0;
  c->view = make_view(c->ws, p);
  // clear the whole workspace once, so that debug views read before the
  // first step are well defined
  const size_t words = p.total / 4;
  hipLaunchKernelGGL(moe_fill_u32_kernel, dim3(256), dim3(256), 0, stream,
                     reinterpret_cast<uint32_t*>(c->ws), words, 0u);
  if (hipGetLastError() != hipSuccess) {
    delete c;
    return MOE_ERR_DEVICE;
  }
  *out = c;
  return MOE_OK;
}

namespace {
// Validates the weights and fills the kernels' argument views for a step of
// `rows` rows of a layer with config `cfg` and plan `p`.
moe_status step_args(const moe_decode_config& cfg, const Plan& p, int rows,
                     const moe_decode_weights* w, Weights* wtp, Dims* dp) {
  if (!w) return MOE_ERR_INVALID_ARG;
  const void* need[] = {w->rms_gamma, w->router_w, w->gate.codes, w->up.codes, w->down.codes};
  for (const void* q : need)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (cfg.routed_fmt != MOE_FMT_Q1_G128) {  // 1-bit blocks hold their own scales
    const void* sc[] = {w->gate.scales, w->up.scales, w->down.scales};
    for (const void* q : sc)
      if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  }
  if (p.Is > 0) {
    const void* sh[] = {w->sh_gate.codes, w->sh_gate.scales, w->sh_up.codes,
                        w->sh_up.scales, w->sh_down.codes, w->sh_down.scales};
    for (const void* q : sh)
      if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  }
  Weights& wt = *wtp;
  wt.gamma = w->rms_gamma;
  wt.router = w->router_w;
  wt.gate_c = static_cast<const uint8_t*>(w->gate.codes);
  wt.up_c = static_cast<const uint8_t*>(w->up.codes);
  wt.down_c = static_cast<const uint8_t*>(w->down.codes);
  wt.gate_s = w->gate.scales;
  wt.up_s = w->up.scales;
  wt.down_s = w->down.scales;
  wt.sg_c = static_cast<const uint8_t*>(w->sh_gate.codes);
  wt.su_c = static_cast<const uint8_t*>(w->sh_up.codes);
  wt.sd_c = static_cast<const uint8_t*>(w->sh_down.codes);
  wt.sg_s = static_cast<const float*>(w->sh_gate.scales);
  wt.su_s = static_cast<const float*>(w->sh_up.scales);
  wt.sd_s = static_cast<const float*>(w->sh_down.scales);

  Dims& d = *dp;
  d.H = p.H;
  d.I = p.I;
  d.E = p.E;
  d.Is = p.Is;
  d.rows = rows;
  d.max_rows = p.R;
  d.imax = p.imax;
  d.ks = p.ks;
  d.no_dedup = (cfg.flags & MOE_F_NO_DEDUP) ? 1 : 0;
  d.eps = cfg.rms_eps;
  d.act_bf16 = cfg.act_fmt == MOE_ACT_BF16 ? 1 : 0;
  d.act_q1 = cfg.routed_fmt == MOE_FMT_Q1_G128 ? 1 : 0;
  const int picks = 8 * rows;
  d.groups = d.no_dedup ? picks : (picks < p.E ? picks : p.E);
  d.wait_ticks = kDefaultWaitTicks;
  d.withhold = 0;
  return MOE_OK;
}

// Groups a step of `rows` rows can produce: at most 8 * rows (and E with dedup).

// Host checks of a step's x and out (rows >= 1).
moe_status check_io(const Plan& p, const uint16_t* x, int rows, const moe_decode_weights* w,
                    const uint16_t* out) {
  if (!x || !w || !out || !aligned16(x) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)rows * p.H * 2;
  const uintptr_t xa = (uintptr_t)x, oa = (uintptr_t)out;
  if (xa < oa + bytes && oa < xa + bytes) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The device address of `scratch` on the current device, looked up once per
// device under a lock and kept.
moe_status scratch_on_device(char** out) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static char* addr[kMaxDevices] = {};
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return MOE_ERR_DEVICE;
    addr[dev] = static_cast<char*>(p);
  }
  *out = addr[dev];
  return MOE_OK;
}

// The step's five launches on `stream` over workspace view `v`; with `ev`,
// an event before the first and after each.
moe_status enqueue_step(int routed_fmt, const Plan& p, const Ws& v, const uint16_t* x,
                        const Weights& wt, const Dims& d, uint16_t* out, hipStream_t stream,
                        hipEvent_t* ev) {
  if (ev && hipEventRecord(ev[0], stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (launch_router(x, wt, v, d, stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (ev && hipEventRecord(ev[1], stream) != hipSuccess) return MOE_ERR_DEVICE;
  // routing, with the up/gate of the shared and the routed experts alongside
  // (or the routing alone, then the up/gate)
  if (launch_route(routed_fmt, wt, v, d, stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (ev && hipEventRecord(ev[2], stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (!fused_route(d) && launch_upgate(routed_fmt, d.groups, wt, v, d, stream) != hipSuccess)
    return MOE_ERR_DEVICE;
  if (ev && hipEventRecord(ev[3], stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (launch_down(routed_fmt, d.groups, wt, v, d, stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (ev && hipEventRecord(ev[4], stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (launch_combine(v, d, out, stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (ev && hipEventRecord(ev[5], stream) != hipSuccess) return MOE_ERR_DEVICE;
  return MOE_OK;
}
}  // namespace

moe_status moe_decode_step(moe_decode_ctx* ctx, const uint16_t* x, int32_t rows,
                           const moe_decode_weights* w, uint16_t* out, hipStream_t stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const Plan& p = ctx->plan;
  if (rows < 0 || rows > p.R) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  moe_status st = check_io(p, x, rows, w, out);
  if (st != MOE_OK) return st;
  Weights wt;
  Dims d;
  st = step_args(ctx->cfg, p, rows, w, &wt, &d);
  if (st != MOE_OK) return st;
  d.wait_ticks = ctx->wait_ticks;
  d.withhold = ctx->withhold;
  ctx->last_rows = rows;
  return enqueue_step(ctx->cfg.routed_fmt, p, ctx->view, x, wt, d, out, stream,
                      ctx->timing ? ctx->events : nullptr);
}

moe_status moe_decode_step_noalloc(const moe_decode_config* cfg, const uint16_t* x,
                                   int32_t rows, const moe_decode_weights* w, uint16_t* out,
                                   hipStream_t stream) {
  Plan p;
  moe_status st = plan_config(cfg, &p);
  if (st != MOE_OK) return st;
  if (p.total > kScratchBytes) return MOE_ERR_WORKSPACE;
  if (rows < 0 || rows > p.R) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  st = check_io(p, x, rows, w, out);
  if (st != MOE_OK) return st;
  Weights wt;
  Dims d;
  st = step_args(*cfg, p, rows, w, &wt, &d);
  if (st != MOE_OK) return st;
  char* base = nullptr;
  st = scratch_on_device(&base);
  if (st != MOE_OK) return st;
  return enqueue_step(cfg->routed_fmt, p, make_view(base, p), x, wt, d, out, stream, nullptr);
}

moe_status moe_decode_debug_view(const moe_decode_ctx* ctx, moe_decode_debug* v) {
  if (!ctx || !v) return MOE_ERR_INVALID_ARG;
  const Ws& w = ctx->view;
  v->logits = w.logits;
  v->rstd = w.rstd;
  v->ids = w.ids;
  v->gates = w.gates;
  v->n_groups = w.n_groups;
  v->grp_expert = w.grp_expert;
  v->grp_owner = w.grp_owner;
  v->grp_mask = w.grp_mask;
  v->grp_slot = w.grp_slot;
  v->act_q = w.act_q;
  v->act_s = w.act_s;
  v->mid = w.mid;
  v->midq = w.midq;
  v->midqs = w.midqs;
  v->y = w.ypart;
  v->max_groups = ctx->plan.groups;
  v->mid_stride = ctx->plan.imax;
  return MOE_OK;
}

moe_status moe_decode_set_timing(moe_decode_ctx* ctx, hipEvent_t* events) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  if (!events) {
    ctx->timing = false;
    return MOE_OK;
  }
  for (int i = 0; i <= MOE_DECODE_N_KERNELS; i++) {
    if (!events[i]) return MOE_ERR_INVALID_ARG;
    ctx->events[i] = events[i];
  }
  ctx->timing = true;
  return MOE_OK;
}

moe_status moe_decode_relaunch(moe_decode_ctx* ctx, int32_t kernel,
                               const moe_decode_weights* w, int32_t reps, hipStream_t stream) {
  if (!ctx || reps < 0) return MOE_ERR_INVALID_ARG;
  if (kernel != MOE_DECODE_K_UPGATE && kernel != MOE_DECODE_K_DOWN) return MOE_ERR_INVALID_ARG;
  if (ctx->last_rows == 0) return MOE_ERR_INVALID_ARG;
  Weights wt;
  Dims d;
  const moe_status st = step_args(ctx->cfg, ctx->plan, ctx->last_rows, w, &wt, &d);
  if (st != MOE_OK) return st;
  d.wait_ticks = ctx->wait_ticks;
  const int rf = ctx->cfg.routed_fmt;
  for (int i = 0; i < reps; i++) {
    hipError_t e;
    if (kernel == MOE_DECODE_K_DOWN)
      e = launch_down(rf, d.groups, wt, ctx->view, d, stream);
    else if (fused_route(d))  // the up/gate runs in the routing launch: relaunch that
      e = launch_route(rf, wt, ctx->view, d, stream);
    else
      e = launch_upgate(rf, d.groups, wt, ctx->view, d, stream);
    if (e != hipSuccess) return MOE_ERR_DEVICE;
  }
  return MOE_OK;
}

moe_status moe_decode_set_wait(moe_decode_ctx* ctx, uint32_t cap_ticks, int32_t withhold) {
  if (!ctx || (withhold != 0 && withhold != 1)) return MOE_ERR_INVALID_ARG;
  ctx->wait_ticks = cap_ticks ? cap_ticks : kDefaultWaitTicks;
  ctx->withhold = withhold;
  return MOE_OK;
}

moe_status moe_decode_wait_timeouts(moe_decode_ctx* ctx, uint32_t* count, hipStream_t stream) {
  if (!ctx || !count) return MOE_ERR_INVALID_ARG;
  if (hipMemcpyAsync(count, ctx->view.wait_timeouts, sizeof(uint32_t), hipMemcpyDeviceToHost,
                     stream) != hipSuccess)
    return MOE_ERR_DEVICE;
  return hipStreamSynchronize(stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

void moe_decode_destroy(moe_decode_ctx* ctx) { delete ctx; }

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or format";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_DEVICE: return "HIP launch error";
  }
  return "unknown status";
}

namespace {
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + bn && y < x + an;
}

// Checks of a GEMV call; *go is set when there is work to launch.
moe_status check_gemv(const lowbit_matrix* w, const uint16_t* x, int32_t rows, const uint16_t* y,
                      bool* go) {
  *go = false;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (w->fmt != MOE_FMT_FP8_E4M3_B128 && w->fmt != MOE_FMT_BF16 && w->fmt != MOE_FMT_Q1_G128)
    return MOE_ERR_UNSUPPORTED;
  if (w->n < 0 || w->k <= 0) return MOE_ERR_INVALID_ARG;
  const bool q1 = w->fmt == MOE_FMT_Q1_G128;
  if (q1) {
    if (w->k % 128 || w->k > 16384) return MOE_ERR_UNSUPPORTED;
  } else if (w->n % 128 || w->k % (w->fmt == MOE_FMT_BF16 ? 64 : 128)) {
    return MOE_ERR_UNSUPPORTED;
  }
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0 || w->n == 0) return MOE_OK;
  // 1-bit, several rows: the MFMA form, which takes K in chunks of 256
  if (rows > 8 || (q1 && rows > 1 && w->k % 256)) return MOE_ERR_UNSUPPORTED;
  if (!w->codes || !x || !y || !aligned16(w->codes) || !aligned16(x)) return MOE_ERR_INVALID_ARG;
  if (q1 ? !aligned16(y) : ((uintptr_t)y & 1u) != 0) return MOE_ERR_INVALID_ARG;
  if (w->fmt == MOE_FMT_FP8_E4M3_B128 && (!w->scales || ((uintptr_t)w->scales & 3u)))
    return MOE_ERR_INVALID_ARG;
  if (overlap(x, (size_t)rows * w->k * 2, y, (size_t)rows * w->n * 2)) return MOE_ERR_INVALID_ARG;
  *go = true;
  return MOE_OK;
}

moe_status enqueue_gemv(const lowbit_matrix* w, const uint16_t* x, int32_t rows, uint16_t* y,
                        const LoraArgs* lora, hipStream_t stream) {
  hipError_t e;
  if (w->fmt == MOE_FMT_FP8_E4M3_B128)
    e = launch_gemv_fp8(static_cast<const uint8_t*>(w->codes), static_cast<const float*>(w->scales),
                        x, y, rows, w->n, w->k, lora, stream);
  else if (w->fmt == MOE_FMT_BF16)
    e = launch_gemv_bf16(static_cast<const uint16_t*>(w->codes), x, y, rows, w->n, w->k, lora, stream);
  else
    e = launch_lowbit_q1(static_cast<const uint8_t*>(w->codes), x, y, rows, w->n, w->k, lora, stream);
  return e == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

// ---- rows grouped by expert

bool sort_shape_ok(int64_t tokens, int top_k, int groups) {
  return tokens >= 0 && top_k >= 1 && top_k <= MOE_MAX_TOP_K && groups >= 1 &&
         groups <= kSortMaxGroups && tokens * top_k <= kSortMaxPicks;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Checks of a row movement; *a is filled when there is work.
moe_status row_args(const moe_row_shape* s, const int32_t* pos, RowArgs* a) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_BF16 && s->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (s->tokens < 0 || s->top_k < 1 || s->hidden < 1 || s->rows < 0) return MOE_ERR_INVALID_ARG;
  if (s->top_k > MOE_MAX_TOP_K || (int64_t)s->tokens * s->top_k > kSortMaxPicks ||
      s->hidden > MOE_MAX_ROW)
    return MOE_ERR_UNSUPPORTED;
  if (s->tokens > 0 && (!pos || !aligned4(pos))) return MOE_ERR_INVALID_ARG;
  a->pos = pos;
  a->tokens = s->tokens;
  a->top_k = s->top_k;
  a->hidden = s->hidden;
  a->rows = s->rows;
  return MOE_OK;
}

struct RowBytes {
  size_t tokens, sorted, picks;  // [tokens, hidden], [rows, hidden], [tokens, top_k] of 4 bytes
};
RowBytes row_bytes(const moe_row_shape* s) {
  const size_t e = (size_t)s->hidden * (s->dtype == MOE_F32 ? 4 : 2);
  return {s->tokens * e, s->rows * e, (size_t)s->tokens * s->top_k * 4};
}

// ---- the experts' step of any number of rows

struct WidePlan {
  size_t actq, acts, actt, order, pos, offsets, counts, tiles, ntiles, midq, mids, y, total;
  int64_t picks;
  int max_tiles;
};

moe_status plan_wide(const moe_decode_config* cfg, int32_t tokens, Plan* p, WidePlan* q) {
  const moe_status st = plan_config(cfg, p);
  if (st != MOE_OK) return st;
  if (cfg->routed_fmt != MOE_FMT_FP8_E4M3_B128 || cfg->act_fmt != MOE_ACT_FP8_B128)
    return MOE_ERR_UNSUPPORTED;
  if (tokens < 0) return MOE_ERR_INVALID_ARG;
  if (tokens > MOE_WIDE_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  const size_t T = tokens, S = 8 * T, R = S + (p->Is ? T : 0);
  q->picks = (int64_t)S;
  q->max_tiles = wide_max_tiles(q->picks, p->E, p->Is ? tokens : 0);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  q->actq = take(T * p->H);
  q->acts = take(T * (p->H / 128) * 4);
  q->actt = take(R * (p->H / 128) * 4);
  q->order = take(S * 4);
  q->pos = take(S * 4);
  q->offsets = take((p->E + 1) * 4);
  q->counts = take(sort_workspace(q->picks, p->E));
  q->tiles = take((size_t)q->max_tiles * sizeof(RowTile));
  q->ntiles = take(4);
  q->midq = take(R * p->I);
  q->mids = take(R * (p->I / 128) * 4);
  q->y = take(R * p->H * 4);
  q->total = o;
  return MOE_OK;
}

// ---- products of rows grouped by expert

moe_status check_product(const moe_product_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_BF16 && s->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (s->n_experts < 1 || s->rows < 0 || s->n < 1 || s->k < 1) return MOE_ERR_INVALID_ARG;
  if (s->n_experts > kProductMaxExperts || s->rows > kProductMaxRows || s->n % 8 || s->k % 8 ||
      s->n > MOE_MAX_PRODUCT_SIDE || s->k > MOE_MAX_PRODUCT_SIDE)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

ProductArgs product_args(const moe_product_shape* s, const int32_t* offsets) {
  ProductArgs a = {};
  a.offsets = offsets;
  a.experts = s->n_experts;
  a.rows = s->rows;
  a.n = s->n;
  a.k = s->k;
  a.f32 = s->dtype == MOE_F32;
  return a;
}

struct ProductBytes {
  size_t x, y, w, offsets;  // [rows, k] and [rows, n] of 2 bytes, [experts, n, k] of 2
};
ProductBytes product_bytes(const moe_product_shape* s) {
  return {(size_t)s->rows * s->k * 2, (size_t)s->rows * s->n * 2, (size_t)s->n_experts * s->n * s->k * 2,
          ((size_t)s->n_experts + 1) * 4};
}

// ---- the LM head's loss

moe_status check_head(const lm_head_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_BF16 && s->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (s->rows < 0 || s->vocab < 1 || s->hidden < 1) return MOE_ERR_INVALID_ARG;
  if (s->rows > MOE_LOSS_MAX_ROWS || s->vocab > MOE_LOSS_MAX_VOCAB || s->hidden % 8 ||
      s->hidden > kLossMaxHidden)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether one of the outputs buf[first] .. overlaps another buffer (null or
// empty ones overlap nothing).
bool any_overlap(const void* const* buf, const size_t* len, int first, int n) {
  for (int i = first; i < n; i++)
    for (int j = 0; j < i; j++)
      if (buf[i] && buf[j] && len[i] && len[j] && overlap(buf[i], len[i], buf[j], len[j])) return true;
  return false;
}

// ---- the embedding

moe_status check_embed(const embed_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_BF16 && s->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (s->rows < 0 || s->vocab < 1 || s->hidden < 1) return MOE_ERR_INVALID_ARG;
  if (s->rows > MOE_EMBED_MAX_ROWS || s->vocab > MOE_EMBED_MAX_VOCAB || s->hidden > MOE_MAX_ROW)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

EmbedArgs embed_args(const embed_shape* s, const int32_t* ids, float scale) {
  return {ids, s->rows, s->vocab, s->hidden, scale, s->dtype == MOE_F32};
}

void launch_zero(void* p, size_t bytes, hipStream_t stream) {  // a multiple of 4
  const size_t words = bytes / 4, blocks = (words + 1023) / 1024;
  hipLaunchKernelGGL(moe_fill_u32_kernel, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream,
                     static_cast<uint32_t*>(p), words, 0u);
}

// ---- adapters

moe_status check_lora_set(const lora_set* l) {
  if (!l) return MOE_ERR_INVALID_ARG;
  if (l->n_adapters < 0 || l->n < 0 || l->k <= 0) return MOE_ERR_INVALID_ARG;
  if (l->n_adapters > kLoraMaxAdapters || l->max_rank < 8 || l->max_rank > kLoraMaxRank ||
      l->max_rank % 8 || l->n % 8 || l->n > MOE_MAX_ROW || l->k % 64 || l->k > 32768)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Pointers of a call with rows >= 1, n >= 1.
moe_status lora_args(const lora_set* l, const uint16_t* x, const int32_t* ids, int32_t rows,
                     const uint16_t* y, void* ws, size_t ws_bytes, LoraArgs* a) {
  if (!x || !ids || !y || !aligned16(x) || !aligned4(ids) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
  if (l->n_adapters > 0 && (!l->a || !l->b || !l->scale || !aligned16(l->a) || !aligned16(l->b) ||
                            !aligned4(l->scale) || !aligned4(l->rank)))
    return MOE_ERR_INVALID_ARG;
  a->adapters = l->n_adapters;
  a->max_rank = l->max_rank;
  a->n = l->n;
  a->k = l->k;
  a->rows = rows;
  const size_t need = lora_plan(a, ws);
  if (!ws || ws_bytes < need || !aligned16(ws)) return MOE_ERR_WORKSPACE;
  const size_t yb = (size_t)rows * l->n * 2;
  if (overlap(x, (size_t)rows * l->k * 2, y, yb) || overlap(ids, (size_t)rows * 4, y, yb) ||
      overlap(ws, need, y, yb) || overlap(ws, need, x, (size_t)rows * l->k * 2) ||
      overlap(ws, need, ids, (size_t)rows * 4))
    return MOE_ERR_INVALID_ARG;
  a->a = l->a;
  a->b = l->b;
  a->rank = l->rank;
  a->scale = l->scale;
  a->ids = ids;
  return MOE_OK;
}
}  // namespace

moe_status lowbit_gemv(const lowbit_matrix* w, const uint16_t* x, int32_t rows, uint16_t* y,
                       hipStream_t stream) {
  bool go;
  const moe_status st = check_gemv(w, x, rows, y, &go);
  if (st != MOE_OK || !go) return st;
  return enqueue_gemv(w, x, rows, y, nullptr, stream);
}

size_t moe_sort_workspace_size(int32_t tokens, int32_t top_k, int32_t n_experts) {
  return sort_shape_ok(tokens, top_k, n_experts) ? sort_workspace((int64_t)tokens * top_k, n_experts) : 0;
}

moe_status moe_sort(const int32_t* ids, int32_t tokens, int32_t top_k, int32_t n_experts,
                    int32_t* offsets, int32_t* order, int32_t* pos, void* workspace,
                    size_t ws_bytes, hipStream_t stream) {
  if (tokens < 0 || top_k < 1 || n_experts < 1) return MOE_ERR_INVALID_ARG;
  if (!sort_shape_ok(tokens, top_k, n_experts)) return MOE_ERR_UNSUPPORTED;
  const int64_t picks = (int64_t)tokens * top_k;
  if (!offsets || !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
  if (picks > 0 && (!ids || !order || !pos || !aligned4(ids) || !aligned4(order) || !aligned4(pos)))
    return MOE_ERR_INVALID_ARG;
  const size_t pb = (size_t)picks * 4, ob = ((size_t)n_experts + 1) * 4;
  const size_t need = sort_workspace(picks, n_experts);
  if (need && (!workspace || ws_bytes < need || !aligned4(workspace))) return MOE_ERR_WORKSPACE;
  const void* buf[] = {ids, offsets, order, pos, workspace};
  const size_t len[] = {pb, ob, pb, pb, need};
  for (int i = 0; i < 5; i++)
    for (int j = i + 1; j < 5; j++)
      if (len[i] && len[j] && overlap(buf[i], len[i], buf[j], len[j])) return MOE_ERR_INVALID_ARG;
  SortArgs a = {};
  a.ids = ids;
  a.picks = picks;
  a.groups = n_experts;
  a.offsets = offsets;
  a.order = order;
  a.pos = pos;
  a.counts = static_cast<int32_t*>(workspace);
  return launch_sort(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

moe_status moe_gather(const moe_row_shape* shape, const void* x, const int32_t* pos, void* xs,
                      hipStream_t stream) {
  RowArgs a;
  const moe_status st = row_args(shape, pos, &a);
  if (st != MOE_OK) return st;
  if (a.tokens == 0 || a.rows == 0) return MOE_OK;
  const RowBytes n = row_bytes(shape);
  if (!x || !xs || !aligned16(x) || !aligned16(xs)) return MOE_ERR_INVALID_ARG;
  if (overlap(x, n.tokens, xs, n.sorted) || overlap(pos, n.picks, xs, n.sorted))
    return MOE_ERR_INVALID_ARG;
  return launch_gather(a, shape->dtype == MOE_F32, x, xs, stream) == hipSuccess ? MOE_OK
                                                                               : MOE_ERR_DEVICE;
}

moe_status moe_gather_backward(const moe_row_shape* shape, const void* dxs, const int32_t* pos,
                               void* dx, hipStream_t stream) {
  RowArgs a;
  const moe_status st = row_args(shape, pos, &a);
  if (st != MOE_OK) return st;
  if (a.tokens == 0) return MOE_OK;
  const RowBytes n = row_bytes(shape);
  if (!dx || !aligned16(dx) || (a.rows > 0 && (!dxs || !aligned16(dxs)))) return MOE_ERR_INVALID_ARG;
  if (overlap(dxs, n.sorted, dx, n.tokens) || overlap(pos, n.picks, dx, n.tokens))
    return MOE_ERR_INVALID_ARG;
  return launch_combine_rows(a, shape->dtype == MOE_F32, dxs, nullptr, nullptr, dx, stream) ==
                 hipSuccess
             ? MOE_OK
             : MOE_ERR_DEVICE;
}

moe_status moe_combine(const moe_row_shape* shape, const void* y, const int32_t* pos,
                       const float* gates, const void* add, void* out, hipStream_t stream) {
  RowArgs a;
  const moe_status st = row_args(shape, pos, &a);
  if (st != MOE_OK) return st;
  if (a.tokens == 0) return MOE_OK;
  const RowBytes n = row_bytes(shape);
  if (!gates || !aligned4(gates) || !out || !aligned16(out) || !aligned16(add) ||
      (a.rows > 0 && (!y || !aligned16(y))))
    return MOE_ERR_INVALID_ARG;
  // out may be add itself: each element is read before it is written
  if (overlap(y, n.sorted, out, n.tokens) || overlap(pos, n.picks, out, n.tokens) ||
      overlap(gates, n.picks, out, n.tokens) ||
      (add && add != out && overlap(add, n.tokens, out, n.tokens)))
    return MOE_ERR_INVALID_ARG;
  return launch_combine_rows(a, shape->dtype == MOE_F32, y, gates, add, out, stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_DEVICE;
}

moe_status moe_combine_backward(const moe_row_shape* shape, const void* dout, const void* y,
                                const int32_t* pos, const float* gates, void* dy, float* dgates,
                                hipStream_t stream) {
  RowArgs a;
  const moe_status st = row_args(shape, pos, &a);
  if (st != MOE_OK) return st;
  if (a.tokens == 0) return MOE_OK;
  const RowBytes n = row_bytes(shape);
  if (!dout || !aligned16(dout) || !gates || !aligned4(gates) || !dgates || !aligned4(dgates) ||
      (a.rows > 0 && (!y || !dy || !aligned16(y) || !aligned16(dy))))
    return MOE_ERR_INVALID_ARG;
  const void* in[] = {dout, y, pos, gates};
  const size_t inb[] = {n.tokens, n.sorted, n.picks, n.picks};
  for (int i = 0; i < 4; i++)
    if (overlap(in[i], inb[i], dy, n.sorted) || overlap(in[i], inb[i], dgates, n.picks))
      return MOE_ERR_INVALID_ARG;
  if (overlap(dy, n.sorted, dgates, n.picks)) return MOE_ERR_INVALID_ARG;
  return launch_combine_bwd(a, shape->dtype == MOE_F32, dout, y, gates, dy, dgates, stream) ==
                 hipSuccess
             ? MOE_OK
             : MOE_ERR_DEVICE;
}

size_t moe_wide_workspace_size(const moe_decode_config* cfg, int32_t tokens) {
  Plan p;
  WidePlan q;
  return plan_wide(cfg, tokens, &p, &q) == MOE_OK ? q.total : 0;
}

moe_status moe_wide_step(const moe_decode_config* cfg, const uint16_t* x, int32_t tokens,
                         const int32_t* ids, const float* gates, const moe_decode_weights* w,
                         uint16_t* out, void* workspace, size_t ws_bytes, hipStream_t stream) {
  Plan p;
  WidePlan q;
  moe_status st = plan_wide(cfg, tokens, &p, &q);
  if (st != MOE_OK) return st;
  if (tokens == 0) return MOE_OK;
  st = check_io(p, x, tokens, w, out);
  if (st != MOE_OK) return st;
  moe_decode_weights ww = *w;
  ww.router_w = ww.rms_gamma;  // not read: the routing is given
  Weights wt;
  Dims d;
  st = step_args(*cfg, p, 1, &ww, &wt, &d);
  if (st != MOE_OK) return st;
  if (!ids || !gates || !aligned4(ids) || !aligned4(gates)) return MOE_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) || ws_bytes < q.total) return MOE_ERR_WORKSPACE;
  const size_t xb = (size_t)tokens * p.H * 2, rb = (size_t)q.picks * 4;
  if (overlap(workspace, q.total, x, xb) || overlap(workspace, q.total, out, xb) ||
      overlap(workspace, q.total, ids, rb) || overlap(workspace, q.total, gates, rb) ||
      overlap(out, xb, ids, rb) || overlap(out, xb, gates, rb))
    return MOE_ERR_INVALID_ARG;
  char* b = static_cast<char*>(workspace);
  WideArgs a;
  a.H = p.H;
  a.I = p.I;
  a.E = p.E;
  a.shared = p.Is > 0;
  a.tokens = tokens;
  a.picks = q.picks;
  a.rows = q.picks + (a.shared ? tokens : 0);
  a.eps = cfg->rms_eps;
  a.act_q = reinterpret_cast<uint8_t*>(b + q.actq);
  a.act_s = reinterpret_cast<float*>(b + q.acts);
  a.act_t = reinterpret_cast<float*>(b + q.actt);
  a.order = reinterpret_cast<int32_t*>(b + q.order);
  a.mid_q = reinterpret_cast<uint8_t*>(b + q.midq);
  a.mid_s = reinterpret_cast<float*>(b + q.mids);
  a.y = reinterpret_cast<float*>(b + q.y);
  a.pos = reinterpret_cast<int32_t*>(b + q.pos);
  a.offsets = reinterpret_cast<int32_t*>(b + q.offsets);
  a.counts = reinterpret_cast<int32_t*>(b + q.counts);
  a.tiles = reinterpret_cast<RowTile*>(b + q.tiles);
  a.n_tiles = reinterpret_cast<int32_t*>(b + q.ntiles);
  a.max_tiles = q.max_tiles;
  const WideWeights v = {wt.gamma, wt.gate_c, wt.up_c, wt.down_c, (const float*)wt.gate_s,
                         (const float*)wt.up_s, (const float*)wt.down_s, wt.sg_c, wt.su_c, wt.sd_c,
                         wt.sg_s, wt.su_s, wt.sd_s};
  return launch_wide(a, v, x, ids, gates, out, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t moe_product_workspace_size(const moe_product_shape* shape) {
  return check_product(shape) == MOE_OK ? product_workspace(product_args(shape, nullptr)) : 0;
}

moe_status moe_product(const moe_product_shape* shape, const uint16_t* x, const uint16_t* w,
                       const int32_t* offsets, void* y, void* workspace, size_t ws_bytes,
                       hipStream_t stream) {
  const moe_status st = check_product(shape);
  if (st != MOE_OK) return st;
  if (shape->rows == 0) return MOE_OK;
  if (!x || !w || !offsets || !y || !aligned16(x) || !aligned16(w) || !aligned4(offsets) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  ProductArgs a = product_args(shape, offsets);
  const size_t need = product_workspace(a);
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace))) return MOE_ERR_WORKSPACE;
  const ProductBytes b = product_bytes(shape);
  const void* buf[] = {x, w, offsets, workspace, y};
  const size_t len[] = {b.x, b.w, b.offsets, need, a.f32 ? 2 * b.y : b.y};
  if (any_overlap(buf, len, 3, 5)) return MOE_ERR_INVALID_ARG;
  a.x = x;
  a.w = w;
  a.y = y;
  a.space = static_cast<float*>(workspace);
  return launch_product(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t moe_product_backward_workspace_size(const moe_product_shape* shape) {
  return check_product(shape) == MOE_OK ? product_backward_workspace(product_args(shape, nullptr)) : 0;
}

moe_status moe_product_backward(const moe_product_shape* shape, const uint16_t* dy,
                                const uint16_t* x, const uint16_t* w, const int32_t* offsets,
                                uint16_t* dx, void* dw, int32_t add, void* workspace,
                                size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_product(shape);
  if (st != MOE_OK) return st;
  if (!dx && !dw) return MOE_OK;
  // without rows dw is all there is, and 0 (x and dy are not read)
  const bool rows = shape->rows > 0;
  if (!offsets || !aligned4(offsets) || (rows && (!dy || !aligned16(dy)))) return MOE_ERR_INVALID_ARG;
  if (dx && rows && (!w || !aligned16(w) || !aligned16(dx))) return MOE_ERR_INVALID_ARG;
  if (dw && (!aligned16(dw) || (rows && (!x || !aligned16(x))))) return MOE_ERR_INVALID_ARG;
  ProductArgs a = product_args(shape, offsets);
  const size_t need = dw ? product_backward_workspace(a) : 0;
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace))) return MOE_ERR_WORKSPACE;
  const ProductBytes b = product_bytes(shape);
  const void* buf[] = {dy, dw ? x : nullptr, dx ? w : nullptr, offsets, workspace, dx, dw};
  const size_t len[] = {b.y, dw ? b.x : 0, dx ? b.w : 0, b.offsets, need, dx ? b.x : 0,
                        dw ? (a.f32 ? 2 * b.w : b.w) : 0};
  if (any_overlap(buf, len, 4, 7)) return MOE_ERR_INVALID_ARG;
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.dx = dx;
  a.dw = dw;
  a.add = add != 0;
  a.space = static_cast<float*>(workspace);
  if (dx && rows && launch_product_dx(a, stream) != hipSuccess) return MOE_ERR_DEVICE;
  if (dw && launch_product_dw(a, stream) != hipSuccess) return MOE_ERR_DEVICE;
  return MOE_OK;
}

size_t lm_head_loss_workspace_size(const lm_head_shape* s) {
  return check_head(s) == MOE_OK && s->rows > 0 ? loss_workspace(s->rows, s->vocab, s->hidden) : 0;
}

moe_status lm_head_loss(const lm_head_shape* shape, const uint16_t* h, const uint16_t* w,
                        const int32_t* targets, float* loss, float* lse, void* workspace,
                        size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_head(shape);
  if (st != MOE_OK) return st;
  if (shape->rows == 0) return MOE_OK;
  if (!h || !w || !targets || !loss || !lse || !aligned16(h) || !aligned16(w) || !aligned4(targets) ||
      !aligned4(loss) || !aligned4(lse))
    return MOE_ERR_INVALID_ARG;
  const size_t need = loss_workspace(shape->rows, shape->vocab, shape->hidden);
  if (!workspace || ws_bytes < need || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  const size_t rb = (size_t)shape->rows * 4;
  const void* buf[] = {h, w, targets, workspace, loss, lse};
  const size_t len[] = {(size_t)shape->rows * shape->hidden * 2, (size_t)shape->vocab * shape->hidden * 2, rb,
                        need, rb, rb};
  if (any_overlap(buf, len, 3, 6)) return MOE_ERR_INVALID_ARG;
  const LossArgs a = {h, w, targets, shape->rows, shape->vocab, shape->hidden, loss, lse};
  return launch_loss(a, workspace, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t lm_head_loss_backward_workspace_size(const lm_head_shape* s) {
  return check_head(s) == MOE_OK && s->rows > 0 ? loss_backward_workspace(s->rows, s->vocab, s->hidden) : 0;
}

moe_status lm_head_loss_backward(const lm_head_shape* shape, const uint16_t* h, const uint16_t* w,
                                 const int32_t* targets, const float* lse, const float* dloss,
                                 uint16_t* dh, void* dw, int32_t add, void* workspace,
                                 size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_head(shape);
  if (st != MOE_OK) return st;
  if (!dh && !dw) return MOE_OK;
  if (!aligned16(dh) || !aligned16(dw)) return MOE_ERR_INVALID_ARG;
  const bool f32 = shape->dtype == MOE_F32;
  const size_t wb = (size_t)shape->vocab * shape->hidden * 2;
  if (shape->rows == 0) {  // a dw of 0
    if (!dw || add) return MOE_OK;
    launch_zero(dw, f32 ? 2 * wb : wb, stream);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
  }
  if (!h || !w || !targets || !lse || !dloss || !aligned16(h) || !aligned16(w) || !aligned4(targets) ||
      !aligned4(lse) || !aligned4(dloss))
    return MOE_ERR_INVALID_ARG;
  const size_t need = loss_backward_workspace(shape->rows, shape->vocab, shape->hidden);
  if (!workspace || ws_bytes < need || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  const size_t rb = (size_t)shape->rows * 4, hb = (size_t)shape->rows * shape->hidden * 2;
  const void* buf[] = {h, w, targets, lse, dloss, workspace, dh, dw};
  const size_t len[] = {hb, wb, rb, rb, rb, need, hb, f32 ? 2 * wb : wb};
  if (any_overlap(buf, len, 5, 8)) return MOE_ERR_INVALID_ARG;
  const LossGradArgs a = {h, w, targets, lse, dloss, shape->rows, shape->vocab, shape->hidden, dh, dw, f32, add != 0};
  return launch_loss_backward(a, workspace, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

moe_status embed(const embed_shape* shape, const int32_t* ids, const void* table, float scale,
                 void* out, hipStream_t stream) {
  const moe_status st = check_embed(shape);
  if (st != MOE_OK) return st;
  if (shape->rows == 0) return MOE_OK;
  if (!ids || !table || !out || !aligned4(ids) || !aligned16(table) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  const size_t rb = (size_t)shape->hidden * (shape->dtype == MOE_F32 ? 4 : 2);
  const void* buf[] = {ids, table, out};
  const size_t len[] = {(size_t)shape->rows * 4, shape->vocab * rb, shape->rows * rb};
  if (any_overlap(buf, len, 2, 3)) return MOE_ERR_INVALID_ARG;
  return launch_embed(embed_args(shape, ids, scale), table, out, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t embed_backward_workspace_size(const embed_shape* shape) {
  return check_embed(shape) == MOE_OK ? embed_backward_workspace(shape->rows, shape->vocab, shape->hidden) : 0;
}

moe_status embed_backward(const embed_shape* shape, const int32_t* ids, const void* dout,
                          float scale, int32_t table_dtype, void* dtable, int32_t add,
                          void* workspace, size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_embed(shape);
  if (st != MOE_OK) return st;
  if (table_dtype != MOE_BF16 && table_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (shape->rows == 0 && add) return MOE_OK;
  if (!dtable || !aligned16(dtable) || (shape->rows > 0 && (!ids || !dout || !aligned4(ids) || !aligned16(dout))))
    return MOE_ERR_INVALID_ARG;
  const size_t need = embed_backward_workspace(shape->rows, shape->vocab, shape->hidden);
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace))) return MOE_ERR_WORKSPACE;
  const size_t h = shape->hidden, rb = h * (shape->dtype == MOE_F32 ? 4 : 2);
  const void* buf[] = {ids, dout, need ? workspace : nullptr, dtable};
  const size_t len[] = {(size_t)shape->rows * 4, shape->rows * rb, need,
                        shape->vocab * h * (table_dtype == MOE_F32 ? 4 : 2)};
  if (any_overlap(buf, len, 2, 4)) return MOE_ERR_INVALID_ARG;
  const EmbedGradArgs a = {embed_args(shape, ids, scale), dout, dtable, table_dtype == MOE_F32, add != 0};
  return launch_embed_backward(a, workspace, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

size_t lora_workspace_size(const lora_set* l, int32_t rows) {
  if (check_lora_set(l) != MOE_OK || rows <= 0 || rows > MOE_LORA_MAX_ROWS) return 0;
  LoraArgs a = {};
  a.adapters = l->n_adapters;
  a.max_rank = l->max_rank;
  a.n = l->n;
  a.k = l->k;
  a.rows = rows;
  return lora_plan(&a, nullptr);
}

moe_status lora_apply(const lora_set* l, const uint16_t* x, const int32_t* ids, int32_t rows,
                      const uint16_t* base, uint16_t* y, void* workspace, size_t ws_bytes,
                      hipStream_t stream) {
  moe_status st = check_lora_set(l);
  if (st != MOE_OK) return st;
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows > MOE_LORA_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || l->n == 0) return MOE_OK;
  LoraArgs a = {};
  st = lora_args(l, x, ids, rows, y, workspace, ws_bytes, &a);
  if (st != MOE_OK) return st;
  const size_t yb = (size_t)rows * l->n * 2;
  if (!base || !aligned16(base) || (base != y && overlap(base, yb, y, yb)) ||
      overlap(workspace, lora_plan(&a, workspace), base, yb))
    return MOE_ERR_INVALID_ARG;
  return launch_lora(a, x, base, y, stream) == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

moe_status lowbit_gemv_lora(const lowbit_matrix* w, const lora_set* l, const uint16_t* x,
                            const int32_t* ids, int32_t rows, uint16_t* y, void* workspace,
                            size_t ws_bytes, hipStream_t stream) {
  bool go;
  moe_status st = check_gemv(w, x, rows, y, &go);
  if (st != MOE_OK) return st;
  st = check_lora_set(l);
  if (st != MOE_OK) return st;
  if (l->n != w->n || l->k != w->k) return MOE_ERR_INVALID_ARG;
  if (!go) return MOE_OK;
  LoraArgs a = {};
  st = lora_args(l, x, ids, rows, y, workspace, ws_bytes, &a);
  if (st != MOE_OK) return st;
  if (launch_lora_shrink(a, x, stream) != hipSuccess) return MOE_ERR_DEVICE;
  return enqueue_gemv(w, x, rows, y, &a, stream);
}

}  // extern "C"
