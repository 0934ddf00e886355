// C ABI entry points of the backward pass (declared in include/moe_null.h): host-side
// argument checks, then stream-ordered launches into the caller's backward workspace.
#include "moe_internal.cuh"

using namespace moe;

#define MOE_CHECK(expr)          \
  do {                           \
    const int _r = (expr);       \
    if (_r != MOE_OK) return _r; \
  } while (0)

static inline cudaStream_t S(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

static int check_pp_inputs(const moe_dims_t* d, const int32_t* topk_idx, const uint16_t* x, const uint16_t* cv) {
  if (d->C + d->V > 0 && (!topk_idx || (d->C > 0 && !x) || (d->V > 0 && !cv))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The five expert GEMMs. With w->w_router set, the router's input gradient ds W_r (from the
// split ds that the router backward left in the workspace) is added to dx_shared inside the
// shared expert's gate/up dgrad. With s8 set, the pre-activations come from its 8-bit blocks,
// and h and h_shared of sv are written from them before the weight gradient reads them.
static int expert_ffn_bwd(const moe_dims_t& d, const moe_weights_t* w, const moe_saved_t* sv, const uint16_t* dys,
                          const uint16_t* dy, uint16_t* dxs, uint16_t* dx_shared, const moe_grads_t* g, void* ws,
                          cudaStream_t st, const moe_saved8_t* s8 = nullptr) {
  const BwdLayout L = bwd_layout(d);
  uint32_t* status = ws_ptr<uint32_t>(ws, L.hdr);
  uint16_t* dh = ws_ptr<uint16_t>(ws, L.dh);
  uint16_t* dhs = ws_ptr<uint16_t>(ws, L.dhs);
  uint16_t* dz = ws_ptr<uint16_t>(ws, L.dz);
  uint16_t* dzs = ws_ptr<uint16_t>(ws, L.dzs);
  float* spart = ws_ptr<float>(ws, L.spart);
  uint16_t* dsplit = nullptr;
  uint16_t* w2 = nullptr;
  if (w->w_router) {
    dsplit = ws_ptr<uint16_t>(ws, L.dsplit);
    w2 = ws_ptr<uint16_t>(ws, L.w2);
    MOE_CHECK(launch_router_split2(d, w->w_router, w2, st));
  }
  MOE_CHECK(launch_dgrad_down(d, sv->offsets, dys, dy, w->w_down, w->shared_down, dh, dhs, status, st));
  if (s8) {
    MOE_CHECK(launch_swiglu_backward8((long long)d.T * d.K, d.F, 1, MOE_DTYPE_BF16, s8->z_codes, s8->z_scales, dh, d.F,
                                      sv->offsets + d.N, dz, 2 * d.F, const_cast<uint16_t*>(sv->h), d.F, status, st));
    MOE_CHECK(launch_swiglu_backward8(d.T, d.F_shared, 1, MOE_DTYPE_BF16, s8->zs_codes, s8->zs_scales, dhs, d.F_shared,
                                      nullptr, dzs, 2 * d.F_shared, const_cast<uint16_t*>(sv->h_shared), d.F_shared,
                                      status, st));
  } else if (sv->z && sv->z_shared)  // training mode: pre-activations saved by the forward
    MOE_CHECK(launch_swiglu_bwd_saved(d, sv->offsets, sv->z, sv->z_shared, dh, dhs, dz, dzs, status, st));
  else
    MOE_CHECK(launch_swiglu_backward(d, sv->offsets, sv->xs, sv->x, w->gate_up, w->shared_gate_up, dh, dhs, dz, dzs,
                                     status, st));
  MOE_CHECK(launch_wgrad_down(d, sv->offsets, dys, dy, sv->h, sv->h_shared, g->dw_down, g->dws_down, spart, status,
                              st));
  MOE_CHECK(launch_dgrad_gate_up(d, sv->offsets, dz, dzs, w->gate_up, w->shared_gate_up, dsplit, w2, dxs, dx_shared,
                                 status, st));
  return launch_wgrad_gate_up(d, sv->offsets, dz, dzs, sv->xs, sv->x, g->dw_gate, g->dw_up, g->dws_gate, g->dws_up,
                              spart, status, st);
}

static int router_wgrad(const moe_dims_t& d, const uint16_t* x, float* dw_router, float* dbias, void* ws,
                        cudaStream_t st) {
  const BwdLayout L = bwd_layout(d);
  float* part = ws_ptr<float>(ws, L.rpart);
  MOE_CHECK(launch_router_wgrad_tc(d, ws_ptr<uint16_t>(ws, L.dsplit), x, part, ws_ptr<uint32_t>(ws, L.hdr), st));
  return launch_router_wgrad_reduce(d, part, router_wgrad_split(d, nullptr), ws_ptr<float>(ws, L.bpart), dw_router,
                                    dbias, st);
}

static bool saved_ok(const moe_saved_t* s, const moe_dims_t* d) {
  return s && s->x && s->logits && s->topk_idx && s->topk_gate && s->offsets && s->slot_row && s->xs && s->h &&
         s->h_shared && s->ys && s->counts_ext && s->t_total >= (int64_t)d->T && s->t_total > 0 &&
         ((s->z != nullptr) == (s->z_shared != nullptr));
}

static bool expert_grads_ok(const moe_grads_t* g) {
  return g && g->dw_gate && g->dw_up && g->dw_down && g->dws_gate && g->dws_up && g->dws_down;
}

static bool weights_ok(const moe_weights_t* w, const moe_dims_t* d) {
  return w && w->w_router && w->gate_up && w->w_down && w->shared_gate_up && w->shared_down &&
         (d->V == 0 || w->const_vectors);
}

static bool saved8_ok(const moe_saved8_t* s, const moe_dims_t* d) {
  return s && s->x && s->logits && s->topk_idx && s->topk_gate && s->offsets && s->slot_row && s->counts_ext &&
         s->t_total >= (int64_t)d->T && s->t_total > 0 && s->z_codes && s->z_scales && s->zs_codes && s->zs_scales &&
         s->ys_codes && s->ys_scales;
}

// Workspace of the backward from an 8-bit checkpoint: moe_backward's, then the gathered rows,
// the activations and (with MoE++ experts, whose combine backward reads them in bf16) the
// routed outputs.
struct Ckpt8Layout {
  size_t xs, h, hs, ys, total;
};
static Ckpt8Layout ckpt8_layout(const moe_dims_t& d) {
  const size_t rcap = (size_t)d.T * d.K, T = (size_t)d.T;
  Ckpt8Layout L{};
  size_t o = align_up(bwd_layout(d).total, 256);
  L.xs = o; o = align_up(o + 2 * rcap * d.d, 256);
  L.h = o; o = align_up(o + 2 * rcap * d.F, 256);
  L.hs = o; o = align_up(o + 2 * T * d.F_shared, 256);
  L.ys = o; o = align_up(o + (d.C + d.V > 0 ? 2 * rcap * d.d : 0), 256);
  L.total = o;
  return L;
}

// The whole backward; with s8, from an 8-bit checkpoint: saved's xs, h, h_shared and ys are
// then workspace buffers that this call fills.
static int backward_run(const moe_dims_t& d, const moe_weights_t* w, const moe_saved_t* saved, const moe_saved8_t* s8,
                        const uint16_t* dy, float alpha, float beta, const moe_grads_t* g, void* ws,
                        cudaStream_t st) {
  const BwdLayout L = bwd_layout(d);
  uint32_t* status = ws_ptr<uint32_t>(ws, L.hdr);
  uint16_t* dys = ws_ptr<uint16_t>(ws, L.dys);
  uint16_t* dxs = ws_ptr<uint16_t>(ws, L.dxs);
  float* dg = ws_ptr<float>(ws, L.dg);
  float* ds = ws_ptr<float>(ws, L.ds);
  MOE_CHECK(cuda_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st)));
  const long long rcap = (long long)d.T * d.K;
  if (s8) {  // the gathered rows again
    MOE_CHECK(launch_spread(d.T, d.K, rcap, d.d, MOE_DTYPE_BF16, saved->x, d.d, nullptr, 0, nullptr, nullptr,
                            saved->slot_row, const_cast<uint16_t*>(saved->xs), d.d, nullptr, status, st));
    if (saved->ys)
      MOE_CHECK(launch_restore8(rcap, d.d, MOE_DTYPE_BF16, s8->ys_codes, s8->ys_scales, saved->offsets + d.N,
                                const_cast<uint16_t*>(saved->ys), d.d, status, st));
  }
  if (s8 && !saved->ys)  // every slot is a real expert or a null copy: the outputs straight from their codes
    MOE_CHECK(launch_spread(d.T, d.K, rcap, d.d, MOE_DTYPE_BF16, dy, d.d, s8->ys_codes, d.d, s8->ys_scales,
                            saved->topk_gate, saved->slot_row, dys, d.d, dg, status, st));
  else
    MOE_CHECK(launch_combine_bwd(d, dy, saved->ys, saved->topk_gate, saved->slot_row, saved->topk_idx, saved->x,
                                 w->const_vectors, dys, dg, status, st));
  MOE_CHECK(launch_router_bwd(d, saved->logits, saved->topk_idx, saved->topk_gate, dg, saved->counts_ext,
                              (long long)saved->t_total, alpha, beta, ds, g->dtok_null_bias,
                              ws_ptr<uint16_t>(ws, L.dsplit), ws_ptr<float>(ws, L.bpart), st));
  MOE_CHECK(router_wgrad(d, saved->x, g->dw_router, g->dbias, ws, st));
  // the shared expert's (and the router's) input gradient goes straight into dx; the input
  // gradient gather then adds the routed and copy-expert terms in place, skipping the tokens
  // that have none
  MOE_CHECK(expert_ffn_bwd(d, w, saved, dys, dy, dxs, g->dx, g, ws, st, s8));
  MOE_CHECK(launch_input_grad(d, g->dx, dxs, saved->slot_row, saved->topk_idx, saved->topk_gate, dy, g->dx, status,
                              st));
  return launch_const_grad(d, saved->topk_idx, saved->topk_gate, dy, g->dconst, st);
}

extern "C" {

size_t moe_backward_workspace_bytes(const moe_dims_t* dims) {
  if (check_dims(dims) != MOE_OK) return 0;
  return bwd_layout(*dims).total;
}

int moe_combine_backward(const moe_dims_t* dims, const uint16_t* dy, const uint16_t* ys, const float* topk_gate,
                         const int32_t* slot_row, const int32_t* topk_idx, const uint16_t* x,
                         const uint16_t* const_vectors, uint16_t* dys, float* dg, void* bwd_workspace,
                         moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!dy || !ys || !topk_gate || !slot_row || !dys || !dg || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  MOE_CHECK(check_pp_inputs(dims, topk_idx, x, const_vectors));
  const BwdLayout L = bwd_layout(*dims);
  return launch_combine_bwd(*dims, dy, ys, topk_gate, slot_row, topk_idx, x, const_vectors, dys, dg,
                            ws_ptr<uint32_t>(bwd_workspace, L.hdr), S(stream));
}

int moe_router_backward(const moe_dims_t* dims, const float* logits, const int32_t* topk_idx, const float* topk_gate,
                        const float* dg, const int32_t* counts_ext, int64_t t_total, float alpha, float beta,
                        float* ds, float* dtok_null_bias, void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_gate || !dg || !counts_ext || !ds || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  if (t_total < (int64_t)dims->T || t_total <= 0) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  return launch_router_bwd(*dims, logits, topk_idx, topk_gate, dg, counts_ext, (long long)t_total, alpha, beta, ds,
                           dtok_null_bias, ws_ptr<uint16_t>(bwd_workspace, L.dsplit),
                           ws_ptr<float>(bwd_workspace, L.bpart), S(stream));
}

int moe_router_weight_grad(const moe_dims_t* dims, const uint16_t* x, float* dw_router, float* dbias,
                           void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (!dw_router) return MOE_ERR_INVALID_ARG;
  const size_t rows = (size_t)router_rows(*dims);
  if (dims->T == 0) {
    MOE_CHECK(cuda_status(cudaMemsetAsync(dw_router, 0, sizeof(float) * rows * dims->d, S(stream))));
    return dbias ? cuda_status(cudaMemsetAsync(dbias, 0, sizeof(float) * rows, S(stream))) : MOE_OK;
  }
  if (!x || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  return router_wgrad(*dims, x, dw_router, dbias, bwd_workspace, S(stream));
}

int moe_expert_ffn_backward(const moe_dims_t* dims, const moe_weights_t* w, const moe_saved_t* saved,
                            const uint16_t* dys, const uint16_t* dy, uint16_t* dxs, uint16_t* dx_shared,
                            const moe_grads_t* g, void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!w || !w->gate_up || !w->w_down || !w->shared_gate_up || !w->shared_down) return MOE_ERR_INVALID_ARG;
  if (!saved || !saved->x || !saved->xs || !saved->offsets || !saved->h || !saved->h_shared) return MOE_ERR_INVALID_ARG;
  if ((saved->z != nullptr) != (saved->z_shared != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!dys || !dy || !dxs || !dx_shared || !expert_grads_ok(g) || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  return expert_ffn_bwd(*dims, w, saved, dys, dy, dxs, dx_shared, g, bwd_workspace, S(stream));
}

// The five GEMM stages of moe_expert_ffn_backward, one launch each (the weight gradients
// add the reduction of the shared expert's K chunks when T needs more than one).
int moe_expert_dgrad_down(const moe_dims_t* dims, const int32_t* offsets, const uint16_t* dys, const uint16_t* dy,
                          const uint16_t* w_down, const uint16_t* shared_down, void* bwd_workspace,
                          moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!offsets || !dys || !dy || !w_down || !shared_down || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  return launch_dgrad_down(*dims, offsets, dys, dy, w_down, shared_down, ws_ptr<uint16_t>(ws, L.dh),
                           ws_ptr<uint16_t>(ws, L.dhs), ws_ptr<uint32_t>(ws, L.hdr), S(stream));
}

int moe_expert_swiglu_backward(const moe_dims_t* dims, const uint16_t* xs, const uint16_t* x, const int32_t* offsets,
                               const uint16_t* gate_up, const uint16_t* shared_gate_up, void* bwd_workspace,
                               moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!xs || !x || !offsets || !gate_up || !shared_gate_up || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  return launch_swiglu_backward(*dims, offsets, xs, x, gate_up, shared_gate_up, ws_ptr<uint16_t>(ws, L.dh),
                                ws_ptr<uint16_t>(ws, L.dhs), ws_ptr<uint16_t>(ws, L.dz), ws_ptr<uint16_t>(ws, L.dzs),
                                ws_ptr<uint32_t>(ws, L.hdr), S(stream));
}

int moe_expert_swiglu_backward_saved(const moe_dims_t* dims, const int32_t* offsets, const uint16_t* z,
                                     const uint16_t* z_shared, void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!offsets || !z || !z_shared || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  return launch_swiglu_bwd_saved(*dims, offsets, z, z_shared, ws_ptr<uint16_t>(ws, L.dh), ws_ptr<uint16_t>(ws, L.dhs),
                                 ws_ptr<uint16_t>(ws, L.dz), ws_ptr<uint16_t>(ws, L.dzs), ws_ptr<uint32_t>(ws, L.hdr),
                                 S(stream));
}

int moe_expert_wgrad_down(const moe_dims_t* dims, const int32_t* offsets, const uint16_t* dys, const uint16_t* dy,
                          const uint16_t* h, const uint16_t* h_shared, uint16_t* dw_down, uint16_t* dws_down,
                          void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!offsets || !dys || !dy || !h || !h_shared || !dw_down || !dws_down || !bwd_workspace)
    return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  return launch_wgrad_down(*dims, offsets, dys, dy, h, h_shared, dw_down, dws_down, ws_ptr<float>(ws, L.spart),
                           ws_ptr<uint32_t>(ws, L.hdr), S(stream));
}

int moe_expert_dgrad_gate_up(const moe_dims_t* dims, const int32_t* offsets, const uint16_t* gate_up,
                             const uint16_t* shared_gate_up, const float* w_router, uint16_t* dxs,
                             uint16_t* dx_shared, void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!offsets || !gate_up || !shared_gate_up || !dxs || !dx_shared || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  uint16_t* dsplit = nullptr;
  uint16_t* w2 = nullptr;
  if (w_router) {
    dsplit = ws_ptr<uint16_t>(ws, L.dsplit);
    w2 = ws_ptr<uint16_t>(ws, L.w2);
    MOE_CHECK(launch_router_split2(*dims, w_router, w2, S(stream)));
  }
  return launch_dgrad_gate_up(*dims, offsets, ws_ptr<uint16_t>(ws, L.dz), ws_ptr<uint16_t>(ws, L.dzs), gate_up,
                              shared_gate_up, dsplit, w2, dxs, dx_shared, ws_ptr<uint32_t>(ws, L.hdr), S(stream));
}

int moe_expert_wgrad_gate_up(const moe_dims_t* dims, const int32_t* offsets, const uint16_t* xs, const uint16_t* x,
                             uint16_t* dw_gate, uint16_t* dw_up, uint16_t* dws_gate, uint16_t* dws_up,
                             void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!offsets || !xs || !x || !dw_gate || !dw_up || !dws_gate || !dws_up || !bwd_workspace)
    return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  void* ws = bwd_workspace;
  return launch_wgrad_gate_up(*dims, offsets, ws_ptr<uint16_t>(ws, L.dz), ws_ptr<uint16_t>(ws, L.dzs), xs, x,
                              dw_gate, dw_up, dws_gate, dws_up, ws_ptr<float>(ws, L.spart),
                              ws_ptr<uint32_t>(ws, L.hdr), S(stream));
}

int moe_input_grad(const moe_dims_t* dims, const uint16_t* dx_shared, const uint16_t* dxs, const int32_t* slot_row,
                   const int32_t* topk_idx, const float* topk_gate, const uint16_t* dy, uint16_t* dx,
                   void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!dx_shared || !dxs || !slot_row || !dx || !bwd_workspace) return MOE_ERR_INVALID_ARG;
  if (dims->C > 0 && (!topk_idx || !topk_gate || !dy)) return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(*dims);
  return launch_input_grad(*dims, dx_shared, dxs, slot_row, topk_idx, topk_gate, dy, dx,
                           ws_ptr<uint32_t>(bwd_workspace, L.hdr), S(stream));
}

int moe_backward(const moe_dims_t* dims, const moe_weights_t* w, const moe_saved_t* saved, const uint16_t* dy,
                 float alpha, float beta, const moe_grads_t* g, void* bwd_workspace, moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!weights_ok(w, dims)) return MOE_ERR_INVALID_ARG;
  if (!saved_ok(saved, dims) || !dy || !expert_grads_ok(g) || !g->dx || !g->dw_router || !bwd_workspace)
    return MOE_ERR_INVALID_ARG;
  if (dims->V > 0 && !g->dconst) return MOE_ERR_INVALID_ARG;
  return backward_run(*dims, w, saved, nullptr, dy, alpha, beta, g, bwd_workspace, S(stream));
}

size_t moe_backward_checkpoint8_workspace_bytes(const moe_dims_t* dims) {
  if (check_dims(dims) != MOE_OK) return 0;
  return ckpt8_layout(*dims).total;
}

int moe_backward_checkpoint8(const moe_dims_t* dims, const moe_weights_t* w, const moe_saved8_t* s8,
                             const uint16_t* dy, float alpha, float beta, const moe_grads_t* g, void* workspace,
                             moe_stream_t stream) {
  MOE_CHECK(check_dims(dims));
  if (dims->T == 0) return MOE_OK;
  if (!weights_ok(w, dims) || !saved8_ok(s8, dims) || !dy || !expert_grads_ok(g) || !g->dx || !g->dw_router ||
      !workspace)
    return MOE_ERR_INVALID_ARG;
  if (dims->V > 0 && !g->dconst) return MOE_ERR_INVALID_ARG;
  const moe_dims_t& d = *dims;
  const Ckpt8Layout L = ckpt8_layout(d);
  moe_saved_t sv{};
  sv.x = s8->x;
  sv.logits = s8->logits;
  sv.topk_idx = s8->topk_idx;
  sv.topk_gate = s8->topk_gate;
  sv.offsets = s8->offsets;
  sv.slot_row = s8->slot_row;
  sv.counts_ext = s8->counts_ext;
  sv.t_total = s8->t_total;
  sv.xs = ws_ptr<uint16_t>(workspace, L.xs);
  sv.h = ws_ptr<uint16_t>(workspace, L.h);
  sv.h_shared = ws_ptr<uint16_t>(workspace, L.hs);
  sv.ys = d.C + d.V > 0 ? ws_ptr<uint16_t>(workspace, L.ys) : nullptr;
  return backward_run(d, w, &sv, s8, dy, alpha, beta, g, workspace, S(stream));
}

}  // extern "C"
