// C ABI of the sequence operators: validation, workspace sizes and launch order.  Validation reads host arguments
// only; nothing is enqueued before it has passed.
#include <stdint.h>

#include "seq.h"

namespace {

using cw::seq_pieces;
using cw::seq_rows;

typedef conv_wgrad_status_t Status;
constexpr int64_t kMaxRows = (int64_t)1 << 30;       // tokens of a sequence, packed rows, sequences, states of a pool
constexpr int64_t kMaxAll = (int64_t)1 << 40;        // rows of all sequences
constexpr int64_t kMaxChannels = (int64_t)1 << 20;
constexpr int64_t kMaxNorm = 16384;                  // channels of a norm: a row stays in registers
using cw::kMaxLanes;

Status of(hipError_t err) { return err == hipSuccess ? CONV_WGRAD_OK : CONV_WGRAD_ERR_HIP; }
bool bad_dtype(int32_t t) { return t != CONV_WGRAD_F32 && t != CONV_WGRAD_BF16 && t != CONV_WGRAD_F16; }
int64_t elem(int32_t t) { return t == CONV_WGRAD_F32 ? 4 : 2; }
bool off(const void* p, int64_t align) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(align - 1)) != 0; }
bool negative(const seq_view_t& v) { return v.batch < 0 || v.row < 0; }
bool fits(int64_t blocks, int64_t threads) { return blocks >= 0 && blocks <= kMaxLanes / threads; }

Status check_tokens(const seq_tokens_t& t) {
  if (t.sequences < 1 || t.rows < 0) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (t.slots ? t.pool < 1 : t.pool < t.sequences) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (t.sequences >= kMaxRows || t.rows >= kMaxRows || t.pool >= kMaxRows) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (!t.offsets && t.rows && t.sequences > kMaxAll / t.rows) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (off(t.offsets, 4) || off(t.slots, 4)) return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

// Pieces of at least 16 tokens: their number has to stay an int.
bool pieces_fit(const seq_tokens_t& t) {
  return t.offsets || t.sequences * (t.rows / 16 + 1) < ((int64_t)1 << 31) - 1;
}

// ---- norm ---------------------------------------------------------------------------------------------------------
Status check_norm(const seq_norm_args_t* a, bool e4m3) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  if (bad_dtype(a->dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a->rows < 0 || a->channels < 1 || a->x_row < 0 || a->residual_row < 0 || !(a->eps >= 0.f))
    return CONV_WGRAD_ERR_BAD_SHAPE;
  const int32_t g = a->group;
  if (e4m3 ? g != 0 && g != 32 && g != 64 && g != 128 && g != 256 : g != 0) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->channels > kMaxNorm || a->rows >= kMaxAll) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (a->rows && (!a->x || !a->w || !a->y || (e4m3 && !a->scale) || (a->h && !a->residual)))
    return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a->dtype);
  if (off(a->x, e) || off(a->residual, e) || off(a->h, e) || off(a->w, 4) || off(a->rstd, 4) || off(a->scale, 4) ||
      (!e4m3 && off(a->y, e)))
    return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_norm_grad(const seq_norm_grad_args_t* a) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  if (bad_dtype(a->dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a->rows < 0 || a->channels < 1 || a->dy_row < 0 || a->h_row < 0 || a->dh_row < 0)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->channels > kMaxNorm || a->rows >= kMaxAll) return CONV_WGRAD_ERR_UNSUPPORTED;
  return CONV_WGRAD_OK;
}

// ---- layer norm ---------------------------------------------------------------------------------------------------
Status check_layer_norm(const seq_layer_norm_args_t* a) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  if (bad_dtype(a->dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a->rows < 0 || a->channels < 1 || a->x_row < 0 || a->residual_row < 0 || !(a->eps >= 0.f))
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->channels > kMaxNorm || a->rows >= kMaxAll) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (a->rows && (!a->x || !a->w || !a->y || (a->h && !a->residual))) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a->dtype);
  if (off(a->x, e) || off(a->residual, e) || off(a->h, e) || off(a->y, e) || off(a->w, 4) || off(a->b, 4) ||
      off(a->mean, 4) || off(a->rstd, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_layer_norm_grad(const seq_layer_norm_grad_args_t* a) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  if (bad_dtype(a->dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a->rows < 0 || a->channels < 1 || a->dy_row < 0 || a->h_row < 0 || a->dh_row < 0)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->channels > kMaxNorm || a->rows >= kMaxAll) return CONV_WGRAD_ERR_UNSUPPORTED;
  return CONV_WGRAD_OK;
}

uint64_t layer_norm_grad_floats(const seq_layer_norm_grad_args_t& a) {
  return (uint64_t)cw::layer_norm_grad_parts(a) * 2 * a.channels;
}

// ---- convolution --------------------------------------------------------------------------------------------------
Status check_conv(const seq_conv_args_t& a, bool step) {
  const Status st = check_tokens(a.tokens);
  if (st != CONV_WGRAD_OK) return st;
  if (bad_dtype(a.dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a.channels < 1 || a.width < 2 || a.width > 4 || negative(a.x) || a.state_stride < 0 || a.state_out_stride < 0)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (step && (a.tokens.offsets || a.tokens.rows != 1)) return CONV_WGRAD_ERR_BAD_SHAPE;
  const int64_t size = (a.width - 1) * a.channels;
  if (a.state_out && a.tokens.pool > 1 && a.state_out_stride < size) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a.state && a.state == a.state_out && a.state_stride != a.state_out_stride) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a.channels > kMaxChannels || !pieces_fit(a.tokens)) return CONV_WGRAD_ERR_UNSUPPORTED;
  // the most workgroups of any of the launches: 4 channels a lane, 64 lanes, one wave a piece of 16 tokens
  const int64_t blocks = (a.channels + 255) / 256;
  const int64_t pieces = seq_pieces(cw::seq_map(a.tokens, 4)) + a.tokens.sequences;
  if (!fits(pieces, 256 * blocks)) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (!a.w || (seq_rows(a.tokens) && !a.x.ptr)) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a.dtype);
  if (off(a.x.ptr, e) || off(a.w, 4) || off(a.bias, 4) || off(a.state, e) || off(a.state_out, e))
    return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_conv_forward(const seq_conv_args_t* a, bool step) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_conv(*a, step);
  if (st != CONV_WGRAD_OK) return st;
  if (negative(a->y)) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (seq_rows(a->tokens) && !a->y.ptr) return CONV_WGRAD_ERR_NULL_ARG;
  return off(a->y.ptr, elem(a->dtype)) ? CONV_WGRAD_ERR_MISALIGNED : CONV_WGRAD_OK;
}

Status check_conv_grad(const seq_conv_grad_args_t* g) {
  if (!g) return CONV_WGRAD_ERR_NULL_ARG;
  seq_conv_args_t f = g->fwd;
  f.state_out = nullptr;
  f.state_out_stride = 0;
  const Status st = check_conv(f, false);
  if (st != CONV_WGRAD_OK) return st;
  return negative(g->dy) || negative(g->dx) ? CONV_WGRAD_ERR_BAD_SHAPE : CONV_WGRAD_OK;
}

uint64_t conv_grad_floats(const seq_conv_grad_args_t& g) {
  return (uint64_t)cw::conv_grad_parts(g) * g.fwd.channels * (g.fwd.width + 1);
}

// ---- scan ---------------------------------------------------------------------------------------------------------
// The sizes and strides that every scan entry reads.
Status check_scan_shape(const seq_scan_args_t& a, bool step) {
  const Status st = check_tokens(a.tokens);
  if (st != CONV_WGRAD_OK) return st;
  if (bad_dtype(a.dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a.channels < 1 || a.groups < 1 || a.channels % a.groups || a.states < 1 || negative(a.u) || negative(a.delta) ||
      negative(a.z) || negative(a.B) || negative(a.C) || a.B_group < 0 || a.C_group < 0 || a.state_stride < 0 ||
      a.state_out_stride < 0)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (step && (a.tokens.offsets || a.tokens.rows != 1)) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a.channels > kMaxChannels || a.states > 32 || !pieces_fit(a.tokens)) return CONV_WGRAD_ERR_UNSUPPORTED;
  if ((step ? cw::scan_step_lanes(a) : cw::scan_lanes(a)) > kMaxLanes) return CONV_WGRAD_ERR_UNSUPPORTED;
  return CONV_WGRAD_OK;
}

Status check_scan_inputs(const seq_scan_args_t& a) {
  if (!a.A || (seq_rows(a.tokens) && (!a.u.ptr || !a.delta.ptr || !a.B.ptr || !a.C.ptr)))
    return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a.dtype);
  if (off(a.u.ptr, e) || off(a.delta.ptr, e) || off(a.z.ptr, e) || off(a.B.ptr, e) || off(a.C.ptr, e) || off(a.A, 4) ||
      off(a.skip, 4) || off(a.delta_bias, 4) || off(a.save, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_scan_forward(const seq_scan_args_t* a, bool step) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  Status st = check_scan_shape(*a, step);
  if (st == CONV_WGRAD_OK) st = check_scan_inputs(*a);
  if (st != CONV_WGRAD_OK) return st;
  if (negative(a->y)) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->state_out && a->tokens.pool > 1 && a->state_out_stride < a->channels * a->states)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->state && a->state == a->state_out && a->state_stride != a->state_out_stride) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (seq_rows(a->tokens) && !a->y.ptr) return CONV_WGRAD_ERR_NULL_ARG;
  if (off(a->y.ptr, elem(a->dtype)) || off(a->state, 4) || off(a->state_out, 4)) return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_scan_grad(const seq_scan_grad_args_t* g) {
  if (!g) return CONV_WGRAD_ERR_NULL_ARG;
  const seq_scan_args_t& a = g->fwd;
  const Status st = check_scan_shape(a, false);
  if (st != CONV_WGRAD_OK) return st;
  if (negative(g->dy)) return CONV_WGRAD_ERR_BAD_SHAPE;
  // the bytes between two rows are 32 bits in the kernel
  for (const seq_view_t* v : {&a.u, &a.delta, &a.z, &a.B, &a.C, &g->dy})
    if (v->row >= (int64_t)1 << 26) return CONV_WGRAD_ERR_UNSUPPORTED;
  return cw::scan_grad_lanes(*g) <= kMaxLanes ? CONV_WGRAD_OK : CONV_WGRAD_ERR_UNSUPPORTED;
}

// ---- gated delta rule -----------------------------------------------------------------------------------------------
// The sizes and strides that every entry reads.
Status check_delta_shape(const seq_delta_args_t& a, bool step) {
  const Status st = check_tokens(a.tokens);
  if (st != CONV_WGRAD_OK) return st;
  if (bad_dtype(a.dtype)) return CONV_WGRAD_ERR_BAD_DTYPE;
  if (a.heads < 1 || a.key_heads < 1 || a.heads % a.key_heads || a.key_dim < 1 || a.value_dim < 1 || negative(a.q) ||
      negative(a.k) || negative(a.v) || negative(a.g) || negative(a.beta) || a.q_head < 0 || a.k_head < 0 || a.v_head < 0 ||
      a.state_stride < 0 || a.state_out_stride < 0)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (step && (a.tokens.offsets || a.tokens.rows != 1)) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a.heads > 65536 || a.key_dim > 256 || a.value_dim > 1024 || !pieces_fit(a.tokens)) return CONV_WGRAD_ERR_UNSUPPORTED;
  // the offsets of a chunk's 64 rows are 32 bits in the kernels, in bytes, for inputs and for dense outputs
  const int64_t most = (int64_t)1 << 24;
  for (const seq_view_t* v : {&a.q, &a.k, &a.v})
    if (v->row >= most) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (a.heads * a.value_dim >= most || a.key_heads * a.key_dim >= most) return CONV_WGRAD_ERR_UNSUPPORTED;
  // a state's heads start at 64-bit offsets; the workspace's sizes have to stay far from overflowing 64 bits
  if (seq_rows(a.tokens) > kMaxAll / 64 || seq_pieces(cw::seq_map(a.tokens, 6)) > ((int64_t)1 << 31) / a.heads)
    return CONV_WGRAD_ERR_UNSUPPORTED;
  return (step ? cw::delta_step_lanes(a) : cw::delta_lanes(a)) <= kMaxLanes ? CONV_WGRAD_OK : CONV_WGRAD_ERR_UNSUPPORTED;
}

Status check_delta_inputs(const seq_delta_args_t& a) {
  if (seq_rows(a.tokens) && (!a.q.ptr || !a.k.ptr || !a.v.ptr || !a.g.ptr || !a.beta.ptr)) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a.dtype);
  if (off(a.q.ptr, e) || off(a.k.ptr, e) || off(a.v.ptr, e) || off(a.g.ptr, 4) || off(a.beta.ptr, 4) || off(a.save, 16))
    return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_delta_forward(const seq_delta_args_t* a, bool step) {
  if (!a) return CONV_WGRAD_ERR_NULL_ARG;
  Status st = check_delta_shape(*a, step);
  if (st == CONV_WGRAD_OK) st = check_delta_inputs(*a);
  if (st != CONV_WGRAD_OK) return st;
  if (negative(a->o)) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->o.row >= (int64_t)1 << 24) return CONV_WGRAD_ERR_UNSUPPORTED;
  if (a->state_out && a->tokens.pool > 1 && a->state_out_stride < a->heads * a->key_dim * a->value_dim)
    return CONV_WGRAD_ERR_BAD_SHAPE;
  if (a->state && a->state == a->state_out && a->state_stride != a->state_out_stride) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (seq_rows(a->tokens) && !a->o.ptr) return CONV_WGRAD_ERR_NULL_ARG;
  if (off(a->o.ptr, elem(a->dtype)) || off(a->state, 4) || off(a->state_out, 4)) return CONV_WGRAD_ERR_MISALIGNED;
  return CONV_WGRAD_OK;
}

Status check_delta_grad(const seq_delta_grad_args_t* g) {
  if (!g) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_delta_shape(g->fwd, false);
  if (st != CONV_WGRAD_OK) return st;
  if (negative(g->dout) || g->dout_head < 0) return CONV_WGRAD_ERR_BAD_SHAPE;
  if (g->dout.row >= (int64_t)1 << 24) return CONV_WGRAD_ERR_UNSUPPORTED;
  return cw::delta_grad_lanes(*g) <= kMaxLanes ? CONV_WGRAD_OK : CONV_WGRAD_ERR_UNSUPPORTED;
}

Status check_space(const void* ws, size_t have, uint64_t floats) {
  if (floats == 0) return CONV_WGRAD_OK;
  if (!ws) return CONV_WGRAD_ERR_NULL_ARG;
  if (have < floats * 4) return CONV_WGRAD_ERR_WORKSPACE;
  return off(ws, 16) ? CONV_WGRAD_ERR_MISALIGNED : CONV_WGRAD_OK;
}

Status size_of(Status st, uint64_t floats, size_t* bytes) {
  if (st == CONV_WGRAD_OK) *bytes = (size_t)(floats * 4);
  return st;
}

}  // namespace

extern "C" {

conv_wgrad_status_t seq_rms_norm(const seq_norm_args_t* args, void* stream) {
  const Status st = check_norm(args, false);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_norm(*args, false, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_rms_norm_e4m3(const seq_norm_args_t* args, void* stream) {
  const Status st = check_norm(args, true);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_norm(*args, true, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_rms_norm_grad_workspace(const seq_norm_grad_args_t* args, size_t* bytes) {
  if (!bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_norm_grad(args);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::norm_grad_parts(*args) * args->channels : 0, bytes);
}

conv_wgrad_status_t seq_rms_norm_grad(const seq_norm_grad_args_t* args, void* workspace, size_t ws_bytes,
                                      void* stream) {
  Status st = check_norm_grad(args);
  if (st != CONV_WGRAD_OK) return st;
  const seq_norm_grad_args_t& a = *args;
  if (!a.w || !a.dw || (a.rows && (!a.dy || !a.h || !a.rstd || !a.dx))) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a.dtype);
  if (off(a.dy, e) || off(a.h, e) || off(a.dh, e) || off(a.dx, e) || off(a.w, 4) || off(a.rstd, 4) || off(a.dw, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  st = check_space(workspace, ws_bytes, (uint64_t)cw::norm_grad_parts(a) * a.channels);
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_norm_grad(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_layer_norm(const seq_layer_norm_args_t* args, void* stream) {
  const Status st = check_layer_norm(args);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_layer_norm(*args, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_layer_norm_grad_workspace(const seq_layer_norm_grad_args_t* args, size_t* bytes) {
  if (!bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_layer_norm_grad(args);
  return size_of(st, st == CONV_WGRAD_OK ? layer_norm_grad_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_layer_norm_grad(const seq_layer_norm_grad_args_t* args, void* workspace, size_t ws_bytes,
                                        void* stream) {
  Status st = check_layer_norm_grad(args);
  if (st != CONV_WGRAD_OK) return st;
  const seq_layer_norm_grad_args_t& a = *args;
  if (!a.w || !a.dw || (a.rows && (!a.dy || !a.h || !a.mean || !a.rstd || !a.dx))) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(a.dtype);
  if (off(a.dy, e) || off(a.h, e) || off(a.dh, e) || off(a.dx, e) || off(a.w, 4) || off(a.mean, 4) || off(a.rstd, 4) ||
      off(a.dw, 4) || off(a.db, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  st = check_space(workspace, ws_bytes, layer_norm_grad_floats(a));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_layer_norm_grad(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_causal_conv(const seq_conv_args_t* args, void* stream) {
  const Status st = check_conv_forward(args, false);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_conv(*args, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_causal_conv_step(const seq_conv_args_t* args, void* stream) {
  const Status st = check_conv_forward(args, true);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_conv_step(*args, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_causal_conv_grad_workspace(const seq_conv_grad_args_t* args, size_t* bytes) {
  if (!bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_conv_grad(args);
  return size_of(st, st == CONV_WGRAD_OK ? conv_grad_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_causal_conv_grad(const seq_conv_grad_args_t* args, void* workspace, size_t ws_bytes,
                                         void* stream) {
  Status st = check_conv_grad(args);
  if (st != CONV_WGRAD_OK) return st;
  const seq_conv_grad_args_t& g = *args;
  if (!g.dw || (seq_rows(g.fwd.tokens) && (!g.dy.ptr || !g.dx.ptr))) return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(g.fwd.dtype);
  if (off(g.dy.ptr, e) || off(g.dx.ptr, e) || off(g.dstate_out, e) || off(g.dstate, e) || off(g.dw, 4) ||
      off(g.dbias, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  st = check_space(workspace, ws_bytes, conv_grad_floats(g));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_conv_grad(g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_selective_scan_save(const seq_scan_args_t* args, size_t* bytes) {
  if (!args || !bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_scan_shape(*args, false);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::scan_save_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_selective_scan_workspace(const seq_scan_args_t* args, size_t* bytes) {
  if (!args || !bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_scan_shape(*args, false);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::scan_ws_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_selective_scan(const seq_scan_args_t* args, void* workspace, size_t ws_bytes, void* stream) {
  Status st = check_scan_forward(args, false);
  if (st == CONV_WGRAD_OK) st = check_space(workspace, ws_bytes, (uint64_t)cw::scan_ws_floats(*args));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_scan(*args, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_selective_scan_step(const seq_scan_args_t* args, void* stream) {
  const Status st = check_scan_forward(args, true);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_scan_step(*args, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_selective_scan_grad_workspace(const seq_scan_grad_args_t* args, size_t* bytes) {
  if (!bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_scan_grad(args);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::scan_grad_ws_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_selective_scan_grad(const seq_scan_grad_args_t* args, void* workspace, size_t ws_bytes,
                                            void* stream) {
  Status st = check_scan_grad(args);
  if (st == CONV_WGRAD_OK) st = check_scan_inputs(args->fwd);
  if (st != CONV_WGRAD_OK) return st;
  const seq_scan_grad_args_t& g = *args;
  if (!g.dA || (seq_rows(g.fwd.tokens) && (!g.dy.ptr || !g.fwd.save || !g.du || !g.ddelta || !g.dB || !g.dC ||
                                           (g.fwd.z.ptr && !g.dz))))
    return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(g.fwd.dtype);
  if (off(g.dy.ptr, e) || off(g.du, e) || off(g.ddelta, e) || off(g.dz, e) || off(g.dB, e) || off(g.dC, e) ||
      off(g.dA, 4) || off(g.dskip, 4) || off(g.ddelta_bias, 4) || off(g.dstate, 4) || off(g.dstate_out, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  st = check_space(workspace, ws_bytes, (uint64_t)cw::scan_grad_ws_floats(g));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_scan_grad(g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_gated_delta_save(const seq_delta_args_t* args, size_t* bytes) {
  if (!args || !bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_delta_shape(*args, false);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::delta_save_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_gated_delta_workspace(const seq_delta_args_t* args, size_t* bytes) {
  if (!args || !bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_delta_shape(*args, false);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::delta_chunk_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_gated_delta(const seq_delta_args_t* args, void* workspace, size_t ws_bytes, void* stream) {
  Status st = check_delta_forward(args, false);
  if (st == CONV_WGRAD_OK) st = check_space(workspace, ws_bytes, (uint64_t)cw::delta_chunk_floats(*args));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_delta(*args, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_gated_delta_step(const seq_delta_args_t* args, void* stream) {
  const Status st = check_delta_forward(args, true);
  return st != CONV_WGRAD_OK ? st : of(cw::launch_delta_step(*args, static_cast<hipStream_t>(stream)));
}

conv_wgrad_status_t seq_gated_delta_grad_workspace(const seq_delta_grad_args_t* args, size_t* bytes) {
  if (!bytes) return CONV_WGRAD_ERR_NULL_ARG;
  const Status st = check_delta_grad(args);
  return size_of(st, st == CONV_WGRAD_OK ? (uint64_t)cw::delta_grad_ws_floats(*args) : 0, bytes);
}

conv_wgrad_status_t seq_gated_delta_grad(const seq_delta_grad_args_t* args, void* workspace, size_t ws_bytes,
                                         void* stream) {
  Status st = check_delta_grad(args);
  if (st == CONV_WGRAD_OK) st = check_delta_inputs(args->fwd);
  if (st != CONV_WGRAD_OK) return st;
  const seq_delta_grad_args_t& g = *args;
  if (seq_rows(g.fwd.tokens) && (!g.dout.ptr || !g.fwd.save || !g.dq || !g.dk || !g.dv || !g.dg || !g.dbeta))
    return CONV_WGRAD_ERR_NULL_ARG;
  const int64_t e = elem(g.fwd.dtype);
  if (off(g.dout.ptr, e) || off(g.dq, e) || off(g.dk, e) || off(g.dv, e) || off(g.dg, 4) || off(g.dbeta, 4) ||
      off(g.dstate, 4) || off(g.dstate_out, 4))
    return CONV_WGRAD_ERR_MISALIGNED;
  st = check_space(workspace, ws_bytes, (uint64_t)cw::delta_grad_ws_floats(g));
  if (st != CONV_WGRAD_OK) return st;
  return of(cw::launch_delta_grad(g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
