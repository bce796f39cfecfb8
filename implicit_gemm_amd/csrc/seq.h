// Internal interface between the C ABI of the sequence operators and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/conv_wgrad.h"
#include "kernels.h"

namespace cw {

constexpr int64_t kMaxLanes = ((int64_t)1 << 32) - 1;   // of a launch

// How tokens are cut into pieces (device side: find_piece).
struct SeqMap {
  const int32_t* offsets;
  int32_t S;       // sequences
  int32_t rows;    // tokens of each, or rows in all with offsets
  int32_t shift;   // 2^shift tokens a piece
  int32_t per;     // pieces of each sequence (without offsets)
};

inline SeqMap seq_map(const seq_tokens_t& t, int shift) {
  const int64_t per = t.rows > 0 ? ((t.rows - 1) >> shift) + 1 : 1;
  return SeqMap{t.offsets, (int32_t)t.sequences, (int32_t)t.rows, shift, t.offsets ? 0 : (int32_t)per};
}
// Numbers that name pieces: with offsets one more sequence, the padding behind the last.
inline int64_t seq_pieces(const SeqMap& m) {
  return m.offsets ? (int64_t)(m.rows >> m.shift) + m.S + 1 : (int64_t)m.S * m.per;
}
inline int64_t seq_rows(const seq_tokens_t& t) { return t.offsets ? t.rows : t.sequences * t.rows; }

// out[e] = sum over p of part[p * stride + e] for e < E, in a fixed order, rounded to dtype (CONV_WGRAD_F32 ..).
struct FoldPart {
  const float* part;
  int64_t stride;
  int32_t count;
  int64_t E;
  void* out;
  int32_t dtype;
};
// Up to five folds in one launch.
struct FoldList {
  FoldPart f[5];
  int32_t n;
};
int64_t fold_lanes(const FoldList& list);   // of the launch
hipError_t launch_seq_fold(const FoldList& list, hipStream_t stream);

hipError_t launch_norm(const seq_norm_args_t& a, bool e4m3, hipStream_t stream);
int norm_grad_parts(const seq_norm_grad_args_t& a);
hipError_t launch_norm_grad(const seq_norm_grad_args_t& a, float* ws, hipStream_t stream);

hipError_t launch_layer_norm(const seq_layer_norm_args_t& a, hipStream_t stream);
int layer_norm_grad_parts(const seq_layer_norm_grad_args_t& a);
hipError_t launch_layer_norm_grad(const seq_layer_norm_grad_args_t& a, float* ws, hipStream_t stream);

hipError_t launch_conv(const seq_conv_args_t& a, hipStream_t stream);
hipError_t launch_conv_step(const seq_conv_args_t& a, hipStream_t stream);
int64_t conv_grad_parts(const seq_conv_grad_args_t& a);
hipError_t launch_conv_grad(const seq_conv_grad_args_t& a, float* ws, hipStream_t stream);

// Tokens between two states that the forward scan saves for the gradient.
constexpr int kSaveShift = 4;
// Blocks of 64 channels, none across two groups.
inline int64_t scan_blocks(const seq_scan_args_t& a) { return (a.channels / a.groups + 63) / 64 * a.groups; }
int64_t scan_save_floats(const seq_scan_args_t& a);
int64_t scan_ws_floats(const seq_scan_args_t& a);
hipError_t launch_scan(const seq_scan_args_t& a, float* ws, hipStream_t stream);
hipError_t launch_scan_step(const seq_scan_args_t& a, hipStream_t stream);
int64_t scan_grad_ws_floats(const seq_scan_grad_args_t& g);
// Lanes of the largest launch of a call.
int64_t scan_lanes(const seq_scan_args_t& a);
int64_t scan_step_lanes(const seq_scan_args_t& a);
int64_t scan_grad_lanes(const seq_scan_grad_args_t& g);
hipError_t launch_scan_grad(const seq_scan_grad_args_t& a, float* ws, hipStream_t stream);

int64_t delta_save_floats(const seq_delta_args_t& a);
int64_t delta_chunk_floats(const seq_delta_args_t& a);
hipError_t launch_delta(const seq_delta_args_t& a, float* ws, hipStream_t stream);
hipError_t launch_delta_step(const seq_delta_args_t& a, hipStream_t stream);
int64_t delta_grad_ws_floats(const seq_delta_grad_args_t& g);
// Lanes of the largest launch of a call.
int64_t delta_lanes(const seq_delta_args_t& a);
int64_t delta_step_lanes(const seq_delta_args_t& a);
int64_t delta_grad_lanes(const seq_delta_grad_args_t& g);
hipError_t launch_delta_grad(const seq_delta_grad_args_t& g, float* ws, hipStream_t stream);

}  // namespace cw
