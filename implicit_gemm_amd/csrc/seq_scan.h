// What the forward scan and its gradient share: how the work is cut, and the carry between pieces.
#pragma once

#include "seq_common.h"

namespace cw {

// A sequence longer than one piece is scanned in three launches: every piece from a zero state (its end state and its
// sum of D, as the product of its decays is e^(A sum D)), the carries of each sequence in order, and every piece again
// from its carry with the outputs.  The gradient runs the same three over the reversed recurrence.
struct ScanArgs {
  seq_scan_args_t a;
  seq_view_t dy;           // gradient only
  const float* last;       // gradient only: dense gradient of the final states, or nullptr
  SeqMap m;
  int32_t pieces;
  int32_t dblocks;         // blocks of 64 channels in a group
  int32_t split;           // the carries are in `carry`
  float* carry;            // [pieces][states][channels]
  float* sums;             // [pieces][channels]: sum of D
};

constexpr int kWholeShift = 30;   // one piece a sequence

struct ScanCut {
  int shift;
  bool split;
};
// Long sequences are cut so that pieces x channel blocks come to about kScanWaves waves, four to a SIMD; a piece has at
// least 16 tokens.  8192 tokens x 2048 channels: 2048 waves 165 us for the three launches, 4096 138, 8192 158 (a piece
// of 32 tokens, whose carries are then as many bytes as the inputs); 5003 x 1536 in 12 sequences: 107, 84 and 102.
// Up to kScanWhole tokens one launch is as quick as three.
constexpr int64_t kScanWaves = 4096, kScanWhole = 64;
ScanCut scan_cut(const seq_scan_args_t& a);
inline int scan_dblocks(const seq_scan_args_t& a) { return (int)((a.channels / a.groups + 63) / 64); }
inline int64_t scan_round(int64_t floats) { return (floats + 63) / 64 * 64; }

// Pieces' aggregates and their combination; backward: over the reversed recurrence.
hipError_t launch_scan_carry(const ScanArgs& k, bool backward, hipStream_t stream);

// Tokens whose loads are issued together, and their elements of B (or C) a lane stages.
constexpr int kScanTile = 8;

// Rows [t, t + kScanTile) of one channel (a lane's own), clamped to the piece.
template <typename T>
struct ChannelTile {
  T v[kScanTile];
  __device__ __forceinline__ void load(const seq_view_t& view, const Piece& p, int t, int d) {
    const T* row = row_at<const T>(view, p, min(max(t, p.t0), p.end - 1));
#pragma unroll
    for (int i = 0; i < kScanTile; ++i) {
      v[i] = load_lane(row, d);
      row += t + i >= p.t0 && t + i + 1 < p.end ? view.row : 0;
    }
  }
  // Zeros past token n.
  __device__ __forceinline__ void cut(int n) {
#pragma unroll
    for (int i = 0; i < kScanTile; ++i)
      if (i >= n) from_f32(0.f, v[i]);
  }
};

// Rows [t, t + kScanTile) of B or C, widened, through registers into LDS ([token][NP]); zeros where there is none.
template <typename T, int NP>
struct StateTile {
  static constexpr int kAll = kScanTile * NP, kEach = (kAll + 63) / 64;
  float v[kEach];
  __device__ __forceinline__ void load(const seq_view_t& view, int64_t group_off, const Piece& p, int t, int N) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * 64 + ((int)threadIdx.x & 63), tok = t + e / NP, n = e % NP;
      v[i] = 0.f;
      if (e < kAll && n < N && tok >= p.t0 && tok < p.end)
        v[i] = to_f32(row_at<const T>(view, p, tok)[group_off + n]);
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * 64 + ((int)threadIdx.x & 63);
      if (e < kAll) lds[e] = v[i];
    }
  }
};

// Lets the waves of a SIMD that have done less go first, in quarters of their work.  Left alone the oldest goes first, and
// when the others have finished the youngest runs by itself, its waits in the open: 60 and 82 us for the aggregates and
// the outputs of 8192 tokens x 2048 channels, against 53 and 74.
__device__ __forceinline__ void yield_by_progress(int done, int all) {
  const int quarter = done * 4 / all;
  if (quarter == 0) __builtin_amdgcn_s_setprio(3);
  else if (quarter == 1) __builtin_amdgcn_s_setprio(2);
  else if (quarter == 2) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

// A log2 e.  Where that is -inf (a state that holds one token's input only) it is fp32's lowest value instead: e^(D A) is
// zero for every D but zero, that of a token past the end, which has to leave the state as it is.
__device__ __forceinline__ float decay_rate(float A) {
  const float v = A * kLog2e;
  return v < -__FLT_MAX__ ? -__FLT_MAX__ : v;
}

// D of a tile's tokens, zero past token n, as is `in`, which repeats its last row there: such a token leaves the state as it
// is, also where that row is infinite.
template <typename T>
__device__ __forceinline__ void step_sizes(float (&dt)[kScanTile], const ChannelTile<T>& delta, float bias,
                                           int32_t with_softplus, int n, ChannelTile<T>& in) {
#pragma unroll
  for (int i = 0; i < kScanTile; ++i) dt[i] = to_f32(delta.v[i]) + bias;
  if (with_softplus) {
#pragma unroll
    for (int i = 0; i < kScanTile; ++i) dt[i] = softplus(dt[i]);
  }
  if (n < kScanTile) {
#pragma unroll
    for (int i = 0; i < kScanTile; ++i) dt[i] = i < n ? dt[i] : 0.f;
    in.cut(n);
  }
}

__device__ __forceinline__ float step_size(float delta, float bias, int32_t with_softplus) {
  const float v = delta + bias;
  return with_softplus ? softplus(v) : v;
}

// The element type and state count of a call as template arguments; the count is rounded up, and the states past the
// call's own have A = B = C = 0.
#define SCAN_DISPATCH_N(call, T, n) \
  ((n) <= 8 ? call(T, 8) : (n) <= 12 ? call(T, 12) : (n) <= 16 ? call(T, 16) : (n) <= 24 ? call(T, 24) : call(T, 32))
#define SCAN_DISPATCH(call, dtype, n)                            \
  switch (dtype) {                                               \
    case CONV_WGRAD_F32: return SCAN_DISPATCH_N(call, float, n); \
    case CONV_WGRAD_BF16: return SCAN_DISPATCH_N(call, Bf16, n); \
    default: return SCAN_DISPATCH_N(call, F16, n);               \
  }
// Kernels that share a channel's states out in fours, and know which states are their own (FULL: all).
#define SCAN_DISPATCH4_N(call, T, n, full)                                                        \
  ((n) <= 8 ? ((full) && (n) == 8 ? call(T, 8, true) : call(T, 8, false))                         \
            : (n) <= 16 ? ((full) && (n) == 16 ? call(T, 16, true) : call(T, 16, false))          \
                        : ((full) && (n) == 32 ? call(T, 32, true) : call(T, 32, false)))
#define SCAN_DISPATCH4(call, dtype, n, full)                            \
  switch (dtype) {                                                      \
    case CONV_WGRAD_F32: return SCAN_DISPATCH4_N(call, float, n, full); \
    case CONV_WGRAD_BF16: return SCAN_DISPATCH4_N(call, Bf16, n, full); \
    default: return SCAN_DISPATCH4_N(call, F16, n, full);               \
  }

}  // namespace cw
