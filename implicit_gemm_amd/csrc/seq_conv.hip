// Short causal convolution over tokens, one filter of 2 .. 4 taps per channel, with its carried window, its gradient
// and its form for one token (gfx950).
//
//   p[t] = bias + sum_k w[k] x[t - (W - 1) + k],  y = p or p sigmoid(p)
//   g[t] = dy[t] (or dy[t] sigmoid(p) (1 + p (1 - sigmoid(p)))),  dx[t] = sum_k w[k] g[t + (W - 1) - k],
//   dw[k] = sum_t g[t] x[t - (W - 1) + k],  dbias = sum_t g[t]
//
// Bound by HBM: every input is read once (W - 1 rows a piece twice) and every output written once.  A lane owns V
// neighbouring channels and walks along the tokens with the window in registers, so the taps cost no loads; a wave
// owns one piece of the tokens.  16384 x 4096 in bf16: 51 us for 268 MB forward (5.2 TB/s, a large copy's rate), 93 us
// for 403 MB backward (4.3 TB/s; its vector ALU is busy 60 % of the time: 34 instructions a token and channel).
#include "seq_common.h"

namespace cw {

namespace {

constexpr int kBatch = 8, kGradBatch = 4;   // tokens whose loads are issued together
// Channels of a lane.  The gradient holds two windows, the filters and their sums for each: with four it takes 180
// registers, two waves a SIMD and 99 us (16384 tokens x 4096 channels, bf16), with two 101 registers and 92 us.
constexpr int kVec = 4, kGradVec = 2;

struct ConvArgs {
  seq_conv_args_t a;
  SeqMap m;
  int32_t pieces;
  int32_t cblocks;
  int32_t window;    // the outgoing windows are written by this launch
};

// V channels of row r of a window; slot -1: zeros.
template <typename T, int V>
__device__ __forceinline__ void load_state(Raw<T, V>& v, const seq_conv_args_t& a, int64_t slot, int r, int c, int nv) {
  v.clear();
  if (a.state != nullptr && slot >= 0 && nv > 0)
    v.load_n(static_cast<const T*>(a.state) + slot * a.state_stride + (int64_t)r * a.channels + c, nv);
}

template <int V, int W>
__device__ __forceinline__ void load_taps(const seq_conv_args_t& a, int c, int nv, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    b[j] = 0.f;
    Raw<float, W> t;
    t.clear();
    if (j < nv) {
      t.load(a.w + (int64_t)(c + j) * W);
      if (a.bias) b[j] = a.bias[c + j];
    }
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][j] = t.get(k);
  }
}

// The window after the last of `len` tokens: its rows are read before any is written, so it may lie on the old one.
template <typename T, int V, int W>
__device__ __forceinline__ void write_window(const seq_conv_args_t& a, const Piece& p, int64_t slot, int c, int nv) {
  Raw<T, V> r[W - 1];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int t = p.len - (W - 1) + i;
    if (t < 0) {
      load_state<T, V>(r[i], a, slot, t + W - 1, c, nv);
    } else {
      r[i].clear();
      if (nv > 0) r[i].load_n(&at_lane(row_at<const T>(a.x, p, t), c), nv);
    }
  }
  if (nv > 0 && slot >= 0) {
    T* out = static_cast<T*>(a.state_out) + slot * a.state_out_stride + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) r[i].store_n(out + (int64_t)i * a.channels, nv);
  }
}

// FULL: the channels fill the blocks of 256, so that no load or store needs a check.
template <typename T, int W, bool FULL>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs k) {
  constexpr int V = kVec, B = kBatch;
  const seq_conv_args_t& a = k.a;
  const int cb = (int)blockIdx.x % k.cblocks;
  const int piece = uniform(((int)blockIdx.x / k.cblocks) * 4 + ((int)threadIdx.x >> 6));
  const int c = (cb * 64 + ((int)threadIdx.x & 63)) * V;
  const int nv = FULL ? V : (int)a.channels - c;   // <= 0: no channel of this lane
  float w[W][V], b[V];
  load_taps<V, W>(a, c, nv, w, b);
  Piece p;
  if (piece >= k.pieces || !find_piece(k.m, piece, p)) return;
  const int n = p.end - p.t0;
  if (p.seq >= k.m.S) {
    Raw<T, V> zero;
    zero.clear();
    for (int i = 0; i < n; ++i)
      if (nv > 0) zero.store_n(&at_lane(row_at<T>(a.y, p, p.t0 + i), c), nv);
    return;
  }
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, p.seq);
  Raw<T, V> x[W - 1 + B], next[B];   // the window and a batch of tokens
  auto fetch = [&](int u0) {
#pragma unroll
    for (int i = 0; i < B; ++i) {   // past the piece's end the last row again
      next[i].clear();
      if (nv > 0) next[i].load_n(&at_lane(row_at<const T>(a.x, p, p.t0 + min(u0 + i, n - 1)), c), nv);
    }
  };
  if (n > 0) fetch(0);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    if (p.t0 == 0) {
      load_state<T, V>(x[i], a, slot, i, c, nv);
    } else {
      x[i].clear();
      if (nv > 0) x[i].load_n(&at_lane(row_at<const T>(a.x, p, p.t0 - (W - 1) + i), c), nv);
    }
  }
  for (int u0 = 0; u0 < n; u0 += B) {
#pragma unroll
    for (int i = 0; i < B; ++i) x[W - 1 + i] = next[i];
    if (u0 + B < n) fetch(u0 + B);
    Raw<T, V> y[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float s = b[j];
#pragma unroll
        for (int q = 0; q < W; ++q) s = __builtin_fmaf(w[q][j], x[i + q].get(j), s);
        o[j] = a.silu ? s * sigmoid(s) : s;
      }
      y[i].pack(o);
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (u0 + i < n && nv > 0) y[i].store_n(&at_lane(row_at<T>(a.y, p, p.t0 + u0 + i), c), nv);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) x[i] = x[B + i];
  }
  if (k.window && p.end == p.len) write_window<T, V, W>(a, p, slot, c, nv);
}

// Outgoing windows on the incoming ones: after the outputs, as other pieces of the sequence read the old window.
template <typename T, int W>
__global__ __launch_bounds__(64) void conv_window_kernel(ConvArgs k) {
  constexpr int V = kVec;
  const int s = (int)blockIdx.x / k.cblocks, cb = (int)blockIdx.x % k.cblocks;
  Piece p;
  p.seq = s;
  p.batch = k.m.offsets ? 0 : s;
  p.first = k.m.offsets ? uniform(seq_start(k.m, s)) : 0;
  p.len = k.m.offsets ? max(uniform(seq_start(k.m, s + 1)) - (int)p.first, 0) : k.m.rows;
  const int c = (cb * 64 + (int)threadIdx.x) * V;
  write_window<T, V, W>(k.a, p, pool_slot(k.a.tokens.slots, k.a.tokens.pool, s), c, (int)k.a.channels - c);
}

// One token of each sequence: four channels a lane, all loads at once; latency is all there is.
template <typename T, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs k) {
  constexpr int V = kVec;
  const seq_conv_args_t& a = k.a;
  const int s = (int)blockIdx.x / k.cblocks, cb = (int)blockIdx.x % k.cblocks;
  const int c = (cb * 256 + (int)threadIdx.x) * V;
  const int nv = (int)a.channels - c;
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, s);
  if (nv <= 0) return;
  Raw<T, V> x[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) load_state<T, V>(x[i], a, slot, i, c, nv);
  x[W - 1].load_n(static_cast<const T*>(a.x.ptr) + s * a.x.batch + c, nv);
  float w[W][V], b[V];
  load_taps<V, W>(a, c, nv, w, b);
  Raw<T, V> y;
  float o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float p = b[j];
#pragma unroll
    for (int q = 0; q < W; ++q) p = __builtin_fmaf(w[q][j], x[q].get(j), p);
    o[j] = a.silu ? p * sigmoid(p) : p;
  }
  y.pack(o);
  y.store_n(static_cast<T*>(a.y.ptr) + s * a.y.batch + c, nv);
  if (slot >= 0 && a.state_out) {
    T* out = static_cast<T*>(a.state_out) + slot * a.state_out_stride + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) x[i + 1].store_n(out + (int64_t)i * a.channels, nv);
  }
}

struct ConvGradArgs {
  seq_conv_grad_args_t g;
  SeqMap m;
  int32_t pieces;
  int32_t cblocks;
  int32_t parts;     // workgroups along the pieces
  float* part;       // [parts][channels * (W + 1)]: dw as [channels][W], then dbias
};

template <typename T, int W, bool FULL>
__global__ __launch_bounds__(256, 4) void conv_grad_kernel(ConvGradArgs k) {
  constexpr int V = kGradVec, B = kGradBatch;
  __shared__ float lds[(W + 1) * V * 64];
  const seq_conv_grad_args_t& g = k.g;
  const seq_conv_args_t& a = g.fwd;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int cb = (int)blockIdx.x % k.cblocks, wg = (int)blockIdx.x / k.cblocks;
  const int c = (cb * 64 + lane) * V;
  const int D = (int)a.channels, nv = FULL ? V : D - c;
  float w[W][V], b[V], dw[W + 1][V];   // dw[W]: the bias
  load_taps<V, W>(a, c, nv, w, b);
#pragma unroll
  for (int q = 0; q <= W; ++q)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[q][j] = 0.f;

  for (int first = wg * 4; first < k.pieces; first += k.parts * 4) {
    const int piece = first + wave;
    Piece p;
    if (piece >= k.pieces || !find_piece(k.m, piece, p)) continue;
    const int n = p.end - p.t0;
    if (p.seq >= k.m.S) {
      Raw<T, V> zero;
      zero.clear();
      for (int i = 0; i < n; ++i)
        if (nv > 0) zero.store_n(&at_lane(row_at<T>(g.dx, p, p.t0 + i), c), nv);
      continue;
    }
    const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, p.seq);
    float xw[W - 1][V], gw[W - 1][V];   // the last W - 1 inputs and g's, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      Raw<T, V> r;
      if (n == 0) {   // no token: its window, whatever it holds, is no part of dw
        r.clear();
      } else if (p.t0 == 0) {
        load_state<T, V>(r, a, slot, i, c, nv);
      } else {
        r.clear();
        if (nv > 0) r.load_n(&at_lane(row_at<const T>(a.x, p, p.t0 - (W - 1) + i), c), nv);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        xw[i][j] = r.get(j);
        gw[i][j] = 0.f;
      }
    }
    // Token t0 + u gives g there and then dx of the token W - 1 before it, for which g is complete.
    const int total = n + W - 1;
    const int inside = min(total, p.len - p.t0);   // of these there is an input
    Raw<T, V> nx[B], ndy[B];
    auto fetch = [&](int u0) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        // past the sequence's end the last row again, whose g is not used
        const int t = p.t0 + min(u0 + i, inside - 1);
        if (nv > 0) {
          nx[i].load_n(&at_lane(row_at<const T>(a.x, p, t), c), nv);
          ndy[i].load_n(&at_lane(row_at<const T>(g.dy, p, t), c), nv);
        }
      }
    };
    // Tokens u0 .. u0 + B - 1 of the piece from rx and rdy.  EDGE: some have no input, are the next piece's for dw, or
    // give dx of a token before the piece or of one that the outgoing window holds.
    auto batch = [&](int u0, const Raw<T, V> (&rx)[B], const Raw<T, V> (&rdy)[B], auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int u = u0 + i;
        if (EDGE && u >= total) break;
        float out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = rx[i].get(j);
          float s = __builtin_fmaf(w[W - 1][j], x, b[j]);
#pragma unroll
          for (int q = 0; q < W - 1; ++q) s = __builtin_fmaf(w[q][j], xw[q][j], s);
          float gr = rdy[i].get(j);
          if (a.silu) {
            const float sg = sigmoid(s);
            gr *= sg * __builtin_fmaf(s, 1.f - sg, 1.f);
          }
          if (EDGE) gr = u < inside ? gr : 0.f;
          const float gm = !EDGE || u < n ? gr : 0.f;
          dw[W][j] += gm;
          dw[W - 1][j] = __builtin_fmaf(gm, x, dw[W - 1][j]);
#pragma unroll
          for (int q = 0; q < W - 1; ++q) dw[q][j] = __builtin_fmaf(gm, xw[q][j], dw[q][j]);
          // dx[tau] = sum_q w[q] g[tau + (W - 1) - q]
          float o = w[0][j] * gr;
#pragma unroll
          for (int q = 1; q < W; ++q) o = __builtin_fmaf(w[q][j], gw[W - 1 - q][j], o);
          out[j] = o;
#pragma unroll
          for (int q = 0; q < W - 2; ++q) {
            xw[q][j] = xw[q + 1][j];
            gw[q][j] = gw[q + 1][j];
          }
          xw[W - 2][j] = x;
          gw[W - 2][j] = gr;
        }
        const int tau = p.t0 + u - (W - 1);
        if (EDGE) {
          // before the piece: another piece's token, or the incoming window
          if (tau < p.t0 && (p.t0 > 0 || !g.dstate)) continue;
          if (g.dstate_out && tau >= p.len - (W - 1) && nv > 0) {
            Raw<T, V> r;
            r.load_n(static_cast<const T*>(g.dstate_out) + ((int64_t)p.seq * (W - 1) + (tau - p.len + W - 1)) * D + c, nv);
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] += r.get(j);
          }
        }
        Raw<T, V> r;
        r.pack(out);
        T* to = !EDGE || tau >= 0 ? row_at<T>(g.dx, p, tau)
                                  : static_cast<T*>(g.dstate) + ((int64_t)p.seq * (W - 1) + tau + W - 1) * D;
        if (nv > 0) r.store_n(&at_lane(to, c), nv);
      }
    };
#pragma unroll
    for (int i = 0; i < B; ++i) {
      nx[i].clear();
      ndy[i].clear();
    }
    if (inside > 0) fetch(0);
    for (int u0 = 0; u0 < total; u0 += B) {
      Raw<T, V> rx[B], rdy[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        rx[i] = nx[i];
        rdy[i] = ndy[i];
      }
      if (u0 + B < inside) fetch(u0 + B);
      if (u0 > 0 && u0 + B <= n) batch(u0, rx, rdy, std::false_type());
      else batch(u0, rx, rdy, std::true_type());
    }
  }
  // The four waves' sums, in order.
  for (int q = 0; q < 4; ++q) {
    if (wave == q) {
#pragma unroll
      for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float& s = lds[(i * V + j) * 64 + lane];
          dw[i][j] += q ? s : 0.f;
          s = dw[i][j];
        }
    }
    __syncthreads();
  }
  if (wave == 3) {
    float* part = k.part + (int64_t)wg * D * (W + 1);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < nv) {
        Raw<float, W> t;
        float f[W];
#pragma unroll
        for (int q = 0; q < W; ++q) f[q] = dw[q][j];
        t.pack(f);
        t.store(part + (int64_t)(c + j) * W);
        part[(int64_t)D * W + c + j] = dw[W][j];
      }
  }
}

// A piece's filters and windows are read once for all its tokens, so pieces grow from 2^shift tokens while kConvWaves
// waves are left.  16384 tokens x 4096 channels, bf16: 16 tokens a piece 65 us, 64 tokens (4096 waves) 52 us, 256 tokens
// 67 us; the gradient with 32 tokens 100 us, with 64 (8192 waves of half as many channels) 92 us.
constexpr int64_t kConvWaves = 4096;
int piece_shift(const seq_conv_args_t& a, int shift, int cblocks) {
  while (shift < 8 && (seq_rows(a.tokens) >> (shift + 1)) * cblocks >= kConvWaves) ++shift;
  return shift;
}
SeqMap grad_map(const seq_conv_args_t& a) {
  return seq_map(a.tokens, piece_shift(a, 5, (int)((a.channels + 64 * kVec - 1) / (64 * kVec))));
}
int cblocks(int64_t channels, int per) { return (int)((channels + per - 1) / per); }

bool whole_blocks(int64_t channels) { return channels % (64 * kVec) == 0; }

template <typename T, int W>
hipError_t conv_tw(const seq_conv_args_t& a, hipStream_t stream) {
  ConvArgs k;
  k.a = a;
  k.cblocks = cblocks(a.channels, 64 * kVec);
  k.m = seq_map(a.tokens, piece_shift(a, 4, k.cblocks));
  k.pieces = (int32_t)seq_pieces(k.m);
  const bool on_itself = a.state_out != nullptr && a.state_out == a.state;
  k.window = a.state_out != nullptr && !on_itself;
  const int64_t groups = ((int64_t)k.pieces + 3) / 4;
  const dim3 grid((unsigned)(groups * k.cblocks));
  hipError_t err = whole_blocks(a.channels) ? launch_kernel(conv_kernel<T, W, true>, grid, dim3(256), k, stream)
                                            : launch_kernel(conv_kernel<T, W, false>, grid, dim3(256), k, stream);
  if (err != hipSuccess || !on_itself) return err;
  return launch_kernel(conv_window_kernel<T, W>, dim3((unsigned)(a.tokens.sequences * k.cblocks)), dim3(64), k, stream);
}

template <typename T, int W>
hipError_t conv_step_tw(const seq_conv_args_t& a, hipStream_t stream) {
  ConvArgs k;
  k.a = a;
  k.m = seq_map(a.tokens, 0);
  k.pieces = 0;
  k.window = 0;
  k.cblocks = cblocks(a.channels, 256 * kVec);
  return launch_kernel(conv_step_kernel<T, W>, dim3((unsigned)(a.tokens.sequences * k.cblocks)), dim3(256), k, stream);
}

template <typename T, int W>
hipError_t conv_grad_tw(const seq_conv_grad_args_t& g, float* ws, hipStream_t stream) {
  ConvGradArgs k;
  k.g = g;
  k.m = grad_map(g.fwd);
  k.pieces = (int32_t)seq_pieces(k.m);
  k.cblocks = cblocks(g.fwd.channels, 64 * kGradVec);
  k.parts = (int32_t)conv_grad_parts(g);
  k.part = ws;
  const dim3 grid((unsigned)(k.parts * k.cblocks));
  return g.fwd.channels % (64 * kGradVec) == 0 ? launch_kernel(conv_grad_kernel<T, W, true>, grid, dim3(256), k, stream)
                                      : launch_kernel(conv_grad_kernel<T, W, false>, grid, dim3(256), k, stream);
}

// The dtype and tap count of a call as template arguments.
#define CONV_DISPATCH(call, dtype, width)                                   \
  switch (dtype) {                                                          \
    case CONV_WGRAD_F32:                                                    \
      return width == 2 ? call(float, 2) : width == 3 ? call(float, 3) : call(float, 4); \
    case CONV_WGRAD_BF16:                                                   \
      return width == 2 ? call(Bf16, 2) : width == 3 ? call(Bf16, 3) : call(Bf16, 4);    \
    default:                                                                \
      return width == 2 ? call(F16, 2) : width == 3 ? call(F16, 3) : call(F16, 4);       \
  }

hipError_t conv_grad_any(const seq_conv_grad_args_t& g, float* ws, hipStream_t stream) {
#define CALL(T, W) conv_grad_tw<T, W>(g, ws, stream)
  CONV_DISPATCH(CALL, g.fwd.dtype, g.fwd.width)
#undef CALL
}

}  // namespace

hipError_t launch_conv(const seq_conv_args_t& a, hipStream_t stream) {
#define CALL(T, W) conv_tw<T, W>(a, stream)
  CONV_DISPATCH(CALL, a.dtype, a.width)
#undef CALL
}

hipError_t launch_conv_step(const seq_conv_args_t& a, hipStream_t stream) {
#define CALL(T, W) conv_step_tw<T, W>(a, stream)
  CONV_DISPATCH(CALL, a.dtype, a.width)
#undef CALL
}

// Workgroups along the pieces, four at a time and each with a partial of dw.  A layer of 4096 channels has 32 blocks of 128:
// the 256 pieces of 16384 tokens give it 64 x 32 = 2048 workgroups, more tokens 8192 at most.
int64_t conv_grad_parts(const seq_conv_grad_args_t& g) {
  const int64_t need = (seq_pieces(grad_map(g.fwd)) + 3) / 4;
  return need < 1 ? 1 : need < 256 ? need : 256;
}

hipError_t launch_conv_grad(const seq_conv_grad_args_t& g, float* ws, hipStream_t stream) {
  const hipError_t err = conv_grad_any(g, ws, stream);
  if (err != hipSuccess) return err;
  const int64_t D = g.fwd.channels, W = g.fwd.width;
  FoldList l;
  l.n = 1;
  l.f[0] = FoldPart{ws, D * (W + 1), (int32_t)conv_grad_parts(g), D * W, g.dw, CONV_WGRAD_F32};
  if (g.dbias)
    l.f[l.n++] = FoldPart{ws + D * W, D * (W + 1), (int32_t)conv_grad_parts(g), D, g.dbias, CONV_WGRAD_F32};
  return launch_seq_fold(l, stream);
}

}  // namespace cw
