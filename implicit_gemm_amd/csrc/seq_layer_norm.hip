// Layer norm with the residual's addition, and its gradient (gfx950).
//
//   h = x + residual (rounded: the next layer reads it back), m = mean(h), r = 1 / sqrt(mean((h - m)^2) + eps)
//   y = (h - m) r w + b
//   with n = (h - m) r and g = dy w:  dx = r (g - mean(g) - n mean(g n)) + dh,  dw = sum dy n,  db = sum dy over rows
//
// Both are bound by HBM: a row is read once, kept in registers between its reductions and its outputs, and written once
// (bf16, 16384 rows of 2048 with a residual: 48.6 us for 268 MB, 5.5 TB/s, the gradient 46.1 + 4.7 for its partial sums;
// 200704 rows of 384: 54.7 us for 308 MB, the gradient 97.6 + 4.8 for 462; calls on 16384 rows of 8192: 118 us for 537 MB,
// the gradient 162 for 805; on 8192 of 16384: 111 and 178; fp32, 8192 of 8192: 102 and 164).  Not so fp32 rows of more than
// 8192 channels forward, whose 64 elements a lane leave registers for one wave a SIMD: 4096 of 16384 153 us for 537 MB, of
// 16383 205.
// The mean is the sum over channels and then, from the registers, the mean of what it leaves: the first sum's rounding is
// 2^-24 of the values, which may be any number of deviations (a row of 10000.1 throughout: y off by 0.3 with the sum alone).
// The squares are summed about both.  The gradient finds the rest of the mean, that its 32 bits leave, from h likewise.  A
// row belongs to a team of 16 lanes (four rows a wave: feature maps of few channels), of 64, of 256, or of 1024 for the
// widest gradients; each lane holds up to 64 elements in 16-byte vectors, and a team of at most a wave needs no barrier.
#include "seq_common.h"

namespace cw {

namespace {

// WHOLE: the channels are a multiple of the vector, so that none is cut short and the branches for that go.  bf16, forward
// and gradient in a captured graph: 6007 rows of 4096 channels with a residual 66.3 us against 72.5, 200704 rows of 384 155.8
// against 176.0.  (Non-temporal stores of y and dx brought the latter from 158 to 137 us, but y then took its reader longer:
// forward and an elementwise use of y 112.4 us against 108.1.)
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void take(Raw<T, V>& r, const T* p, int n) {
  if constexpr (WHOLE) r.load(p);
  else r.load_n(p, n);
}
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void give(const Raw<T, V>& r, T* p, int n) {
  if constexpr (WHOLE) r.store(p);
  else r.store_n(p, n);
}

// Channels from a vector on: hidden from the compiler where vectors are cut short, so that it keeps no masks of their
// elements from one loop over a row to the next (fp32, 4096 rows of 16383 channels: 205 us against 231; the same for whole
// vectors of 16384 167 against 150).
template <bool WHOLE>
__device__ __forceinline__ int left_of(int n) {
  return WHOLE ? n : opaque(n);
}

// The sums of N values over a team, with 3 TEAM / 64 floats of lds for a team of more than a wave.
template <int TEAM, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float* lds) {
  static_assert(N <= 3, "size of lds");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_reduce<AddOp>(v[i], TEAM < 64 ? TEAM : 64);
  if constexpr (TEAM > 64) {
    constexpr int kWaves = TEAM / 64;
    __syncthreads();  // the last reduction's reads are done
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i * kWaves + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_reduce<AddOp>(lds[i * kWaves + threadIdx.x % kWaves], kWaves);
  }
}

template <typename T, int TEAM, int NE, bool WHOLE>
__global__ __launch_bounds__(256) void layer_norm_kernel(seq_layer_norm_args_t a) {
  constexpr int V = 16 / sizeof(T), NV = NE / V, kTeams = 256 / TEAM;
  __shared__ float lds[4];
  const int lane = threadIdx.x % TEAM;
  const int C = (int)a.channels;
  for (int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM; row < a.rows; row += (int64_t)gridDim.x * kTeams) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    Raw<T, V> raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      if (c < C) take<WHOLE>(raw[v], x + c, C - c);
      else raw[v].clear();
    }
    if (a.residual) {
      const T* p = static_cast<const T*>(a.residual) + row * a.residual_row;
      Raw<T, V> res[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TEAM + lane) * V;
        if (c < C) take<WHOLE>(res[v], p + c, C - c);
        else res[v].clear();
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = raw[v].get(i) + res[v].get(i);
        raw[v].pack(s);
      }
      if (a.h) {
        T* h = static_cast<T*>(a.h) + row * C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = (v * TEAM + lane) * V;
          if (c < C) give<WHOLE>(raw[v], h + c, C - c);
        }
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < V; ++i) sum += raw[v].get(i);
    const float mean = team_reduce<AddOp, TEAM>(sum, lds) / (float)C;
    float left = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = left_of<WHOLE>(C - (v * TEAM + lane) * V);
#pragma unroll
      for (int i = 0; i < V; ++i) left += (WHOLE ? 0 : i) < n ? raw[v].get(i) - mean : 0.f;
    }
    const float rest = team_reduce<AddOp, TEAM>(left, lds) / (float)C;
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = left_of<WHOLE>(C - (v * TEAM + lane) * V);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = (WHOLE ? 0 : i) < n ? (raw[v].get(i) - mean) - rest : 0.f;
        ss = __builtin_fmaf(d, d, ss);
      }
    }
    const float r = 1.f / sqrtf(team_reduce<AddOp, TEAM>(ss, lds) / (float)C + a.eps);
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean + rest;
      if (a.rstd) a.rstd[row] = r;
    }
    T* y = static_cast<T*>(a.y) + row * C;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      if (c < C) {
        Raw<float, V> w, b;
        take<WHOLE>(w, a.w + c, C - c);
        b.clear();
        if (a.b) take<WHOLE>(b, a.b + c, C - c);
        Raw<T, V> o;
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = __builtin_fmaf(((raw[v].get(i) - mean) - rest) * r, w.get(i), b.get(i));
        o.pack(s);
        give<WHOLE>(o, y + c, C - c);
      }
    }
  }
}

struct LayerNormGradArgs {
  seq_layer_norm_grad_args_t a;
  float* part;   // [gridDim.x][2][channels]: partial sums of dw and db
};

template <typename T, int TEAM, int NE, bool WHOLE>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void layer_norm_grad_kernel(LayerNormGradArgs args) {
  constexpr int V = 16 / sizeof(T), NV = NE / V, kThreads = TEAM > 256 ? TEAM : 256, kTeams = kThreads / TEAM;
  __shared__ float lds[TEAM > 64 ? 3 * TEAM / 64 : 2 * TEAM * NE];
  const seq_layer_norm_grad_args_t& a = args.a;
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int C = (int)a.channels;
  float w[NV][V], accw[NV][V], accb[NV][V];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TEAM + lane) * V;
    Raw<float, V> t;
    t.clear();
    if (c < C) take<WHOLE>(t, a.w + c, C - c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[v][i] = t.get(i);
      accw[v][i] = accb[v][i] = 0.f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * kTeams + team; row < a.rows; row += (int64_t)gridDim.x * kTeams) {
    const T* pdy = static_cast<const T*>(a.dy) + row * a.dy_row;
    const T* ph = static_cast<const T*>(a.h) + row * a.h_row;
    const T* pdh = static_cast<const T*>(a.dh) + row * a.dh_row;
    Raw<T, V> dy[NV], h[NV], dh[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      dy[v].clear();
      h[v].clear();
      dh[v].clear();
      if (c < C) {
        take<WHOLE>(dy[v], pdy + c, C - c);
        take<WHOLE>(h[v], ph + c, C - c);
        if (a.dh) take<WHOLE>(dh[v], pdh + c, C - c);
      }
    }
    const float mean = a.mean[row], r = a.rstd[row];
    // Channels past the end have dy = w = 0; their n is a number that no output takes.
    float sums[3] = {0.f, 0.f, 0.f};       // of g, g (h - mean) and h - mean
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = opaque(C - (v * TEAM + lane) * V);     // no masks kept over the rows' loop
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = dy[v].get(i) * w[v][i], c = h[v].get(i) - mean;
        sums[0] += g;
        sums[1] = __builtin_fmaf(g, c, sums[1]);
        sums[2] += (WHOLE ? 0 : i) < n ? c : 0.f;
      }
    }
    team_sums<TEAM>(sums, lds);
    const float rest = sums[2] / (float)C, s1 = sums[0] / (float)C, s2 = (sums[1] - rest * sums[0]) * r / (float)C;
    T* dx = static_cast<T*>(a.dx) + row * C;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      Raw<T, V> o;
      float s[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = dy[v].get(i), n = ((h[v].get(i) - mean) - rest) * r;
        s[i] = __builtin_fmaf(r, __builtin_fmaf(d, w[v][i], -s1) - n * s2, dh[v].get(i));
        accw[v][i] = __builtin_fmaf(d, n, accw[v][i]);
        accb[v][i] += d;
      }
      o.pack(s);
      if (c < C) give<WHOLE>(o, dx + c, C - c);
    }
  }
  float* part = args.part + (int64_t)blockIdx.x * 2 * C;
  if constexpr (kTeams > 1) {
    // The teams' sums are added in order through LDS.
    for (int q = 0; q < kTeams; ++q) {
      if (team == q) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float& sw = lds[(v * V + i) * TEAM + lane];
            float& sb = lds[TEAM * NE + (v * V + i) * TEAM + lane];
            accw[v][i] += q ? sw : 0.f;
            accb[v][i] += q ? sb : 0.f;
            sw = accw[v][i];
            sb = accb[v][i];
          }
      }
      __syncthreads();
    }
    if (team != kTeams - 1) return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TEAM + lane) * V;
    Raw<float, V> ow, ob;
    ow.pack(accw[v]);
    ob.pack(accb[v]);
    if (c < C) {
      give<WHOLE>(ow, part + c, C - c);
      give<WHOLE>(ob, part + C + c, C - c);
    }
  }
}

// Which team.  Times of a call in us, forward / gradient, in a captured graph, the operands in the last-level cache up to
// 256 MB:
//
// 16 lanes against a wave, bf16        8192 rows            65536 rows           131072 rows
//   128 channels                     3.3 /  8.8 against     8.5 / 17.8 against  15.1 / 25.2 against
//                                    4.9 /  9.3            21.8 / 38.8          39.1 / 71.5
//   384                              4.7 / 15.2 against    19.6 / 35.6 against  33.5 / 58.9 against
//                                    5.4 / 10.6            27.0 / 40.9          49.1 / 95.4
//   512                              5.5 / 18.5 against    24.5 / 45.7 against  44.4 / 88.8 against
//                                    5.7 / 10.8            27.9 / 42.3          52.8 / 99.5
// (fp32 by bytes: 256 channels as bf16's 512.)  Rows of up to 768 bytes go to 16 lanes where there are enough of them; of
// 1024 bytes they would gain forward and lose in the gradient up to 65536 rows.
//
// A wave against 256 lanes, bf16        256 rows             1024 rows            8192 rows            65536 rows
//   512 channels                     2.9 /  6.0 against    3.0 /  6.4 against   5.7 / 10.9 against   28.5 /  42.4 against
//                                    3.4 /  6.2            4.0 /  8.6          12.2 / 25.0           74.3 / 174.8
//   2048                             4.1 /  8.8 against    4.6 / 11.0 against  15.5 / 25.3 against  107.4 / 155.7 against
//                                    3.5 /  8.0            4.4 / 11.2          16.9 / 31.6          126.8 / 225.6
template <typename T>
constexpr bool by_sixteen(int64_t C, int64_t rows, int64_t least) { return C * (int64_t)sizeof(T) <= 768 && rows >= least; }
template <typename T>
constexpr bool by_wave(int64_t C, int64_t rows) { return C * (int64_t)sizeof(T) <= 4096 && rows >= 1024; }

template <typename T, bool WHOLE>
hipError_t layer_norm_t(const seq_layer_norm_args_t& a, hipStream_t stream) {
  const int64_t C = a.channels;
  const bool narrow = by_sixteen<T>(C, a.rows, 4096), wave = by_wave<T>(C, a.rows);
  const int64_t teams = narrow ? 16 : wave ? 4 : 1;
  const int64_t most = 1 << 20;
  const int64_t blocks = (a.rows + teams - 1) / teams;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(256);
  if (narrow) {
    if (C <= 16 * 8) return launch_kernel(layer_norm_kernel<T, 16, 8, WHOLE>, grid, block, a, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 16 * 16) return launch_kernel(layer_norm_kernel<T, 16, 24, WHOLE>, grid, block, a, stream);
    }
    return launch_kernel(layer_norm_kernel<T, 16, 16, WHOLE>, grid, block, a, stream);
  }
  if (wave) {
    if (C <= 64 * 8) return launch_kernel(layer_norm_kernel<T, 64, 8, WHOLE>, grid, block, a, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 64 * 16) return launch_kernel(layer_norm_kernel<T, 64, 32, WHOLE>, grid, block, a, stream);
    }
    return launch_kernel(layer_norm_kernel<T, 64, 16, WHOLE>, grid, block, a, stream);
  }
  if (C <= 256 * 8) return launch_kernel(layer_norm_kernel<T, 256, 8, WHOLE>, grid, block, a, stream);
  if (C <= 256 * 16) return launch_kernel(layer_norm_kernel<T, 256, 16, WHOLE>, grid, block, a, stream);
  if (C <= 256 * 32) return launch_kernel(layer_norm_kernel<T, 256, 32, WHOLE>, grid, block, a, stream);
  return launch_kernel(layer_norm_kernel<T, 256, 64, WHOLE>, grid, block, a, stream);
}

// Lanes of a row's team in the gradient.
template <typename T>
int grad_team(const seq_layer_norm_grad_args_t& a) {
  return by_sixteen<T>(a.channels, a.rows, 32768) ? 16 : by_wave<T>(a.channels, a.rows) ? 64 : 256;
}

template <typename T, bool WHOLE>
hipError_t layer_norm_grad_t(const seq_layer_norm_grad_args_t& a, float* ws, hipStream_t stream) {
  const int64_t C = a.channels;
  const LayerNormGradArgs k{a, ws};
  const dim3 grid((unsigned)layer_norm_grad_parts(a)), block(256);
  const int team = grad_team<T>(a);
  if (team == 16) {
    if (C <= 16 * 8) return launch_kernel(layer_norm_grad_kernel<T, 16, 8, WHOLE>, grid, block, k, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 16 * 16) return launch_kernel(layer_norm_grad_kernel<T, 16, 24, WHOLE>, grid, block, k, stream);
    }
    return launch_kernel(layer_norm_grad_kernel<T, 16, 16, WHOLE>, grid, block, k, stream);
  }
  if (team == 64) {
    if (C <= 64 * 8) return launch_kernel(layer_norm_grad_kernel<T, 64, 8, WHOLE>, grid, block, k, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 64 * 16) return launch_kernel(layer_norm_grad_kernel<T, 64, 32, WHOLE>, grid, block, k, stream);
    }
    return launch_kernel(layer_norm_grad_kernel<T, 64, 16, WHOLE>, grid, block, k, stream);
  }
  if constexpr (sizeof(T) == 4) {
    if (C <= 256 * 8) return launch_kernel(layer_norm_grad_kernel<T, 256, 8, WHOLE>, grid, block, k, stream);
  }
  if (C <= 256 * 16) return launch_kernel(layer_norm_grad_kernel<T, 256, 16, WHOLE>, grid, block, k, stream);
  if (C <= 256 * 32) return launch_kernel(layer_norm_grad_kernel<T, 256, 32, WHOLE>, grid, block, k, stream);
  return launch_kernel(layer_norm_grad_kernel<T, 1024, 16, WHOLE>, grid, dim3(1024), k, stream);
}

template <typename T>
hipError_t layer_norm_of(const seq_layer_norm_args_t& a, hipStream_t stream) {
  return a.channels % (16 / (int)sizeof(T)) == 0 ? layer_norm_t<T, true>(a, stream) : layer_norm_t<T, false>(a, stream);
}
template <typename T>
hipError_t layer_norm_grad_of(const seq_layer_norm_grad_args_t& a, float* ws, hipStream_t stream) {
  return a.channels % (16 / (int)sizeof(T)) == 0 ? layer_norm_grad_t<T, true>(a, ws, stream) : layer_norm_grad_t<T, false>(a, ws, stream);
}

}  // namespace

hipError_t launch_layer_norm(const seq_layer_norm_args_t& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  switch (a.dtype) {
    case CONV_WGRAD_F32: return layer_norm_of<float>(a, stream);
    case CONV_WGRAD_BF16: return layer_norm_of<Bf16>(a, stream);
    default: return layer_norm_of<F16>(a, stream);
  }
}

// Workgroups of the gradient, each with its own partial dw and db: up to 256 as many as the rows need, then at least four
// rows a team (1024 rows of 4096 channels in bf16: 15.5 us with 256 workgroups against 23.9 with 1024, whose sums take
// longer to add than the rows), up to 512 (against 1024 and 256: 16384 rows of 4096 channels in bf16 86.8 against 89.0 and
// 120.5 us, 65536 of 2048 in fp32 295 against 337 and 370, 200704 of 384 in bf16 forward and gradient 156 against 166 and 170).
int layer_norm_grad_parts(const seq_layer_norm_grad_args_t& a) {
  const int teams = 256 / (a.dtype == CONV_WGRAD_F32 ? grad_team<float>(a) : grad_team<Bf16>(a));
  const int64_t need = (a.rows + teams - 1) / teams, some = (need + 3) / 4;
  const int64_t parts = need <= 256 ? need : some < 256 ? 256 : some;
  return (int)(parts < 1 ? 1 : parts < 512 ? parts : 512);
}

hipError_t launch_layer_norm_grad(const seq_layer_norm_grad_args_t& a, float* ws, hipStream_t stream) {
  hipError_t err;
  switch (a.dtype) {
    case CONV_WGRAD_F32: err = layer_norm_grad_of<float>(a, ws, stream); break;
    case CONV_WGRAD_BF16: err = layer_norm_grad_of<Bf16>(a, ws, stream); break;
    default: err = layer_norm_grad_of<F16>(a, ws, stream); break;
  }
  if (err != hipSuccess) return err;
  FoldList l;
  const int parts = layer_norm_grad_parts(a);
  l.n = a.db ? 2 : 1;
  l.f[0] = FoldPart{ws, 2 * a.channels, parts, a.channels, a.dw, CONV_WGRAD_F32};
  l.f[1] = FoldPart{ws + a.channels, 2 * a.channels, parts, a.channels, a.db, CONV_WGRAD_F32};
  return launch_seq_fold(l, stream);
}

}  // namespace cw
