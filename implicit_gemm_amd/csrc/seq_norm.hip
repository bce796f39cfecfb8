// Root-mean-square norm with the residual's addition, its 8-bit output and its gradient (gfx950).
//
//   h = x + residual (rounded: the next layer reads it back), r = 1 / sqrt(mean(h^2) + eps), y = h r w
//   8 bits: scale = max|y| / 448 over a group of channels, q = e4m3(y / scale)
//   dx = r (dy w - h r^2 mean(dy w h)) + dh,   dw = sum over rows of dy h r
//
// All three are bound by HBM: a row is read once, kept in registers between its reduction and its outputs, and written
// once.  A row belongs to a team of 64 or 256 lanes (1024 for the widest gradients), each lane holding up to 64
// elements in 16-byte vectors; a team of one wave needs no barrier.  16384 x 2048 in bf16: 46 us for 268 MB forward (5.8
// TB/s), 45 us for 268 MB backward; 6007 x 4096 in fp16 to 8 bits: 34 us for 172 MB (a copy of 1 GiB reaches 5.2 TB/s).
#include "seq_common.h"

namespace cw {

namespace {

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// NE elements a lane.
template <typename T, int TEAM, int NE, bool E4M3>
__global__ __launch_bounds__(256) void norm_kernel(seq_norm_args_t a) {
  constexpr int V = 16 / sizeof(T), NV = NE / V, kTeams = 256 / TEAM;
  __shared__ float lds[4];
  const int lane = threadIdx.x % TEAM;
  const int C = (int)a.channels;
  for (int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM; row < a.rows; row += (int64_t)gridDim.x * kTeams) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    Raw<T, V> raw[NV], res[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      if (c < C) raw[v].load_n(x + c, C - c);
      else raw[v].clear();
    }
    if (a.residual) {
      const T* r = static_cast<const T*>(a.residual) + row * a.residual_row;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TEAM + lane) * V;
        if (c < C) res[v].load_n(r + c, C - c);
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
          if (c < C) raw[v].store_n(h + c, C - c);
        }
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < V; ++i) ss = __builtin_fmaf(raw[v].get(i), raw[v].get(i), ss);
    ss = team_reduce<AddOp, TEAM>(ss, lds);
    const float r = 1.f / sqrtf(ss / (float)C + a.eps);
    if constexpr (!E4M3) {
      if (a.rstd && lane == 0) a.rstd[row] = r;
      T* y = static_cast<T*>(a.y) + row * C;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TEAM + lane) * V;
        if (c < C) {
          Raw<float, V> w;
          w.load_n(a.w + c, C - c);
          Raw<T, V> o;
          float s[V];
#pragma unroll
          for (int i = 0; i < V; ++i) s[i] = raw[v].get(i) * r * w.get(i);
          o.pack(s);
          o.store_n(y + c, C - c);
        }
      }
    } else {
      float y[NV][V], top[NV];
      float all = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TEAM + lane) * V;
        Raw<float, V> w;
        w.clear();
        if (c < C) w.load_n(a.w + c, C - c);
        top[v] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[v][i] = c + i < C ? raw[v].get(i) * r * w.get(i) : 0.f;
          top[v] = MaxBitsOp::of(top[v], fabsf(y[v][i]));
        }
        all = MaxBitsOp::of(all, top[v]);
      }
      const int group = a.group;
      const int nscale = group ? (C + group - 1) / group : 1;
      if (group == 0) {
        all = team_reduce<MaxBitsOp, TEAM>(all, lds);
#pragma unroll
        for (int v = 0; v < NV; ++v) top[v] = all;
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) top[v] = lanes_reduce<MaxBitsOp>(top[v], group / V);
      }
      uint8_t* q = static_cast<uint8_t*>(a.y) + row * C;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TEAM + lane) * V;
        // top / 448 underflows to zero for the smallest denormals too; a denormal scale can be so much smaller than top /
        // 448 that the quotient passes 464, whose code is NaN: there it is held to 448 (and is a number, as top is).
        float scale = top[v] / 448.f;
        scale = scale == 0.f ? 1.f : scale;
        const bool rough = scale < __FLT_MIN__;
        if (c < C) {
          if (group == 0 ? c == 0 : c % group == 0) a.scale[row * nscale + (group ? c / group : 0)] = scale;
          float f[V];
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = y[v][i] / scale;
          if (__any(rough)) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = rough ? __builtin_amdgcn_fmed3f(f[i], -448.f, 448.f) : f[i];
          }
          uint32_t packed[V / 4];
#pragma unroll
          for (int i = 0; i < V; i += 4) packed[i / 4] = e4m3x4(f[i], f[i + 1], f[i + 2], f[i + 3]);
          if (c + V <= C) {
            __builtin_memcpy(q + c, packed, V);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (c + i < C) q[c + i] = (uint8_t)(packed[i / 4] >> (8 * (i % 4)));
          }
        }
      }
    }
  }
}

struct NormGradArgs {
  seq_norm_grad_args_t a;
  float* part;   // [gridDim.x][channels]: partial sums of dw
};

template <typename T, int TEAM, int NE>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void norm_grad_kernel(NormGradArgs args) {
  constexpr int V = 16 / sizeof(T), NV = NE / V, kThreads = TEAM > 256 ? TEAM : 256, kTeams = kThreads / TEAM;
  __shared__ float lds[TEAM > 64 ? TEAM / 64 : TEAM * NE];
  const seq_norm_grad_args_t& a = args.a;
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int C = (int)a.channels;
  float w[NV][V], acc[NV][V];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TEAM + lane) * V;
    Raw<float, V> t;
    t.clear();
    if (c < C) t.load_n(a.w + c, C - c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[v][i] = t.get(i);
      acc[v][i] = 0.f;
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
        dy[v].load_n(pdy + c, C - c);
        h[v].load_n(ph + c, C - c);
        if (a.dh) dh[v].load_n(pdh + c, C - c);
      }
    }
    const float r = a.rstd[row];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < V; ++i) s = __builtin_fmaf(dy[v].get(i) * w[v][i], h[v].get(i), s);
    s = team_reduce<AddOp, TEAM>(s, lds);
    const float k = s / (float)C * r * r;
    T* dx = static_cast<T*>(a.dx) + row * C;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TEAM + lane) * V;
      Raw<T, V> o;
      float s[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = dy[v].get(i), hv = h[v].get(i);
        s[i] = r * (g * w[v][i] - hv * k) + dh[v].get(i);
        acc[v][i] = __builtin_fmaf(g * hv, r, acc[v][i]);
      }
      o.pack(s);
      if (c < C) o.store_n(dx + c, C - c);
    }
  }
  float* part = args.part + (int64_t)blockIdx.x * C;
  if constexpr (kTeams > 1) {
    // The teams' sums are added in order through LDS.
    for (int q = 0; q < kTeams; ++q) {
      if (team == q) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float& s = lds[(v * V + i) * TEAM + lane];
            acc[v][i] += q ? s : 0.f;
            s = acc[v][i];
          }
      }
      __syncthreads();
    }
    if (team != kTeams - 1) return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TEAM + lane) * V;
    Raw<float, V> o;
    o.pack(acc[v]);
    if (c < C) o.store_n(part + c, C - c);
  }
}

// One wave a row needs no barrier and keeps the most rows in flight, up to 4 KB a row (four vectors a lane); wider rows
// take four waves.  16384 x 2048 in bf16: norm 46 us by waves, 49 by fours, gradient 44 and 49; 3136 x 1537 in fp32: 20
// and 17, 21 and 18.  Few rows take four waves a row in any case, for the latency of one.
template <typename T>
constexpr bool by_wave(int64_t C) { return C * (int64_t)sizeof(T) <= 4096; }

template <typename T, bool E4M3>
hipError_t norm_t(const seq_norm_args_t& a, hipStream_t stream) {
  const int64_t C = a.channels;
  const bool wave = by_wave<T>(C) && a.rows >= 1024;
  const int64_t teams = wave ? 4 : 1;
  const int64_t most = 1 << 20;
  const int64_t blocks = (a.rows + teams - 1) / teams;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(256);
  if (wave) {
    if (C <= 64 * 8) return launch_kernel(norm_kernel<T, 64, 8, E4M3>, grid, block, a, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 64 * 16) return launch_kernel(norm_kernel<T, 64, 32, E4M3>, grid, block, a, stream);
    }
    return launch_kernel(norm_kernel<T, 64, 16, E4M3>, grid, block, a, stream);
  }
  if (C <= 256 * 8) return launch_kernel(norm_kernel<T, 256, 8, E4M3>, grid, block, a, stream);
  if (C <= 256 * 16) return launch_kernel(norm_kernel<T, 256, 16, E4M3>, grid, block, a, stream);
  if (C <= 256 * 32) return launch_kernel(norm_kernel<T, 256, 32, E4M3>, grid, block, a, stream);
  return launch_kernel(norm_kernel<T, 256, 64, E4M3>, grid, block, a, stream);
}

bool grad_by_wave(const seq_norm_grad_args_t& a) {
  return a.dtype == CONV_WGRAD_F32 ? by_wave<float>(a.channels) : by_wave<Bf16>(a.channels);
}

template <typename T>
hipError_t norm_grad_t(const seq_norm_grad_args_t& a, float* ws, hipStream_t stream) {
  const int64_t C = a.channels;
  const NormGradArgs k{a, ws};
  const dim3 grid((unsigned)norm_grad_parts(a));
  if (by_wave<T>(C)) {
    if (C <= 64 * 8) return launch_kernel(norm_grad_kernel<T, 64, 8>, grid, dim3(256), k, stream);
    if constexpr (sizeof(T) == 2) {
      if (C > 64 * 16) return launch_kernel(norm_grad_kernel<T, 64, 32>, grid, dim3(256), k, stream);
    }
    return launch_kernel(norm_grad_kernel<T, 64, 16>, grid, dim3(256), k, stream);
  }
  if constexpr (sizeof(T) == 4) {
    if (C <= 256 * 8) return launch_kernel(norm_grad_kernel<T, 256, 8>, grid, dim3(256), k, stream);
  }
  if (C <= 256 * 16) return launch_kernel(norm_grad_kernel<T, 256, 16>, grid, dim3(256), k, stream);
  if (C <= 256 * 32) return launch_kernel(norm_grad_kernel<T, 256, 32>, grid, dim3(256), k, stream);
  return launch_kernel(norm_grad_kernel<T, 1024, 16>, grid, dim3(1024), k, stream);
}

}  // namespace

hipError_t launch_norm(const seq_norm_args_t& a, bool e4m3, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  switch (a.dtype) {
    case CONV_WGRAD_F32: return e4m3 ? norm_t<float, true>(a, stream) : norm_t<float, false>(a, stream);
    case CONV_WGRAD_BF16: return e4m3 ? norm_t<Bf16, true>(a, stream) : norm_t<Bf16, false>(a, stream);
    default: return e4m3 ? norm_t<F16, true>(a, stream) : norm_t<F16, false>(a, stream);
  }
}

// Workgroups of the gradient, each with its own partial dw: as many as rows need, up to 2048 waves, or 4096 where four
// share a row.
int norm_grad_parts(const seq_norm_grad_args_t& a) {
  const int64_t teams = grad_by_wave(a) ? 4 : 1;
  const int64_t need = (a.rows + teams - 1) / teams;
  const int64_t most = teams == 4 ? 512 : 1024;
  return (int)(need < 1 ? 1 : need < most ? need : most);
}

hipError_t launch_norm_grad(const seq_norm_grad_args_t& a, float* ws, hipStream_t stream) {
  hipError_t err;
  switch (a.dtype) {
    case CONV_WGRAD_F32: err = norm_grad_t<float>(a, ws, stream); break;
    case CONV_WGRAD_BF16: err = norm_grad_t<Bf16>(a, ws, stream); break;
    default: err = norm_grad_t<F16>(a, ws, stream); break;
  }
  if (err != hipSuccess) return err;
  FoldList l;
  l.n = 1;
  l.f[0] = FoldPart{ws, a.channels, norm_grad_parts(a), a.channels, a.dw, CONV_WGRAD_F32};
  return launch_seq_fold(l, stream);
}

}  // namespace cw
