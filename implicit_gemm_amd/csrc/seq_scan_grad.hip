// Gradients of the selective state space scan (gfx950).
//
// With do = dy z sigmoid(z) and the reversed recurrence  g[t] = do[t] C[t] + c[t],  c[t - 1] = e^(D[t] A) g[t]:
//   dC[t] = sum_d do h[t],  dB[t] = sum_d g D u,  du = skip do + D sum_n g B,
//   dD = sum_n A c[t - 1] h[t - 1] + u sum_n g B,  ddelta = dD sigmoid(delta + bias),  dA = sum_t D c[t - 1] h[t - 1]
// and dz from o = sum_n h C + skip u.  All of it needs the states again: the forward saved one state of every 16 tokens
// (4 bytes a token and channel for 16 states; scanning forward once more to find them would cost as much as the first
// of the three forward launches, about twice what writing and reading them does).
//
// Bound by the vector ALU.  A workgroup takes a piece of a sequence and 64 channels, 16 tokens at a time from the last:
// what a token and channel need (D, D u, do) is computed once by the lane that loads it and passed through LDS; then
// NG lanes share a channel, four states each, and keep e^(D A) and h of the 16 tokens in registers (128 of them), so
// the reversed sweep recomputes nothing.  Sums over states are taken inside a group of NG lanes, sums over channels by
// exchanging halves of the wave (each step halves the values a lane holds), then over the waves through LDS and over
// the channel blocks by a fold, in a fixed order.
#include "seq_scan.h"

namespace cw {

namespace {

constexpr int kTile = 1 << kSaveShift;

struct GradArgs {
  ScanArgs s;
  seq_scan_grad_args_t g;   // outputs; g.fwd is s.a
  int32_t parts;            // workgroups along the pieces
  float* part_bc;           // [dblocks][2][rows * groups * states]: dB, dC
  float* part_a;            // [parts][channels * states]
  float* part_s;            // [parts][2][channels]: dskip, ddelta_bias
};

// The value of the lane 4 away inside each half row of 8 lanes.
__device__ __forceinline__ float xor4(float v) {
  const int b = __builtin_bit_cast(int, v);
  int r = __builtin_amdgcn_update_dpp(0, b, 0x104, 0xf, 0x5, false);    // row_shl:4 into banks 0 and 2
  r = __builtin_amdgcn_update_dpp(r, b, 0x114, 0xf, 0xa, false);        // row_shr:4 into banks 1 and 3
  return __builtin_bit_cast(float, r);
}
constexpr int kXor8 = 0x128;   // row_ror:8

// Sums v[0 .. 7] over the lanes that differ in bits 3 .. 5 and, for NG < 8, 2 (and 1); lane l gets value
// 4 b5 + 2 b4 + b3 of its bits.
template <int NG>
__device__ __forceinline__ float channels_reduce(const float (&v)[8]) {
  float r4[4], r2[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2 p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
    r4[i] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32x2 p = __builtin_amdgcn_permlane16_swap(__float_as_uint(r4[i]), __float_as_uint(r4[i + 2]), false, false);
    r2[i] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  const bool b3 = threadIdx.x & 8;
  float r = (b3 ? r2[1] : r2[0]) + dpp<kXor8>(b3 ? r2[0] : r2[1]);
  if constexpr (NG < 8) r += xor4(r);
  if constexpr (NG < 4) r += dpp<kXor2>(r);
  return r;
}

// What the lanes of a workgroup pass each other of one tile.
template <int NG>
struct GradTile {
  alignas(16) float dt[kTile][64], x[kTile][64], dov[kTile][64];   // D, D u, do
  float o[kTile][64], gb[kTile][64], da[kTile][64];                // sums over states: h C, g B, A c[t - 1] h[t - 1]
  alignas(16) float B[kTile][4 * NG], C[kTile][4 * NG];
  float bias[64], skip[64];
  float bc[NG][kTile][8 * NG];                                     // each wave's sums over its channels: dB, dC
};

template <typename T, int NG, bool FULL>
__global__ __launch_bounds__(64 * NG) void scan_grad_kernel(GradArgs k) {
  constexpr int NP = 4 * NG, kWaveCh = 64 / NG, V = 16 / NG;
  __shared__ GradTile<NG> m;
  const seq_scan_args_t& a = k.s.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int N = a.states, D = (int)a.channels, Dg = D / (int)a.groups;
  const int blocks = k.s.dblocks * (int)a.groups;
  const int part = (int)blockIdx.x / blocks, block = (int)blockIdx.x % blocks;
  const int g = block / k.s.dblocks, cblock = block % k.s.dblocks;
  const int c0 = cblock * 64;               // first channel of the block in its group
  const int nch = min(64, Dg - c0);         // channels of the block
  const int d0 = g * Dg + c0;
  // As a lane of the sweeps: one channel, four states.
  const int ch = wave * kWaveCh + lane / NG, n0 = (lane % NG) * 4, nv = N - n0;
  const bool on = ch < nch;
  const int d = d0 + min(ch, nch - 1);
  // As a lane of the loads and outputs: one token, V channels.
  const int it = tid / (64 / V), ic = tid % (64 / V) * V, iv = nch - ic;   // iv <= 0: none
  const bool gated = a.z.ptr != nullptr;

  float A2[4], dA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = FULL || i < nv ? a.A[(int64_t)d * N + n0 + i] * kLog2e : 0.f;
  float dskip[V], dbias[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dskip[j] = dbias[j] = 0.f;
  if (tid < 64) {
    m.bias[tid] = a.delta_bias && tid < nch ? a.delta_bias[d0 + tid] : 0.f;
    m.skip[tid] = a.skip && tid < nch ? a.skip[d0 + tid] : 0.f;
  }
  __syncthreads();
  const int64_t all_rows = k.s.m.offsets ? k.s.m.rows : (int64_t)k.s.m.S * k.s.m.rows;
  const int64_t bc = all_rows * a.groups * N;   // floats of dB

  for (int piece = part; piece < k.s.pieces; piece += k.parts) {
    Piece p;
    if (!find_piece(k.s.m, piece, p)) continue;
    const int64_t row0 = k.s.m.offsets ? p.first : (int64_t)p.seq * k.s.m.rows;   // dense row of the first token
    const bool real = p.seq < k.s.m.S;
    const int tiles = (p.end - p.t0 + kTile - 1) / kTile;
    const int64_t tile0 = k.s.m.offsets ? (p.first >> kSaveShift) + p.seq
                                        : (int64_t)p.seq * (((k.s.m.rows - 1) >> kSaveShift) + 1);
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0.f;
      if (real && (FULL || i < nv)) {
        if (k.s.split) c[i] = k.s.carry[((int64_t)piece * N + n0 + i) * D + d];
        else if (k.s.last) c[i] = k.s.last[((int64_t)p.seq * D + d) * N + n0 + i];
      }
    }
    Raw<T, V> u, dl, z, dy;
    float h0[4], eB, eC;
    const int eT = tid / NP, eN = tid % NP;   // the element of B and C that this lane stages
    auto fetch = [&](int j) {                 // the inputs of tile j
      const int t = p.t0 + j * kTile;
      u.clear();
      dl.clear();
      z.clear();
      dy.clear();
      eB = eC = 0.f;
      if (j < 0 || !real) return;
      if (t + it < p.end && iv > 0) {
        u.load_n(row_at<const T>(a.u, p, t + it) + d0 + ic, iv);
        dl.load_n(row_at<const T>(a.delta, p, t + it) + d0 + ic, iv);
        dy.load_n(row_at<const T>(k.s.dy, p, t + it) + d0 + ic, iv);
        if (gated) z.load_n(row_at<const T>(a.z, p, t + it) + d0 + ic, iv);
      }
      if (t + eT < p.end && eN < N) {
        eB = to_f32(row_at<const T>(a.B, p, t + eT)[g * a.B_group + eN]);
        eC = to_f32(row_at<const T>(a.C, p, t + eT)[g * a.C_group + eN]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h0[i] = FULL || i < nv ? a.save[((tile0 + (t >> kSaveShift)) * D + d) * N + n0 + i] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) h0[i] = 0.f;
    fetch(tiles - 1);
    for (int j = tiles - 1; j >= 0; --j) {
      const int t = p.t0 + j * kTile;
      const int nt = min(kTile, p.end - t);
      // What the sweeps need of this lane's own token and channels; its raw inputs are kept for its outputs.
      const Raw<T, V> cu = u, cdl = dl, cz = z, cdy = dy;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float raw = cdl.get(q) + m.bias[ic + q];
        // Tokens past the piece's end pass state and gradient on unchanged.
        const float dt = it >= nt ? 0.f : a.softplus ? softplus(raw) : raw;
        float dov = cdy.get(q);
        if (gated) dov *= cz.get(q) * sigmoid(cz.get(q));
        m.dt[it][ic + q] = dt;
        m.x[it][ic + q] = dt * cu.get(q);
        m.dov[it][ic + q] = dov;
      }
      m.B[eT][eN] = eB;
      m.C[eT][eN] = eC;
      float hs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) hs[i] = h0[i];
      __syncthreads();
      fetch(j - 1);

      float e[kTile][4], h[kTile][4];
#pragma unroll
      for (int q = 0; q < kTile; ++q) {
          const float dt = m.dt[q][ch], x = m.x[q][ch];
          float o = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[q][i] = __builtin_amdgcn_exp2f(dt * A2[i]);
            const float b = FULL || i < nv ? x * m.B[q][n0 + i] : 0.f;
            h[q][i] = __builtin_fmaf(e[q][i], q ? h[q ? q - 1 : 0][i] : hs[i], b);
            o = __builtin_fmaf(h[q][i], FULL || i < nv ? m.C[q][n0 + i] : 0.f, o);
          }
          o = lanes_reduce<AddOp>(o, NG);
          if (n0 == 0) m.o[q][ch] = o;
        __builtin_amdgcn_sched_barrier(0);
      }
      // Read B, C, D and D u again: kept from the sweep above they would take 160 registers more.  The compiler is
      // not to know that these are the same indices.
      int ch2 = ch, n2 = n0;
      asm volatile("" : "+v"(ch2), "+v"(n2));
#pragma unroll
      for (int q = kTile - 1; q >= 0; --q) {
          const float dt = m.dt[q][ch2], x = m.x[q][ch2], dov = m.dov[q][ch2];
          const float4 Bv = *reinterpret_cast<const float4*>(&m.B[q][n2]);
          const float4 Cv = *reinterpret_cast<const float4*>(&m.C[q][n2]);
          const float B4[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, C4[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
          float gb = 0.f, da = 0.f, v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float gi = FULL || i < nv ? __builtin_fmaf(dov, C4[i], c[i]) : 0.f;
            v[i] = gi * x;                // lanes without a channel: x and do are zero
            v[4 + i] = dov * h[q][i];
            gb = __builtin_fmaf(gi, B4[i], gb);
            c[i] = e[q][i] * gi;
            const float r = c[i] * (q ? h[q ? q - 1 : 0][i] : hs[i]);
            da = __builtin_fmaf(r, A2[i], da);
            dA[i] = __builtin_fmaf(r, dt, dA[i]);
          }
          gb = lanes_reduce<AddOp>(gb, NG);
          da = lanes_reduce<AddOp>(da, NG);
          if (n0 == 0) {
            m.gb[q][ch2] = gb;
            m.da[q][ch2] = da * kLn2;   // A2 = A log2 e
          }
          const float r = channels_reduce<NG>(v);
          // bits 3 .. 5 name the value; the bits below that are not the state's have the same sum
          if ((lane & 7) < NG) m.bc[wave][q][(lane >> 5) * NP + n0 + ((lane >> 3) & 3)] = r;
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      if (it < nt && iv > 0) {
        float du[V], dd[V], dz[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const float dov = m.dov[it][ic + q], dt = m.dt[it][ic + q], gb = m.gb[it][ic + q], uv = cu.get(q);
          du[q] = __builtin_fmaf(dt, gb, m.skip[ic + q] * dov);
          dd[q] = __builtin_fmaf(uv, gb, m.da[it][ic + q]);
          if (a.softplus) dd[q] *= sigmoid(cdl.get(q) + m.bias[ic + q]);
          dskip[q] = __builtin_fmaf(dov, uv, dskip[q]);
          dbias[q] += dd[q];
          if (gated) {
            const float zv = cz.get(q), sg = sigmoid(zv);
            dz[q] = cdy.get(q) * __builtin_fmaf(m.skip[ic + q], uv, m.o[it][ic + q]) * (sg * __builtin_fmaf(zv, 1.f - sg, 1.f));
          } else {
            dz[q] = 0.f;
          }
        }
        const int64_t at = (row0 + t + it) * D + d0 + ic;
        Raw<T, V> r;
        r.pack(du);
        r.store_n(static_cast<T*>(k.g.du) + at, iv);
        r.pack(dd);
        r.store_n(static_cast<T*>(k.g.ddelta) + at, iv);
        if (gated) {
          r.pack(dz);
          r.store_n(static_cast<T*>(k.g.dz) + at, iv);
        }
      }
      // dB and dC of the block's channels: two values a lane, the waves in order.
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int q = tid / NP, n = tid % NP;
        if (q < nt && n < N) {
          float r = m.bc[0][q][i * NP + n];
#pragma unroll
          for (int w = 1; w < NG; ++w) r += m.bc[w][q][i * NP + n];
          k.part_bc[(cblock * 2 + i) * bc + ((row0 + t + q) * a.groups + g) * N + n] = real ? r : 0.f;
        }
      }
      __syncthreads();
    }
    if (real && p.t0 == 0 && k.g.dstate && on) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (FULL || i < nv) k.g.dstate[((int64_t)p.seq * D + d) * N + n0 + i] = c[i];
    }
  }
  if (on) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (FULL || i < nv) k.part_a[(int64_t)part * D * N + (int64_t)d * N + n0 + i] = dA[i];
  }
#pragma unroll
  for (int q = 0; q < V; ++q) {
    m.dt[it][ic + q] = dskip[q];
    m.x[it][ic + q] = dbias[q];
  }
  __syncthreads();
  if (tid < nch) {
    float s = 0.f, b = 0.f;
    for (int q = 0; q < kTile; ++q) {
      s += m.dt[q][tid];
      b += m.x[q][tid];
    }
    k.part_s[(int64_t)part * 2 * D + d0 + tid] = s;
    k.part_s[(int64_t)part * 2 * D + D + d0 + tid] = b;
  }
}

template <typename T, int NP, bool FULL>
hipError_t grad_t(const GradArgs& k, hipStream_t stream) {
  const int64_t grid = (int64_t)k.parts * k.s.dblocks * k.s.a.groups;
  return launch_kernel(scan_grad_kernel<T, NP / 4, FULL>, dim3((unsigned)grid), dim3(64 * (NP / 4)), k, stream);
}

hipError_t grad_any(const GradArgs& k, hipStream_t stream) {
#define CALL(T, NP, FULL) grad_t<T, NP, FULL>(k, stream)
  SCAN_DISPATCH(CALL, k.s.a.dtype, k.s.a.states)
#undef CALL
}

// Workgroups along the pieces: one a piece, but no more than give about 4096 workgroups (each has a partial of dA).
int32_t grad_parts(const seq_scan_args_t& a, int64_t pieces) {
  const int64_t blocks = (int64_t)scan_dblocks(a) * a.groups;
  int64_t most = 4096 / blocks;
  if (most < 16) most = 16;
  return (int32_t)(pieces < most ? pieces : most);
}

struct GradSpace {
  int64_t carry, sums, bc, a, s, total;   // offsets in floats
  int64_t pieces;
  int32_t parts;
};
GradSpace grad_space(const seq_scan_args_t& a) {
  const ScanCut cut = scan_cut(a);
  GradSpace w;
  w.pieces = seq_pieces(seq_map(a.tokens, cut.shift));
  w.parts = grad_parts(a, w.pieces);
  const int64_t dn = a.channels * a.states;
  int64_t at = 0;
  w.carry = at;
  at += cut.split ? scan_round(w.pieces * dn) : 0;
  w.sums = at;
  at += cut.split ? scan_round(w.pieces * a.channels) : 0;
  w.bc = at;
  at += scan_round(2 * scan_dblocks(a) * seq_rows(a.tokens) * a.groups * a.states);
  w.a = at;
  at += scan_round(w.parts * dn);
  w.s = at;
  at += scan_round(w.parts * 2 * a.channels);
  w.total = at;
  return w;
}

}  // namespace

int64_t scan_grad_ws_floats(const seq_scan_grad_args_t& g) { return grad_space(g.fwd).total; }

hipError_t launch_scan_grad(const seq_scan_grad_args_t& g, float* ws, hipStream_t stream) {
  const seq_scan_args_t& a = g.fwd;
  const ScanCut cut = scan_cut(a);
  const GradSpace w = grad_space(a);
  GradArgs k{};
  k.s.a = a;
  k.s.dy = g.dy;
  k.s.last = g.dstate_out;
  k.s.m = seq_map(a.tokens, cut.shift);
  k.s.pieces = (int32_t)w.pieces;
  k.s.dblocks = scan_dblocks(a);
  k.s.split = cut.split;
  k.s.carry = ws + w.carry;
  k.s.sums = ws + w.sums;
  k.g = g;
  k.parts = w.parts;
  k.part_bc = ws + w.bc;
  k.part_a = ws + w.a;
  k.part_s = ws + w.s;
  hipError_t err;
  if (cut.split && (err = launch_scan_carry(k.s, true, stream)) != hipSuccess) return err;
  if ((err = grad_any(k, stream)) != hipSuccess) return err;
  const int64_t D = a.channels, bc = seq_rows(a.tokens) * a.groups * a.states;
  FoldList l;
  l.n = 0;
  l.f[l.n++] = FoldPart{k.part_bc, 2 * bc, k.s.dblocks, bc, g.dB, a.dtype};
  l.f[l.n++] = FoldPart{k.part_bc + bc, 2 * bc, k.s.dblocks, bc, g.dC, a.dtype};
  l.f[l.n++] = FoldPart{k.part_a, D * a.states, w.parts, D * a.states, g.dA, CONV_WGRAD_F32};
  if (g.dskip) l.f[l.n++] = FoldPart{k.part_s, 2 * D, w.parts, D, g.dskip, CONV_WGRAD_F32};
  if (g.ddelta_bias) l.f[l.n++] = FoldPart{k.part_s + D, 2 * D, w.parts, D, g.ddelta_bias, CONV_WGRAD_F32};
  return launch_seq_fold(l, stream);
}

}  // namespace cw
