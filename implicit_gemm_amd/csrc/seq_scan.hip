// Selective state space scan for prompts and for one token of each sequence (gfx950).
//
//   D = softplus(delta + bias),  h[t] = e^(D A) h[t - 1] + D u B[t],  y = (sum_n h C[t] + skip u) z sigmoid(z)
//
// Bound by the vector ALU: every (token, channel, state) costs one exponential (8 cycles a wave, twice an instruction)
// and four multiply-adds, 16 states to the 8 bytes that a token and channel move.  A lane owns one channel with all its
// states in registers, so the sum over states stays in the lane; a wave owns 64 channels and one piece of a sequence,
// with B and C of its tokens broadcast from LDS in fp32.  Channels alone give a long prompt too few waves, so its tokens
// are split as well (seq_scan.h).  8192 tokens x 2048 channels x 16 states in bf16: aggregates 54 us, their join 10,
// outputs 75; the vector ALU is busy 84 % and 76 % of the first and the last.  The rank-1 update h <- e h + x B and the
// sum h C on the matrix pipe (v_mfma_f32_4x4x1) were slower, 67 -> 75 and 99 -> 120 us when tried: its products take issue
// slots and their results come late.
#include "seq_scan.h"

namespace cw {

namespace {

// Waves of a workgroup, each with a piece and channels of its own: workgroups of one wave are not spread evenly over
// the four SIMDs of a CU.
constexpr int kScanGroup = 4;

// Channel of this lane within its group's blocks; lanes past the group's end repeat its last channel.
struct Lane {
  int d;
  int g;
  bool on;
};
__device__ __forceinline__ Lane lane_channel(const ScanArgs& k, int block) {
  const int Dg = (int)(k.a.channels / k.a.groups);
  const int c = (block % k.dblocks) * 64 + ((int)threadIdx.x & 63);
  const int g = block / k.dblocks;
  return Lane{g * Dg + min(c, Dg - 1), g, c < Dg};
}

// Decay rates of a channel, zero for the states past N.  The lanes' rows lie 4 N bytes apart, and a load takes a cycle for
// each of the 64 lines that it touches: four states a load where they come in fours.
template <int NP>
__device__ __forceinline__ void load_decay(const seq_scan_args_t& a, int d, float (&A2)[NP]) {
  const float* row = a.A + (int64_t)d * a.states;
  if (a.states % 4 == 0) {
#pragma unroll
    for (int n = 0; n < NP; n += 4) {
      Raw<float, 4> r;
      r.clear();
      if (n < a.states) r.load(row + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) A2[n + i] = decay_rate(r.get(i));
    }
  } else {
#pragma unroll
    for (int n = 0; n < NP; ++n) A2[n] = n < a.states ? decay_rate(row[n]) : 0.f;
  }
}

template <typename T, int NP>
__global__ __launch_bounds__(64 * kScanGroup) void scan_kernel(ScanArgs k) {
  typedef StateTile<T, NP> Tile;
  __shared__ __align__(16) float l_B[kScanGroup][2][Tile::kAll], l_C[kScanGroup][2][Tile::kAll];
  const seq_scan_args_t& a = k.a;
  const int blocks = k.dblocks * (int)a.groups, wave = uniform((int)threadIdx.x >> 6);
  const int job = (int)blockIdx.x * kScanGroup + wave, piece = job / blocks;
  const Lane l = lane_channel(k, job % blocks);
  Piece p;
  if (piece >= k.pieces || !find_piece(k.m, piece, p)) return;
  auto& lb = l_B[wave];
  auto& lc = l_C[wave];
  if (p.seq >= k.m.S) {
    T zero;
    from_f32(0.f, zero);
    for (int t = p.t0; t < p.end; ++t)
      if (l.on) row_at<T>(a.y, p, t)[l.d] = zero;
    return;
  }
  const int N = a.states, D = (int)a.channels;
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, p.seq);
  float A2[NP], h[NP];
  load_decay<NP>(a, l.d, A2);
  const float bias = a.delta_bias ? a.delta_bias[l.d] : 0.f;
  const float skip = a.skip ? a.skip[l.d] : 0.f;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    h[n] = 0.f;
    if (n < N) {
      if (k.split) h[n] = k.carry[((int64_t)piece * N + n) * D + l.d];
      else if (a.state && slot >= 0) h[n] = a.state[slot * a.state_stride + (int64_t)l.d * N + n];
    }
  }
  // Where the states of this sequence's 16-token tiles are saved.
  const int64_t tile0 = k.m.offsets ? (p.first >> kSaveShift) + p.seq
                                    : (int64_t)p.seq * (((k.m.rows - 1) >> kSaveShift) + 1);
  if (p.end > p.t0) {
    const int64_t gb = l.g * a.B_group, gc = l.g * a.C_group;
    ChannelTile<T> u, z, nu, ndl;   // z is not needed before the tile's end: it is not loaded ahead
    Tile sb, sc;
    nu.load(a.u, p, p.t0, l.d);
    ndl.load(a.delta, p, p.t0, l.d);
    sb.load(a.B, gb, p, p.t0, N);
    sc.load(a.C, gc, p, p.t0, N);
    int buf = 0;
    for (int t = p.t0; t < p.end; t += kScanTile, buf ^= 1) {
      const int valid = p.end - t;
      yield_by_progress(t - p.t0, p.end - p.t0);
      sb.put(lb[buf]);
      sc.put(lc[buf]);
      u = nu;
      float dt[kScanTile], o[kScanTile];
      step_sizes<T>(dt, ndl, bias, a.softplus, valid, u);
      wave_sync();
      nu.load(a.u, p, t + kScanTile, l.d);
      ndl.load(a.delta, p, t + kScanTile, l.d);
      if (a.z.ptr) z.load(a.z, p, t, l.d);
      sb.load(a.B, gb, p, t + kScanTile, N);
      sc.load(a.C, gc, p, t + kScanTile, N);
      if (a.save && (t & ((1 << kSaveShift) - 1)) == 0 && l.on) {
        float* s = a.save + (tile0 + (t >> kSaveShift)) * D * N + l.d;   // [tile][state][channel]
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (n < N) s[(int64_t)n * D] = h[n];
      }
      // No branch from here to the outputs, and four states at a time with the next four's B and C read ahead (88 -> 83 us
      // for 8192 tokens x 2048 channels: the compiler by itself reads more of them at once and has fewer waves).
      float4 nb = *reinterpret_cast<const float4*>(&lb[buf][0]), nc = *reinterpret_cast<const float4*>(&lc[buf][0]);
#pragma unroll
      for (int i = 0; i < kScanTile; ++i) {
        const float uv = to_f32(u.v[i]), x = dt[i] * uv;
        float part[2] = {skip * uv, 0.f};
#pragma unroll
        for (int v = 0; v < NP; v += 4) {
          const float b4[4] = {nb.x, nb.y, nb.z, nb.w}, c4[4] = {nc.x, nc.y, nc.z, nc.w};
          const int at = v + 4 < NP ? i * NP + v + 4 : min(i + 1, kScanTile - 1) * NP;
          nb = *reinterpret_cast<const float4*>(&lb[buf][at]);
          nc = *reinterpret_cast<const float4*>(&lc[buf][at]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float e = __builtin_amdgcn_exp2f(dt[i] * A2[v + r]);
            h[v + r] = __builtin_fmaf(e, h[v + r], x * b4[r]);
            part[r & 1] = __builtin_fmaf(h[v + r], c4[r], part[r & 1]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        o[i] = part[0] + part[1];
      }
      if (a.z.ptr) {
#pragma unroll
        for (int i = 0; i < kScanTile; ++i) {
          const float zv = to_f32(z.v[i]);
          o[i] *= zv * sigmoid(zv);
        }
      }
      if (l.on) {
        T y[kScanTile];
#pragma unroll
        for (int i = 0; i < kScanTile; ++i) from_f32(o[i], y[i]);
        T* row = row_at<T>(a.y, p, t);
        if (valid >= kScanTile) {
#pragma unroll
          for (int i = 0; i < kScanTile; ++i, row += a.y.row) store_lane(row, l.d, y[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kScanTile; ++i, row += a.y.row)
            if (i < valid) store_lane(row, l.d, y[i]);
        }
      }
    }
  }
  if (a.state_out && p.end == p.len && slot >= 0 && l.on) {
    float* s = a.state_out + slot * a.state_out_stride + (int64_t)l.d * N;
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < N) s[n] = h[n];
  }
}

// A piece from a zero carry.  Forward: its end state.  Backward: what its first token passes to the token before,
// from g[t] = dy z sigmoid(z) C[t] + c, c = e^(D A) g[t].  The last (first) piece of a sequence passes nothing on.
template <typename T, int NP, bool BACK>
__global__ __launch_bounds__(64 * kScanGroup) void scan_carry_kernel(ScanArgs k) {
  typedef StateTile<T, NP> Tile;
  __shared__ __align__(16) float l_side[kScanGroup][2][Tile::kAll];
  const seq_scan_args_t& a = k.a;
  const int blocks = k.dblocks * (int)a.groups, wave = uniform((int)threadIdx.x >> 6);
  const int job = (int)blockIdx.x * kScanGroup + wave, piece = job / blocks;
  const Lane l = lane_channel(k, job % blocks);
  Piece p;
  if (piece >= k.pieces || !find_piece(k.m, piece, p) || p.seq >= k.m.S) return;
  auto& lds = l_side[wave];
  if (p.end == p.t0 || (BACK ? p.t0 == 0 : p.end == p.len)) return;
  const int N = a.states, D = (int)a.channels;
  float A2[NP], c[NP], sum = 0.f;
  load_decay<NP>(a, l.d, A2);
  const float bias = a.delta_bias ? a.delta_bias[l.d] : 0.f;
#pragma unroll
  for (int n = 0; n < NP; ++n) c[n] = 0.f;
  const seq_view_t in = BACK ? k.dy : a.u, side = BACK ? a.C : a.B;
  const int64_t goff = l.g * (BACK ? a.C_group : a.B_group);
  const int tiles = (p.end - p.t0 + kScanTile - 1) / kScanTile;
  ChannelTile<T> nu, ndl, nz;
  Tile s;
  const int t1 = BACK ? p.t0 + (tiles - 1) * kScanTile : p.t0;
  nu.load(in, p, t1, l.d);
  ndl.load(a.delta, p, t1, l.d);
  if (BACK && a.z.ptr) {
    nz.load(a.z, p, t1, l.d);
    nz.cut(p.end - t1);   // the only tile that can pass the end
  }
  s.load(side, goff, p, t1, N);
  for (int j = 0; j < tiles; ++j) {
    const int t = BACK ? t1 - j * kScanTile : t1 + j * kScanTile;
    const int next = BACK ? t - kScanTile : t + kScanTile;
    yield_by_progress(j, tiles);
    s.put(lds[j & 1]);
    float dt[kScanTile], x[kScanTile];
    step_sizes<T>(dt, ndl, bias, a.softplus, p.end - t, nu);
#pragma unroll
    for (int i = 0; i < kScanTile; ++i) x[i] = to_f32(nu.v[i]);
    if constexpr (BACK) {
      if (a.z.ptr) {
#pragma unroll
        for (int i = 0; i < kScanTile; ++i) {
          const float zv = to_f32(nz.v[i]);
          x[i] *= zv * sigmoid(zv);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kScanTile; ++i) x[i] *= dt[i];
    }
    wave_sync();
    nu.load(in, p, next, l.d);
    ndl.load(a.delta, p, next, l.d);
    if (BACK && a.z.ptr) nz.load(a.z, p, next, l.d);
    s.load(side, goff, p, next, N);
    // Four states at a time, the next four's B (C) read ahead: left to itself the compiler reads a token's all at once and
    // waits for them, 69 us against 66.  It is zero for a token past the end.
    float4 ahead = *reinterpret_cast<const float4*>(&lds[j & 1][(BACK ? kScanTile - 1 : 0) * NP]);
#pragma unroll
    for (int q = 0; q < kScanTile; ++q) {
      const int i = BACK ? kScanTile - 1 - q : q;
      sum += dt[i];
#pragma unroll
      for (int v = 0; v < NP; v += 4) {
        const float4 cur = ahead;
        const int follows = BACK ? max(i - 1, 0) : min(i + 1, kScanTile - 1);
        ahead = *reinterpret_cast<const float4*>(&lds[j & 1][v + 4 < NP ? i * NP + v + 4 : follows * NP]);
        const float b4[4] = {cur.x, cur.y, cur.z, cur.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(dt[i] * A2[v + r]);
          c[v + r] = BACK ? e * __builtin_fmaf(x[i], b4[r], c[v + r]) : __builtin_fmaf(e, c[v + r], x[i] * b4[r]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (l.on) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < N) k.carry[((int64_t)piece * N + n) * D + l.d] = c[n];
    k.sums[(int64_t)piece * D + l.d] = sum;
  }
}

// The carry into every piece of a sequence, in place of the pieces' aggregates; a lane owns one channel and state.
// WAVES waves take 16 consecutive pieces each, all their aggregates in registers after one wait for memory; what the
// waves before pass on comes through LDS.  Four waves for the shortest wait, one where sequences have few pieces and the
// workgroups fill the GPU by themselves (join_few).
//
// A decay is 2^x, x = A log2 e sum D, of a whole piece (or of sixteen).  Where A D is positive, states grow, and over a piece
// by more than fp32 holds though the state itself stays small, or zero (inf x 0): so 2^x h is 2^(x/2) (2^(x/2) h), for x up
// to 254, past which any state that is not zero overflows.
constexpr int kJoinEach = 16;
// 2^half; a sum of D that is NaN comes with an end state that is.
__device__ __forceinline__ float half_decay(float half) { return __builtin_amdgcn_exp2f(fminf(half, 127.f)); }
template <bool BACK, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void scan_join_kernel(ScanArgs k) {
  __shared__ float l_end[WAVES][64], l_decay[WAVES][64];
  const seq_scan_args_t& a = k.a;
  const int N = a.states, D = (int)a.channels;
  const int dblocks = (D + 63) / 64;
  const int db = (int)blockIdx.x % dblocks, n = (int)blockIdx.x / dblocks % N, s = (int)blockIdx.x / dblocks / N;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int d = min(db * 64 + lane, D - 1);
  const bool on = db * 64 + lane < D;
  int first, len;
  if (k.m.offsets) {
    const int start = seq_start(k.m, s);
    first = (start >> k.m.shift) + s;
    len = max(seq_start(k.m, s + 1) - start, 0);
  } else {
    first = s * k.m.per;
    len = k.m.rows;
  }
  const int count = max(1, ((len - 1) >> k.m.shift) + 1);   // len 0: one piece
  const float half = 0.5f * decay_rate(a.A[(int64_t)d * N + n]);
  float h = 0.f;
  if (BACK) {
    if (k.last) h = k.last[((int64_t)s * D + d) * N + n];
  } else {
    const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, s);
    if (a.state && slot >= 0) h = a.state[slot * a.state_stride + (int64_t)d * N + n];
  }
  for (int j0 = 0; j0 < count; j0 += WAVES * kJoinEach) {
    const int mine = j0 + wave * kJoinEach;
    float e[kJoinEach], q[kJoinEach];   // end state, sum of D: zeros (which change nothing) where no piece follows
#pragma unroll
    for (int i = 0; i < kJoinEach; ++i) {
      const int j = mine + i;
      e[i] = q[i] = 0.f;
      if (j < count - 1) {
        const int64_t at = first + (BACK ? count - 1 - j : j);
        e[i] = k.carry[(at * N + n) * D + d];
        q[i] = k.sums[at * D + d];
      }
    }
    float end = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinEach; ++i) {
      sum += q[i];
      q[i] = half_decay(half * q[i]);
      end = __builtin_fmaf(q[i], q[i] * end, e[i]);
    }
    l_end[wave][lane] = end;
    l_decay[wave][lane] = half_decay(half * sum);
    __syncthreads();
    float c = h;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w == wave) c = h;
      h = __builtin_fmaf(l_decay[w][lane], l_decay[w][lane] * h, l_end[w][lane]);
    }
#pragma unroll
    for (int i = 0; i < kJoinEach; ++i) {
      const int j = mine + i;
      if (j < count && on) k.carry[((int64_t)(first + (BACK ? count - 1 - j : j)) * N + n) * D + d] = c;
      c = __builtin_fmaf(q[i], q[i] * c, e[i]);
    }
    __syncthreads();
  }
}

// One token of each sequence: NP / 4 lanes a channel with four states each, so that the states of a wave's channels
// are one contiguous read and write of 16 bytes a lane.  Bound by those bytes.
template <typename T, int NP, bool FULL>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs k) {
  constexpr int NG = NP / 4, kChannels = 256 / NG;
  const seq_scan_args_t& a = k.a;
  const int N = a.states, D = (int)a.channels;
  const int blocks = (D + kChannels - 1) / kChannels;
  const int s = (int)blockIdx.x / blocks;
  const int c = ((int)blockIdx.x % blocks) * kChannels + (int)threadIdx.x / NG;
  const int n0 = ((int)threadIdx.x % NG) * 4;
  const bool on = c < D;
  const int d = min(c, D - 1);
  const int g = d / (D / (int)a.groups);
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, s);
  const int nv = N - n0;   // states of this lane, <= 0: none
  Raw<float, 4> A, h;
  Raw<T, 4> B, C;
  A.clear();
  h.clear();
  B.clear();
  C.clear();
  if (FULL || nv > 0) {
    const int v = FULL ? 4 : nv;
    if (a.state && slot >= 0) h.load_n(a.state + slot * a.state_stride + (int64_t)d * N + n0, v);
    A.load_n(a.A + (int64_t)d * N + n0, v);
    B.load_n(static_cast<const T*>(a.B.ptr) + s * a.B.batch + g * a.B_group + n0, v);
    C.load_n(static_cast<const T*>(a.C.ptr) + s * a.C.batch + g * a.C_group + n0, v);
  }
  const float u = to_f32(static_cast<const T*>(a.u.ptr)[s * a.u.batch + d]);
  const float delta = to_f32(static_cast<const T*>(a.delta.ptr)[s * a.delta.batch + d]);
  const float dt = step_size(delta, a.delta_bias ? a.delta_bias[d] : 0.f, a.softplus);
  const float x = dt * u;
  float o = 0.f, out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] = 0.f;
    if (FULL || i < nv) {
      out[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(dt * decay_rate(A.get(i))), h.get(i), x * B.get(i));
      o = __builtin_fmaf(out[i], C.get(i), o);
    }
  }
  o = lanes_reduce<AddOp>(o, NG);
  if (!on) return;
  if (a.state_out && slot >= 0 && (FULL || nv > 0)) {
    h.pack(out);
    h.store_n(a.state_out + slot * a.state_out_stride + (int64_t)d * N + n0, FULL ? 4 : nv);
  }
  if (n0 == 0) {
    float y = __builtin_fmaf(a.skip ? a.skip[d] : 0.f, u, o);
    if (a.z.ptr) {
      const float zv = to_f32(static_cast<const T*>(a.z.ptr)[s * a.z.batch + d]);
      y *= zv * sigmoid(zv);
    }
    from_f32(y, static_cast<T*>(a.y.ptr)[s * a.y.batch + d]);
  }
}

int64_t scan_groups(int64_t pieces, const seq_scan_args_t& a) { return (pieces * scan_blocks(a) + kScanGroup - 1) / kScanGroup; }
unsigned scan_grid(const ScanArgs& k) { return (unsigned)scan_groups(k.pieces, k.a); }

template <typename T, int NP>
hipError_t scan_t(const ScanArgs& k, hipStream_t stream) {
  return launch_kernel(scan_kernel<T, NP>, dim3(scan_grid(k)), dim3(64 * kScanGroup), k, stream);
}

template <typename T, int NP>
hipError_t carry_t(const ScanArgs& k, bool back, hipStream_t stream) {
  const dim3 grid(scan_grid(k)), block(64 * kScanGroup);
  if (back) return launch_kernel(scan_carry_kernel<T, NP, true>, grid, block, k, stream);
  return launch_kernel(scan_carry_kernel<T, NP, false>, grid, block, k, stream);
}

// Workgroups of the single-token kernel, `lanes` lanes a channel.
int64_t step_grid(const seq_scan_args_t& a, int lanes) {
  return (a.channels * lanes + 255) / 256 * a.tokens.sequences;
}

template <typename T, int NP, bool FULL>
hipError_t step_t(const ScanArgs& k, hipStream_t stream) {
  return launch_kernel(scan_step_kernel<T, NP, FULL>, dim3((unsigned)step_grid(k.a, NP / 4)), dim3(256), k, stream);
}

hipError_t scan_any(const ScanArgs& k, hipStream_t stream) {
#define CALL(T, NP) scan_t<T, NP>(k, stream)
  SCAN_DISPATCH(CALL, k.a.dtype, k.a.states)
#undef CALL
}

hipError_t carry_any(const ScanArgs& k, bool back, hipStream_t stream) {
#define CALL(T, NP) carry_t<T, NP>(k, back, stream)
  SCAN_DISPATCH(CALL, k.a.dtype, k.a.states)
#undef CALL
}

}  // namespace

// Tokens of the longest sequence, as far as the host knows.
static int64_t scan_longest(const seq_scan_args_t& a) {
  return a.tokens.offsets && a.longest > 0 && a.longest < a.tokens.rows ? a.longest : a.tokens.rows;
}

static int64_t join_groups(const seq_scan_args_t& a) { return (a.channels + 63) / 64 * a.states * a.tokens.sequences; }

ScanCut scan_cut(const seq_scan_args_t& a) {
  const int64_t waves = scan_blocks(a), rows = seq_rows(a.tokens);
  const int64_t longest = scan_longest(a);
  int shift = kSaveShift;
  while (shift < kWholeShift && (rows >> shift) * waves > kScanWaves) ++shift;
  const int64_t piece = (int64_t)1 << shift;
  if (longest <= (piece > kScanWhole ? piece : kScanWhole)) return ScanCut{kWholeShift, false};
  // 2^24 sequences x channels / 64 x states: waves enough without a cut, and past what a launch of the join can hold.
  if (join_groups(a) > kMaxLanes / 256) return ScanCut{kWholeShift, false};
  return ScanCut{shift, true};
}

int64_t scan_save_floats(const seq_scan_args_t& a) {
  return seq_pieces(seq_map(a.tokens, kSaveShift)) * a.channels * a.states;
}

int64_t scan_ws_floats(const seq_scan_args_t& a) {
  const ScanCut cut = scan_cut(a);
  if (!cut.split) return 0;
  const int64_t pieces = seq_pieces(seq_map(a.tokens, cut.shift));
  return scan_round(pieces * a.channels * a.states) + scan_round(pieces * a.channels);
}

// One wave a workgroup: for sequences of up to 16 pieces, which are one wave's, and up to 32 where workgroups fill the GPU
// by themselves.  us with one and with four (16 states): 16 pieces, 240 workgroups 4.2 and 3.7, 480 4.4 and 4.7, 1024 5.1 and
// 6.3, 2048 7.3 and 10.5; 32 pieces, 768 8.2 and 6.8, 1152 8.2 and 7.7, 1536 8.6 and 9.1, 2048 9.2 and 10.1, but a whole
// training step of that size 450.0 and 449.3; packed, up to 29 pieces, 4608 12 and 17; 64 pieces, 1024 11.6 and 8.8.
static bool join_few(const seq_scan_args_t& a, int shift) {
  const int64_t pieces = ((scan_longest(a) - 1) >> shift) + 1;
  return pieces <= kJoinEach || (pieces <= 2 * kJoinEach && join_groups(a) > 2048);
}

// The join has fewer than kMaxLanes: scan_cut.
int64_t scan_lanes(const seq_scan_args_t& a) {
  return scan_groups(seq_pieces(seq_map(a.tokens, scan_cut(a).shift)), a) * 64 * kScanGroup;
}

int64_t scan_step_lanes(const seq_scan_args_t& a) {
  return step_grid(a, a.states <= 8 ? 2 : a.states <= 16 ? 4 : 8) * 256;
}

hipError_t launch_scan_carry(const ScanArgs& k, bool backward, hipStream_t stream) {
  const hipError_t err = carry_any(k, backward, stream);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)join_groups(k.a));
  const bool few = join_few(k.a, k.m.shift);
  if (backward)
    return few ? launch_kernel(scan_join_kernel<true, 1>, grid, dim3(64), k, stream)
               : launch_kernel(scan_join_kernel<true, 4>, grid, dim3(256), k, stream);
  return few ? launch_kernel(scan_join_kernel<false, 1>, grid, dim3(64), k, stream)
             : launch_kernel(scan_join_kernel<false, 4>, grid, dim3(256), k, stream);
}

hipError_t launch_scan(const seq_scan_args_t& a, float* ws, hipStream_t stream) {
  const ScanCut cut = scan_cut(a);
  ScanArgs k{};
  k.a = a;
  k.m = seq_map(a.tokens, cut.shift);
  k.pieces = (int32_t)seq_pieces(k.m);
  k.dblocks = scan_dblocks(a);
  k.split = cut.split;
  if (cut.split) {
    k.carry = ws;
    k.sums = ws + scan_round((int64_t)k.pieces * a.channels * a.states);
    const hipError_t err = launch_scan_carry(k, false, stream);
    if (err != hipSuccess) return err;
  }
  return scan_any(k, stream);
}

hipError_t launch_scan_step(const seq_scan_args_t& a, hipStream_t stream) {
  ScanArgs k{};
  k.a = a;
#define CALL(T, NP, FULL) step_t<T, NP, FULL>(k, stream)
  SCAN_DISPATCH4(CALL, a.dtype, a.states, true)
#undef CALL
}

}  // namespace cw
