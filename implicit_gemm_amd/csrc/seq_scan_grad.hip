// Gradients of the selective state space scan (gfx950).
//
// With do = dy z sigmoid(z) and the reversed recurrence  g[t] = do[t] C[t] + c[t],  c[t - 1] = e^(D[t] A) g[t]:
//   dC[t] = sum_d do h[t],  dB[t] = sum_d g D u,  du = skip do + D sum_n g B,
//   dD = sum_n A c[t - 1] h[t - 1] + u sum_n g B,  ddelta = dD sigmoid(delta + bias),  dA = sum_t D c[t - 1] h[t - 1]
// and dz from o = sum_n h C + skip u.  All of it needs the states again: the forward saved one state of every 16 tokens
// (4 bytes a token and channel for 16 states; scanning forward once more to find them would cost as much as the first
// of the three forward launches, 54 us where writing and reading them costs 10 and 14).
//
// Bound by the vector ALU.  A workgroup takes a piece of a sequence and 64 channels, 16 tokens at a time from the last:
// what a token and channel need (D, D u, do) is computed once by the lane that loads it and passed through LDS; then
// NG lanes share a channel, four states each, and keep h of the 16 tokens in 64 registers for the reversed sweep.
// Keeping all of e^(D A) too would save its second evaluation (3 of about 26 instructions a state) but 64 registers more
// leave one wave a SIMD.  With two, what one token reads of LDS is read a token ahead, and the 256 registers then hold
// e^(D A) of the last 8 tokens (8192 tokens x 2048 channels x 16 states in bf16: kept for no token 280 us, for 8 257,
// for 12 but read where needed 272).  Sums over states are taken inside a group of NG lanes, each of which keeps one of
// NG tokens' results; sums over channels by exchanging halves of the wave (each step halves the values a lane holds),
// then over the waves through LDS and over the channel blocks by a fold, all in a fixed order.  The vector ALU is busy
// 86 % of the kernel's 261 us.
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

// One step of a sum over lanes that shares its results out: of values a and b, lanes whose bit is clear get the sum of
// a over themselves and their partner, the others that of b; `from` brings the partner's value.
template <class From>
__device__ __forceinline__ float halve(bool bit, float a, float b, From from) {
  return (bit ? b : a) + from(bit ? a : b);
}

// Sums v[0 .. 7] over the lanes that differ in bits 3 .. 5; lane l gets value 4 b5 + 2 b4 + b3 of its bits.
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
  return halve(threadIdx.x & 8, r2[0], r2[1], [](float f) { return dpp<kXor8>(f); });
}

// The rest of that sum, over bits 2 (NG = 4) or 2 and 1 (NG = 2) that name channels too, shared out over 8 / NG tokens:
// lane l gets token bit 2 (+ 2 bit 1).
template <int NG>
__device__ __forceinline__ float tokens_reduce(const float (&r)[8 / NG]) {
  const bool b2 = threadIdx.x & 4;
  auto four = [](float f) { return xor4(f); };
  if constexpr (NG == 8) {
    return r[0];
  } else if constexpr (NG == 4) {
    return halve(b2, r[0], r[1], four);
  } else {
    const float lo = halve(b2, r[0], r[1], four), hi = halve(b2, r[2], r[3], four);
    return halve(threadIdx.x & 2, lo, hi, [](float f) { return dpp<kXor2>(f); });
  }
}

// The tensors whose rows a tile reads.
enum { kU, kDelta, kDy, kZ, kB, kC, kInputs };

// What the lanes of a workgroup pass each other of one tile.
template <int NG>
struct GradTile {
  alignas(16) float dt[kTile][64], x[kTile][64], dov[kTile][64];   // D, D u, do
  // Sums over states: h C, g B, A c[t - 1] h[t - 1].  NG lanes write NG rows of 64 / NG channels: no two in one bank.
  alignas(16) float o[kTile][64 + 64 / NG], gb[kTile][64 + 64 / NG], da[kTile][64 + 64 / NG];
  alignas(16) float B[kTile][4 * NG], C[kTile][4 * NG];
  float bias[64], skip[64];
  // Address of a piece's first row (the block's channels, the group's states) and bytes between two rows, per input: in
  // LDS, as six 64-bit products a tile would be a third of all instructions and six addresses too many scalar registers.
  uint64_t base[kInputs];
  uint32_t step[kInputs];
  float bc[NG][kTile][8 * NG];                                     // each wave's sums over its channels: dB, dC
};

// The kernel's arguments, to be loaded where they are used: held through the sweeps they need more scalar registers than
// there are, and the compiler would keep them in vector lanes, an instruction for each use.
typedef const __attribute__((address_space(4))) GradArgs* ArgsPtr;
__device__ __forceinline__ ArgsPtr args_again() {
  ArgsPtr p = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// V floats of a row of LDS, in as few accesses as there are.
template <int V>
__device__ __forceinline__ void put_row(float* to, const float (&v)[V]) {
  if constexpr (V == 2) {
    *reinterpret_cast<float2*>(to) = float2{v[0], v[1]};
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(to + i) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  }
}

// What a sweep reads of one token: D, D u, do of the lane's channel, B and C of its states.
template <int NG>
struct Token {
  float dt, x, dov;
  float4 B, C;
  __device__ __forceinline__ void read(const GradTile<NG>& m, int q, int ch, int ng) {
    dt = m.dt[q][ch];
    x = m.x[q][ch];
    dov = m.dov[q][ch];
    B = reinterpret_cast<const float4*>(&m.B[q][0])[ng];
    C = reinterpret_cast<const float4*>(&m.C[q][0])[ng];
  }
};

// FULL: every lane has a channel and four states (channels of a group a multiple of 64, states of 4 NG).
template <typename T, int NG, bool FULL>
__global__ __launch_bounds__(64 * NG, 2) void scan_grad_kernel(GradArgs k) {
  constexpr int NP = 4 * NG, kWaveCh = 64 / NG, V = 16 / NG, kShare = 8 / NG;
  constexpr int kHeld = NG == 2 ? 0 : sizeof(T) == 2 ? 8 : 4;   // tokens whose e^(D A) is kept, as registers allow
  constexpr bool kEarly = NG > 2;   // the next tile's inputs fit the registers (eight channels a lane do not)
  __shared__ GradTile<NG> m;
  const seq_scan_args_t& a = k.s.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int N = FULL ? NP : a.states, D = (int)a.channels, Dg = D / (int)a.groups;
  const int blocks = k.s.dblocks * (int)a.groups;
  const int part = (int)blockIdx.x / blocks, block = (int)blockIdx.x % blocks;
  const int g = block / k.s.dblocks, cblock = block % k.s.dblocks;
  const int nch = FULL ? 64 : min(64, Dg - cblock * 64);   // channels of the block
  const int d0 = g * Dg + cblock * 64;                     // the first
  // As a lane of the sweeps: one channel, four states.
  const int ch = wave * kWaveCh + lane / NG, ng = lane % NG, n0 = ng * 4, nv = N - n0;
  const bool on = FULL || ch < nch;
  const int chc = FULL ? ch : min(ch, nch - 1);
  // As a lane of the loads and outputs: one token, V channels; and one element of B and C.
  const int it = tid / (64 / V), ic = tid % (64 / V) * V, iv = nch - ic;   // iv <= 0: none
  const int eT = tid / NP, eN = tid % NP;
  const bool gated = a.z.ptr != nullptr, with_softplus = a.softplus != 0;

  float A2[4], dA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = FULL || i < nv ? decay_rate(a.A[(int64_t)(d0 + chc) * N + n0 + i]) : 0.f;
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
  const uint32_t bc_row = (uint32_t)a.groups * (uint32_t)N;

  for (int piece = part; piece < k.s.pieces; piece += k.parts) {
    Piece p;
    if (!find_piece(k.s.m, piece, p)) continue;
    const int tiles = (p.end - p.t0 + kTile - 1) / kTile;
    // Dense row of the piece's first token, and where this lane writes in it.
    const int64_t row0 = (k.s.m.offsets ? p.first : (int64_t)p.seq * k.s.m.rows) + p.t0;
    float* const bc0 = k.part_bc + (int64_t)cblock * 2 * bc + (row0 * a.groups + g) * N;
    if (p.seq >= k.s.m.S) {   // padding behind the last sequence
      for (int j = 0; j < tiles; ++j) {
        const int nt = min(kTile, p.end - p.t0 - j * kTile);
        if (it < nt && iv > 0) {
          Raw<T, V> zero;
          zero.clear();
          const int64_t at = (row0 + j * kTile + it) * D + d0 + ic;
          zero.store_n(static_cast<T*>(k.g.du) + at, iv);
          zero.store_n(static_cast<T*>(k.g.ddelta) + at, iv);
          if (gated) zero.store_n(static_cast<T*>(k.g.dz) + at, iv);
        }
        if (eT < nt && eN < N) {
          float* const to = bc0 + (int64_t)(j * kTile + eT) * bc_row + eN;
          to[0] = to[bc] = 0.f;
        }
      }
      continue;
    }
    if (tid < kInputs) {
      const seq_view_t& v = tid == kU ? a.u : tid == kDelta ? a.delta : tid == kDy ? k.s.dy : tid == kZ ? a.z : tid == kB ? a.B : a.C;
      const int64_t from = tid == kB ? g * a.B_group : tid == kC ? g * a.C_group : d0;
      m.base[tid] = reinterpret_cast<uint64_t>(row_at<const T>(v, p, p.t0) + from);
      m.step[tid] = (uint32_t)v.row * (uint32_t)sizeof(T);
    }
    __syncthreads();
    const int64_t tile0 = (k.s.m.offsets ? (p.first >> kSaveShift) + p.seq
                                         : (int64_t)p.seq * (((k.s.m.rows - 1) >> kSaveShift) + 1)) +
                          (p.t0 >> kSaveShift);
    const uint32_t state_off = (uint32_t)(n0 * D + chc);   // of this lane's first state in [states][channels]
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0.f;
      if (FULL || i < nv) {
        if (k.s.split) c[i] = (k.s.carry + (int64_t)piece * N * D + d0)[state_off + i * D];
        else if (k.s.last) c[i] = k.s.last[((int64_t)p.seq * D + d0 + chc) * N + n0 + i];
      }
    }
    Raw<T, V> u, dl, z, dy;
    float h0[4];
    T eB, eC;
    from_f32(0.f, eB);
    from_f32(0.f, eC);
    u.clear();
    dl.clear();
    z.clear();
    dy.clear();
    // Row `r` of tile j of an input, from element `e` on.
    auto row_of = [&](int input, int j, int r, int e) {
      return reinterpret_cast<const T*>(m.base[input] + (uint64_t)(uint32_t)(j * kTile + r) * m.step[input] +
                                        (uint32_t)e * (uint32_t)sizeof(T));
    };
    // This lane's token and channels of tile j; rows past the end repeat the last one.
    auto fetch_items = [&](int j, Raw<T, V>& u, Raw<T, V>& dl, Raw<T, V>& z, Raw<T, V>& dy) {
      const int r = min(it, min(kTile, p.end - p.t0 - j * kTile) - 1);
      if (FULL || iv > 0) {
        const int nvec = FULL ? V : iv;
        u.load_n(row_of(kU, j, r, ic), nvec);
        dl.load_n(row_of(kDelta, j, r, ic), nvec);
        dy.load_n(row_of(kDy, j, r, ic), nvec);
        if (gated) z.load_n(row_of(kZ, j, r, ic), nvec);
      }
    };
    // The inputs of tile j.
    auto fetch = [&](int j) {
      fetch_items(j, u, dl, z, dy);
      const int e = min(eT, min(kTile, p.end - p.t0 - j * kTile) - 1);
      if (FULL || eN < N) {
        eB = *row_of(kB, j, e, eN);
        eC = *row_of(kC, j, e, eN);
      }
      const ArgsPtr q = args_again();
      const float* const from = q->s.a.save + (tile0 + j) * D * N + d0;
#pragma unroll
      for (int i = 0; i < 4; ++i) h0[i] = FULL || i < nv ? from[state_off + i * D] : 0.f;
    };
    if (kEarly && tiles) fetch(tiles - 1);
    for (int j = tiles - 1; j >= 0; --j) {
      if constexpr (!kEarly) fetch(j);
      yield_by_progress(tiles - 1 - j, tiles);   // 273 us without, 267 with
      const int nt = min(kTile, p.end - p.t0 - j * kTile);
      // What the sweeps need of this lane's own token and channels; its raw inputs are kept for its outputs (eight
      // channels a lane do not fit the registers: read again).  Tokens past the piece's end pass state and gradient on
      // unchanged.
      Raw<T, V> cu = u, cdl = dl, cz = z, cdy = dy;
      const bool valid = it < nt;
      float pdt[V], pdo[V];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        pdt[q] = cdl.get(q) + m.bias[ic + q];
        pdo[q] = cdy.get(q);
      }
      if (with_softplus) {
#pragma unroll
        for (int q = 0; q < V; ++q) pdt[q] = softplus(pdt[q]);
      }
      if (gated) {
#pragma unroll
        for (int q = 0; q < V; ++q) pdo[q] *= cz.get(q) * sigmoid(cz.get(q));
      }
      float px[V];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        pdt[q] = valid ? pdt[q] : 0.f;
        px[q] = valid ? pdt[q] * cu.get(q) : 0.f;
        pdo[q] = valid ? pdo[q] : 0.f;
      }
      put_row(&m.dt[it][ic], pdt);
      put_row(&m.x[it][ic], px);
      put_row(&m.dov[it][ic], pdo);
      m.B[eT][eN] = to_f32(eB);
      m.C[eT][eN] = to_f32(eC);
      float hs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) hs[i] = h0[i];
      __syncthreads();
      if (kEarly && j > 0) fetch(j - 1);

      float h[kTile][4], held[kHeld > 0 ? kHeld : 1][4];
      float keep = 0.f;
      Token<NG> ahead;
      ahead.read(m, 0, ch, ng);
#pragma unroll
      for (int q = 0; q < kTile; ++q) {
        const Token<NG> now = ahead;
        if (q + 1 < kTile) ahead.read(m, q + 1, ch, ng);
        const float dt = now.dt, x = now.x;
        const float B4[4] = {now.B.x, now.B.y, now.B.z, now.B.w}, C4[4] = {now.C.x, now.C.y, now.C.z, now.C.w};
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(dt * A2[i]);
          if (q >= kTile - kHeld) held[q >= kTile - kHeld ? q - (kTile - kHeld) : 0][i] = e;
          h[q][i] = __builtin_fmaf(e, q ? h[q ? q - 1 : 0][i] : hs[i], x * B4[i]);
          o = __builtin_fmaf(h[q][i], C4[i], o);
        }
        o = lanes_reduce<AddOp>(o, NG);
        keep = ng == q % NG ? o : keep;
        if (q % NG == NG - 1) m.o[q - (NG - 1) + ng][ch] = keep;
        __builtin_amdgcn_sched_barrier(0);
      }
      // Read B, C, D and D u again: kept from the sweep above they would take 160 registers more.  The compiler is
      // not to know that these are the same indices.
      int ch2 = ch, ng2 = ng;
      asm volatile("" : "+v"(ch2), "+v"(ng2));
      float keep_gb = 0.f, keep_da = 0.f, sums[kShare];
      Token<NG> before;
      before.read(m, kTile - 1, ch2, ng2);
#pragma unroll
      for (int q = kTile - 1; q >= 0; --q) {
        const Token<NG> now = before;
        if (q > 0) before.read(m, q - 1, ch2, ng2);
        const float dt = now.dt, x = now.x, dov = now.dov;
        const float B4[4] = {now.B.x, now.B.y, now.B.z, now.B.w}, C4[4] = {now.C.x, now.C.y, now.C.z, now.C.w};
        float gb = 0.f, da = 0.f, v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gi = __builtin_fmaf(dov, C4[i], c[i]);
          v[i] = gi * x;                // lanes without a channel: x and do are zero
          v[4 + i] = dov * h[q][i];
          gb = __builtin_fmaf(gi, B4[i], gb);
          const float e = q >= kTile - kHeld ? held[q >= kTile - kHeld ? q - (kTile - kHeld) : 0][i]
                                             : __builtin_amdgcn_exp2f(dt * A2[i]);
          c[i] = e * gi;
          const float r = c[i] * (q ? h[q ? q - 1 : 0][i] : hs[i]);
          da = __builtin_fmaf(r, A2[i], da);
          dA[i] = __builtin_fmaf(r, dt, dA[i]);
        }
        gb = lanes_reduce<AddOp>(gb, NG);
        da = lanes_reduce<AddOp>(da, NG);
        keep_gb = ng == q % NG ? gb : keep_gb;
        keep_da = ng == q % NG ? da : keep_da;
        if (q % NG == 0) {
          m.gb[q + ng][ch2] = keep_gb;
          m.da[q + ng][ch2] = keep_da * kLn2;   // A2 = A log2 e
        }
        sums[q % kShare] = channels_reduce(v);
        if (q % kShare == 0) {
          const int to = NG == 8 ? 0 : NG == 4 ? (lane >> 2) & 1 : ((lane >> 2) & 1) + (lane & 2);
          m.bc[wave][q + to][(lane >> 5) * NP + n0 + ((lane >> 3) & 3)] = tokens_reduce<NG>(sums);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      if constexpr (NG == 2) fetch_items(j, cu, cdl, cz, cdy);
      if (valid && (FULL || iv > 0)) {
        const ArgsPtr w = args_again();
        float du[V], dd[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const float dov = m.dov[it][ic + q], dt = m.dt[it][ic + q], gb = m.gb[it][ic + q], uv = cu.get(q);
          du[q] = __builtin_fmaf(dt, gb, m.skip[ic + q] * dov);
          dd[q] = __builtin_fmaf(uv, gb, m.da[it][ic + q]);
          dskip[q] = __builtin_fmaf(dov, uv, dskip[q]);
        }
        if (with_softplus) {
#pragma unroll
          for (int q = 0; q < V; ++q) dd[q] *= sigmoid(cdl.get(q) + m.bias[ic + q]);
        }
#pragma unroll
        for (int q = 0; q < V; ++q) dbias[q] += dd[q];
        const int64_t at = (row0 + j * kTile) * D + d0;
        const uint32_t off = (uint32_t)(it * D + ic);
        const int nvec = FULL ? V : iv;
        Raw<T, V> r;
        r.pack(du);
        r.store_n(static_cast<T*>(w->g.du) + at + off, nvec);
        r.pack(dd);
        r.store_n(static_cast<T*>(w->g.ddelta) + at + off, nvec);
        if (gated) {
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const float zv = cz.get(q), sg = sigmoid(zv);
            du[q] = cdy.get(q) * __builtin_fmaf(m.skip[ic + q], cu.get(q), m.o[it][ic + q]) *
                    (sg * __builtin_fmaf(zv, 1.f - sg, 1.f));
          }
          r.pack(du);
          r.store_n(static_cast<T*>(w->g.dz) + at + off, nvec);
        }
      }
      // dB and dC of the block's channels: one state of one token a lane, the waves in order.
      if (eT < nt && (FULL || eN < N)) {
        float* const to = bc0 + (int64_t)j * kTile * bc_row + (uint32_t)eT * bc_row + eN;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float r = m.bc[0][eT][i * NP + eN];
#pragma unroll
          for (int w = 1; w < NG; ++w) r += m.bc[w][eT][i * NP + eN];
          to[i * bc] = r;
        }
      }
      __syncthreads();
    }
    if (p.t0 == 0 && k.g.dstate && on) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (FULL || i < nv) k.g.dstate[((int64_t)p.seq * D + d0 + ch) * N + n0 + i] = c[i];
    }
  }
  if (on) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (FULL || i < nv) k.part_a[(int64_t)part * D * N + (int64_t)(d0 + ch) * N + n0 + i] = dA[i];
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
  const bool whole = k.s.a.channels / k.s.a.groups % 64 == 0;
  SCAN_DISPATCH4(CALL, k.s.a.dtype, k.s.a.states, whole)
#undef CALL
}

// Workgroups along the pieces: one a piece, but no more than give about 2048 workgroups (each has a partial of dA).
int32_t grad_parts(const seq_scan_args_t& a, int64_t pieces) {
  const int64_t blocks = (int64_t)scan_dblocks(a) * a.groups;
  int64_t most = 2048 / blocks;
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

// The sums over channel blocks and workgroups, from the partial results.
FoldList grad_folds(const seq_scan_grad_args_t& g, const GradSpace& w, const float* ws) {
  const seq_scan_args_t& a = g.fwd;
  const int64_t D = a.channels, bc = seq_rows(a.tokens) * a.groups * a.states;
  const float *part_bc = ws + w.bc, *part_a = ws + w.a, *part_s = ws + w.s;
  FoldList l;
  l.n = 0;
  l.f[l.n++] = FoldPart{part_bc, 2 * bc, scan_dblocks(a), bc, g.dB, a.dtype};
  l.f[l.n++] = FoldPart{part_bc + bc, 2 * bc, scan_dblocks(a), bc, g.dC, a.dtype};
  l.f[l.n++] = FoldPart{part_a, D * a.states, w.parts, D * a.states, g.dA, CONV_WGRAD_F32};
  if (g.dskip) l.f[l.n++] = FoldPart{part_s, 2 * D, w.parts, D, g.dskip, CONV_WGRAD_F32};
  if (g.ddelta_bias) l.f[l.n++] = FoldPart{part_s + D, 2 * D, w.parts, D, g.ddelta_bias, CONV_WGRAD_F32};
  return l;
}

}  // namespace

int64_t scan_grad_lanes(const seq_scan_grad_args_t& g) {
  const GradSpace w = grad_space(g.fwd);
  const int64_t n = g.fwd.states, lanes = 64 * (n <= 8 ? 2 : n <= 16 ? 4 : 8);
  const int64_t sweep = w.parts * scan_blocks(g.fwd) * lanes, fold = fold_lanes(grad_folds(g, w, nullptr));
  const int64_t before = scan_lanes(g.fwd);   // aggregates and join of the same cut
  return sweep > fold ? sweep > before ? sweep : before : fold > before ? fold : before;
}

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
  return launch_seq_fold(grad_folds(g, w, ws), stream);
}

}  // namespace cw
