// The gated delta rule forward (gfx950): the triangular systems of all chunks, the chunks of each sequence in order, and
// the single token.  seq_delta.h has the formulas.
#include "seq_delta.h"

namespace cw {

namespace {

// ---- the chunks' systems ----------------------------------------------------------------------------------------------
// Bound by HBM and the write path where there are many chunks (8192 tokens of 32 heads of 128 in bf16: 151 MB read and 153
// written in 62 us, 4.9 TB/s; what is written are the systems, which the walk's slices of columns, eight there, then share).
// One workgroup a chunk and head.  Wave r multiplies rows 16 r .. of K and Q with K of the tiles before it; (1 + M)^-1
// comes from its 16 x 16 diagonal blocks, each solved row by row by one wave, doubled twice: the block below the diagonal
// of [[A, 0], [C, B]]^-1 is -B^-1 C A^-1, in 32-bit matrix products.
constexpr int kSquarePitch = kChunk + 4;   // floats of an LDS row

__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// acc += the 16 x 16 block of a at (ar, ac) times the one of b at (br, bc).
__device__ __forceinline__ f32x4 block_product(const float (*a)[kSquarePitch], int ar, int ac, const float (*b)[kSquarePitch],
                                               int br, int bc, int lane, f32x4 acc) {
  const int lr = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = mfma32(a[ar + lr][ac + 4 * s + lg], b[br + 4 * s + lg][bc + lr], acc);
  return acc;
}
__device__ __forceinline__ void block_store(float (*c)[kSquarePitch], int r, int col, int lane, f32x4 v, float sign) {
#pragma unroll
  for (int x = 0; x < 4; ++x) c[r + 4 * (lane >> 4) + x][col + (lane & 15)] = sign * v[x];
}

constexpr int kPanel = 128;                // dimensions of K and Q that are staged at a time

template <typename T>
union ChunkLds {
  static constexpr int kPitch = kPanel + 16 / (int)sizeof(T);
  struct Panel {
    T key[kChunk][kPitch], query[kChunk][kPitch];
  } panel;
  struct Squares {
    float M[kChunk][kSquarePitch], I[kChunk][kSquarePitch];
  } squares;
};

// EIGHTS: Dk is a multiple of 8, so that no load has a branch (the long prompt, with the walk's WHOLE for Dk = KP: 302 us
// in a captured graph against 344 without both).
template <typename T, bool GRAD, bool EIGHTS>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) void delta_chunk_kernel(DeltaArgs k) {
  constexpr int N = ElemPieces<T>::n;
  __shared__ __attribute__((aligned(16))) char bytes[sizeof(ChunkLds<T>)];
  __shared__ ChunkDecay d;
  ChunkLds<T>& L = *reinterpret_cast<ChunkLds<T>*>(bytes);
  auto& M = L.squares.M;
  auto& I = L.squares.I;
  const seq_delta_args_t& a = k.a;
  const int tid = threadIdx.x, lane = tid & 63, r = uniform(tid >> 6), lr = lane & 15, lg = lane >> 4;
  const int heads = (int)a.heads, piece = blockIdx.x / heads, head = blockIdx.x % heads;
  Piece p;
  if (!find_piece(k.m, piece, p)) return;
  const int n = p.end - p.t0, Dk = a.key_dim;
  if (p.seq == k.m.S) {            // padding behind the last sequence
    if constexpr (!GRAD) {
      const int Dv = a.value_dim;
      for (int i = tid; i < n * Dv; i += 256)
        from_f32(0.f, row_at<T>(a.o, p, p.t0 + i / Dv)[(int64_t)head * Dv + i % Dv]);
    }
    return;
  }
  if (n <= 0) return;                // an empty sequence has a number too
  const int64_t at = chunk_head(k, piece, head);
  const int64_t kh = head / (heads / (int)a.key_heads);
  const ChunkRows<const T> key(a.k, kh * a.k_head, p, p.t0), query(a.q, kh * a.q_head, p, p.t0);
  f32x4 kk[4], qk[4];
  clear(kk);
  clear(qk);
  for (int c0 = 0; c0 < Dk; c0 += kPanel) {
    // 64 rows of 16 groups of 8 dimensions, four groups a lane.  Rows past the chunk's end read its last one: what they
    // give is thrown away below.
    Eight<T> ek[4], eq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = min(tid / 16 + 16 * i, n - 1), c = c0 + 8 * (tid & 15);
      if constexpr (EIGHTS) {
        ek[i].raw.load(&key.at(row, c < Dk ? c : 0));
        eq[i].raw.load(&query.at(row, c < Dk ? c : 0));
      } else {
        ek[i].load(&key.at(row, c), Dk - c);
        eq[i].load(&query.at(row, c), Dk - c);
      }
    }
    if (c0 == 0 && r == 0) {
      chunk_decay(a, p, head, lane, d);
      k.decay[at * 2 * kChunk + lane] = d.first[lane];
      k.decay[(at * 2 + 1) * kChunk + lane] = d.last[lane] * d.beta[lane];
    }
    if (c0) __syncthreads();         // the last panel's reads are done
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = tid / 16 + 16 * i, c = 8 * (tid & 15);
      if (EIGHTS && c0 + c >= Dk) {
        ek[i].raw.clear();
        eq[i].raw.clear();
      }
      ek[i].put(&L.panel.key[row][c]);
      eq[i].put(&L.panel.query[row][c]);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kPanel / 32; ++c)
      if (c0 + 32 * c < Dk) {
        Eight<T> e;
        s16x8 ka[N], qa[N];
        e.raw.load(&L.panel.key[16 * r + lr][32 * c + 8 * lg]);
        e.pieces(ka);
        e.raw.load(&L.panel.query[16 * r + lr][32 * c + 8 * lg]);
        e.pieces(qa);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (t <= r) {
            s16x8 kb[N];
            e.raw.load(&L.panel.key[16 * t + lr][32 * c + 8 * lg]);
            e.pieces(kb);
            mfma_pieces<kPieces>(ka, kb, kk[t]);
            mfma_pieces<kPieces>(qa, kb, qk[t]);
          }
      }
  }
  __syncthreads();
  {
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&d.hi[16 * r + 4 * lg]), lo = *reinterpret_cast<const f32x4*>(&d.lo[16 * r + 4 * lg]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t > r) continue;
      const int j = 16 * t + lr;
      const float hj = d.hi[j], lj = d.lo[j], beta = d.beta[j], scaled = a.scale * beta;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 16 * r + 4 * lg + x;
        const bool live = i < n && j <= i;
        const float e = exp_of(hi[x] - hj, lo[x] - lj);
        M[i][j] = live && j < i ? e * beta * kk[t][x] : 0.f;
        qk[t][x] = live ? e * scaled * qk[t][x] : 0.f;
      }
    }
    // The blocks beside the diagonal's that share an operand block with it.
    if ((r & 1) == 0) block_store(I, 16 * r, 16 * r + 16, lane, zero4(), 1.f);
  }
  wave_sync();                       // a diagonal block is read by the wave that wrote it
  {
    float x[16];                     // column lr of the inverse of block r; the four groups of lanes do the same
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i == lr ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < i) x[i] = __builtin_fmaf(-M[16 * r + i][16 * r + j], x[j], x[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & 3) == lg) I[16 * r + i][16 * r + lr] = x[i];
  }
  __syncthreads();
  // Y = C A^-1 goes through the block of M above the diagonal, which is zero and not read.
  if ((r & 1) == 0) block_store(M, 16 * r, 16 * r + 16, lane, block_product(M, 16 * r + 16, 16 * r, I, 16 * r, 16 * r, lane, zero4()), 1.f);
  __syncthreads();
  if ((r & 1) == 0)
    block_store(I, 16 * r + 16, 16 * r, lane, block_product(I, 16 * r + 16, 16 * r + 16, M, 16 * r, 16 * r + 16, lane, zero4()), -1.f);
  __syncthreads();
  {
    const int u = 16 * (r >> 1), v = 16 * (r & 1);
    f32x4 y = zero4();
    if (v == 0) y = block_product(M, 32 + u, 0, I, 0, 0, lane, y);
    y = block_product(M, 32 + u, 16, I, 16, v, lane, y);
    block_store(M, u, 32 + v, lane, y, 1.f);
    __syncthreads();
    f32x4 z = block_product(I, 32 + u, 32, M, 0, 32 + v, lane, zero4());
    if (u == 16) z = block_product(I, 48, 48, M, 16, 32 + v, lane, z);
    block_store(I, 32 + u, v, lane, z, -1.f);
  }
  __syncthreads();
  // M has served: P takes its place.
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (t <= (r | 1)) block_store(M, 16 * r, 16 * t, lane, qk[t], 1.f);      // zero past the diagonal
  if (GRAD) __syncthreads();         // columns are read, of all waves' rows
  else wave_sync();
  const int row = 16 * r + lr;
  uint16_t* inv = k.inverse + at * kMatrix;
  uint16_t* inn = k.inner + at * kMatrix;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (GRAD ? s < r / 2 : s > r / 2) continue;
    const int b = GRAD ? upper_frag(r, s) : lower_frag(r, s);
    float fi[8], fp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 32 * s + 8 * lg + i;
      fi[i] = GRAD ? I[c][row] : I[row][c];
      fp[i] = GRAD ? M[c][row] : M[row][c];
    }
    s16x8 pi[kPieces], pp[kPieces];
    split8<kPieces>(fi, pi);
    split8<kPieces>(fp, pp);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      *reinterpret_cast<s16x8*>(&at_lane(inv + (b * kPieces + i) * kFragElems, lane * 8)) = pi[i];
      *reinterpret_cast<s16x8*>(&at_lane(inn + (b * kPieces + i) * kFragElems, lane * 8)) = pp[i];
    }
  }
}

// ---- the chunks of a sequence in order ------------------------------------------------------------------------------
// Bound by the chain's latency: a chunk is three products that wait for each other, each behind an exchange through LDS.
// 8192 tokens of 32 heads of 128 x 128 in bf16 are 128 chunks in 265 us (2.1 us a chunk; the chain alone 1.4, with its loads
// 1.65), with one workgroup a CU, the vector ALU 26 %, LDS 29 % and the matrix units 19 % busy.  So the chain has waves of
// its own, nothing that waits for memory between two exchanges, and operands in LDS in the order that a wave reads them.
// Outputs take all three pieces of S, P and Z (two, 16 bits, took 246 us and left 0.3 % of bf16 and 1.9 % of fp16 outputs a
// step off).  Measured and slower: the state only in registers with partial sums of K S exchanged (315 against 262 us then),
// 32 columns a workgroup (spills), Q S after the first exchange (half of it 275 us against 274, all 288).  4 x 2048 tokens of
// 16 heads, two workgroups a CU: 120 us, and 172 with the 240 MB that the gradient needs (kept by columns in 16-byte stores:
// no change).
//
// A workgroup has 16 NT columns of one sequence's and head's state.  Waves 0 .. 3 walk the chain: wave r has the
// chunk's tokens 16 r .. and the state's rows r KP / 4 .., in registers; the state's pieces go to all waves through LDS.
// Waves 4 .. 7 make the outputs of the same tokens beside them.  Three exchanges a chunk: the state, X, and Z; global
// loads are one chunk ahead.
template <typename T, int KP, int NT>
struct WalkLds {
  static constexpr int N = ElemPieces<T>::n;
  Operand<KP> S[kPieces][NT];
  Operand<kChunk> X[kPieces][NT], W[kPieces][NT], Z[kPieces][NT];
  Staged<T, KP> K;
};
template <typename T, int KP, int NT, bool SAVE, bool WHOLE>
__device__ __forceinline__ void walk_chain(const DeltaArgs& k, const Walk& w, WalkLds<T, KP, NT>& L, int r, int lane) {
  typedef WalkLds<T, KP, NT> Lds;
  constexpr int N = Lds::N, KS = KP / 32, MT = KP / 64;
  const seq_delta_args_t& a = k.a;
  const int lr = lane & 15, lg = lane >> 4, heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, w.seq);
  const int64_t place = (int64_t)w.head * Dk * Dv;
  f32x4 S[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = w.col0 + 16 * t + lr;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 16 * (r * MT + m) + 4 * lg + x;
        S[m][t][x] = a.state && slot >= 0 && (WHOLE || row < Dk) && c < Dv
                         ? at_lane(a.state + slot * a.state_stride + place, row * Dv + c) : 0.f;
      }
    }
  auto share_state = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        u32x2 u[kPieces];
        split4<kPieces>(S[m][t], u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) L.S[i][t].four(16 * (r * MT + m) + 4 * lg, lr) = u[i];
      }
  };
  auto keep_state = [&](float* to) __attribute__((always_inline)) {
    const int row0 = opaque(16 * MT * r + 4 * lg);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = w.col0 + 16 * t + lr;
      if (c < Dv) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (WHOLE || row0 + 16 * m + x < Dk) at_lane(to, (row0 + 16 * m + x) * Dv + c) = S[m][t][x];
      }
    }
  };
  Eight<T> rows[KS];
  T v[NT][4];
  s16x8 square[2][kPieces];
  float4 first, last;
  float whole;
  auto keys = [&](int j) __attribute__((always_inline)) {
    return ChunkRows<const T>(a.k, w.key_head * a.k_head, w.p, kChunk * j);
  };
  auto load_rows = [&](int j) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < KS; ++c) load_row<T, KP, WHOLE>(keys(j), w.p.len - kChunk * j, 16 * r + lr, lg, Dk, c, rows[c]);
  };
  auto load_values = [&](int j) __attribute__((always_inline)) {
    const int n = w.p.len - kChunk * j;
    const ChunkRows<const T> from(a.v, w.head * a.v_head, w.p, kChunk * j);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int t = 0; t < NT; ++t) v[t][x] = from.at(min(16 * r + 4 * lg + x, n - 1), min(w.col0 + 16 * t + lr, Dv - 1));
  };
  auto load_square = [&](int j) __attribute__((always_inline)) {
    const uint16_t* from = k.inverse + (w.number + (int64_t)j * heads) * kMatrix;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        square[c][i] = *reinterpret_cast<const s16x8*>(&at_lane(from + (lower_frag(r, min(c, r / 2)) * kPieces + i) * kFragElems, lane * 8));
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    const float* from = k.decay + (w.number + (int64_t)j * heads) * 2 * kChunk;
    first = *reinterpret_cast<const float4*>(from + 16 * r + 4 * lg);
    last = *reinterpret_cast<const float4*>(from + kChunk + 16 * r + 4 * lg);
    whole = from[kChunk - 1];
  };
  if (w.chunks > 0) {
    load_rows(0);
    load_values(0);
    load_decay(0);
    load_square(0);
  }
  share_state();
  lds_barrier();
#pragma unroll 1
  for (int j = 0; j < w.chunks; ++j) {
    const int n = w.p.len - kChunk * j;      // tokens that are left
    const int next = min(j + 1, w.chunks - 1);
    const float f[4] = {first.x, first.y, first.z, first.w}, l[4] = {last.x, last.y, last.z, last.w};
    const float keep = whole;
    if (SAVE) keep_state(k.states + (w.number + (int64_t)j * heads) * Dk * Dv);
    // X = V - e^G (K S)
    {
      f32x4 sum[NT][kPieces];
#pragma unroll
      for (int t = 0; t < NT; ++t) clear(sum[t]);
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        s16x8 e[N];
        rows[c].pieces(e);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.S[i][t].eight(c, lane);
          mfma_pieces<kPieces>(e, b, sum[t]);
        }
        if (c & 1) __builtin_amdgcn_sched_barrier(0);     // two blocks' operands in registers at a time
      }
#pragma unroll
      for (int c = 0; c < KS; ++c) rows[c].put(&L.K.at[16 * r + lr][32 * c + 8 * lg]);
      load_rows(next);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4 kS = total(sum[t]);
        f32x4 x;
        u32x2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d = __builtin_fmaf(-f[i], kS[i], to_f32(v[t][i]));
          x[i] = 16 * r + 4 * lg + i < n && w.col0 + 16 * t + lr < Dv ? d : 0.f;
        }
        split4<kPieces>(x, u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) L.X[i][t].four(16 * r + 4 * lg, lr) = u[i];
      }
    }
    load_values(next);
    lds_barrier();
    // Z = (1 + M)^-1 X
    f32x4 z[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 sum[kPieces];
      clear(sum);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c <= r / 2) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.X[i][t].eight(c, lane);
          mfma_pieces<kPieces>(square[c], b, sum);
        }
      z[t] = total(sum);
      u32x2 u[kPieces];
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = l[i] * z[t][i];
      split4<kPieces>(x, u);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) L.W[i][t].four(16 * r + 4 * lg, lr) = u[i];
      split4<kPieces>(z[t], u);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) L.Z[i][t].four(16 * r + 4 * lg, lr) = u[i];
    }
    lds_barrier();
    if (SAVE) {
      float* to = k.errors + ((w.p.batch * k.m.rows + w.p.first + kChunk * j) * heads + w.head) * Dv + w.col0;
#pragma unroll
      for (int c = 0; c < NT; ++c)
        if (w.col0 + 16 * c + lr < Dv) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = opaque(16 * r + 4 * lg) + i;
            if (t < n) at_lane(to, t * heads * Dv + 16 * c + lr) = z[c][i];
          }
        }
    }
    load_decay(next);
    if (N == 1) load_square(next);
    // S' = e^G_C S + K^T W
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f32x4 sum[NT][kPieces];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        clear(sum[t]);
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[t][0][x] = keep * S[m][t][x];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s16x8 e[N];
        L.K.transposed(r * MT + m, c, lane, e);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.W[i][t].eight(c, lane);
          mfma_pieces<kPieces>(e, b, sum[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) S[m][t] = total(sum[t]);
    }
    if (N > 1) {                             // fp32 and fp16 K take their pieces' registers: only now are enough free
      __builtin_amdgcn_sched_barrier(0);
      load_square(next);
    }
    share_state();
    lds_barrier();
  }
  if (a.state_out && slot >= 0) keep_state(a.state_out + slot * a.state_out_stride + place);
}

template <typename T, int KP, int NT, bool WHOLE>
__device__ __forceinline__ void walk_outputs(const DeltaArgs& k, const Walk& w, WalkLds<T, KP, NT>& L, int r, int lane) {
  typedef WalkLds<T, KP, NT> Lds;
  constexpr int N = Lds::N, KS = KP / 32;
  const seq_delta_args_t& a = k.a;
  const int lr = lane & 15, lg = lane >> 4, heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  Eight<T> rows[KS];
  s16x8 square[2][kPieces];
  float4 first;
  auto queries = [&](int j) __attribute__((always_inline)) {
    return ChunkRows<const T>(a.q, w.key_head * a.q_head, w.p, kChunk * j);
  };
  auto load_rows = [&](int j) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < KS; ++c) load_row<T, KP, WHOLE>(queries(j), w.p.len - kChunk * j, 16 * r + lr, lg, Dk, c, rows[c]);
  };
  auto load_square = [&](int j) __attribute__((always_inline)) {
    const uint16_t* from = k.inner + (w.number + (int64_t)j * heads) * kMatrix;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        square[c][i] = *reinterpret_cast<const s16x8*>(&at_lane(from + (lower_frag(r, min(c, r / 2)) * kPieces + i) * kFragElems, lane * 8));
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    first = *reinterpret_cast<const float4*>(k.decay + (w.number + (int64_t)j * heads) * 2 * kChunk + 16 * r + 4 * lg);
  };
  if (w.chunks > 0) {
    load_rows(0);
    load_decay(0);
    load_square(0);
  }
  lds_barrier();
#pragma unroll 1
  for (int j = 0; j < w.chunks; ++j) {
    const int n = w.p.len - kChunk * j;
    const int next = min(j + 1, w.chunks - 1);
    f32x4 o[NT][kPieces];
#pragma unroll
    for (int t = 0; t < NT; ++t) clear(o[t]);
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      s16x8 e[N];
      rows[c].pieces(e);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s16x8 b[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) b[i] = L.S[i][t].eight(c, lane);
        mfma_pieces<kPieces>(e, b, o[t]);
      }
    }
    lds_barrier();
    const float f[4] = {first.x, first.y, first.z, first.w};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 qS = total(o[t]);
      clear(o[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][0][i] = a.scale * f[i] * qS[i];
    }
    load_rows(next);
    load_decay(next);
    lds_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c <= r / 2) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.Z[i][t].eight(c, lane);
          mfma_pieces<kPieces>(square[c], b, o[t]);
        }
    load_square(next);
    const ChunkRows<T> out(a.o, (int64_t)w.head * Dv, w.p, kChunk * j);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 v = total(o[t]);
      const int col = w.col0 + 16 * t + lr;
      if (col < Dv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * r + 4 * lg + i;
          if (row < n) from_f32(v[i], out.at(row, col));
        }
      }
    }
    lds_barrier();
  }
}

// Four waves a SIMD, that is two workgroups a CU, wherever they fit without spills: fp16 keys of 65 .. 127 dimensions would
// take 129 registers when they save (4 x 2048 tokens of 16 heads of 100 x 100, a saving call in a captured graph: 242 us
// against 307; of one sequence of 8192, which leaves CUs empty, 552 against 526; the others have at most 128 by themselves,
// or, fp32 over 64 and all over 128 dimensions, far more).
template <class Lds, int KP>
constexpr int walk_waves() { return KP <= 128 && KP * Lds::N <= 256 ? 4 : 2; }

template <typename T, int KP, int NT, bool SAVE, bool WHOLE>
__global__ __launch_bounds__(512, (walk_waves<WalkLds<T, KP, NT>, KP>())) void delta_kernel(DeltaArgs k) {
  typedef WalkLds<T, KP, NT> Lds;
  __shared__ __attribute__((aligned(16))) char bytes[sizeof(Lds)];
  Lds& L = *reinterpret_cast<Lds*>(bytes);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  Walk w;
  if (!find_walk<16 * NT>(k, w)) return;
  if (wave < 4) walk_chain<T, KP, NT, SAVE, WHOLE>(k, w, L, wave, lane);
  else walk_outputs<T, KP, NT, WHOLE>(k, w, L, wave - 4, lane);
}

// ---- one token ----------------------------------------------------------------------------------------------------------
// A workgroup has one sequence's head and up to 4 LANES columns of its state, four to a lane; its 256 lanes are groups of
// LANES that share the state's rows.  The state is read once, held in registers between the two sums over its rows, and
// written once: bound by HBM.
//
// States stream past the caches (64 sequences of 32 heads of 128 x 128, 268 MB a call, four sets in turn: 51.4 us against
// 59.7 with ordinary loads and stores, a copy of the same size 49.9; 8 sequences of 16 heads 6.7 against 7.6): the next
// token comes when the model's other layers have gone through the caches.  WHOLE: Dv is a multiple of 4, so that a lane
// has all of its columns or none (without the branches for that 70.7 us became 59.7).
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void stream_in(Raw<float, 4>& r, const float* p) {
  const f32x4_u v = __builtin_nontemporal_load(reinterpret_cast<const f32x4_u*>(p));
  const float f[4] = {v[0], v[1], v[2], v[3]};
  r.pack(f);
}
__device__ __forceinline__ void stream_out(const Raw<float, 4>& r, float* p) {
  __builtin_nontemporal_store(f32x4_u{r.get(0), r.get(1), r.get(2), r.get(3)}, reinterpret_cast<f32x4_u*>(p));
}

template <typename T, int LANES, int ROWS, bool WHOLE>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs k) {
  constexpr int kGroups = 256 / LANES;
  __shared__ float sums[kGroups][LANES * 4 + 1];
  __shared__ float key[256], query[256];
  const seq_delta_args_t& a = k.a;
  const int heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  const int64_t unit = blockIdx.x / k.slices;
  const int col0 = (int)(blockIdx.x % k.slices) * LANES * 4;
  const int s = uniform((int)(unit / heads)), head = uniform((int)(unit % heads));
  const int64_t kh = head / (heads / (int)a.key_heads);
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, s);
  const int tid = threadIdx.x, c = tid % LANES * 4, g = tid / LANES;
  const int left = Dv - col0 - c;              // columns from this lane's on
  const int64_t place = (int64_t)head * Dk * Dv + col0 + c;
  Piece p;
  p.batch = s;
  p.first = 0;
  if (tid < Dk) {
    key[tid] = to_f32(row_at<const T>(a.k, p, 0)[kh * a.k_head + tid]);
    query[tid] = to_f32(row_at<const T>(a.q, p, 0)[kh * a.q_head + tid]) * a.scale;
  }
  const float decay = exp_of(log_decay(row_at<const float>(a.g, p, 0)[head]), 0.f), beta = row_at<const float>(a.beta, p, 0)[head];
  Raw<float, 4> S[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = g + i * kGroups;
    S[i].clear();
    if (a.state && slot >= 0 && row < Dk && left > 0) {
      const float* from = a.state + slot * a.state_stride + place + (int64_t)row * Dv;
      if constexpr (WHOLE) stream_in(S[i], from);
      else S[i].load_n(from, left);
    }
  }
  __syncthreads();
  // Sum over the rows of x S, in every lane; the groups' sums are added in order.
  auto over_rows = [&](const float* x, float (&out)[4]) __attribute__((always_inline)) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int row = g + i * kGroups;
      const float w = row < Dk ? x[row] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = __builtin_fmaf(w, S[i].get(e), t[e]);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[g][c + e] = t[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = 0.f;
      for (int i = 0; i < kGroups; ++i) out[e] += sums[i][c + e];
    }
  };
  float kS[4], w[4], o[4];
  over_rows(key, kS);
  const T* v = row_at<const T>(a.v, p, 0) + head * a.v_head + col0 + c;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = e < left ? beta * (to_f32(v[e]) - decay * kS[e]) : 0.f;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = g + i * kGroups;
    const float x = row < Dk ? key[row] : 0.f;
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = __builtin_fmaf(x, w[e], decay * S[i].get(e));
    S[i].pack(t);
    if (a.state_out && slot >= 0 && row < Dk && left > 0) {
      float* to = a.state_out + slot * a.state_out_stride + place + (int64_t)row * Dv;
      if constexpr (WHOLE) stream_out(S[i], to);
      else S[i].store_n(to, left);
    }
  }
  over_rows(query, o);
  if (g == 0) {
    T* to = row_at<T>(a.o, p, 0) + (int64_t)head * Dv + col0 + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) from_f32(o[e], to[e]);
  }
}

template <typename T, int LANES, bool WHOLE>
hipError_t step_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 grid((unsigned)(k.a.tokens.sequences * k.a.heads * k.slices)), block(256);
  constexpr int kGroups = 256 / LANES;
  if (k.a.key_dim <= 64) return launch_kernel(delta_step_kernel<T, LANES, 64 / kGroups, WHOLE>, grid, block, k, stream);
  if (k.a.key_dim <= 128) return launch_kernel(delta_step_kernel<T, LANES, 128 / kGroups, WHOLE>, grid, block, k, stream);
  return launch_kernel(delta_step_kernel<T, LANES, 256 / kGroups, WHOLE>, grid, block, k, stream);
}
// 64 columns at most leave half of 32 lanes without work (64 sequences of 16 heads of 128 x 64: 12.6 us against 13.1; of 72 x
// 41: 10.9 against 12.2).
template <typename T>
hipError_t step_t(const DeltaArgs& k, hipStream_t stream) {
  if (k.a.value_dim <= 64) return k.a.value_dim % 4 == 0 ? step_n<T, 16, true>(k, stream) : step_n<T, 16, false>(k, stream);
  return k.a.value_dim % 4 == 0 ? step_n<T, 32, true>(k, stream) : step_n<T, 32, false>(k, stream);
}

template <typename T, int KP, int NT, bool WHOLE>
hipError_t delta_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 grid((unsigned)shares(k.a.tokens.sequences * k.a.heads, k.slices)), block(512);
  if (k.states) return launch_kernel(delta_kernel<T, KP, NT, true, WHOLE>, grid, block, k, stream);
  return launch_kernel(delta_kernel<T, KP, NT, false, WHOLE>, grid, block, k, stream);
}
template <typename T, int KP>
hipError_t delta_k(const DeltaArgs& k, hipStream_t stream) {
  if (k.a.key_dim == KP) return delta_n<T, KP, 1, true>(k, stream);
  return delta_n<T, KP, 1, false>(k, stream);
}
template <typename T>
hipError_t delta_t(const DeltaArgs& k, hipStream_t stream) {
  if (k.a.key_dim <= 64) return delta_k<T, 64>(k, stream);
  if (k.a.key_dim <= 128) return delta_k<T, 128>(k, stream);
  return delta_k<T, 256>(k, stream);
}

template <typename T>
hipError_t chunks_t(const DeltaArgs& k, bool gradient, hipStream_t stream) {
  const dim3 grid((unsigned)(k.pieces * k.a.heads)), block(256);
  if (k.a.key_dim % 8 == 0)
    return gradient ? launch_kernel(delta_chunk_kernel<T, true, true>, grid, block, k, stream)
                    : launch_kernel(delta_chunk_kernel<T, false, true>, grid, block, k, stream);
  return gradient ? launch_kernel(delta_chunk_kernel<T, true, false>, grid, block, k, stream)
                  : launch_kernel(delta_chunk_kernel<T, false, false>, grid, block, k, stream);
}

int64_t round16(int64_t floats) { return (floats + 15) / 16 * 16; }
constexpr int kStepCols = 128;
int step_slices(const seq_delta_args_t& a) { return (a.value_dim + kStepCols - 1) / kStepCols; }

}  // namespace

int delta_slices(const seq_delta_args_t& a) { return (a.value_dim + 15) / 16; }

// Floats of the chunks' systems and decays; the operand blocks come first, 16-byte aligned.
int64_t delta_chunk_floats(const seq_delta_args_t& a) {
  return seq_pieces(seq_map(a.tokens, kChunkShift)) * a.heads * (kMatrix + 2 * kChunk);
}
int64_t delta_save_floats(const seq_delta_args_t& a) {
  return round16(seq_pieces(seq_map(a.tokens, kChunkShift)) * a.heads * a.key_dim * a.value_dim) +
         seq_rows(a.tokens) * a.heads * a.value_dim;
}
DeltaArgs delta_args(const seq_delta_args_t& a, float* ws) {
  DeltaArgs k{};
  k.a = a;
  k.m = seq_map(a.tokens, kChunkShift);
  k.pieces = (int32_t)seq_pieces(k.m);
  k.slices = delta_slices(a);
  const int64_t all = (int64_t)k.pieces * a.heads;
  k.inverse = reinterpret_cast<uint16_t*>(ws);
  k.inner = k.inverse + all * kMatrix;
  k.decay = reinterpret_cast<float*>(k.inner + all * kMatrix);
  k.states = a.save;
  k.errors = a.save ? a.save + round16(all * a.key_dim * a.value_dim) : nullptr;
  return k;
}

// Lanes of the largest launch.
int64_t delta_lanes(const seq_delta_args_t& a) {
  const int64_t chunks = seq_pieces(seq_map(a.tokens, kChunkShift)) * a.heads * 256;
  const int64_t order = shares(a.tokens.sequences * a.heads, delta_slices(a)) * 512;
  return chunks > order ? chunks : order;
}
int64_t delta_step_lanes(const seq_delta_args_t& a) { return a.tokens.sequences * a.heads * step_slices(a) * 256; }

hipError_t launch_delta_chunks(const DeltaArgs& k, bool gradient, hipStream_t stream) {
  switch (k.a.dtype) {
    case CONV_WGRAD_F32: return chunks_t<float>(k, gradient, stream);
    case CONV_WGRAD_BF16: return chunks_t<Bf16>(k, gradient, stream);
    default: return chunks_t<F16>(k, gradient, stream);
  }
}

hipError_t launch_delta(const seq_delta_args_t& a, float* ws, hipStream_t stream) {
  const DeltaArgs k = delta_args(a, ws);
  if (seq_rows(a.tokens) > 0) {
    const hipError_t err = launch_delta_chunks(k, false, stream);
    if (err != hipSuccess) return err;
  }
  switch (a.dtype) {
    case CONV_WGRAD_F32: return delta_t<float>(k, stream);
    case CONV_WGRAD_BF16: return delta_t<Bf16>(k, stream);
    default: return delta_t<F16>(k, stream);
  }
}

hipError_t launch_delta_step(const seq_delta_args_t& a, hipStream_t stream) {
  DeltaArgs k{};
  k.a = a;
  k.slices = step_slices(a);
  switch (a.dtype) {
    case CONV_WGRAD_F32: return step_t<float>(k, stream);
    case CONV_WGRAD_BF16: return step_t<Bf16>(k, stream);
    default: return step_t<F16>(k, stream);
  }
}

}  // namespace cw
