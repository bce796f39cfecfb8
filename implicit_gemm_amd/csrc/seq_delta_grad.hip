// The gated delta rule's gradient (gfx950).  With the forward's notation (seq_delta.h), do' = scale do, and walking the
// chunks of a sequence backwards:
//
//   dZ = beta e^(G_C - G) (K dS') + P^T do,  dX = (1 + M)^-T dZ  (also dv),
//   dS = e^G_C dS' + (e^G Q)^T do' - (e^G K)^T dX
//
// and then for all chunks at once, with E = e . (do' Z^T) on and below the diagonal, R = e . (dX Z^T) below it:
//
//   dq = e^G (do' S^T) + (E beta) K
//   dk = reads + beta w,   reads = -e^G (dX S^T) - (R beta) K,   w = e^(G_C - G) (Z dS'^T) + E^T Q - R^T K
//   dbeta = k . w,   dG = q . dq + k . reads - beta dbeta,   dg[t] = sum of dG from t on + <dS', S'>
//
// <dS', S'> follows from S' = e^G_C S + K^T (beta e^(G_C - G) Z) without reading S'.
#include "seq_delta.h"

namespace cw {

namespace {

// ---- the chunks of a sequence, last to first ------------------------------------------------------------------------
// The mirror of the forward's walk: 16 NT columns of one sequence's and head's dS a workgroup, waves 0 .. 3 the chain
// (K dS', dX, K^T dX), waves 4 .. 7 what does not wait for it: P^T do of the chunk to come and Q^T do' of this one.
template <typename T, int KP, int NT>
__global__ __launch_bounds__(512) void delta_back_kernel(DeltaArgs k) {
  constexpr int N = ElemPieces<T>::n, KS = KP / 32, MT = KP / 64;
  constexpr int kKeyPitch = KP + 8;
  constexpr bool kStage = N == 1 || KP * N <= 256;     // K's and Q's pieces fit the LDS beside the rest
  constexpr int kCols = 16 * NT;
  constexpr bool kAhead = N == 1 || KP <= 128;     // K's and Q's rows of the next chunk fit the registers
  __shared__ __attribute__((aligned(16))) uint16_t sS[kPieces][kCols][kKeyPitch], sX[kPieces][kCols][kTokenPitch],
      sW[kPieces][kCols][kTokenPitch], sD[kPieces][kCols][kTokenPitch], sO[N][kCols][kTokenPitch],
      sK[2][kStage ? N : 1][kStage ? kChunk : 1][kKeyPitch];
  __shared__ f32x4 sR[4][NT][64], sQ[KP / 16][NT][64];
  const seq_delta_args_t& a = k.a;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = wave & 3, lr = lane & 15, lg = lane >> 4;
  const bool chain = wave < 4;
  const int heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  const Share share = share_of(blockIdx.x, k.slices);
  if (share.unit >= k.m.S * heads) return;
  const int s = uniform(share.unit / heads), head = uniform(share.unit % heads), col0 = share.slice * kCols;
  const int64_t kh = head / (heads / (int)a.key_heads);
  Piece p;
  p.seq = s;
  if (k.m.offsets) {
    const int start = uniform(seq_start(k.m, s)), stop = uniform(seq_start(k.m, s + 1));
    p.batch = 0;
    p.first = start;
    p.len = max(stop - start, 0);
  } else {
    p.batch = s;
    p.first = 0;
    p.len = k.m.rows;
  }
  const int chunks = (p.len + kChunk - 1) >> kChunkShift;
  const int64_t number = chunk_head(k, chunk_number(k.m, s, (int)p.first, 0), head);
  const int64_t place = ((int64_t)s * heads + head) * Dk * Dv;

  f32x4 S[MT][NT];
  if (chain) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = col0 + 16 * t + lr;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 16 * (r * MT + m) + 4 * lg + x;
          S[m][t][x] = k.last && row < Dk && c < Dv ? at_lane(k.last + place, row * Dv + c) : 0.f;
        }
      }
  }
  auto share_state = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint2 u[kPieces];
        split4<kPieces>(S[m][t], u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          *reinterpret_cast<uint2*>(&sS[i][16 * t + lr][16 * (r * MT + m) + 4 * lg]) = u[i];
      }
  };
  auto keep_state = [&](float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = col0 + 16 * t + lr;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 16 * (r * MT + m) + 4 * lg + x;
          if (row < Dk && c < Dv) at_lane(to, row * Dv + c) = S[m][t][x];
        }
      }
  };

  Eight<T> rows[kAhead ? KS : 1];                 // chain: K, beside: Q
  T now[NT][4], next[NT][4];         // beside: do of this chunk and of the one to come
  s16x8 square[2][kPieces];          // chain: (1 + M)^-T, beside: P^T of the chunk to come
  float4 first, last;
  float whole;
  auto load_row = [&](int j, int c, Eight<T>& to) __attribute__((always_inline)) {
    const int n = p.len - kChunk * j, t = 16 * r + lr;
    const ChunkRows<const T> from(chain ? a.k : a.q, kh * (chain ? a.k_head : a.q_head), p, kChunk * j);
    to.load(&from.at(min(t, n - 1), 32 * c + 8 * lg), t < n ? Dk - 32 * c - 8 * lg : 0);
  };
  auto load_rows = [&](int j) __attribute__((always_inline)) {
    if constexpr (kAhead) {
#pragma unroll
      for (int c = 0; c < KS; ++c) load_row(j, c, rows[c]);
    }
  };
  auto row_pieces = [&](int j, int c, s16x8 (&e)[N]) __attribute__((always_inline)) {
    if constexpr (kAhead) {
      rows[c].pieces(e);
    } else {
      Eight<T> row;
      load_row(j, c, row);
      row.pieces(e);
    }
  };
  auto load_do = [&](int j, T (&v)[NT][4]) __attribute__((always_inline)) {
    const int n = p.len - kChunk * j;
    const ChunkRows<const T> from(k.dout, head * k.dout_head, p, kChunk * j);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int t = 16 * r + 4 * lg + x;
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const int col = col0 + 16 * c + lr;
        if (t < n && col < Dv) v[c][x] = from.at(t, col);
        else from_f32(0.f, v[c][x]);
      }
    }
  };
  auto load_square = [&](int j) __attribute__((always_inline)) {
    const uint16_t* from = (chain ? k.inverse : k.inner) + (number + (int64_t)j * heads) * kMatrix + lane * 8;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (c >= r / 2) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          square[c][i] = *reinterpret_cast<const s16x8*>(from + (upper_frag(r, c) * kPieces + i) * kFragElems);
      }
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    const float* from = k.decay + (number + (int64_t)j * heads) * 2 * kChunk;
    first = *reinterpret_cast<const float4*>(from + 16 * r + 4 * lg);
    last = *reinterpret_cast<const float4*>(from + kChunk + 16 * r + 4 * lg);
    whole = from[kChunk - 1];
  };
  // beside: do as an operand
  auto share_do = [&](const T (&v)[NT][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint2 u[N];
      split4<N>(f32x4{to_f32(v[t][0]), to_f32(v[t][1]), to_f32(v[t][2]), to_f32(v[t][3])}, u);
#pragma unroll
      for (int i = 0; i < N; ++i) *reinterpret_cast<uint2*>(&sO[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
    }
  };
  // beside: P^T do
  auto inner_part = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 lead = zero4(), rest = zero4();
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c >= r / 2) {
          s16x8 b[N];
#pragma unroll
          for (int i = 0; i < N; ++i) b[i] = lds8(&sO[i][16 * t + lr][32 * c + 8 * lg]);
          mfma_pieces<kPieces>(square[c], b, lead, rest);
        }
      sR[r][t][lane] = lead + rest;
    }
  };
  // Operand of K^T or Q^T: rows of the state, terms are tokens.
  auto transposed = [&](int which, const seq_view_t& view, int64_t at, int j, int m, int c, s16x8 (&e)[N]) __attribute__((always_inline)) {
    if constexpr (kStage) {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = lds8_trans(&sK[which][i][32 * c][16 * m] + trans_place(lane, kKeyPitch), kKeyPitch);
    } else {
      const ChunkRows<const T> from(view, at, p, kChunk * j);
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = opaque(32 * c + 8 * lg) + i, row = 16 * m + lr;
        g[i] = kChunk * j + t < p.len && row < Dk ? to_f32(from.at(t, row)) : 0.f;
      }
      split8<N>(g, e);
    }
  };

  if (chunks > 0) {
    load_rows(chunks - 1);
    load_square(chunks - 1);
    load_decay(chunks - 1);
    if (!chain) {
      load_do(chunks - 1, now);
      share_do(now);
      if (chunks > 1) load_do(chunks - 2, next);
    }
  }
  if (chain) share_state();
  lds_barrier();
  if (chunks > 0 && !chain) {
    inner_part();
    if (chunks > 1) load_square(chunks - 2);
  }
  lds_barrier();

  for (int j = chunks - 1; j >= 0; --j) {
    const int n = p.len - kChunk * j;
    const bool more = j > 0;
    const float f[4] = {first.x, first.y, first.z, first.w}, l[4] = {last.x, last.y, last.z, last.w};
    const float keep = whole;
    if (chain) {
      keep_state(k.dstates + (number + (int64_t)j * heads) * Dk * Dv);
      f32x4 lead[NT], rest[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) lead[t] = rest[t] = zero4();
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        s16x8 e[N];
        row_pieces(j, c, e);
        if (kStage) {
#pragma unroll
          for (int i = 0; i < N; ++i) *reinterpret_cast<s16x8*>(&sK[0][i][kStage ? 16 * r + lr : 0][32 * c + 8 * lg]) = e[i];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = lds8(&sS[i][16 * t + lr][32 * c + 8 * lg]);
          mfma_pieces<kPieces>(e, b, lead[t], rest[t]);
        }
      }
      if (more) load_rows(j - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 z = sR[r][t][lane];
        uint2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __builtin_fmaf(l[i], lead[t][i] + rest[t][i], z[i]);
        split4<kPieces>(z, u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint2*>(&sX[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
      }
    } else {
      if (kStage) {
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          s16x8 e[N];
          row_pieces(j, c, e);
#pragma unroll
          for (int i = 0; i < N; ++i) *reinterpret_cast<s16x8*>(&sK[1][i][kStage ? 16 * r + lr : 0][32 * c + 8 * lg]) = e[i];
        }
        if (more) load_rows(j - 1);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 x;
        uint2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a.scale * f[i] * to_f32(now[t][i]);
        split4<kPieces>(x, u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint2*>(&sD[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
      }
      if (more) {
        share_do(next);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) now[t][i] = next[t][i];
        if (j > 1) load_do(j - 2, next);
        load_decay(j - 1);
      }
    }
    lds_barrier();
    if (chain) {
      f32x4 dx[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 lead = zero4(), rest = zero4();
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c >= r / 2) {
            s16x8 b[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) b[i] = lds8(&sX[i][16 * t + lr][32 * c + 8 * lg]);
            mfma_pieces<kPieces>(square[c], b, lead, rest);
          }
        dx[t] = lead + rest;
        f32x4 x;
        uint2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = -f[i] * dx[t][i];
        split4<kPieces>(x, u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint2*>(&sW[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
      }
      if (more) {
        load_square(j - 1);
        load_decay(j - 1);
      }
      const int64_t at = ((p.batch * k.m.rows + p.first + kChunk * j) * heads + head) * Dv + col0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * r + 4 * lg + i;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (t < n && col0 + 16 * c + lr < Dv) {
            at_lane(k.dx + at, t * heads * Dv + 16 * c + lr) = dx[c][i];
            from_f32(dx[c][i], at_lane(static_cast<T*>(k.dv) + at, t * heads * Dv + 16 * c + lr));
          }
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 lead[NT], rest[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) lead[t] = rest[t] = zero4();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s16x8 e[N];
          transposed(1, a.q, kh * a.q_head, j, r * MT + m, c, e);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            s16x8 b[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) b[i] = lds8(&sD[i][16 * t + lr][32 * c + 8 * lg]);
            mfma_pieces<kPieces>(e, b, lead[t], rest[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) sQ[r * MT + m][t][lane] = lead[t] + rest[t];
      }
    }
    lds_barrier();
    if (chain) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 low[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          low[t] = sQ[r * MT + m][t][lane];
#pragma unroll
          for (int x = 0; x < 4; ++x) S[m][t][x] *= keep;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s16x8 e[N];
          transposed(0, a.k, kh * a.k_head, j, r * MT + m, c, e);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            s16x8 b[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) b[i] = lds8(&sW[i][16 * t + lr][32 * c + 8 * lg]);
            mfma_pieces<kPieces>(e, b, S[m][t], low[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) S[m][t] += low[t];
      }
      share_state();
    } else if (more) {
      inner_part();
      if (j > 1) load_square(j - 2);
    }
    lds_barrier();
  }
  if (chain && k.dstate) keep_state(k.dstate + place);
}

// ---- queries, keys and decays -----------------------------------------------------------------------------------------
// A workgroup has a chunk and a key head, and goes through the value heads that share it.  Four waves have 16 tokens
// each; keys of more than 64 dimensions go to two such sets of waves, half of the dimensions each.  First the products over
// the value's dimension (do S^T, dX S^T, Z dS'^T, do Z^T, dX Z^T), 32 columns of S, dS' and Z at a time as pieces in LDS,
// then those over the chunk's tokens (with E and R, through LDS).
constexpr int kPanelPitch = 40;      // 16-bit elements of an LDS row of 32 columns

template <typename T, int KP>
struct InputGradLds {
  static constexpr bool kStage = ElemPieces<T>::n == 1;
  struct Panels {
    uint16_t S[kPieces][KP][kPanelPitch], D[kPieces][KP][kPanelPitch], Z[kPieces][kChunk][kPanelPitch];
  };
  struct Squares {
    uint16_t E[kPieces][kChunk][kTokenPitch], R[kPieces][kChunk][kTokenPitch];     // [j][i]
    uint16_t key[kStage ? kChunk : 1][KP + 8], query[kStage ? kChunk : 1][KP + 8];
  };
  union {
    Panels panels;
    Squares squares;
  };
  ChunkDecay d;
  float dots[2][kChunk], db[2][kChunk], part[8];
};

template <bool FIRST, class A, class B>
__device__ __forceinline__ auto& pick(A& a, B& b) {
  if constexpr (FIRST) return a;
  else return b;
}

// How the value heads of a key head are gone through: there is one, all in one launch with the sums in registers, or a
// launch each with the sums in the workspace (keys of 256 dimensions leave no registers for them).
enum Sharing { kAlone, kTogether, kInTurn };

template <typename T, int KP, Sharing SHARING>
__global__ __launch_bounds__(KP > 64 ? 512 : 256) void delta_input_grad_kernel(DeltaArgs k) {
  constexpr int N = ElemPieces<T>::n, kParts = KP > 64 ? 2 : 1, kThreads = 256 * kParts, KT = KP / 16 / kParts;
  typedef InputGradLds<T, KP> Lds;
  __shared__ __attribute__((aligned(16))) char bytes[sizeof(Lds)];
  Lds& L = *reinterpret_cast<Lds*>(bytes);
  const seq_delta_args_t& a = k.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = wave & 3, part = wave >> 2;
  int lr = lane & 15, lg = lane >> 4;
  const int heads = (int)a.heads, key_heads = (int)a.key_heads, group = heads / key_heads, Dk = a.key_dim, Dv = a.value_dim;
  const int piece = blockIdx.x / key_heads, kh = blockIdx.x % key_heads;
  Piece p;
  if (!find_piece(k.m, piece, p)) return;
  const int n = p.end - p.t0;
  const int64_t row0 = p.batch * k.m.rows + p.first + p.t0;      // of the dense outputs
  if (p.seq == k.m.S) {              // padding behind the last sequence
    for (int i = tid; i < n * Dk; i += kThreads) {
      const int64_t at = ((row0 + i / Dk) * key_heads + kh) * Dk + i % Dk;
      from_f32(0.f, static_cast<T*>(k.dq)[at]);
      from_f32(0.f, static_cast<T*>(k.dk)[at]);
    }
    for (int64_t i = tid; i < (int64_t)n * group * Dv; i += kThreads)
      from_f32(0.f, static_cast<T*>(k.dv)[((row0 + i / (group * Dv)) * heads + (int64_t)kh * group) * Dv + i % (group * Dv)]);
    for (int i = tid; i < n * group; i += kThreads) {
      const int64_t at = (row0 + i / group) * heads + (int64_t)kh * group + i % group;
      k.dg[at] = 0.f;
      k.dbeta[at] = 0.f;
    }
    return;
  }
  if (n <= 0) return;                // an empty sequence has a number too
  const int tile0 = part * KT;       // first of this wave's 16-column tiles of the key's dimension
  constexpr bool kHeld = SHARING == kTogether;
  f32x4 dq[kHeld ? KT : 1], dk[kHeld ? KT : 1];
  if constexpr (kHeld) {
#pragma unroll
    for (int t = 0; t < KT; ++t) dq[t] = dk[t] = zero4();
  }
  const ChunkRows<const T> key(a.k, kh * a.k_head, p, p.t0), query(a.q, kh * a.q_head, p, p.t0);
  // K or Q as the second operand: columns are the key's dimension, terms are tokens.
  auto transposed = [&](const uint16_t* staged, const ChunkRows<const T>& from, int t, int c, s16x8 (&e)[N]) __attribute__((always_inline)) {
    if constexpr (Lds::kStage) {
      e[0] = lds8_trans(staged + 32 * c * (KP + 8) + 16 * (tile0 + t) + trans_place(lane, KP + 8), KP + 8);
    } else {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = opaque(32 * c + 8 * lg) + i, col = 16 * (tile0 + t) + lr;
        g[i] = tok < n && col < Dk ? to_f32(from.at(tok, col)) : 0.f;
      }
      split8<N>(g, e);
    }
  };
  // Element (token 16 r + 4 lg + i, column 16 t + lr) of K or Q.
  auto element = [&](const ChunkRows<const T>& from, int t, int i) __attribute__((always_inline)) {
    const int row = opaque(16 * r + 4 * lg) + i, col = 16 * (tile0 + t) + lr;
    return row < n && col < Dk ? to_f32(from.at(row, col)) : 0.f;
  };
  for (int h = 0; h < (kHeld ? group : 1); ++h) {
    const int head = kh * group + (SHARING == kInTurn ? k.turn : h);
    if constexpr (kHeld) {           // offsets made from these are not kept over the loop
      lr = opaque(lr);
      lg = opaque(lg);
    }
    const int mine = 16 * r + lr;    // the token whose row this lane loads
    const int64_t at = chunk_head(k, piece, head);
    const float* pS = k.states + at * Dk * Dv;
    const float* pD = k.dstates + at * Dk * Dv;
    if (wave == 0) chunk_decay(a, p, head, lane, L.d);
    f32x4 Q[KT], R[KT], W[KT], oz[4], other[kParts == 1 ? 4 : 1];     // do Z^T and dX Z^T; two sets of waves have one each
    f32x4 (&xz)[4] = pick<kParts == 1>(other, oz);
#pragma unroll
    for (int t = 0; t < KT; ++t) Q[t] = R[t] = W[t] = zero4();
#pragma unroll
    for (int t = 0; t < 4; ++t) oz[t] = xz[t] = zero4();
    float inside = 0.f;              // <dS', S>
#pragma unroll 1
    for (int c0 = 0; c0 < Dv; c0 += 32) {
#pragma unroll
      for (int i = 0; i < KP * 8 / kThreads; ++i) {
        const int row = (tid + kThreads * i) >> 3, c = 4 * (tid & 7);
        Raw<float, 4> s, d;
        s.clear();
        d.clear();
        if (row < Dk && c0 + c < Dv) {
          s.load_n(&at_lane(pS, row * Dv + c0 + c), Dv - c0 - c);
          d.load_n(&at_lane(pD, row * Dv + c0 + c), Dv - c0 - c);
        }
        uint2 us[kPieces], ud[kPieces];
        split4<kPieces>(f32x4{s.get(0), s.get(1), s.get(2), s.get(3)}, us);
        split4<kPieces>(f32x4{d.get(0), d.get(1), d.get(2), d.get(3)}, ud);
#pragma unroll
        for (int e = 0; e < 4; ++e) inside = __builtin_fmaf(s.get(e), d.get(e), inside);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
          *reinterpret_cast<uint2*>(&L.panels.S[e][row][c]) = us[e];
          *reinterpret_cast<uint2*>(&L.panels.D[e][row][c]) = ud[e];
        }
      }
#pragma unroll
      for (int i = 0; i < kChunk * 8 / kThreads; ++i) {
        const int row = (tid + kThreads * i) >> 3, c = 4 * (tid & 7);
        Raw<float, 4> z;
        z.clear();
        if (row < n && c0 + c < Dv) z.load_n(&at_lane(k.errors + (row0 * heads + head) * Dv, row * heads * Dv + c0 + c), Dv - c0 - c);
        uint2 u[kPieces];
        split4<kPieces>(f32x4{z.get(0), z.get(1), z.get(2), z.get(3)}, u);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) *reinterpret_cast<uint2*>(&L.panels.Z[e][row][c]) = u[e];
      }
      s16x8 o[N], x[kPieces], z[kPieces];
      {
        const int left = mine < n ? Dv - c0 - 8 * lg : 0;
        Eight<T> eo;
        Eight<float> ex;
        eo.load(&ChunkRows<const T>(k.dout, head * k.dout_head, p, p.t0).at(min(mine, n - 1), c0 + 8 * lg), left);
        ex.load(&at_lane(k.dx + (row0 * heads + head) * Dv, min(mine, n - 1) * heads * Dv + c0 + 8 * lg), left);
        eo.pieces(o);
        ex.pieces(x);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kPieces; ++e) z[e] = lds8(&L.panels.Z[e][mine][8 * lg]);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        s16x8 b[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.S[e][16 * (tile0 + t) + lr][8 * lg]);
        mfma_pieces<kPieces>(o, b, Q[t], Q[t]);
        mfma_pieces<kPieces>(x, b, R[t], R[t]);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.D[e][16 * (tile0 + t) + lr][8 * lg]);
        mfma_pieces<kPieces>(z, b, W[t], W[t]);
        if (t & 1) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= r) {
          s16x8 b[kPieces];
#pragma unroll
          for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.Z[e][16 * t + lr][8 * lg]);
          if (part == 0) mfma_pieces<kPieces>(o, b, oz[t], oz[t]);
          if (part == kParts - 1) mfma_pieces<kPieces>(x, b, xz[t], xz[t]);
        }
      __syncthreads();
    }
    // E and R (with the sign that R's products have), and the parts that the states give
    float first[4], last[4], beta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * r + 4 * lg + i;
      first[i] = L.d.first[row];
      last[i] = L.d.last[row];
      beta[i] = L.d.beta[row];
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * r + 4 * lg + i, j = 16 * t + lr;
        const bool live = row < n && j <= row;
        const float e = live ? decay_between(L.d, row, j) : 0.f;
        if (part == 0) oz[t][i] = live ? a.scale * e * oz[t][i] : 0.f;
        if (part == kParts - 1) xz[t][i] = live && j < row ? -e * xz[t][i] : 0.f;
      }
    auto share_square = [&](const f32x4 (&m)[4], uint16_t (*to)[kChunk][kTokenPitch], bool weighted) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int j = 16 * t + lr;
        const float w = weighted ? L.d.beta[j] : 1.f;
        uint2 u[kPieces];
        split4<kPieces>(f32x4{w * m[t][0], w * m[t][1], w * m[t][2], w * m[t][3]}, u);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) *reinterpret_cast<uint2*>(&to[e][j][16 * r + 4 * lg]) = u[e];
      }
    };
    auto share_squares = [&](bool weighted) __attribute__((always_inline)) {
      if (part == 0) share_square(oz, L.squares.E, weighted);
      if (part == kParts - 1) share_square(xz, L.squares.R, weighted);
    };
    share_squares(true);
    if constexpr (Lds::kStage) {
#pragma unroll
      for (int c = 0; c < KT / 2; ++c) {
        const int col = 16 * tile0 + 32 * c + 8 * lg, left = mine < n ? Dk - col : 0;
        Eight<T> e;
        s16x8 u[N];
        e.load(&key.at(min(mine, n - 1), col), left);
        e.pieces(u);
        *reinterpret_cast<s16x8*>(&L.squares.key[mine][col]) = u[0];
        e.load(&query.at(min(mine, n - 1), col), left);
        e.pieces(u);
        *reinterpret_cast<s16x8*>(&L.squares.query[mine][col]) = u[0];
      }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Q[t][i] *= a.scale * first[i];
        R[t][i] *= -first[i];
        W[t][i] *= last[i];
      }
    __syncthreads();
    const uint16_t* staged_key = &L.squares.key[0][0];
    const uint16_t* staged_query = &L.squares.query[0][0];
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (c <= r / 2) {
        s16x8 e[kPieces], x[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          e[i] = lds8_trans(&L.squares.E[i][32 * c][16 * r] + trans_place(lane, kTokenPitch), kTokenPitch);
          x[i] = lds8_trans(&L.squares.R[i][32 * c][16 * r] + trans_place(lane, kTokenPitch), kTokenPitch);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          s16x8 b[N];
          transposed(staged_key, key, t, c, b);
          mfma_pieces<kPieces>(e, b, Q[t], Q[t]);
          mfma_pieces<kPieces>(x, b, R[t], R[t]);
          if (!Lds::kStage) __builtin_amdgcn_sched_barrier(0);
        }
      }
    __syncthreads();
    share_squares(false);
    // <dS', S'>: e^G_C <dS', S> and what the chunk itself writes, beta k . (e^(G_C - G) Z dS'^T)
    float tail = L.d.first[kChunk - 1] * inside, dots[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float kv = element(key, t, i), qv = element(query, t, i);
        tail = __builtin_fmaf(beta[i] * kv, W[t][i], tail);
        dots[i] = __builtin_fmaf(qv, Q[t][i], __builtin_fmaf(kv, R[t][i], dots[i]));
      }
      if (t & 1) __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (c >= r / 2) {
        s16x8 e[kPieces], x[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          e[i] = lds8(&L.squares.E[i][mine][32 * c + 8 * lg]);
          x[i] = lds8(&L.squares.R[i][mine][32 * c + 8 * lg]);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          s16x8 b[N];
          transposed(staged_query, query, t, c, b);
          mfma_pieces<kPieces>(e, b, W[t], W[t]);
          transposed(staged_key, key, t, c, b);
          mfma_pieces<kPieces>(x, b, W[t], W[t]);
          if (!Lds::kStage) __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) db[i] = __builtin_fmaf(element(key, t, i), W[t][i], db[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) R[t][i] = __builtin_fmaf(beta[i], W[t][i], R[t][i]);
      if constexpr (kHeld) {
        dq[t] += Q[t];
        dk[t] += R[t];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      db[i] = lanes_reduce<AddOp>(db[i], 16);
      dots[i] = lanes_reduce<AddOp>(dots[i], 16);
    }
    tail = lanes_reduce<AddOp>(tail, 64);
    if (lane == 0) L.part[wave] = tail;
    if (lr == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        L.dots[part][16 * r + 4 * lg + i] = dots[i];
        L.db[part][16 * r + 4 * lg + i] = db[i];
      }
    }
    __syncthreads();
    if (wave == 0) {
      float b = L.db[0][lane], dot = L.dots[0][lane], end = 0.f;
      if constexpr (kParts == 2) {
        b += L.db[1][lane];
        dot += L.dots[1][lane];
      }
      double sum = lane < n ? __builtin_fmaf(-L.d.beta[lane], b, dot) : 0.f;
#pragma unroll
      for (int step = 1; step < 64; step *= 2) {
        const double from = __shfl_down(sum, step);
        if (lane + step < 64) sum += from;
      }
#pragma unroll
      for (int i = 0; i < 4 * kParts; ++i) end += L.part[i];
      if (lane < n) {
        k.dg[(row0 + lane) * heads + head] = (float)(sum + end);
        k.dbeta[(row0 + lane) * heads + head] = b;
      }
    }
    if (!kHeld || h == group - 1) {
      const int64_t to = (row0 * key_heads + kh) * Dk;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * r + 4 * lg + i, col = 16 * (tile0 + t) + lr;
          if (row < n && col < Dk) {
            const int e = row * key_heads * Dk + col;
            float vq = kHeld ? dq[kHeld ? t : 0][i] : Q[t][i], vk = kHeld ? dk[kHeld ? t : 0][i] : R[t][i];
            if constexpr (SHARING == kInTurn) {
              float& sq = at_lane(k.sums + to, e);
              float& sk = at_lane(k.sums + k.sums_stride + to, e);
              if (k.turn > 0) {
                vq += sq;
                vk += sk;
              }
              sq = vq;
              sk = vk;
            }
            if (SHARING != kInTurn || k.turn == group - 1) {
              from_f32(vq, at_lane(static_cast<T*>(k.dq) + to, e));
              from_f32(vk, at_lane(static_cast<T*>(k.dk) + to, e));
            }
          }
        }
    }
    if constexpr (kHeld) __syncthreads();
  }
}

template <typename T, int KP>
hipError_t grad_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 order((unsigned)shares(k.a.tokens.sequences * k.a.heads, k.slices));
  const hipError_t err = launch_kernel(delta_back_kernel<T, KP, 1>, order, dim3(512), k, stream);
  if (err != hipSuccess || seq_rows(k.a.tokens) == 0) return err;
  const dim3 grid((unsigned)(k.pieces * k.a.key_heads)), block(KP > 64 ? 512 : 256);
  const int group = (int)(k.a.heads / k.a.key_heads);
  if (group == 1) return launch_kernel(delta_input_grad_kernel<T, KP, kAlone>, grid, block, k, stream);
  if constexpr (KP <= 128) {
    return launch_kernel(delta_input_grad_kernel<T, KP, kTogether>, grid, block, k, stream);
  } else {
    DeltaArgs one = k;
    for (one.turn = 0; one.turn < group; ++one.turn) {
      const hipError_t e = launch_kernel(delta_input_grad_kernel<T, KP, kInTurn>, grid, block, one, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
}
template <typename T>
hipError_t grad_t(const DeltaArgs& k, hipStream_t stream) {
  if (k.a.key_dim <= 64) return grad_n<T, 64>(k, stream);
  if (k.a.key_dim <= 128) return grad_n<T, 128>(k, stream);
  return grad_n<T, 256>(k, stream);
}

int64_t round16(int64_t floats) { return (floats + 15) / 16 * 16; }
int64_t sums_floats(const seq_delta_args_t& a) {
  return a.heads > a.key_heads && a.key_dim > 128 ? seq_rows(a.tokens) * a.key_heads * a.key_dim : 0;
}

}  // namespace

int64_t delta_grad_ws_floats(const seq_delta_grad_args_t& g) {
  const seq_delta_args_t& a = g.fwd;
  return delta_chunk_floats(a) + round16(seq_pieces(seq_map(a.tokens, kChunkShift)) * a.heads * a.key_dim * a.value_dim) +
         round16(seq_rows(a.tokens) * a.heads * a.value_dim) + 2 * sums_floats(a);
}

int64_t delta_grad_lanes(const seq_delta_grad_args_t& g) {
  const int64_t inputs = seq_pieces(seq_map(g.fwd.tokens, kChunkShift)) * g.fwd.key_heads * (g.fwd.key_dim > 64 ? 512 : 256);
  const int64_t others = delta_lanes(g.fwd);
  return inputs > others ? inputs : others;
}

hipError_t launch_delta_grad(const seq_delta_grad_args_t& g, float* ws, hipStream_t stream) {
  DeltaArgs k = delta_args(g.fwd, ws);
  k.dout = g.dout;
  k.dout_head = g.dout_head;
  k.last = g.dstate_out;
  k.dstates = ws + delta_chunk_floats(g.fwd);
  k.dx = k.dstates + round16((int64_t)k.pieces * g.fwd.heads * g.fwd.key_dim * g.fwd.value_dim);
  k.sums = k.dx + round16(seq_rows(g.fwd.tokens) * g.fwd.heads * g.fwd.value_dim);
  k.sums_stride = sums_floats(g.fwd);
  k.dq = g.dq;
  k.dk = g.dk;
  k.dv = g.dv;
  k.dg = g.dg;
  k.dbeta = g.dbeta;
  k.dstate = g.dstate;
  if (seq_rows(g.fwd.tokens) > 0) {
    const hipError_t err = launch_delta_chunks(k, true, stream);
    if (err != hipSuccess) return err;
  }
  switch (g.fwd.dtype) {
    case CONV_WGRAD_F32: return grad_t<float>(k, stream);
    case CONV_WGRAD_BF16: return grad_t<Bf16>(k, stream);
    default: return grad_t<F16>(k, stream);
  }
}

}  // namespace cw
