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
// Bound by the chain's latency as the forward's walk is: 4 x 2048 tokens of 16 heads of 128 x 128 in bf16 in 180 us, 177 MB
// read and 237 written, the vector ALU and LDS 26 % busy, the matrix units 13 %.
//
// The mirror of the forward's walk: 16 NT columns of one sequence's and head's dS a workgroup, waves 0 .. 3 the chain
// (K dS', dX, K^T dX), waves 4 .. 7 what does not wait for it: P^T do of the chunk to come and Q^T do' of this one.
template <typename T, int KP, int NT>
struct BackLds {
  static constexpr int N = ElemPieces<T>::n;
  static constexpr bool kStage = sizeof(T) == 2 || KP <= 128;     // K and Q fit beside the rest
  Operand<KP> S[kPieces][NT];
  Operand<kChunk> X[kPieces][NT], W[kPieces][NT], D[kPieces][NT], O[N][NT];
  Staged<T, kStage ? KP : 0> K, Q;
  f32x4 back[KP / 16][NT][64];       // Q^T do', each lane's as the chain's lane takes it
  // P^T do of the chunk to come, where the chain's wave r is to put its part of dZ: its tokens' 16 x 16 blocks of two
  // pieces of X, free from the one exchange to the other.
  __device__ __forceinline__ f32x4& inner(int r, int t, int lane) {
    return *reinterpret_cast<f32x4*>(&X[lane >> 5][t].at[2 * r + ((lane >> 4) & 1)][lane & 15][0]);
  }
};
template <typename T, int KP, int NT, bool WHOLE>
__device__ __forceinline__ void back_chain(const DeltaArgs& k, const Walk& w, BackLds<T, KP, NT>& L, int r, int lane) {
  typedef BackLds<T, KP, NT> Lds;
  constexpr int N = Lds::N, KS = KP / 32, MT = KP / 64;
  const seq_delta_args_t& a = k.a;
  const int lr = lane & 15, lg = lane >> 4, heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  const int64_t place = ((int64_t)w.seq * heads + w.head) * Dk * Dv;
  f32x4 S[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = w.col0 + 16 * t + lr;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 16 * (r * MT + m) + 4 * lg + x;
        S[m][t][x] = k.last && (WHOLE || row < Dk) && c < Dv ? at_lane(k.last + place, row * Dv + c) : 0.f;
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
  auto load_square = [&](int j) __attribute__((always_inline)) {
    const uint16_t* from = k.inverse + (w.number + (int64_t)j * heads) * kMatrix;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        square[c][i] = *reinterpret_cast<const s16x8*>(&at_lane(from + (upper_frag(r, max(c, r / 2)) * kPieces + i) * kFragElems, lane * 8));
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    const float* from = k.decay + (w.number + (int64_t)j * heads) * 2 * kChunk;
    first = *reinterpret_cast<const float4*>(from + 16 * r + 4 * lg);
    last = *reinterpret_cast<const float4*>(from + kChunk + 16 * r + 4 * lg);
    whole = from[kChunk - 1];
  };
  if (w.chunks > 0) {
    load_rows(w.chunks - 1);
    load_decay(w.chunks - 1);
    load_square(w.chunks - 1);
  }
  share_state();
  lds_barrier();
  lds_barrier();
#pragma unroll 1
  for (int j = w.chunks - 1; j >= 0; --j) {
    const int n = w.p.len - kChunk * j, next = max(j - 1, 0);
    const float f[4] = {first.x, first.y, first.z, first.w}, l[4] = {last.x, last.y, last.z, last.w};
    const float keep = whole;
    keep_state(k.dstates + (w.number + (int64_t)j * heads) * Dk * Dv);
    // dZ
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
        if (c & 1) __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (Lds::kStage) {
#pragma unroll
        for (int c = 0; c < KS; ++c) rows[c].put(&L.K.at[16 * r + lr][32 * c + 8 * lg]);
      }
      load_rows(next);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4 kS = total(sum[t]);
        f32x4 z = L.inner(r, t, lane);
        u32x2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = 16 * r + 4 * lg + i < n ? __builtin_fmaf(l[i], kS[i], z[i]) : 0.f;
        split4<kPieces>(z, u);
        wave_sync();                 // what `inner` holds is read by then
#pragma unroll
        for (int i = 0; i < kPieces; ++i) L.X[i][t].four(16 * r + 4 * lg, lr) = u[i];
      }
    }
    lds_barrier();
    // dX
    f32x4 dx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 sum[kPieces];
      clear(sum);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c >= r / 2) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.X[i][t].eight(c, lane);
          mfma_pieces<kPieces>(square[c], b, sum);
        }
      dx[t] = total(sum);
      f32x4 x;
      u32x2 u[kPieces];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = -f[i] * dx[t][i];
      split4<kPieces>(x, u);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) L.W[i][t].four(16 * r + 4 * lg, lr) = u[i];
    }
    lds_barrier();
    {
      const int64_t at = ((w.p.batch * k.m.rows + w.p.first + kChunk * j) * heads + w.head) * Dv + w.col0;
#pragma unroll
      for (int c = 0; c < NT; ++c)
        if (w.col0 + 16 * c + lr < Dv) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = opaque(16 * r + 4 * lg) + i;
            if (t < n) {
              at_lane(k.dx + at, t * heads * Dv + 16 * c + lr) = dx[c][i];
              from_f32(dx[c][i], at_lane(static_cast<T*>(k.dv) + at, t * heads * Dv + 16 * c + lr));
            }
          }
        }
    }
    load_decay(next);
    if (N == 1) load_square(next);
    // dS
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f32x4 sum[NT][kPieces];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        clear(sum[t]);
        sum[t][1] = L.back[r * MT + m][t][lane];
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[t][0][x] = keep * S[m][t][x];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s16x8 e[N];
        if constexpr (Lds::kStage) L.K.transposed(r * MT + m, c, lane, e);
        else transposed_rows<T>(keys(j), n, Dk, r * MT + m, c, lane, e);
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
    if (N > 1) {                     // fp32 and fp16 K take their pieces' registers: only now are enough free
      __builtin_amdgcn_sched_barrier(0);
      load_square(next);
    }
    share_state();
    lds_barrier();
  }
  if (k.dstate) keep_state(k.dstate + place);
}

template <typename T, int KP, int NT, bool WHOLE>
__device__ __forceinline__ void back_beside(const DeltaArgs& k, const Walk& w, BackLds<T, KP, NT>& L, int r, int lane) {
  typedef BackLds<T, KP, NT> Lds;
  constexpr int N = Lds::N, KS = KP / 32, MT = KP / 64;
  const seq_delta_args_t& a = k.a;
  const int lr = lane & 15, lg = lane >> 4, heads = (int)a.heads, Dk = a.key_dim, Dv = a.value_dim;
  Eight<T> rows[KS];
  T now[NT][4], next[NT][4];         // do of this chunk and of the one to come
  s16x8 square[2][kPieces];
  float4 first;
  auto queries = [&](int j) __attribute__((always_inline)) {
    return ChunkRows<const T>(a.q, w.key_head * a.q_head, w.p, kChunk * j);
  };
  auto load_rows = [&](int j) __attribute__((always_inline)) {
    if constexpr (Lds::kStage) {
#pragma unroll
      for (int c = 0; c < KS; ++c) load_row<T, KP, WHOLE>(queries(j), w.p.len - kChunk * j, 16 * r + lr, lg, Dk, c, rows[c]);
    }
  };
  auto load_do = [&](int j, T (&v)[NT][4]) __attribute__((always_inline)) {
    const int n = w.p.len - kChunk * j;
    const ChunkRows<const T> from(k.dout, w.head * k.dout_head, w.p, kChunk * j);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int t = 0; t < NT; ++t) v[t][x] = from.at(min(16 * r + 4 * lg + x, n - 1), min(w.col0 + 16 * t + lr, Dv - 1));
  };
  auto load_square = [&](int j) __attribute__((always_inline)) {
    const uint16_t* from = k.inner + (w.number + (int64_t)j * heads) * kMatrix;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        square[c][i] = *reinterpret_cast<const s16x8*>(&at_lane(from + (upper_frag(r, max(c, r / 2)) * kPieces + i) * kFragElems, lane * 8));
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    first = *reinterpret_cast<const float4*>(k.decay + (w.number + (int64_t)j * heads) * 2 * kChunk + 16 * r + 4 * lg);
  };
  // do of chunk j times a number per token, zeros past the sequence's end
  auto values = [&](int j, const T (&v)[NT][4], int t, float (&by)[4]) __attribute__((always_inline)) {
    f32x4 x;
    const int n = w.p.len - kChunk * j;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 16 * r + 4 * lg + i < n && w.col0 + 16 * t + lr < Dv ? by[i] * to_f32(v[t][i]) : 0.f;
    return x;
  };
  auto share_do = [&](int j, const T (&v)[NT][4]) __attribute__((always_inline)) {
    float one[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      u32x2 u[N];
      split4<N>(values(j, v, t, one), u);
#pragma unroll
      for (int i = 0; i < N; ++i) L.O[i][t].four(16 * r + 4 * lg, lr) = u[i];
    }
  };
  auto inner_part = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 sum[kPieces];
      clear(sum);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c >= r / 2) {
          s16x8 b[N];
#pragma unroll
          for (int i = 0; i < N; ++i) b[i] = L.O[i][t].eight(c, lane);
          mfma_pieces<kPieces>(square[c], b, sum);
        }
      L.inner(r, t, lane) = total(sum);
    }
  };
  if (w.chunks > 0) {
    load_do(w.chunks - 1, now);
    load_square(w.chunks - 1);
    load_rows(w.chunks - 1);
    load_decay(w.chunks - 1);
    load_do(max(w.chunks - 2, 0), next);
    share_do(w.chunks - 1, now);
  }
  lds_barrier();
  if (w.chunks > 0) {
    inner_part();
    load_square(max(w.chunks - 2, 0));
  }
  lds_barrier();
#pragma unroll 1
  for (int j = w.chunks - 1; j >= 0; --j) {
    const int n = w.p.len - kChunk * j, after = max(j - 1, 0);
    if constexpr (Lds::kStage) {
#pragma unroll
      for (int c = 0; c < KS; ++c) rows[c].put(&L.Q.at[16 * r + lr][32 * c + 8 * lg]);
    }
    {
      float by[4] = {a.scale * first.x, a.scale * first.y, a.scale * first.z, a.scale * first.w};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        u32x2 u[kPieces];
        split4<kPieces>(values(j, now, t, by), u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) L.D[i][t].four(16 * r + 4 * lg, lr) = u[i];
      }
    }
    share_do(after, next);
    lds_barrier();
    load_rows(after);
    load_decay(after);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) now[t][i] = next[t][i];
    load_do(max(j - 2, 0), next);
    // Q^T do'
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f32x4 sum[NT][kPieces];
#pragma unroll
      for (int t = 0; t < NT; ++t) clear(sum[t]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s16x8 e[N];
        if constexpr (Lds::kStage) L.Q.transposed(r * MT + m, c, lane, e);
        else transposed_rows<T>(queries(j), n, Dk, r * MT + m, c, lane, e);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s16x8 b[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i) b[i] = L.D[i][t].eight(c, lane);
          mfma_pieces<kPieces>(e, b, sum[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) L.back[r * MT + m][t][lane] = total(sum[t]);
    }
    lds_barrier();
    inner_part();                    // of the chunk to come; after the first chunk nobody takes it
    load_square(max(j - 2, 0));
    lds_barrier();
  }
}

// Two workgroups a CU where they fit without spills, as in the forward: fp16 keys of 65 .. 128 dimensions would take up to
// 139 registers (4 x 2048 tokens of 16 heads of 100 x 100, the whole gradient: 520 us against 603; of 128 x 128 448 against 480).
template <class Lds, int KP>
constexpr int back_waves() { return KP <= 128 && KP * Lds::N <= 256 ? 4 : 2; }

template <typename T, int KP, int NT, bool WHOLE>
__global__ __launch_bounds__(512, (back_waves<BackLds<T, KP, NT>, KP>())) void delta_back_kernel(DeltaArgs k) {
  typedef BackLds<T, KP, NT> Lds;
  __shared__ __attribute__((aligned(16))) char bytes[sizeof(Lds)];
  Lds& L = *reinterpret_cast<Lds*>(bytes);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  Walk w;
  if (!find_walk<16 * NT>(k, w)) return;
  if (wave < 4) back_chain<T, KP, NT, WHOLE>(k, w, L, wave, lane);
  else back_beside<T, KP, NT, WHOLE>(k, w, L, wave - 4, lane);
}

// ---- queries, keys and decays -----------------------------------------------------------------------------------------
// The same tokens and heads: 229 us, 514 MB read and 75 written, the vector ALU 31 %, LDS 30 % (44 % of it conflicts) and the
// matrix units 18 % busy: one workgroup a CU fits LDS and registers, and loads, pieces and products take turns in it.  The
// panels' loads run one panel ahead where the registers allow it (the whole gradient 431 us against 451).  Measured and
// not kept: 16 waves (270 against 254 us then), two workgroups with 128 registers a lane (spills, 315), panels in the order
// of the reads (no change).
//
// A workgroup has a chunk and a key head, and goes through the value heads that share it.  Four waves have 16 tokens
// each; keys of more than 64 dimensions go to two such sets of waves, half of the dimensions each.  First the products over
// the value's dimension (do S^T, dX S^T, Z dS'^T, do Z^T, dX Z^T), 32 columns of S, dS' and Z at a time as pieces in LDS,
// then those over the chunk's tokens (with E and R, through LDS).
constexpr int kPanelPitch = 40;      // 16-bit elements of an LDS row of 32 columns

template <typename T, int KP>
struct InputGradLds {
  // K and Q lie beside the rest, or in its place after the first products, or nowhere (fp32 keys of 256 dimensions).
  static constexpr bool kBeside = KP <= 128, kStage = kBeside || sizeof(T) == 2;
  struct Keys {
    Staged<T, KP> key, query;
  };
  struct Nothing {};
  struct Panels {
    uint16_t S[kPieces][KP][kPanelPitch], D[kPieces][KP][kPanelPitch], Z[kPieces][kChunk][kPanelPitch];
  };
  struct Squares {
    uint16_t E[kPieces][kChunk][kTokenPitch], R[kPieces][kChunk][kTokenPitch];     // [j][i]
    typename std::conditional<kStage && !kBeside, Keys, Nothing>::type keys;
  };
  union {
    Panels panels;
    Squares squares;
  };
  typename std::conditional<kBeside, Keys, Nothing>::type beside;
  ChunkDecay d;
  float dots[2][kChunk], db[2][kChunk], part[8];
  __device__ __forceinline__ Keys& keys() {
    if constexpr (kBeside) return beside;
    else return squares.keys;
  }
};

template <bool FIRST, class A, class B>
__device__ __forceinline__ auto& pick(A& a, B& b) {
  if constexpr (FIRST) return a;
  else return b;
}

// How the value heads of a key head are gone through: there is one, all in one launch with the sums in registers, or a
// launch each with the sums in the workspace (keys of 256 dimensions leave no registers for them, one head or more).
enum Sharing { kAlone, kTogether, kInTurn };

// WHOLE: Dk is KP and Dv a multiple of 32, so that no load has a branch (8192 tokens of 16 heads of 128 in bf16, the whole
// gradient: 413.8 us against 432.0).  Rows past the chunk's end are then its last one: what they meet is masked or not
// written.

template <typename T, int KP, Sharing SHARING, bool WHOLE>
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
  auto transposed = [&](bool keys, int t, int c, s16x8 (&e)[N]) __attribute__((always_inline)) {
    if constexpr (Lds::kStage) (keys ? L.keys().key : L.keys().query).transposed(tile0 + t, c, lane, e);
    else transposed_rows<T>(keys ? key : query, n, Dk, tile0 + t, c, lane, e);
  };
  // Element (token 16 r + 4 lg + i, column 16 t + lr) of K or Q.
  auto element = [&](bool keys, int t, int i) __attribute__((always_inline)) {
    const int row = opaque(16 * r + 4 * lg) + i, col = 16 * (tile0 + t) + lr;
    float v;
    if constexpr (Lds::kStage) v = to_f32((keys ? L.keys().key : L.keys().query).at[row][col]);
    else v = to_f32((keys ? key : query).at(min(row, n - 1), min(col, Dk - 1)));
    return row < n && col < Dk ? v : 0.f;
  };
  auto stage_keys = [&]() __attribute__((always_inline)) {
    if constexpr (Lds::kStage) {
      const int row = 16 * r + lr;
#pragma unroll
      for (int c = 0; c < KT / 2; ++c) {
        const int col = 16 * tile0 + 32 * c + 8 * lg;
        Eight<T> e, f;
        e.load(&key.at(min(row, n - 1), col), Dk - col);
        f.load(&query.at(min(row, n - 1), col), Dk - col);
        e.put(&L.keys().key.at[row][col]);
        f.put(&L.keys().query.at[row][col]);
      }
    }
  };
  if constexpr (Lds::kBeside) stage_keys();
  for (int h = 0; h < (kHeld ? group : 1); ++h) {
    const int head = kh * group + (SHARING == kInTurn ? k.turn : h);
    lr = opaque(lr);                 // offsets made from these are not kept over the loop, nor from one part to the next
    lg = opaque(lg);
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
    // 32 columns: what this lane brings to the panels, and its own operands.
    constexpr int kRows = KP * 8 / kThreads, kErrors = kChunk * 8 / kThreads;
    constexpr bool kAhead = KP <= 128 && !(kHeld && KP * N > 256);         // the next panel's loads fit the registers
    Raw<float, 4> vS[kRows], vD[kRows], vZ[kErrors];
    Eight<T> vO;
    Eight<float> vX;
    auto load_panel = [&](int c0) __attribute__((always_inline)) {
      const int lane8 = opaque(tid), c = c0 + 4 * (lane8 & 7), left = Dv - c;
      const float* z = k.errors + (row0 * heads + head) * Dv;
      const float* x = k.dx + (row0 * heads + head) * Dv;
      const ChunkRows<const T> dout(k.dout, head * k.dout_head, p, p.t0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = (lane8 + kThreads * i) >> 3;
        if constexpr (WHOLE) {
          vS[i].load(&at_lane(pS, row * Dv + c));
          vD[i].load(&at_lane(pD, row * Dv + c));
        } else {
          vS[i].clear();
          vD[i].clear();
          if (row < Dk && left > 0) {
            vS[i].load_n(&at_lane(pS, row * Dv + c), left);
            vD[i].load_n(&at_lane(pD, row * Dv + c), left);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kErrors; ++i) {
        const int row = (lane8 + kThreads * i) >> 3;
        if constexpr (WHOLE) {
          vZ[i].load(&at_lane(z, min(row, n - 1) * heads * Dv + c));
        } else {
          vZ[i].clear();
          if (row < n && left > 0) vZ[i].load_n(&at_lane(z, row * heads * Dv + c), left);
        }
      }
      const int from = min(mine, n - 1), own = mine < n ? Dv - c0 - 8 * lg : 0;
      if constexpr (WHOLE) {
        vO.raw.load(&dout.at(from, c0 + 8 * lg));
        vX.raw.load(&at_lane(x, from * heads * Dv + c0 + 8 * lg));
      } else {
        vO.load(&dout.at(from, c0 + 8 * lg), own);
        vX.load(&at_lane(x, from * heads * Dv + c0 + 8 * lg), own);
      }
    };
    if (kAhead) load_panel(0);
#pragma unroll 1
    for (int c0 = 0; c0 < Dv; c0 += 32) {
      if (!kAhead) load_panel(c0);
      s16x8 o[N], x[kPieces], z[kPieces];
      vO.pieces(o);
      vX.pieces(x);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = (tid + kThreads * i) >> 3, c = 4 * (tid & 7);
        u32x2 us[kPieces], ud[kPieces];
        split4<kPieces>(f32x4{vS[i].get(0), vS[i].get(1), vS[i].get(2), vS[i].get(3)}, us);
        split4<kPieces>(f32x4{vD[i].get(0), vD[i].get(1), vD[i].get(2), vD[i].get(3)}, ud);
#pragma unroll
        for (int e = 0; e < 4; ++e) inside = __builtin_fmaf(vS[i].get(e), vD[i].get(e), inside);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
          *reinterpret_cast<u32x2*>(&L.panels.S[e][row][c]) = us[e];
          *reinterpret_cast<u32x2*>(&L.panels.D[e][row][c]) = ud[e];
        }
      }
#pragma unroll
      for (int i = 0; i < kErrors; ++i) {
        const int row = (tid + kThreads * i) >> 3, c = 4 * (tid & 7);
        u32x2 u[kPieces];
        split4<kPieces>(f32x4{vZ[i].get(0), vZ[i].get(1), vZ[i].get(2), vZ[i].get(3)}, u);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) *reinterpret_cast<u32x2*>(&L.panels.Z[e][row][c]) = u[e];
      }
      lds_barrier();
      if (kAhead) load_panel(WHOLE ? min(c0 + 32, Dv - 32) : c0 + 32);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) z[e] = lds8(&L.panels.Z[e][mine][8 * lg]);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        s16x8 b[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.S[e][16 * (tile0 + t) + lr][8 * lg]);
        mfma_pieces<kPieces>(o, b, Q[t]);
        mfma_pieces<kPieces>(x, b, R[t]);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.D[e][16 * (tile0 + t) + lr][8 * lg]);
        mfma_pieces<kPieces>(z, b, W[t]);
        if ((t & 1) || KP * N > 256) __builtin_amdgcn_sched_barrier(0);     // operands in registers at a time
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= r) {
          s16x8 b[kPieces];
#pragma unroll
          for (int e = 0; e < kPieces; ++e) b[e] = lds8(&L.panels.Z[e][16 * t + lr][8 * lg]);
          if (part == 0) mfma_pieces<kPieces>(o, b, oz[t]);
          if (part == kParts - 1) mfma_pieces<kPieces>(x, b, xz[t]);
        }
      lds_barrier();
    }
    // E and R (with the sign that R's products have), and the parts that the states give
    lr = opaque(lr);
    lg = opaque(lg);
    auto of_rows = [&](const float (&v)[kChunk]) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4*>(&v[opaque(16 * r + 4 * lg)]);
    };
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
        u32x2 u[kPieces];
        split4<kPieces>(f32x4{w * m[t][0], w * m[t][1], w * m[t][2], w * m[t][3]}, u);
#pragma unroll
        for (int e = 0; e < kPieces; ++e) *reinterpret_cast<u32x2*>(&to[e][j][16 * r + 4 * lg]) = u[e];
      }
    };
    auto share_squares = [&](bool weighted) __attribute__((always_inline)) {
      if (part == 0) share_square(oz, L.squares.E, weighted);
      if (part == kParts - 1) share_square(xz, L.squares.R, weighted);
    };
    share_squares(true);
    if constexpr (Lds::kStage && !Lds::kBeside) stage_keys();
    const f32x4 first = of_rows(L.d.first), last = of_rows(L.d.last);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Q[t][i] *= a.scale * first[i];
        R[t][i] *= -first[i];
        W[t][i] *= last[i];
      }
    __syncthreads();
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
          transposed(true, t, c, b);
          mfma_pieces<kPieces>(e, b, Q[t]);
          mfma_pieces<kPieces>(x, b, R[t]);
          if (!Lds::kStage || KP * N > 256) __builtin_amdgcn_sched_barrier(0);
        }
      }
    __syncthreads();
    share_squares(false);
    // <dS', S'>: e^G_C <dS', S> and what the chunk itself writes, beta k . (e^(G_C - G) Z dS'^T)
    f32x4 beta = of_rows(L.d.beta);
    float tail = L.d.first[kChunk - 1] * inside, dots[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float kv = element(true, t, i), qv = element(false, t, i);
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
          transposed(false, t, c, b);
          mfma_pieces<kPieces>(e, b, W[t]);
          transposed(true, t, c, b);
          mfma_pieces<kPieces>(x, b, W[t]);
          if (!Lds::kStage || KP * N > 256) __builtin_amdgcn_sched_barrier(0);
        }
      }
    beta = of_rows(L.d.beta);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) db[i] = __builtin_fmaf(element(true, t, i), W[t][i], db[i]);
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
            if (SHARING == kInTurn && group > 1) {
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

template <typename T, int KP, bool WHOLE>
hipError_t inputs_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 grid((unsigned)(k.pieces * k.a.key_heads)), block(KP > 64 ? 512 : 256);
  const int group = (int)(k.a.heads / k.a.key_heads);
  if constexpr (KP <= 128) {
    if (group == 1) return launch_kernel(delta_input_grad_kernel<T, KP, kAlone, WHOLE>, grid, block, k, stream);
    return launch_kernel(delta_input_grad_kernel<T, KP, kTogether, WHOLE>, grid, block, k, stream);
  } else {
    DeltaArgs one = k;
    for (one.turn = 0; one.turn < group; ++one.turn) {
      const hipError_t e = launch_kernel(delta_input_grad_kernel<T, KP, kInTurn, WHOLE>, grid, block, one, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
}
template <typename T, int KP>
hipError_t grad_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 order((unsigned)shares(k.a.tokens.sequences * k.a.heads, k.slices));
  const hipError_t err = k.a.key_dim == KP ? launch_kernel(delta_back_kernel<T, KP, 1, true>, order, dim3(512), k, stream)
                                           : launch_kernel(delta_back_kernel<T, KP, 1, false>, order, dim3(512), k, stream);
  if (err != hipSuccess || seq_rows(k.a.tokens) == 0) return err;
  if (k.a.key_dim == KP && k.a.value_dim % 32 == 0) return inputs_n<T, KP, true>(k, stream);
  return inputs_n<T, KP, false>(k, stream);
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
