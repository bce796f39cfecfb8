// The gated delta rule forward (gfx950): the triangular systems of all chunks, the chunks of each sequence in order, and
// the single token.  seq_delta.h has the formulas.
#include "seq_delta.h"

namespace cw {

namespace {

// ---- the chunks' systems ----------------------------------------------------------------------------------------------
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

template <typename T, bool GRAD>
__global__ __launch_bounds__(256) void delta_chunk_kernel(DeltaArgs k) {
  constexpr int N = ElemPieces<T>::n;
  __shared__ __attribute__((aligned(16))) float M[kChunk][kSquarePitch], P[kChunk][kSquarePitch], I[kChunk][kSquarePitch];
  __shared__ ChunkDecay d;
  const seq_delta_args_t& a = k.a;
  const int lane = threadIdx.x & 63, r = uniform(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4;
  const int heads = (int)a.heads, piece = blockIdx.x / heads, head = blockIdx.x % heads;
  Piece p;
  if (!find_piece(k.m, piece, p)) return;
  if (p.seq == k.m.S) {            // padding behind the last sequence
    if constexpr (!GRAD) {
      const int Dv = a.value_dim;
      for (int i = threadIdx.x; i < (p.end - p.t0) * Dv; i += 256)
        from_f32(0.f, row_at<T>(a.o, p, p.t0 + i / Dv)[(int64_t)head * Dv + i % Dv]);
    }
    return;
  }
  const int n = p.end - p.t0, Dk = a.key_dim;
  if (n <= 0) return;                // an empty sequence has a number too
  const int64_t at = chunk_head(k, piece, head);
  if (r == 0) {
    chunk_decay(a, p, head, lane, d);
    k.decay[at * 2 * kChunk + lane] = d.first[lane];
    k.decay[(at * 2 + 1) * kChunk + lane] = d.last[lane] * d.beta[lane];
  }
  const int64_t kh = head / (heads / (int)a.key_heads);
  const int row = 16 * r + lr;
  // Rows past the chunk's end read its last one: what they give is multiplied by zero or thrown away below.
  const ChunkRows<const T> key(a.k, kh * a.k_head, p, p.t0), query(a.q, kh * a.q_head, p, p.t0);
  f32x4 kk[4][2], qk[4][2];
#pragma unroll
  for (int t = 0; t < 4; ++t) kk[t][0] = kk[t][1] = qk[t][0] = qk[t][1] = zero4();
  for (int c = 8 * lg; c - 8 * lg < Dk; c += 32) {
    Eight<T> e;
    s16x8 ka[N], qa[N];
    e.load(&key.at(min(row, n - 1), c), Dk - c);
    e.pieces(ka);
    e.load(&query.at(min(row, n - 1), c), Dk - c);
    e.pieces(qa);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t <= r) {
        s16x8 kb[N];
        e.load(&key.at(min(16 * t + lr, n - 1), c), Dk - c);
        e.pieces(kb);
        mfma_pieces<kPieces>(ka, kb, kk[t][0], kk[t][1]);
        mfma_pieces<kPieces>(qa, kb, qk[t][0], qk[t][1]);
      }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int j = 16 * t + lr;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = 16 * r + 4 * lg + x;
      const bool live = i < n && j <= i;
      const float e = live ? decay_between(d, i, j) * d.beta[j] : 0.f;
      M[i][j] = live && j < i ? e * (kk[t][0][x] + kk[t][1][x]) : 0.f;
      P[i][j] = live ? e * (qk[t][0][x] + qk[t][1][x]) * a.scale : 0.f;
      I[i][j] = 0.f;
    }
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
    f32x4 y = block_product(M, 32 + u, 0, I, 0, v, lane, zero4());
    y = block_product(M, 32 + u, 16, I, 16, v, lane, y);
    block_store(M, u, 32 + v, lane, y, 1.f);
    __syncthreads();
    f32x4 z = block_product(I, 32 + u, 32, M, 0, 32 + v, lane, zero4());
    z = block_product(I, 32 + u, 48, M, 16, 32 + v, lane, z);
    block_store(I, 32 + u, v, lane, z, -1.f);
  }
  __syncthreads();
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
      fp[i] = GRAD ? P[c][row] : P[row][c];
    }
    s16x8 pi[kPieces], pp[kPieces];
    split8<kPieces>(fi, pi);
    split8<kPieces>(fp, pp);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      *reinterpret_cast<s16x8*>(inv + (b * kPieces + i) * kFragElems + lane * 8) = pi[i];
      *reinterpret_cast<s16x8*>(inn + (b * kPieces + i) * kFragElems + lane * 8) = pp[i];
    }
  }
}

// ---- the chunks of a sequence in order ------------------------------------------------------------------------------
// A workgroup has 16 NT columns of one sequence's and head's state.  Waves 0 .. 3 walk the chain: wave r has the
// chunk's tokens 16 r .. and the state's rows r KP / 4 .., in registers; the state's pieces go to all waves through LDS.
// Waves 4 .. 7 make the outputs of the same tokens beside them.  Three exchanges a chunk: the state, X, and Z; global
// loads are one chunk ahead.
template <typename T, int KP, int NT, bool SAVE>
__global__ __launch_bounds__(512) void delta_kernel(DeltaArgs k) {
  constexpr int N = ElemPieces<T>::n, NO = OutPieces<T>::n, KS = KP / 32, MT = KP / 64;
  constexpr int kKeyPitch = KP + 8;
  constexpr bool kStage = N == 1 || KP <= 128;     // K's pieces fit the LDS beside the rest
  constexpr int kCols = 16 * NT;
  constexpr bool kAhead = N == 1 || KP <= 128;     // K's and Q's rows of the next chunk fit the registers
  __shared__ __attribute__((aligned(16))) uint16_t sS[kPieces][kCols][kKeyPitch], sX[kPieces][kCols][kTokenPitch],
      sW[kPieces][kCols][kTokenPitch], sZ[NO][kCols][kTokenPitch], sK[kStage ? N : 1][kStage ? kChunk : 1][kKeyPitch];
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
  const int64_t slot = pool_slot(a.tokens.slots, a.tokens.pool, s);

  // ---- the state
  f32x4 S[MT][NT];
  const int64_t place = (int64_t)head * Dk * Dv;
  if (chain) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = col0 + 16 * t + lr;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 16 * (r * MT + m) + 4 * lg + x;
          S[m][t][x] = a.state && slot >= 0 && row < Dk && c < Dv ? a.state[slot * a.state_stride + place + (int64_t)row * Dv + c] : 0.f;
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

  // ---- what is loaded a chunk ahead
  Eight<T> rows[kAhead ? KS : 1];                 // chain: K, outputs: Q
  T v[NT][4];                        // chain: V
  s16x8 square[2][kPieces];          // chain: (1 + M)^-1, outputs: P
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
  auto load_values = [&](int j) __attribute__((always_inline)) {
    const int n = p.len - kChunk * j;
    const ChunkRows<const T> from(a.v, head * a.v_head, p, kChunk * j);
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
      if (c <= r / 2) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (i < (NO > 2 ? kPieces : 2) || chain)
            square[c][i] = *reinterpret_cast<const s16x8*>(from + (lower_frag(r, c) * kPieces + i) * kFragElems);
      }
  };
  auto load_decay = [&](int j) __attribute__((always_inline)) {
    const float* from = k.decay + (number + (int64_t)j * heads) * 2 * kChunk;
    first = *reinterpret_cast<const float4*>(from + 16 * r + 4 * lg);
    last = *reinterpret_cast<const float4*>(from + kChunk + 16 * r + 4 * lg);
    whole = from[kChunk - 1];
  };
  if (chunks > 0) {
    load_rows(0);
    if (chain) load_values(0);
    load_square(0);
    load_decay(0);
  }
  if (chain) share_state();
  lds_barrier();

  for (int j = 0; j < chunks; ++j) {
    const int n = p.len - kChunk * j;      // tokens that are left
    const bool more = j + 1 < chunks;
    const float f[4] = {first.x, first.y, first.z, first.w}, l[4] = {last.x, last.y, last.z, last.w};
    const float keep = whole;
    f32x4 lead[NT], rest[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) lead[t] = rest[t] = zero4();
    // K S or Q S
    if (SAVE && chain) keep_state(k.states + (number + (int64_t)j * heads) * Dk * Dv);
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      s16x8 e[N];
      row_pieces(j, c, e);
      if (kStage && chain) {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<s16x8*>(&sK[i][kStage ? 16 * r + lr : 0][32 * c + 8 * lg]) = e[i];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s16x8 b[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (chain || i < NO) b[i] = lds8(&sS[i][16 * t + lr][32 * c + 8 * lg]);
        if (chain) mfma_pieces<kPieces>(e, b, lead[t], rest[t]);
        else mfma_pieces<NO>(e, b, lead[t], rest[t]);
      }
    }
    if (more) load_rows(j + 1);
    if (chain) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 x;
        uint2 u[kPieces];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __builtin_fmaf(-f[i], lead[t][i] + rest[t][i], to_f32(v[t][i]));
        split4<kPieces>(x, u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint2*>(&sX[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
      }
      if (more) load_values(j + 1);
    }
    lds_barrier();
    if (chain) {
      // Z
      f32x4 z[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        lead[t] = rest[t] = zero4();
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c <= r / 2) {
            s16x8 b[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) b[i] = lds8(&sX[i][16 * t + lr][32 * c + 8 * lg]);
            mfma_pieces<kPieces>(square[c], b, lead[t], rest[t]);
          }
        z[t] = lead[t] + rest[t];
        uint2 u[kPieces], w[kPieces];
        split4<kPieces>(z[t], u);
#pragma unroll
        for (int i = 0; i < NO; ++i) *reinterpret_cast<uint2*>(&sZ[i][16 * t + lr][16 * r + 4 * lg]) = u[i];
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = l[i] * z[t][i];
        split4<kPieces>(x, w);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint2*>(&sW[i][16 * t + lr][16 * r + 4 * lg]) = w[i];
      }
      if (SAVE) {
        float* to = k.errors + ((p.batch * k.m.rows + p.first + kChunk * j) * heads + head) * Dv + col0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * r + 4 * lg + i;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (t < n && col0 + 16 * c + lr < Dv) at_lane(to, t * heads * Dv + 16 * c + lr) = z[c][i];
        }
      }
      if (more) {
        load_square(j + 1);
        load_decay(j + 1);
      }
    }
    lds_barrier();
    if (chain) {
      // S' = e^G_C S + K^T W
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 low[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          low[t] = zero4();
#pragma unroll
          for (int x = 0; x < 4; ++x) S[m][t][x] *= keep;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s16x8 e[N];
          if constexpr (kStage) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              e[i] = lds8_trans(&sK[i][32 * c][16 * (r * MT + m)] + trans_place(lane, kKeyPitch), kKeyPitch);
          } else {
            const ChunkRows<const T> key(a.k, kh * a.k_head, p, kChunk * j);
            float g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int t = opaque(32 * c + 8 * lg) + i, row = 16 * (r * MT + m) + lr;
              g[i] = t < n && row < Dk ? to_f32(key.at(t, row)) : 0.f;
            }
            split8<N>(g, e);
          }
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
    } else {
      // O
      const ChunkRows<T> out(a.o, (int64_t)head * Dv, p, kChunk * j);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 o, low = zero4();
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a.scale * f[i] * (lead[t][i] + rest[t][i]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c <= r / 2) {
            s16x8 b[NO];
#pragma unroll
            for (int i = 0; i < NO; ++i) b[i] = lds8(&sZ[i][16 * t + lr][32 * c + 8 * lg]);
            mfma_pieces<NO>(square[c], b, o, low);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * r + 4 * lg + i, col = col0 + 16 * t + lr;
          if (row < n && col < Dv) from_f32(o[i] + low[i], out.at(row, col));
        }
      }
      if (more) {
        load_square(j + 1);
        load_decay(j + 1);
      }
    }
    lds_barrier();
  }
  if (chain && a.state_out && slot >= 0) keep_state(a.state_out + slot * a.state_out_stride + place);
}

// ---- one token ----------------------------------------------------------------------------------------------------------
// A workgroup has one sequence's head and up to 128 columns of its state, four to a lane; its 256 lanes are 32 / (columns
// / 4) .. groups that share the state's rows.  The state is read once, held in registers between the two sums over its
// rows, and written once.
template <typename T, int LANES, int ROWS>
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
    if (a.state && slot >= 0 && row < Dk && left > 0)
      S[i].load_n(a.state + slot * a.state_stride + place + (int64_t)row * Dv, left);
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
    if (a.state_out && slot >= 0 && row < Dk && left > 0)
      S[i].store_n(a.state_out + slot * a.state_out_stride + place + (int64_t)row * Dv, left);
  }
  over_rows(query, o);
  if (g == 0) {
    T* to = row_at<T>(a.o, p, 0) + (int64_t)head * Dv + col0 + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) from_f32(o[e], to[e]);
  }
}

template <typename T>
hipError_t step_t(const DeltaArgs& k, hipStream_t stream) {
  const dim3 grid((unsigned)(k.a.tokens.sequences * k.a.heads * k.slices)), block(256);
  // 32 lanes x 4 columns, 8 groups
  if (k.a.key_dim <= 64) return launch_kernel(delta_step_kernel<T, 32, 8>, grid, block, k, stream);
  if (k.a.key_dim <= 128) return launch_kernel(delta_step_kernel<T, 32, 16>, grid, block, k, stream);
  return launch_kernel(delta_step_kernel<T, 32, 32>, grid, block, k, stream);
}

template <typename T, int KP, int NT>
hipError_t delta_n(const DeltaArgs& k, hipStream_t stream) {
  const dim3 grid((unsigned)shares(k.a.tokens.sequences * k.a.heads, k.slices)), block(512);
  if (k.states) return launch_kernel(delta_kernel<T, KP, NT, true>, grid, block, k, stream);
  return launch_kernel(delta_kernel<T, KP, NT, false>, grid, block, k, stream);
}
template <typename T>
hipError_t delta_t(const DeltaArgs& k, hipStream_t stream) {
  if (k.a.key_dim <= 64) return delta_n<T, 64, 1>(k, stream);
  if (k.a.key_dim <= 128) return delta_n<T, 128, 1>(k, stream);
  return delta_n<T, 256, 1>(k, stream);
}

template <typename T>
hipError_t chunks_t(const DeltaArgs& k, bool gradient, hipStream_t stream) {
  const dim3 grid((unsigned)(k.pieces * k.a.heads)), block(256);
  if (gradient) return launch_kernel(delta_chunk_kernel<T, true>, grid, block, k, stream);
  return launch_kernel(delta_chunk_kernel<T, false>, grid, block, k, stream);
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
