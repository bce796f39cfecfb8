// What the gated delta rule's kernels share: how tokens are cut, how numbers are held, and what a chunk's decays are.
//
//   S[t] = a S[t-1] + beta k (v - (a S[t-1])^T k)^T,   o[t] = scale S[t]^T q,   a = e^g,   S [Dk, Dv] a head
//
// In a chunk of 64 tokens with G = the running sum of g, e_ij = e^(G_i - G_j), what the tokens write is the solution of
// a unit triangular system:
//
//   M_ij = e_ij (k_i . k_j) beta_j (j < i),  X = V - e^G (K S),  Z = (1 + M)^-1 X  (the errors v - (a S)^T k),
//   O = scale e^G (Q S) + P Z,  P_ij = scale e_ij (q_i . k_j) beta_j (j <= i),
//   S' = e^G_C S + K^T (beta e^(G_C - G) Z).
//
// (1 + M)^-1 and P need no state: one launch makes them for all chunks at once, and only the three products with S and
// Z follow one another from chunk to chunk.  The columns of S (and of V, Z, O) are independent, so a sequence and head
// is shared out over workgroups by columns.
//
// Numbers.  The products run on the bf16 matrix instructions.  A 32-bit number is held as up to three bf16 pieces whose
// sum it is (24 bits), a product of two such numbers is the six products of pieces above 2^-24 of it, all summed in 32
// bits; bf16 inputs are one piece, fp16 ones two (exact).  So states, corrections, outputs and sums keep 32-bit accuracy
// from chunk to chunk at a sixth to a third of the bf16 rate, two and a half to five times the fp32 instructions' rate.
#pragma once

#include "seq_common.h"

namespace cw {

constexpr int kChunkShift = 6, kChunk = 1 << kChunkShift;
constexpr int kPieces = 3;             // of a 32-bit number
constexpr int kFrags = 6;              // 16 x 32 blocks of a triangular 64 x 64 matrix that are not zero
constexpr int kFragElems = 64 * 8;     // of one piece of one block
constexpr int kMatrix = kFrags * kPieces * kFragElems;   // 16-bit elements of such a matrix
constexpr int kTokenPitch = kChunk + 8;                  // 16-bit elements of an LDS row of tokens (input gradients)

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Pieces that hold an element exactly.
template <typename T>
struct ElemPieces {
  static constexpr int n = __is_same(T, Bf16) ? 1 : __is_same(T, F16) ? 2 : kPieces;
};

struct DeltaArgs {
  seq_delta_args_t a;
  SeqMap m;
  int32_t pieces;          // chunks' numbers
  int32_t slices;          // workgroups that share a head's columns
  uint16_t* inverse;       // [pieces][heads][kMatrix]: (1 + M)^-1 (gradient: transposed), blocks in operand order
  uint16_t* inner;         // the same for P
  float* decay;            // [pieces][heads][2][kChunk]: e^G, beta e^(G_C - G)
  float* states;           // [pieces][heads][Dk][Dv]: where each chunk begins, or nullptr
  float* errors;           // [rows][heads][Dv]: Z, or nullptr
  // gradient
  seq_view_t dout;
  int64_t dout_head;
  const float* last;       // gradient of the final states, or nullptr
  float* dstates;          // [pieces][heads][Dk][Dv]: gradient of where each chunk ends
  float* dx;               // [rows][heads][Dv]: gradient of X
  float* sums;             // [2][rows][key_heads][Dk]: dq and dk summed over value heads, where registers do not hold them
  int64_t sums_stride;
  int32_t turn;            // which of a key head's value heads, where each has a launch
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dstate;
};

// ---- pieces ---------------------------------------------------------------------------------------------------------
// Two numbers rounded to bf16 in one instruction.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
// Two numbers as pairs of pieces; what a piece leaves is exact in 32 bits.
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    out[i] = bf16_pair(a, b);
    if (i + 1 < N) {
      a -= __uint_as_float(out[i] << 16);
      b -= __uint_as_float(out[i] & 0xffff0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void split4(f32x4 v, u32x2 (&out)[N]) {
  uint32_t lo[N], hi[N];
  split2<N>(v[0], v[1], lo);
  split2<N>(v[2], v[3], hi);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = u32x2{lo[i], hi[i]};
}
template <int N>
__device__ __forceinline__ void split8(const float (&f)[8], s16x8 (&out)[N]) {
  uint32_t u[4][N];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<N>(f[2 * i], f[2 * i + 1], u[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __builtin_bit_cast(s16x8, uint4{u[0][i], u[1][i], u[2][i], u[3][i]});
}

// Eight elements of a row, and as pieces.
template <typename T>
struct Eight {
  Raw<T, 8> raw;
  __device__ __forceinline__ void load(const T* p, int n) {   // the first n, the others zero
    if (n > 0) raw.load_n(p, n);
    else raw.clear();
  }
  __device__ __forceinline__ void put(T* p) const {           // 16-byte aligned
    *reinterpret_cast<uint4*>(p) = uint4{raw.u[0], raw.u[1], raw.u[2], raw.u[3]};
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(p)[1] = uint4{raw.u[4], raw.u[5], raw.u[6], raw.u[7]};
  }
  __device__ __forceinline__ void pieces(s16x8 (&out)[ElemPieces<T>::n]) const {
    if constexpr (__is_same(T, Bf16)) {
      out[0] = __builtin_bit_cast(s16x8, uint4{raw.u[0], raw.u[1], raw.u[2], raw.u[3]});
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = raw.get(i);
      split8<ElemPieces<T>::n>(f, out);
    }
  }
};

// A chunk of a view: where its first row's head begins, the same in the whole wave, and elements from there, whose offsets
// are 32 bits (rows lie less than 2^24 elements apart).
template <typename T>
struct ChunkRows {
  T* base;
  uint32_t row;
  __device__ __forceinline__ ChunkRows(const seq_view_t& v, int64_t head, const Piece& p, int t0)
      : base(row_at<T>(v, p, t0) + head), row((uint32_t)v.row) {}
  __device__ __forceinline__ T& at(int token, int c) const { return at_lane(base, (int)(token * row + c)); }
};

// ---- matrix instructions ----------------------------------------------------------------------------------------------
// 16 x 16 += 16 x 32 times 32 x 16.  Lane l holds row (column) l % 16 and terms 8 (l / 16) .. + 7 of an operand, column
// l % 16 and rows 4 (l / 16) .. + 3 of the result.
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// The products of pieces above 2^-8N of the whole, each order of magnitude in a sum of its own, so that N chains run.
template <int N, int NA, int NB>
__device__ __forceinline__ void mfma_pieces(const s16x8 (&a)[NA], const s16x8 (&b)[NB], f32x4 (&sum)[N]) {
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i + j < N) sum[i + j] = mfma(a[i], b[j], sum[i + j]);
}
// The same into one sum, where there are enough others to fill the time between two steps of a chain.
template <int N, int NA, int NB>
__device__ __forceinline__ void mfma_pieces(const s16x8 (&a)[NA], const s16x8 (&b)[NB], f32x4& sum) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < N) sum = mfma(a[i], b[j], sum);
}
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
template <int N>
__device__ __forceinline__ void clear(f32x4 (&sum)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = zero4();
}
template <int N>
__device__ __forceinline__ f32x4 total(const f32x4 (&sum)[N]) {
  f32x4 t = sum[N - 1];
#pragma unroll
  for (int i = N - 2; i >= 0; --i) t += sum[i];
  return t;
}

// A second operand of D terms and 16 columns in LDS, in the order that a wave reads it: eight terms of a column, column by
// column.  One read of a wave is 1 KB on end, whatever lanes the LDS serves together.
template <int D>
struct Operand {
  alignas(16) uint16_t at[D / 8][16][8];
  // Four terms from term d on, and a lane's part of terms 32 c ...
  __device__ __forceinline__ u32x2& four(int d, int col) { return *reinterpret_cast<u32x2*>(&at[d >> 3][col][d & 4]); }
  __device__ __forceinline__ s16x8 eight(int c, int lane) const {
    return *reinterpret_cast<const s16x8*>(&at[4 * c + (lane >> 4)][lane & 15][0]);
  }
};

// Eight 16-bit elements of LDS at p; and a transposed operand: terms are LDS rows of `pitch` elements, p is lane's place
// as trans_place gives it.
__device__ __forceinline__ s16x8 lds8(const uint16_t* p) { return *reinterpret_cast<const s16x8*>(p); }
__device__ __forceinline__ int trans_place(int lane, int pitch) {
  return (8 * (lane >> 4) + ((lane & 15) >> 2)) * pitch + 4 * (lane & 3);
}
__device__ __forceinline__ s16x8 lds8_trans(const uint16_t* p, int pitch) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * pitch));
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// K or Q of a chunk in LDS as it lies in memory, a few elements' padding a row.
template <typename T, int KP>
struct Staged {
  static constexpr int kPitch = KP + 16 / (int)sizeof(T);
  alignas(16) T at[kChunk][kPitch];
  // Its transpose as an operand: rows (columns) are dimensions 16 m .., terms are tokens 32 c ...
  __device__ __forceinline__ void transposed(int m, int c, int lane, s16x8 (&e)[ElemPieces<T>::n]) const {
    if constexpr (sizeof(T) == 2) {
      const s16x8 raw = lds8_trans(reinterpret_cast<const uint16_t*>(&at[32 * c][16 * m]) + trans_place(lane, kPitch), kPitch);
      if constexpr (__is_same(T, Bf16)) {
        e[0] = raw;
      } else {
        Eight<T> v;
        __builtin_memcpy(v.raw.u, &raw, sizeof(raw));
        v.pieces(e);
      }
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_f32(at[32 * c + 8 * (lane >> 4) + i][16 * m + (lane & 15)]);
      split8<ElemPieces<T>::n>(f, e);
    }
  }
};
// The same from memory, where the LDS is full; n tokens are the chunk's.
template <typename T>
__device__ __forceinline__ void transposed_rows(const ChunkRows<const T>& from, int n, int Dk, int m, int c, int lane,
                                                s16x8 (&e)[ElemPieces<T>::n]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = opaque(32 * c + 8 * (lane >> 4)) + i, d = 16 * m + (lane & 15);
    f[i] = t < n && d < Dk ? to_f32(from.at(t, d)) : 0.f;
  }
  split8<ElemPieces<T>::n>(f, e);
}

// Block (row tile r of 16, terms 32 s ..) of a lower triangular matrix, and of an upper one.
__host__ __device__ constexpr int lower_frag(int r, int s) { return r < 2 ? r : 2 * r - 2 + s; }
__host__ __device__ constexpr int upper_frag(int r, int s) { return r < 2 ? 2 * r + s : r + 2; }

// ---- decays -----------------------------------------------------------------------------------------------------------
// e^(hi + lo), |lo| far below |hi|; the argument's rounding is put back to first order.
__device__ __forceinline__ float exp_of(float hi, float lo) {
  const float t = hi * kLog2e;
  float r = __builtin_fmaf(hi, kLog2e, -t);
  r = __builtin_fmaf(hi, 1.92596299e-8f, r);     // what kLog2e leaves of log2 e
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, __builtin_fmaf(r, kLn2, lo), e);
}

// A token whose g is below -200 forgets everything in any case (e^-104 is zero in 32 bits), which keeps -inf out of the
// differences.  NaN stays.
__device__ __forceinline__ float log_decay(float g) { return g < -200.f ? -200.f : g; }
// The running sum of g as two floats (48 bits: differences of it are good to 32 bits however far it has run), e^G, e^(G_C
// - G) and beta of a chunk's tokens, zeros behind its end.
struct alignas(16) ChunkDecay {
  float hi[kChunk], lo[kChunk], first[kChunk], last[kChunk], beta[kChunk];
};
// By one wave, lane = token; n of them are the chunk's.
__device__ __forceinline__ void chunk_decay(const seq_delta_args_t& a, const Piece& p, int64_t head, int lane, ChunkDecay& d) {
  const int n = p.end - p.t0;
  float g = 0.f, beta = 0.f;
  if (lane < n) {
    g = log_decay(row_at<const float>(a.g, p, p.t0 + lane)[head]);
    beta = row_at<const float>(a.beta, p, p.t0 + lane)[head];
  }
  double sum = g;
#pragma unroll
  for (int step = 1; step < 64; step *= 2) {
    const double from = __shfl_up(sum, step);
    if (lane >= step) sum += from;
  }
  const double all = __shfl(sum, 63);
  const float hi = (float)sum, lo = (float)(sum - (double)hi);
  const double left = all - sum;
  const float lhi = (float)left;
  d.hi[lane] = hi;
  d.lo[lane] = lo;
  d.beta[lane] = beta;
  d.first[lane] = exp_of(hi, lo);
  d.last[lane] = exp_of(lhi, (float)(left - (double)lhi));
}
__device__ __forceinline__ float decay_between(const ChunkDecay& d, int i, int j) {
  return exp_of(d.hi[i] - d.hi[j], d.lo[i] - d.lo[j]);
}

// ---- places -----------------------------------------------------------------------------------------------------------
__device__ __forceinline__ int64_t chunk_head(const DeltaArgs& k, int piece, int head) {
  return (int64_t)piece * k.a.heads + head;
}
// The number of chunk j of sequence s that begins at row `start`.
__device__ __forceinline__ int chunk_number(const SeqMap& m, int s, int start, int j) {
  return m.offsets ? (start >> kChunkShift) + s + j : s * m.per + j;
}
// Workgroup b of units x slices: a unit's slices on one XCD (workgroup b runs on b % 8), whose L2 holds what they share.
struct Share {
  int unit, slice;
};
__device__ __forceinline__ Share share_of(unsigned b, int slices) {
  const unsigned i = b >> 3;
  return Share{(int)(i / slices * 8 + (b & 7)), (int)(i % slices)};
}
inline int64_t shares(int64_t units, int64_t slices) { return (units + 7) / 8 * 8 * slices; }

// What a workgroup that walks along a sequence has: COLS columns of one head's state.
struct Walk {
  int seq, head, col0, chunks;
  int64_t key_head, number;      // number: chunk_head of the sequence's first chunk
  Piece p;
};
// False for a workgroup past the last one.
template <int COLS>
__device__ __forceinline__ bool find_walk(const DeltaArgs& k, Walk& w) {
  const int heads = (int)k.a.heads;
  const Share share = share_of(blockIdx.x, k.slices);
  if (share.unit >= k.m.S * heads) return false;
  w.seq = uniform(share.unit / heads);
  w.head = uniform(share.unit % heads);
  w.col0 = share.slice * COLS;
  w.key_head = w.head / (heads / (int)k.a.key_heads);
  w.p.seq = w.seq;
  if (k.m.offsets) {
    const int start = uniform(seq_start(k.m, w.seq)), stop = uniform(seq_start(k.m, w.seq + 1));
    w.p.batch = 0;
    w.p.first = start;
    w.p.len = max(stop - start, 0);
  } else {
    w.p.batch = w.seq;
    w.p.first = 0;
    w.p.len = k.m.rows;
  }
  w.chunks = (w.p.len + kChunk - 1) >> kChunkShift;
  w.number = chunk_head(k, chunk_number(k.m, w.seq, (int)w.p.first, 0), w.head);
  return true;
}

// A wave's 16 rows of K or Q in a chunk as loaded, lane by lane: row 16 r + l % 16, dimensions 32 c + 8 (l / 16) .. + 7.
// Rows past the sequence's end are its last one: what they meet is zero or thrown away.  WHOLE: Dk is KP.
template <typename T, int KP, bool WHOLE>
__device__ __forceinline__ void load_row(const ChunkRows<const T>& from, int n, int row, int lg, int Dk, int c, Eight<T>& to) {
  const int d = 32 * c + 8 * lg;
  if constexpr (WHOLE) to.raw.load(&from.at(min(row, n - 1), d));
  else to.load(&from.at(min(row, n - 1), d), Dk - d);
}

DeltaArgs delta_args(const seq_delta_args_t& a, float* ws);
hipError_t launch_delta_chunks(const DeltaArgs& k, bool gradient, hipStream_t stream);

}  // namespace cw
