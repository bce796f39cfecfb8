// Device helpers of the sequence operators (norm, short causal convolution, selective scan).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "seq.h"

namespace cw {

// ---- elements -----------------------------------------------------------------------------------------------------
// Round to nearest even; NaN stays NaN (gfx950 converts bf16 in one instruction).
__device__ __forceinline__ void from_f32(float v, float& out) { out = v; }
__device__ __forceinline__ void from_f32(float v, Bf16& out) { out.bits = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void from_f32(float v, F16& out) { out.v = (_Float16)v; }

// V consecutive elements as they lie in memory.  The copy claims the element's alignment only: gfx950 loads and stores
// up to 16 bytes at any element-aligned global address in one instruction, so odd strides need no form of their own.
// They are held as 32-bit words (two 16-bit elements in one register) until get() widens one.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  static_assert(V * sizeof(T) % 4 == 0, "whole words");
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(u, p, sizeof(u)); }
  __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, u, sizeof(u)); }
  // The first n >= 1 elements, the others zero.
  __device__ __forceinline__ void load_n(const T* p, int n) {
    if (n >= V) {
      load(p);
    } else {
      clear();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(p[i]);
          else u[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i & 1));
        }
    }
  }
  __device__ __forceinline__ void store_n(T* p, int n) const {
    if (n >= V) {
      store(p);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 4) p[i] = __uint_as_float(u[i]);
          else p[i] = __builtin_bit_cast(T, (uint16_t)(u[i / 2] >> (16 * (i & 1))));
        }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else if constexpr (__is_same(T, Bf16)) return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)(u[i / 2] >> (16 * (i & 1))));
  }
  __device__ __forceinline__ void pack(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        u[i] = __float_as_uint(f[i]);
      } else {
        T lo, hi;
        from_f32(f[2 * i], lo);
        from_f32(f[2 * i + 1], hi);
        u[i] = __builtin_bit_cast(uint16_t, lo) | (uint32_t)__builtin_bit_cast(uint16_t, hi) << 16;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = 0;
  }
};

// ---- functions ----------------------------------------------------------------------------------------------------
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// 1 / (1 + e^-v).  The exponential's argument is rounded once, which costs |v| 2^-24 of it: at v = -8 half a millionth
// of a value of 3e-4.  NaN stays, infinities give 0 and 1.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e));
}
// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1].  log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3; unlike
// log(1 + e) this keeps the leading bits for small e.  atanh(s) / s is a polynomial in s^2, fitted for the least
// relative error on [0, 1/9]: 8e-9 with these fp32 coefficients.  e itself is 2^t with the rounding error of t = -|v|
// log2 e put back to first order, as every step of a sequence multiplies by it.
__device__ __forceinline__ float softplus(float v) {
  const float a = __builtin_amdgcn_fmed3f(-fabsf(v), -100.f, 0.f);
  const float t = a * kLog2e;
  const float r = __builtin_fmaf(a, kLog2e, -t) * kLn2;
  float e = __builtin_amdgcn_exp2f(t);
  e = __builtin_fmaf(e, r, e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = 0.14089183509349823f;
  p = __builtin_fmaf(p, q, 0.1398029774427414f);
  p = __builtin_fmaf(p, q, 0.2001245617866516f);
  p = __builtin_fmaf(p, q, 0.3333315849304199f);
  p = __builtin_fmaf(p, q, 1.f);
  return __builtin_fmaf(s + s, p, v < 0.f ? 0.f : v);
}

// ---- lanes --------------------------------------------------------------------------------------------------------
// The value of the lane that DPP pattern kCtrl names.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

struct AddOp {
  __device__ __forceinline__ static float of(float a, float b) { return a + b; }
};
// Larger of two non-negative values; NaN, whose bits lie above infinity's, wins.
struct MaxBitsOp {
  __device__ __forceinline__ static float of(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  }
};
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
// Combines the values of n consecutive lanes (n a power of two, 1 .. 64, the same in all lanes); every lane gets the
// result.  Lanes 1 and 2 apart are swapped inside a quad; quads and rows are mirrored, which is enough as all lanes of
// a quad (half row) are equal by then; rows and halves are exchanged by the lane swaps of gfx950.
template <class Op>
__device__ __forceinline__ float lanes_reduce(float v, int n) {
  if (n > 1) v = Op::of(v, dpp<kXor1>(v));
  if (n > 2) v = Op::of(v, dpp<kXor2>(v));
  if (n > 4) v = Op::of(v, dpp<kHalfMirror>(v));
  if (n > 8) v = Op::of(v, dpp<kMirror>(v));
  if (n > 16) {
    const unsigned u = __float_as_uint(v);
    const u32x2 p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = Op::of(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if (n > 32) {
    const unsigned u = __float_as_uint(v);
    const u32x2 p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = Op::of(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}

// Combines the values of a team of TEAM lanes (16 or 64: part of a wave or a whole one; more: the waves of a workgroup,
// all of which call it, with TEAM / 64 floats of lds).
template <class Op, int TEAM>
__device__ __forceinline__ float team_reduce(float v, float* lds) {
  v = lanes_reduce<Op>(v, TEAM < 64 ? TEAM : 64);
  if constexpr (TEAM > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the last reduction's reads are done
    if ((threadIdx.x & 63) == 0) lds[w] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < TEAM / 64; ++i) v = Op::of(v, lds[i]);
  }
  return v;
}

// An integer that the compiler cannot see through: keeps what is computed from it inside of a loop.
__device__ __forceinline__ int opaque(int v) {
  asm("" : "+v"(v));
  return v;
}

// Orders a wave's LDS accesses before and after it.  The LDS serves one wave's accesses in order, so this costs nothing.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- sequences ----------------------------------------------------------------------------------------------------
// The tokens are cut into pieces of 2^shift tokens, no piece holding two sequences.  Equal lengths: `per` pieces each.
// Packed rows: piece j of sequence s is piece (offsets[s] >> shift) + s + j; as (o + n >> shift) + 1 >= (o >> shift) +
// ceil(n / 2^shift), no two sequences meet in one piece, and no prefix sum over the lengths is needed.  Rows past the
// last sequence are those of one more "sequence" S, which has no state.  An empty sequence still has its piece j = 0.
struct Piece {
  int seq;         // S: rows past the last sequence
  int64_t batch;   // index along the batch stride
  int64_t first;   // row of the sequence's first token
  int len;         // tokens of the sequence
  int t0;          // first token of the piece
  int end;         // one past its last token
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Where sequence s of packed rows begins; any offsets give a row in [0, rows].
__device__ __forceinline__ int seq_start(const SeqMap& m, int s) {
  return min(max(m.offsets[s], 0), m.rows);
}

// Finds a piece; false for a number that names none.  All 64 lanes of the wave call it with the same number.
__device__ __forceinline__ bool find_piece(const SeqMap& m, int piece, Piece& p) {
  int j;
  if (m.offsets == nullptr) {
    p.seq = uniform(piece / m.per);
    if (p.seq >= m.S) return false;
    j = piece - p.seq * m.per;
    p.batch = p.seq;
    p.first = 0;
    p.len = m.rows;
  } else {
    // The last s with seq_base(s) <= piece among 0 .. S, 64 candidates at a time; where it begins and ends is with the
    // last round's lanes, unless the next sequence is beyond them.
    const int lane = threadIdx.x & 63;
    int lo = 0, n = m.S + 1, step, cnt, v, had;
    do {
      had = n;
      step = (n + 63) >> 6;
      v = lane * step < n ? seq_start(m, lo + lane * step) : 0;
      cnt = __popcll(__ballot(lane * step < n && (v >> m.shift) + lo + lane * step <= piece));
      if (cnt == 0) return false;
      lo = uniform(lo + (cnt - 1) * step);
      n = uniform(min(step, n - (cnt - 1) * step));
    } while (n > 1);
    const int start = __builtin_amdgcn_readlane(v, cnt - 1);
    int stop = m.rows;
    if (lo < m.S)
      stop = step == 1 && cnt < min(had, 64) ? __builtin_amdgcn_readlane(v, cnt) : uniform(seq_start(m, lo + 1));
    p.seq = lo;
    p.batch = 0;
    p.first = start;
    p.len = max(stop - start, 0);
    j = piece - ((start >> m.shift) + lo);
  }
  if (j < 0 || (j > 0 && ((int64_t)j << m.shift) >= p.len)) return false;
  p.t0 = j << m.shift;
  p.end = min(p.len, p.t0 + (1 << m.shift));
  return true;
}

// The state that sequence s has in its pool, or -1: none (a slot outside the pool marks a row of padding).
__device__ __forceinline__ int64_t pool_slot(const int32_t* slots, int64_t pool, int s) {
  if (slots == nullptr) return s;
  const int v = uniform(slots[s]);
  return v >= 0 && v < pool ? v : -1;
}

// Element `c` of a row: the row's address is the same in the whole wave, so the lane's part is a 32-bit offset.
template <typename T>
__device__ __forceinline__ T& at_lane(T* row, int c) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
  return *reinterpret_cast<T*>(reinterpret_cast<Byte*>(row) + (uint32_t)c * (uint32_t)sizeof(T));
}
// The same for one element, with the row's address held to scalar registers: the compiler would rather add it to the
// lane's part, a 64-bit vector addition a row.
template <typename T>
struct Bits {
  typedef typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type Word;
  typedef __attribute__((address_space(1))) Word Global;
};
__device__ __forceinline__ uint64_t scalar_address(const void* row) {
  uint64_t b = reinterpret_cast<uint64_t>(row);
  asm("" : "+s"(b));
  return b;
}
template <typename T>
__device__ __forceinline__ T load_lane(const T* row, int c) {
  typedef const typename Bits<T>::Global G;
  return __builtin_bit_cast(T, (typename Bits<T>::Word)*(G*)(scalar_address(row) + (uint32_t)c * (uint32_t)sizeof(T)));
}
template <typename T>
__device__ __forceinline__ void store_lane(T* row, int c, T v) {
  typedef typename Bits<T>::Global G;
  *(G*)(scalar_address(row) + (uint32_t)c * (uint32_t)sizeof(T)) = __builtin_bit_cast(typename Bits<T>::Word, v);
}

template <typename T>
__device__ __forceinline__ T* row_at(const seq_view_t& v, const Piece& p, int64_t t) {
  return static_cast<T*>(v.ptr) + p.batch * v.batch + (p.first + t) * v.row;
}

}  // namespace cw
