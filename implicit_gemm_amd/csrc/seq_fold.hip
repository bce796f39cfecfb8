// Fixed-order sums of partial results: the last step of every gradient that is summed over tokens or channel blocks.
// out[e] = sum_p part[p][e].  A workgroup of kCols x kGroups lanes owns kCols outputs; group g sums the partials g,
// g + kGroups, ... with eight loads in flight, and the group sums are added in order through LDS.  Few partials
// (<= 64) take 64 columns x 4 groups, or 256 x 4 beside a fold of many in the same launch; many take 32 x 32: the longest
// chain of dependent loads stays at a few.
#include "seq_common.h"

namespace cw {

namespace {

struct FoldArgs {
  FoldList l;
  int32_t first[6];   // first workgroup of each fold
};

template <int kCols, int kGroups>
__device__ __forceinline__ void fold(const FoldPart& f, int block, float* lds) {
  const int c = threadIdx.x % kCols, g = threadIdx.x / kCols;
  const int64_t e = (int64_t)block * kCols + c;
  float acc = 0.f;
  if (e < f.E && g < kGroups) {
    const float* s = f.part + e;
    int p = g;
    for (; p + 7 * kGroups < f.count; p += 8 * kGroups) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s[(int64_t)(p + i * kGroups) * f.stride];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += v[i];
    }
    for (; p < f.count; p += kGroups) acc += s[(int64_t)p * f.stride];
  }
  if (g < kGroups) lds[g * kCols + c] = acc;
  __syncthreads();
  if (g == 0 && e < f.E) {
    float r = lds[c];
    for (int i = 1; i < kGroups; ++i) r += lds[i * kCols + c];
    if (f.dtype == CONV_WGRAD_F32) static_cast<float*>(f.out)[e] = r;
    else if (f.dtype == CONV_WGRAD_BF16) from_f32(r, static_cast<Bf16*>(f.out)[e]);
    else from_f32(r, static_cast<F16*>(f.out)[e]);
  }
}

constexpr int kFewMax = 64;

template <int kThreads>
__global__ __launch_bounds__(kThreads) void seq_fold_kernel(FoldArgs a) {
  __shared__ float lds[kThreads];
  int k = 0;
  while (k + 1 < a.l.n && (int)blockIdx.x >= a.first[k + 1]) ++k;
  const int block = (int)blockIdx.x - a.first[k];
  if constexpr (kThreads == 256) fold<64, 4>(a.l.f[k], block, lds);
  else if (a.l.f[k].count <= kFewMax) fold<256, 4>(a.l.f[k], block, lds);
  else fold<32, 32>(a.l.f[k], block, lds);
}

}  // namespace

namespace {

bool all_few(const FoldList& list) {
  for (int i = 0; i < list.n; ++i)
    if (list.f[i].count > kFewMax) return false;
  return true;
}

// Workgroups of fold i.
int64_t fold_blocks(const FoldList& list, int i, bool few) {
  const int cols = few ? 64 : list.f[i].count <= kFewMax ? 256 : 32;
  return (list.f[i].E + cols - 1) / cols;
}

}  // namespace

int64_t fold_lanes(const FoldList& list) {
  const bool few = all_few(list);
  int64_t blocks = 0;
  for (int i = 0; i < list.n; ++i) blocks += fold_blocks(list, i, few);
  return blocks * (few ? 256 : 1024);
}

hipError_t launch_seq_fold(const FoldList& list, hipStream_t stream) {
  FoldArgs a;
  a.l = list;
  const bool few = all_few(list);
  int64_t blocks = 0;
  for (int i = 0; i < list.n; ++i) {
    a.first[i] = (int32_t)blocks;
    blocks += fold_blocks(list, i, few);
  }
  if (blocks == 0) return hipSuccess;
  if (few) return launch_kernel(seq_fold_kernel<256>, dim3((unsigned)blocks), dim3(256), a, stream);
  return launch_kernel(seq_fold_kernel<1024>, dim3((unsigned)blocks), dim3(1024), a, stream);
}

}  // namespace cw
