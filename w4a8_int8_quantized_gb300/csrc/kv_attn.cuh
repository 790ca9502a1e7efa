// The cache attention kernels' common end: a row's sums to its output.
#pragma once

#include <math_constants.h>

#include "kv_common.cuh"

namespace w8a8 {

// Four elements d .. d + 3 of a row from its unnormalised sums x and its sum
// of weights l, both against reference m (base 2).
template <int D>
__device__ __forceinline__ void store_row4(const KvAttnParams &p, long long row, int d, float4 x,
                                           float m, float l) {
  const float r = l == 0.f ? 0.f : 1.f / l;
  const __half2 a = __floats2half2_rn(x.x * r, x.y * r), b = __floats2half2_rn(x.z * r, x.w * r);
  uint2 o;
  o.x = *reinterpret_cast<const uint32_t *>(&a);
  o.y = *reinterpret_cast<const uint32_t *>(&b);
  *reinterpret_cast<uint2 *>(p.out + row * D + d) = o;
  if (d == 0 && p.lse != nullptr)
    p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// Rows per kv head and sequence up to which the few-row kernel runs, else the
// tensor-memory one.
constexpr int kFewRows = 64;

size_t kv_decode_workspace(int D, long long rows);
int launch_kv_decode(const KvAttnParams &p, int bits, int D, cudaStream_t s);
size_t kv_prefill_workspace(int D);
int launch_kv_prefill(const KvAttnParams &p, int bits, int D, cudaStream_t s);

}  // namespace w8a8
