// The cache attention kernels' common end: a row's sums to its output.
#pragma once

#include <math_constants.h>

#include "kv_common.cuh"

namespace w8a8 {

// Two outputs as fp16.  They are averages of values of at most 65504, which the weights'
// rounding to fp16 may take past 65520, where a plain rounding gives infinity: the largest
// finite value stands for those.  NaN stays NaN.
__device__ __forceinline__ uint32_t output2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Four elements d .. d + 3 of a row from its unnormalised sums x and its sum
// of weights l, both against reference m (base 2).
template <int D>
__device__ __forceinline__ void store_row4(const KvAttnParams &p, long long row, int d, float4 x,
                                           float m, float l) {
  const float r = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2 *>(p.out + row * D + d) = make_uint2(output2(x.x * r, x.y * r), output2(x.z * r, x.w * r));
  if (d == 0 && p.lse != nullptr)
    p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// Rows that no sequence owns: before the first, after the last (padding of a batch, say),
// and beyond max_q queries of one (reported).
__device__ __forceinline__ int offset_of(const int *q_offsets, int T, long long b) {
  return min(max(__ldg(q_offsets + b), 0), T);
}
// Whether there are any, as far as this thread's share of the sequences tells.  Asked after
// the offsets were read for the ranges, from L1 then: at the kernel's start it cost a
// round trip to L2, 0.5 us.
__device__ __forceinline__ bool some_unowned(const KvAttnParams &p) {
  if (p.q_offsets == nullptr) return false;
  bool any = offset_of(p.q_offsets, p.T, 0) > 0 || offset_of(p.q_offsets, p.T, p.B) < p.T;
  for (long long b = blockIdx.x + static_cast<long long>(threadIdx.x) * gridDim.x; b < p.B;
       b += static_cast<long long>(gridDim.x) * blockDim.x)
    any |= offset_of(p.q_offsets, p.T, b + 1) - offset_of(p.q_offsets, p.T, b) > p.max_q;
  return any;
}
// They get 0 and -inf, by the warps in which some thread found any: all threads, who all
// see them, share the rows before and after; a sequence's are the warp's that looked at
// it.  (A call with few arguments: inlined, it spilled in the many-row kernel.)
template <int D>
__device__ __noinline__ void blank_unowned(__half *out, float *lse, const int *q_offsets, int T, int Hq, int B,
                                           int max_q) {
  auto blank = [&](long long r0, long long r1, long long at, long long step) {
#pragma unroll 1
    for (long long i = r0 * Hq * (D / 8) + at; i < r1 * Hq * (D / 8); i += step)
      reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (long long i = r0 * Hq + at; i < r1 * Hq && lse != nullptr; i += step) lse[i] = -CUDART_INF_F;
  };
  const long long at = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  blank(0, offset_of(q_offsets, T, 0), at, step);
  blank(max(offset_of(q_offsets, T, B - 1), offset_of(q_offsets, T, B)), T, at, step);
  const int lane = threadIdx.x & 31;
  for (long long k = threadIdx.x - lane; blockIdx.x + k * gridDim.x < B; k += blockDim.x)
    for (int i = 0; i < 32 && blockIdx.x + (k + i) * gridDim.x < B; ++i) {
      const long long b = blockIdx.x + (k + i) * gridDim.x;
      blank(static_cast<long long>(offset_of(q_offsets, T, b)) + max_q, offset_of(q_offsets, T, b + 1), lane, 32);
    }
}

// Partial results of an item cut by ranges: block i of the line left two slots of
// ROWS rows' D sums each (in the kernel's own order), then (reference, sum of
// weights) per row; its item's first piece is in slot 1, any other in slot 0.
template <int D, int ROWS>
struct Partials {
  static constexpr long long SIZE = static_cast<long long>(ROWS) * (D + 2);
  const float *parts;
  int first;  // range of the item's first piece
  __device__ __forceinline__ const float *slot(int i) const {
    return parts + (static_cast<long long>(i) * 2 + (i == first ? 1 : 0)) * SIZE;
  }
};

// A row's sums against reference m, and its sum of weights.
template <int V>
struct JoinedRow {
  float4 o[V];
  float m = kNoRef, l = 0.f;
  __device__ __forceinline__ JoinedRow() {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
};

// Adds row r of the pieces i, i + step, ... (U of them, none beyond `last`), in that
// order: the V times four sums at `at`, `at` + `stride`, ... of a slot (none if
// negative).  All are fetched before the first is used.
template <int U, int D, int ROWS, int V>
__device__ __forceinline__ void join_pieces(const Partials<D, ROWS> &ps, int r, int at, int stride, int i,
                                            int step, int last, JoinedRow<V> &x) {
  float4 y[U][V];
  float2 s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = make_float2(kNoRef, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) y[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i + u * step <= last) {
      const float *p = ps.slot(i + u * step);
      s[u] = *reinterpret_cast<const float2 *>(p + ROWS * D + 2 * r);
      if (at >= 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) y[u][v] = *reinterpret_cast<const float4 *>(p + at + v * stride);
      }
    }
  }
  float top = x.m;
#pragma unroll
  for (int u = 0; u < U; ++u) top = fmaxf(top, s[u].x);
  const float a = exp2_fast(x.m - top);
#pragma unroll
  for (int v = 0; v < V; ++v) x.o[v] = make_float4(x.o[v].x * a, x.o[v].y * a, x.o[v].z * a, x.o[v].w * a);
  x.l *= a;
  x.m = top;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float b = exp2_fast(s[u].x - top);
    x.l = fmaf(b, s[u].y, x.l);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x.o[v].x = fmaf(b, y[u][v].x, x.o[v].x);
      x.o[v].y = fmaf(b, y[u][v].y, x.o[v].y);
      x.o[v].z = fmaf(b, y[u][v].z, x.o[v].z);
      x.o[v].w = fmaf(b, y[u][v].w, x.o[v].w);
    }
  }
}

// Rows per kv head and sequence up to which the few-row kernel runs, else the
// tensor-memory one.  It works through 16 rows at a time, so its time goes up in
// steps of 16.  Measured with 8 kv heads, 16 sequences of 4000 tokens (us, few rows
// against many):
//              16 rows   24 to 32   33 to 64
//   4 bits, 128   37, 60    57, 61    98, 62
//   8 bits, 128   46, 68    72, 68   129, 69
//   4 bits,  64   37, 51    55, 51    93, 52
//   8 bits,  64   29, 51    43, 51    71, 51
// (the bytes alone: 10.3, 19.9, 5.4 and 10.3).  One sequence of 32768 tokens and 64 of
// 1000 give the same picture.
constexpr int few_rows(int bits, int D) { return bits * D == 512 ? 32 : 16; }

int launch_kv_blank(__half *out, float *lse, long long rows, int D, cudaStream_t s);
size_t kv_decode_workspace(int D, long long rows);
int launch_kv_decode(const KvAttnParams &p, int bits, int D, cudaStream_t s);
size_t kv_prefill_workspace(int D);
int launch_kv_prefill(const KvAttnParams &p, int bits, int D, cudaStream_t s);

}  // namespace w8a8
