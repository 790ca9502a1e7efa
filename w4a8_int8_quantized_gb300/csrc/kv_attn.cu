// Attention over the quantized key/value cache, one warp per query row.
//
// Row (t, head) at position p of its sequence, keys j visible to it:
//   S_j = scale * s_k[j] * (q . code_k[j]),  o = sum_j softmax(S)_j s_v[j] code_v[j],
//   lse = ln sum_j exp S_j,
// in one pass with the running maximum and sum.  A row that sees nothing
// gives o = 0 and lse = -inf.
#include <math_constants.h>

#include "common.cuh"
#include "kv_attn.cuh"
#include "kv_common.cuh"

namespace w8a8 {
namespace {

// E = D / 32 consecutive codes of lane `lane` of a row, as fp32
template <int BITS, int E>
__device__ __forceinline__ void codes_of(const uint8_t *row, int lane, float (&c)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int d = lane * E + i;
    if (BITS == 8)
      c[i] = static_cast<float>(static_cast<int8_t>(row[d]));
    else
      c[i] = static_cast<float>(static_cast<int>(static_cast<uint32_t>(row[d / 2]) << (d & 1 ? 24 : 28)) >> 28);
  }
}

template <int BITS, int D>
__global__ void __launch_bounds__(128) kv_attn_row_kernel(const KvAttnParams p) {
  constexpr int E = D / 32, ROW = D * BITS / 8;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int hq = static_cast<int>(item % p.Hq);
  const long long rest = item / p.Hq;
  const int i = static_cast<int>(rest % p.max_q);
  const long long b = rest / p.max_q;
  if (b >= p.B) return;
  int q0, nq, len, lo, hi;
  seq_of(p, static_cast<int>(b), q0, nq, len);
  if (i >= nq) return;
  const long long t = q0 + i;
  visible(p, len - nq + i, len, lo, hi);
  const int h = hq / p.group;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __half2float(p.q[t * p.q_ts + hq * p.q_hs + lane * E + e]);
    o[e] = 0.f;
  }
  float m = -CUDART_INF_F, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int page = page_of(p, static_cast<int>(b), j >> p.kv.page_shift);
    if (page < 0) continue;
    const long long row = p.kv.row(page, h) + (j & ((1 << p.kv.page_shift) - 1));
    float c[E];
    codes_of<BITS, E>(p.kv.kc + row * ROW, lane, c);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], c[e], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.kv.ks[row] * p.scale;
    const float mn = fmaxf(m, s);
    const float a = m == mn ? 1.f : expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * a + w;
    codes_of<BITS, E>(p.kv.vc + row * ROW, lane, c);
    const float ws = w * p.kv.vs[row];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(ws, c[e], o[e] * a);
  }
  const float r = l > 0.f ? 1.f / l : 0.f;
  const long long at = t * p.Hq + hq;
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[at * D + lane * E + e] = __float2half_rn(o[e] * r);
  if (p.lse != nullptr && lane == 0) p.lse[at] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace

size_t kv_attn_workspace(int T, int Hq, int max_q, int B, long long max_len, const KvView &kv,
                         int bits, int D) {
  const long long rows = static_cast<long long>(max_q) * (Hq / kv.heads);
  return rows <= kFewRows ? kv_decode_workspace(D, rows) : 0;
}

int launch_kv_attn(const KvAttnParams &p, int bits, int D, cudaStream_t s) {
  if (static_cast<long long>(p.max_q) * p.group <= kFewRows) return launch_kv_decode(p, bits, D, s);
  const long long items = static_cast<long long>(p.B) * p.max_q * p.Hq;
  const long long blocks = (items + 3) / 4;
  if (blocks > 0x7fffffffLL) return W8A8_ERR_INVALID_ARG;
  const unsigned g = static_cast<unsigned>(blocks);
  if (bits == 4)
    D == 64 ? kv_attn_row_kernel<4, 64><<<g, 128, 0, s>>>(p)
            : kv_attn_row_kernel<4, 128><<<g, 128, 0, s>>>(p);
  else
    D == 64 ? kv_attn_row_kernel<8, 64><<<g, 128, 0, s>>>(p)
            : kv_attn_row_kernel<8, 128><<<g, 128, 0, s>>>(p);
  return launch_status();
}

}  // namespace w8a8
