// The quantized key/value cache: tokens quantized as they are written, and
// read back.
//
// Rule (the library's symmetric per-token rule, one scale per token and kv
// head): a = max |x| over the head's D elements, s = a / qmax (one IEEE fp32
// division), q = clamp(rint(x / s), -qmax, qmax) (see quant_rule.cuh); read
// back as fp16_rn(q * s).  The cache holds finite values only: NaN is stored
// as 0 and +-Inf as +-65504, so that no position that attention masks out can
// reach a result through 0 * NaN.
//
// Both kernels stream (no reuse): 4 D bytes of fp16 k and v per token and
// head against D bits / 4 + 8 of the cache.  D / 8 lanes own a row, one
// 16-byte vector each, and a thread has the K and the V vector of kUnroll
// tokens in flight.  blockIdx.y is the head, so that a block's rows are
// consecutive tokens of one head: consecutive slots are consecutive rows of
// the cache, and their 64-byte (4 bits, D = 128) code rows and 4-byte scales
// fill whole sectors, while the fp16 side moves in 2 D-byte rows whatever the
// strides.
#include "common.cuh"
#include "kv_common.cuh"
#include "quant_rule.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

// Largest magnitude of the 8 fp16 values as fp16 bits (the order of the bits
// is that of the magnitudes, with Inf and NaN above all finite values).
__device__ __forceinline__ uint32_t max_bits8(const uint4 &v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// NaN -> 0, +-Inf -> +-65504
__device__ __noinline__ uint4 finite8(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t e = (w[i] >> (16 * h)) & 0xffffu;
      if ((e & 0x7fffu) > 0x7c00u) e = 0;
      if ((e & 0x7fffu) == 0x7c00u) e = (e & 0x8000u) | 0x7bffu;
      o |= e << (16 * h);
    }
    w[i] = o;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t pack_i4x8(const float (&r)[8]) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o |= (static_cast<uint32_t>(__float2int_rn(r[i])) & 0xfu) << (4 * i);
  return o;
}

// Slot of a token as (page, offset); false if it is not stored.
__device__ __forceinline__ bool find_slot(const KvView &c, long long slot, long long &page,
                                          int &off) {
  if (slot < 0) return false;
  page = slot >> c.page_shift;
  off = static_cast<int>(slot) & ((1 << c.page_shift) - 1);
  if (page < c.pages) return true;
  if (c.err != nullptr) atomicCAS(c.err, 0u, static_cast<unsigned>(kDevErrIndex));
  return false;
}

// Quantizes one row held as one vector per lane of an L-lane team.
template <int BITS, int L>
__device__ __forceinline__ void store_row(uint4 v, uint8_t *codes, float *scale, long long row,
                                          int lane, bool keep) {
  uint32_t m = max_bits8(v);
  if (m >= 0x7c00u) {
    v = finite8(v);
    m = max_bits8(v);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!keep) return;
  constexpr float qmax = BITS == 8 ? 127.f : 7.f;
  const float s = __fdiv_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(m))), qmax);
  const float rcp = s > 0.f ? __frcp_rn(s) : 0.f;
  float r[8];
  quant_vec8(v, s, rcp, r);
  constexpr int ROW = L * BITS;  // bytes: 8 L elements
  if (BITS == 8)
    *reinterpret_cast<uint2 *>(codes + row * ROW + lane * 8) = pack_i8x8(r);
  else
    *reinterpret_cast<uint32_t *>(codes + row * ROW + lane * 4) = pack_i4x8(r);
  if (lane == 0) scale[row] = s;
}

struct WriteParams {
  KvView kv;
  const __half *k, *v;
  long long k_ts, k_hs, v_ts, v_hs;  // element strides: token, head
  const long long *slots;
  int T;
};

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const WriteParams p) {
  constexpr int L = D / 8, TEAMS = kThreads / L;
  const int lane = threadIdx.x % L, team = threadIdx.x / L, h = blockIdx.y;
  const long long step = static_cast<long long>(gridDim.x) * TEAMS * kUnroll;
  for (long long t0 = static_cast<long long>(blockIdx.x) * TEAMS * kUnroll; t0 < p.T; t0 += step) {
    uint4 k[kUnroll], v[kUnroll];
    long long slot[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long t = t0 + u * TEAMS + team;
      slot[u] = -1;
      k[u] = v[u] = make_uint4(0, 0, 0, 0);
      if (t < p.T) {
        slot[u] = __ldg(p.slots + t);
        k[u] = __ldcs(reinterpret_cast<const uint4 *>(p.k + t * p.k_ts + h * p.k_hs) + lane);
        v[u] = __ldcs(reinterpret_cast<const uint4 *>(p.v + t * p.v_ts + h * p.v_hs) + lane);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      long long page = 0;
      int off = 0;
      const bool keep = find_slot(p.kv, slot[u], page, off);
      const long long row = p.kv.row(page, h) + off;
      store_row<BITS, L>(k[u], p.kv.kc, p.kv.ks, row, lane, keep);
      store_row<BITS, L>(v[u], p.kv.vc, p.kv.vs, row, lane, keep);
    }
  }
}

// 8 codes of a row times its scale, rounded to fp16 once
template <int BITS>
__device__ __forceinline__ uint4 values8(uint2 w, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int a, b;
    if (BITS == 8) {
      const uint32_t x = i < 2 ? w.x : w.y;
      a = static_cast<int8_t>(x >> (16 * (i & 1)));
      b = static_cast<int8_t>(x >> (16 * (i & 1) + 8));
    } else {
      a = static_cast<int>(w.x << (28 - 8 * i)) >> 28;
      b = static_cast<int>(w.x << (24 - 8 * i)) >> 28;
    }
    const __half2 h = __floats2half2_rn(__fmul_rn(static_cast<float>(a), s),
                                        __fmul_rn(static_cast<float>(b), s));
    o[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct ReadParams {
  KvView kv;
  __half *k, *v;  // [T, heads, D]
  const long long *slots;
  int T;
};

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
  constexpr int L = D / 8, TEAMS = kThreads / L;
  const int lane = threadIdx.x % L, team = threadIdx.x / L, h = blockIdx.y;
  constexpr int ROW = L * BITS;
  const long long step = static_cast<long long>(gridDim.x) * TEAMS * kUnroll;
  for (long long t0 = static_cast<long long>(blockIdx.x) * TEAMS * kUnroll; t0 < p.T; t0 += step) {
    uint2 k[kUnroll], v[kUnroll];
    float ks[kUnroll], vs[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long t = t0 + u * TEAMS + team;
      k[u] = v[u] = make_uint2(0, 0);
      ks[u] = vs[u] = 0.f;
      long long page;
      int off;
      if (t < p.T && find_slot(p.kv, __ldg(p.slots + t), page, off)) {
        const long long row = p.kv.row(page, h) + off;
        if (BITS == 8) {
          k[u] = *reinterpret_cast<const uint2 *>(p.kv.kc + row * ROW + lane * 8);
          v[u] = *reinterpret_cast<const uint2 *>(p.kv.vc + row * ROW + lane * 8);
        } else {
          k[u].x = *reinterpret_cast<const uint32_t *>(p.kv.kc + row * ROW + lane * 4);
          v[u].x = *reinterpret_cast<const uint32_t *>(p.kv.vc + row * ROW + lane * 4);
        }
        ks[u] = p.kv.ks[row];
        vs[u] = p.kv.vs[row];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long t = t0 + u * TEAMS + team;
      if (t < p.T) {
        const long long o = (t * p.kv.heads + h) * L + lane;
        __stcs(reinterpret_cast<uint4 *>(p.k) + o, values8<BITS>(k[u], ks[u]));
        __stcs(reinterpret_cast<uint4 *>(p.v) + o, values8<BITS>(v[u], vs[u]));
      }
    }
  }
}

// blocks along the tokens: enough for every token, at most a few waves
dim3 token_grid(int T, int heads, int D) {
  const int per = kThreads / (D / 8) * kUnroll;
  const int most = ceil_div(kNumSMsGB300 * 16, heads);
  const int want = ceil_div(T, per);
  return dim3(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(heads));
}

}  // namespace

int launch_kv_write(const KvView &kv, int bits, int D, const __half *k, long long k_ts,
                    long long k_hs, const __half *v, long long v_ts, long long v_hs,
                    const long long *slots, int T, cudaStream_t s) {
  const WriteParams p{kv, k, v, k_ts, k_hs, v_ts, v_hs, slots, T};
  const dim3 grid = token_grid(T, kv.heads, D);
  if (bits == 4)
    D == 64 ? kv_write_kernel<4, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_write_kernel<4, 128><<<grid, kThreads, 0, s>>>(p);
  else
    D == 64 ? kv_write_kernel<8, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_write_kernel<8, 128><<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

int launch_kv_read(const KvView &kv, int bits, int D, const long long *slots, int T, __half *k,
                   __half *v, cudaStream_t s) {
  const ReadParams p{kv, k, v, slots, T};
  const dim3 grid = token_grid(T, kv.heads, D);
  if (bits == 4)
    D == 64 ? kv_read_kernel<4, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_read_kernel<4, 128><<<grid, kThreads, 0, s>>>(p);
  else
    D == 64 ? kv_read_kernel<8, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_read_kernel<8, 128><<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

}  // namespace w8a8
