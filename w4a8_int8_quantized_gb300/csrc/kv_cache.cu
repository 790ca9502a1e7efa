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
// head against D bits / 4 + 8 of the cache.  D / 16 lanes own a row when
// writing, two 16-byte vectors each, D / 8 when reading, one vector each, and a
// thread has the K and the V vectors of kUnroll rows in flight.  Alone, 32771 tokens of 8
// heads at 8 / 4 bits take 42 / 40 us to write and 35 / 32 to read (bytes: 30 / 25).
// Writing, neighbouring rows are the heads of a token, so
// that the fp16 side is read in runs of heads x 2 D bytes (32771 tokens of 8
// heads at 8 bits took 56 us with a head per block, whose 256-byte rows lie
// 12 KB apart in a fused projection); a block's tokens follow one another, so
// the code rows and 4-byte scales that it writes to each head's part of a page
// fill whole sectors in L2.  Reading, a block keeps to one head: the cache
// side is then read in runs, and the fp16 side written in whole 2 D-byte rows.
#include "common.cuh"
#include "kv_common.cuh"
#include "quant_rule.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

// Larger magnitude of two pairs of fp16 values, NaN above all (the sign bits of
// both are 0).
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// Magnitudes of a vector's 8 values, the larger ones of 4 pairs of pairs.
__device__ __forceinline__ uint32_t max_pair8(const uint4 &v) {
  return max_pair(max_pair(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                  max_pair(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
// Inf or NaN in either half
__device__ __forceinline__ bool not_finite(uint32_t pair) {
  return (pair & 0x7c00u) == 0x7c00u || (pair & 0x7c000000u) == 0x7c000000u;
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

// a / QMAX correctly rounded, for every finite fp16 value a >= 0: Markstein's
// correction of the product with the rounded reciprocal (one residual, one
// multiply-add); equal to the IEEE quotient for all of them.
template <int QMAX>
__device__ __forceinline__ float scale_of(float a) {
  constexpr float r = 1.f / QMAX;
  const float q = a * r;
  return fmaf(fmaf(-static_cast<float>(QMAX), q, a), r, q);
}

// The codes of one vector: rint(x / s), packed (8 bytes, or 4).  As in
// quant_rule.cuh, t = x * (1 / s) decides unless it is within 2^-14 of a tie,
// where the IEEE quotient does; here 1 / s is within one unit in the last
// place, so t is within |x / s| (2^-23 + 2^-24) <= 2.3e-5 of x / s, the IEEE
// quotient within 7.6e-6, together still under 2^-14.  Rounding to an integer
// is the addition of 1.5 * 2^23 (round to nearest, ties to even), which leaves
// the integer in the low bits: no conversion instruction is needed, whose rate
// is a quarter of an addition's (they held the kernel at 56 us for 32771
// tokens of 8 heads at 8 bits, 49 without).  At 4 bits, two codes go through one such
// addition: 16 hi + lo + 136 has (hi + 8, lo + 8) as its nibbles.
template <int BITS>
__device__ __forceinline__ uint2 quant8(const uint4 &v, float s, float rcp) {
  constexpr float M = 12582912.f;
  const __half2 *h = reinterpret_cast<const __half2 *>(&v);
  float z[8], r[8], far = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __half22float2(h[j]);
    const float2 t = mul2_rn(x, make_float2(rcp, rcp));
    z[2 * j] = __fadd_rn(t.x, M);
    z[2 * j + 1] = __fadd_rn(t.y, M);
    r[2 * j] = __fadd_rn(z[2 * j], -M);
    r[2 * j + 1] = __fadd_rn(z[2 * j + 1], -M);
    far = fmaxf(far, fmaxf(fabsf(t.x - r[2 * j]), fabsf(t.y - r[2 * j + 1])));
  }
  if (far >= 0.49993896484375f) {  // 1/2 - 2^-14: some element is near a tie
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = __half2float(reinterpret_cast<const __half *>(&v)[j]);
      if (s > 0.f) r[j] = rintf(__fdiv_rn(x, s));
      z[j] = __fadd_rn(r[j], M);
    }
  }
  uint32_t w[2];
  if (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __byte_perm(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]), 0x0040);
      const uint32_t b = __byte_perm(__float_as_uint(z[4 * i + 2]), __float_as_uint(z[4 * i + 3]), 0x0040);
      w[i] = __byte_perm(a, b, 0x5410);
    }
  } else {
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = __float_as_uint(__fadd_rn(fmaf(r[2 * j + 1], 16.f, r[2 * j]), M + 136.f));
    w[0] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410) ^ 0x88888888u;
    w[1] = 0;
  }
  return make_uint2(w[0], w[1]);
}

// Slot of a token as (page, offset); false if it is not stored.
__device__ __forceinline__ bool find_slot(const KvView &c, long long slot, long long &page,
                                          int &off) {
  if (slot < 0) return false;
  page = slot >> c.page_shift;
  off = static_cast<int>(slot) & ((1 << c.page_shift) - 1);
  if (page < c.pages) return true;
  report_index(c.err);
  return false;
}

// Quantizes one row of D = 16 L elements, held by an L-lane team as two vectors a
// lane (vectors lane and lane + L).
template <int BITS, int L>
__device__ __forceinline__ void store_row(uint4 (&v)[2], uint8_t *codes, float *scale, long long row,
                                          int lane, bool keep) {
  uint32_t m = max_pair(max_pair8(v[0]), max_pair8(v[1]));
  if (not_finite(m)) {
    v[0] = finite8(v[0]);
    v[1] = finite8(v[1]);
    m = max_pair(max_pair8(v[0]), max_pair8(v[1]));
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max_pair(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!keep) return;
  m = max(m & 0xffffu, m >> 16);  // the order of finite magnitudes is that of their bits
  const float s = scale_of<BITS == 8 ? 127 : 7>(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
  float rcp;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rcp) : "f"(s));
  if (s == 0.f) rcp = 0.f;
  constexpr int ROW = 2 * L * BITS;  // bytes: 16 L elements
  uint8_t *at = codes + row * ROW + lane * BITS;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 q = quant8<BITS>(v[i], s, rcp);
    if (BITS == 8)
      *reinterpret_cast<uint2 *>(at + i * L * 8) = q;
    else
      *reinterpret_cast<uint32_t *>(at + i * L * 4) = q.x;
  }
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
  // two vectors a lane: the row's scale, slot and addresses cost as much as
  // quantizing one (one vector a lane: 79 us for 32771 tokens at 8 bits with the
  // reading back, two: 72)
  constexpr int L = D / 16, TEAMS = kThreads / L;
  const int lane = threadIdx.x % L, team = threadIdx.x / L, H = p.kv.heads;
  const long long rows = static_cast<long long>(p.T) * H;  // row t H + h
  const long long step = static_cast<long long>(gridDim.x) * TEAMS * kUnroll;
  for (long long r0 = static_cast<long long>(blockIdx.x) * TEAMS * kUnroll; r0 < rows; r0 += step) {
    // the block's first row; what follows it is counted in 32 bits
    const int t0 = static_cast<int>(r0 / H), h0 = static_cast<int>(r0 - static_cast<long long>(t0) * H);
    uint4 k[kUnroll][2], v[kUnroll][2];
    long long slot[kUnroll];
    int h[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const unsigned at = h0 + u * TEAMS + team, dt = at / static_cast<unsigned>(H);
      const long long t = static_cast<long long>(t0) + dt;
      h[u] = at - dt * H;
      slot[u] = -1;
      k[u][0] = k[u][1] = v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (t < p.T) {
        slot[u] = __ldg(p.slots + t);
        const uint4 *kp = reinterpret_cast<const uint4 *>(p.k + t * p.k_ts + h[u] * p.k_hs) + lane;
        const uint4 *vp = reinterpret_cast<const uint4 *>(p.v + t * p.v_ts + h[u] * p.v_hs) + lane;
        k[u][0] = __ldcs(kp);
        k[u][1] = __ldcs(kp + L);
        v[u][0] = __ldcs(vp);
        v[u][1] = __ldcs(vp + L);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      long long page = 0;
      int off = 0;
      const bool keep = find_slot(p.kv, slot[u], page, off);
      const long long row = p.kv.row(page, h[u]) + off;
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

// blocks for `rows` rows, `per` at a time: enough for every row, at most a few waves
int blocks_for(long long rows, int per, int most) {
  const long long want = (rows + per - 1) / per;
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

int launch_kv_write(const KvView &kv, int bits, int D, const __half *k, long long k_ts,
                    long long k_hs, const __half *v, long long v_ts, long long v_hs,
                    const long long *slots, int T, cudaStream_t s) {
  const WriteParams p{kv, k, v, k_ts, k_hs, v_ts, v_hs, slots, T};
  const int grid = blocks_for(static_cast<long long>(T) * kv.heads, kThreads / (D / 16) * kUnroll, kNumSMsGB300 * 16);
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
  const dim3 grid(blocks_for(T, kThreads / (D / 8) * kUnroll, ceil_div(kNumSMsGB300 * 16, kv.heads)), kv.heads);
  if (bits == 4)
    D == 64 ? kv_read_kernel<4, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_read_kernel<4, 128><<<grid, kThreads, 0, s>>>(p);
  else
    D == 64 ? kv_read_kernel<8, 64><<<grid, kThreads, 0, s>>>(p)
            : kv_read_kernel<8, 128><<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

}  // namespace w8a8
