// Root-mean-square norm of fp16 rows with the residual's addition, as fp16
// values or straight as 8-bit codes with scales; and the 8-bit float
// quantizer, which is the same kernel without the norm.
//
//   h = fp16(x + r)                      (the new residual, h = x without one)
//   v = (h w) * (1 / sqrt(mean(h^2) + eps))
//   y = fp16(v), or codes and scales of v
//
// h is rounded to fp16 because that is what the residual stream holds: the
// norm of the stored row and of the row in flight are the same.  h w is exact
// in fp32 (11 + 11 bits) and v is rounded once, so the codes are those of the
// fp32 value; it is never rounded to fp16 on the way.  max|v| of a row or
// group is max|h w| / rms (rounding is monotonic), so one reduction gives the
// sum of squares and the maximum together.  An INT8 code v / (max|v| / 127) is
// round(h w 127 / max|h w|), rounded once behind the factor 127 / max|h w|
// (2^-24): 1 / rms cancels, and only a quotient within 2^-16 of a tie can go
// either way.
//
// Design (HBM-bound, one pass): a block of T threads owns a row, V 16-byte
// vectors a thread in registers.  A persistent grid: a block fetches its next
// row before it reduces the current one.  Vector i of thread t covers elements
// [8 (i T + t), + 8), so a warp's load is 512 consecutive bytes and a group of
// 64 / 128 elements is 8 / 16 neighbouring lanes.
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "quant_rule.cuh"

namespace w8a8 {
namespace {

enum NormFormat { kInt8 = 0, kHalf = 1, kFp8 = 2, kValues = 3 };

struct NormParams {
  const uint4 *x, *r, *w;
  uint4 *h;      // new residual, or nullptr
  void *out;
  void *scale;   // fp32 (INT8 codes) or e8m0 bytes
  long rows;
  int K, gs;
  float eps;
};

// a b + c of two lanes, each rounded once
__device__ __forceinline__ float2 fma2_rn(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\n"
      "mov.b64 a, {%2, %3};\n"
      "mov.b64 b, {%4, %5};\n"
      "mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\n"
      "mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// 1.5 2^23: x + kRound is x rounded to an integer, in the low mantissa bits
constexpr float kRound = 12582912.f;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float most_of(const float2 (&p)[4]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(p[j].x), fabsf(p[j].y)));
  return m;
}

__device__ __forceinline__ uint4 hadd8(const uint4 &a, const uint4 &b) {
  uint4 c;
  const __half2 *x = reinterpret_cast<const __half2 *>(&a), *y = reinterpret_cast<const __half2 *>(&b);
  __half2 *z = reinterpret_cast<__half2 *>(&c);
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = __hadd2(x[j], y[j]);
  return c;
}

// h w of eight elements (h alone without a norm), in fp32: exact
template <bool NORM>
__device__ __forceinline__ void products(const uint4 &h, const uint4 &w, float2 (&p)[4]) {
  const __half2 *a = reinterpret_cast<const __half2 *>(&h), *b = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = NORM ? mul2_rn(__half22float2(a[j]), __half22float2(b[j])) : __half22float2(a[j]);
}

constexpr int kMaxThreads = 512;

// EARLY: the kernels that follow may start (they wait for this grid before
// they read what it writes).  Never where a caller gets 8-bit codes: they have a
// weight's type and format (a product of two activations reads them as one), and
// the few-row products request weights before they wait.  Nor may a kernel between
// the two, which starts only when this grid has ended, pass an early start on.
//
// T threads at most.  Registers for three blocks of 256 an SM or two of 512 (17089
// x 4096 with the residual to INT8 codes: 75 us; held to 64 registers 82, free 82).
template <int FORMAT, bool NORM, bool RES, bool EARLY, int V, int MOST>
__global__ void __launch_bounds__(MOST, V > 4 ? 1 : MOST == 256 ? 3 : 2) norm_kernel(const NormParams par) {
  // a second row in registers only where it fits
  constexpr bool AHEAD = V <= 2;
  if (EARLY) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float2 red[2][kMaxThreads / 32];
  const int nvec = par.K >> 3, t = threadIdx.x, T = blockDim.x, lane = t & 31;
  const int width = FORMAT == kFp8 ? kFp8Group / 8 : par.gs >> 3;  // lanes of a group; 0: the row
  // everything is read after the previous kernel: its output may be any of it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (NORM && AHEAD && i * T + t < nvec) w[i] = par.w[i * T + t];
  }

  auto load = [&](long row, uint4 (&x)[V], uint4 (&r)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vi = i * T + t;
      x[i] = make_uint4(0, 0, 0, 0);
      if (RES) r[i] = make_uint4(0, 0, 0, 0);
      if (row < par.rows && vi < nvec) {
        x[i] = __ldcs(par.x + row * nvec + vi);
        if (RES) r[i] = __ldcs(par.r + row * nvec + vi);
      }
    }
  };

  uint4 x[V], r[V];
  if (AHEAD) load(blockIdx.x, x, r);
  int parity = 0;
  for (long row = blockIdx.x; row < par.rows; row += gridDim.x, parity ^= 1) {
    if (!AHEAD) load(row, x, r);
    uint4 h[V];
    float2 p[V][4];  // kept between the passes where there is room (AHEAD)
    float2 sums = make_float2(0.f, 0.f);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] = RES ? hadd8(x[i], r[i]) : x[i];
      const int vi = i * T + t;
      if (RES && vi < nvec) par.h[row * nvec + vi] = h[i];
    }
    if (AHEAD) load(row + gridDim.x, x, r);
    float inv = 1.f;
    if (NORM) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const __half2 *a = reinterpret_cast<const __half2 *>(&h[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(a[j]);
          sums = fma2_rn(f, f, sums);
        }
        if (FORMAT < kFp8 && width == 0) {
          if (!AHEAD) w[i] = i * T + t < nvec ? __ldg(par.w + i * T + t) : make_uint4(0, 0, 0, 0);
          products<true>(h[i], w[i], p[i]);
          top = fmaxf(top, most_of(p[i]));
        }
      }
      float sum = sums.x + sums.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (FORMAT < kFp8) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (T > 32) {
        if (lane == 0) red[parity][t >> 5] = make_float2(sum, top);
        __syncthreads();
        sum = 0.f;
        top = 0.f;
        for (int i = 0; i < (T >> 5); ++i) {
          sum += red[parity][i].x;
          top = fmaxf(top, red[parity][i].y);
        }
      }
      const float mean = sum / static_cast<float>(par.K) + par.eps;
      inv = mean > 0.f ? 1.f / sqrtf(mean) : mean == 0.f ? 0.f : mean;  // a row of zeros, eps 0: zeros
    }
    float c = 0.f;  // INT8: code = round(p c), c = 127 / max|p|
    if (FORMAT < kFp8 && width == 0) {
      c = top == 0.f ? 0.f : __fdiv_rn(127.f, top);
      if (t == 0) static_cast<float *>(par.scale)[row] = __fdiv_rn(top * inv, 127.f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vi = i * T + t;
      // a group's lanes agree whether they are past the row's end only by the
      // whole warp: those past it stay for the exchange
      if (i * T + (t & ~31) >= nvec) break;
      const bool in = vi < nvec;
      if (!(AHEAD && FORMAT < kFp8 && width == 0)) {
        if (NORM && !AHEAD) w[i] = in ? __ldg(par.w + vi) : make_uint4(0, 0, 0, 0);
        products<NORM>(h[i], w[i], p[i]);
      }
      if (FORMAT == kFp8) {
        float most = most_of(p[i]);
#pragma unroll
        for (int o = kFp8Group / 16; o > 0; o >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        // v / 2^e is rounded once: the power of two joins 1 / rms exactly
        const uint32_t byte = fp8_scale_byte(most * inv);
        const float2 m = both(inv * fp8_scale_inverse(byte));
        float2 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = mul2_rn(p[i][j], m);
        if (in) {
          static_cast<uint2 *>(par.out)[row * nvec + vi] = make_uint2(fp8_pack4(q[0].x, q[0].y, q[1].x, q[1].y),
                                                                    fp8_pack4(q[2].x, q[2].y, q[3].x, q[3].y));
          if ((lane & 15) == 0)
            static_cast<uint8_t *>(par.scale)[row * ((nvec + 15) >> 4) + (vi >> 4)] = static_cast<uint8_t>(byte);
        }
      } else if (FORMAT == kValues) {
        uint4 o;
        __half2 *a = reinterpret_cast<__half2 *>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __float22half2_rn(mul2_rn(p[i][j], both(inv)));
        if (in) static_cast<uint4 *>(par.out)[row * nvec + vi] = o;
      } else {
        if (width != 0) {
          float most = most_of(p[i]);
          for (int o = width >> 1; o > 0; o >>= 1)
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          c = most == 0.f ? 0.f : __fdiv_rn(127.f, most);
          if (in && (lane & (width - 1)) == 0)
            static_cast<float *>(par.scale)[row * (par.K / par.gs) + (vi << 3) / par.gs] = __fdiv_rn(most * inv, 127.f);
        }
        float2 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = fma2_rn(p[i][j], both(c), both(kRound));
        if (in) {
          if (FORMAT == kHalf) {
            uint4 o;
            __half2 *a = reinterpret_cast<__half2 *>(&o);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = __float22half2_rn(sub2_rn(q[j], both(kRound)));
            static_cast<uint4 *>(par.out)[row * nvec + vi] = o;
          } else {
            auto low = [](const float2 &a, const float2 &b) {  // four low bytes
              const uint32_t ab = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
              return __byte_perm(ab, __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
            };
            static_cast<uint2 *>(par.out)[row * nvec + vi] = make_uint2(low(q[0], q[1]), low(q[2], q[3]));
          }
        }
      }
    }
  }
}

template <int FORMAT, bool NORM, bool RES, bool EARLY, int V, int MOST>
int launch_v(const NormParams &p, int T, cudaStream_t s) {
  // blocks that are resident at once, per device and block size
  static int resident[64][kMaxThreads / 32] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W8A8_ERR_CUDA;
  int most = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    int &known = resident[dev][T / 32 - 1];
    if (known == 0) {
      int sms = 0, occ = 0;
      if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, norm_kernel<FORMAT, NORM, RES, EARLY, V, MOST>,
                                                        T, 0) != cudaSuccess || occ < 1)
        return W8A8_ERR_CUDA;
      known = sms * occ;
    }
    most = known;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows < most ? p.rows : most));
  cfg.blockDim = dim3(static_cast<unsigned>(T));
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, norm_kernel<FORMAT, NORM, RES, EARLY, V, MOST>, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  return launch_status();
}

template <int FORMAT, bool NORM, bool RES, bool EARLY>
int launch_f(const NormParams &p, cudaStream_t s) {
  const int nvec = p.K >> 3;
  // the fewest vectors a thread that a block of at most 512 covers the row with
  int V = 1;
  while (V * kMaxThreads < nvec) V <<= 1;
  if (V == 1 && nvec > 128) V = 2;
  const int T = ((nvec + V - 1) / V + 31) & ~31;
  switch (V) {
    case 1: return launch_v<FORMAT, NORM, RES, EARLY, 1, 256>(p, T, s);
    case 2: return T <= 256 ? launch_v<FORMAT, NORM, RES, EARLY, 2, 256>(p, T, s) : launch_v<FORMAT, NORM, RES, EARLY, 2, 512>(p, T, s);
    case 4: return launch_v<FORMAT, NORM, RES, EARLY, 4, 512>(p, T, s);
    case 8: return launch_v<FORMAT, NORM, RES, EARLY, 8, 512>(p, T, s);
    default: return W8A8_ERR_INVALID_ARG;  // K > 32768
  }
}

NormParams params(const __half *x, const __half *r, const __half *w, long rows, int K, float eps,
                  int gs, __half *h, void *out, void *scale) {
  NormParams p;
  p.x = reinterpret_cast<const uint4 *>(x);
  p.r = reinterpret_cast<const uint4 *>(r);
  p.w = reinterpret_cast<const uint4 *>(w);
  p.h = reinterpret_cast<uint4 *>(h);
  p.out = out;
  p.scale = scale;
  p.rows = rows;
  p.K = K;
  p.gs = gs;
  p.eps = eps;
  return p;
}

template <int FORMAT>
int launch_n(const NormParams &p, cudaStream_t s) {
  constexpr bool EARLY = FORMAT == kValues || FORMAT == kHalf;  // fp16: nothing that a product takes for weights
  return p.r != nullptr ? launch_f<FORMAT, true, true, EARLY>(p, s)
                        : launch_f<FORMAT, true, false, EARLY>(p, s);
}

}  // namespace

int launch_rms_norm(const __half *x, const __half *r, const __half *w, int M, int K, float eps,
                    __half *h, __half *y, cudaStream_t s) {
  return launch_n<kValues>(params(x, r, w, M, K, eps, 0, h, y, nullptr), s);
}

int launch_rms_norm_quant(const __half *x, const __half *r, const __half *w, int M, int K,
                          float eps, int format, int group_size, __half *h, void *q, void *scale,
                          cudaStream_t s) {
  const NormParams p = params(x, r, w, M, K, eps, group_size, h, q, scale);
  switch (format) {
    case W8A8_CODES_INT8: return launch_n<kInt8>(p, s);
    case W8A8_CODES_HALF: return launch_n<kHalf>(p, s);
    default: return launch_n<kFp8>(p, s);
  }
}

int launch_quant_fp8(const __half *x, long rows, int K, bool early, uint8_t *q, uint8_t *scale,
                     cudaStream_t s) {
  const NormParams p = params(x, nullptr, nullptr, rows, K, 0.f, 0, nullptr, q, scale);
  return early ? launch_f<kFp8, false, false, true>(p, s) : launch_f<kFp8, false, false, false>(p, s);
}

}  // namespace w8a8
