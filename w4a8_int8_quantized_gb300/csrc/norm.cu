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
// sum of squares and the maximum together.
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

// Codes of eight fp32 values by the rule of the fp16 quantizer (v / s rounded
// to nearest even): v * (1 / s) decides, but within 2^-14 of a tie the IEEE
// quotient does.  |v| <= max|v| = 127 s up to rounding, so no clamp.
__device__ __forceinline__ void quant8(const float (&v)[8], float s, float rcp, float (&q)[8]) {
  bool any_near = false;
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t[j] = v[j] * rcp;
    q[j] = rintf(t[j]);
    any_near |= near_half(t[j], q[j]);
  }
  if (any_near) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (near_half(t[j], q[j])) q[j] = rintf(__fdiv_rn(v[j], s));
  }
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
__device__ __forceinline__ void products(const uint4 &h, const uint4 &w, float (&p)[8]) {
  const __half2 *a = reinterpret_cast<const __half2 *>(&h), *b = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __half22float2(a[j]);
    if (NORM) {
      const float2 y = __half22float2(b[j]);
      p[2 * j] = x.x * y.x;
      p[2 * j + 1] = x.y * y.y;
    } else {
      p[2 * j] = x.x;
      p[2 * j + 1] = x.y;
    }
  }
}

constexpr int kMaxThreads = 512;

// EARLY: the kernels that follow may start (they wait for this grid before
// they read what it writes); never when the codes are weights, which the
// few-row kernels request before they wait.
template <int FORMAT, bool NORM, bool RES, bool EARLY, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p) {
  // a second row in registers only where it fits
  constexpr bool AHEAD = V <= 2;
  if (EARLY) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float2 red[2][kMaxThreads / 32];
  const int nvec = p.K >> 3, t = threadIdx.x, T = blockDim.x, lane = t & 31;
  const int width = FORMAT == kFp8 ? kFp8Group / 8 : p.gs >> 3;  // lanes of a group; 0: the row
  // everything is read after the previous kernel: its output may be any of it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (NORM && AHEAD && i * T + t < nvec) w[i] = p.w[i * T + t];
  }

  auto load = [&](long row, uint4 (&x)[V], uint4 (&r)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vi = i * T + t;
      x[i] = make_uint4(0, 0, 0, 0);
      if (RES) r[i] = make_uint4(0, 0, 0, 0);
      if (row < p.rows && vi < nvec) {
        x[i] = __ldcs(p.x + row * nvec + vi);
        if (RES) r[i] = __ldcs(p.r + row * nvec + vi);
      }
    }
  };

  uint4 x[V], r[V];
  if (AHEAD) load(blockIdx.x, x, r);
  int parity = 0;
  for (long row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    if (!AHEAD) load(row, x, r);
    uint4 h[V];
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] = RES ? hadd8(x[i], r[i]) : x[i];
      const int vi = i * T + t;
      if (RES && vi < nvec) p.h[row * nvec + vi] = h[i];
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
          sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
        }
        if (FORMAT < kFp8 && width == 0) {
          if (!AHEAD) w[i] = i * T + t < nvec ? __ldg(p.w + i * T + t) : make_uint4(0, 0, 0, 0);
          float q[8];
          products<true>(h[i], w[i], q);
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(q[j]));
        }
      }
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
      const float mean = sum / static_cast<float>(p.K) + p.eps;
      inv = mean > 0.f ? 1.f / sqrtf(mean) : mean == 0.f ? 0.f : mean;  // a row of zeros, eps 0: zeros
    }
    float s = 1.f, rcp = 1.f;
    if (FORMAT < kFp8 && width == 0) {
      s = __fdiv_rn(top * inv, 127.f);
      rcp = s == 0.f ? 0.f : __frcp_rn(s);
      if (t == 0) static_cast<float *>(p.scale)[row] = s;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vi = i * T + t;
      // a group's lanes agree whether they are past the row's end only by the
      // whole warp: those past it stay for the exchange
      if (i * T + (t & ~31) >= nvec) break;
      const bool in = vi < nvec;
      if (NORM && !AHEAD) w[i] = in ? __ldg(p.w + vi) : make_uint4(0, 0, 0, 0);
      float v[8];
      products<NORM>(h[i], w[i], v);
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (NORM) v[j] *= inv;
        most = fmaxf(most, fabsf(v[j]));
      }
      if (FORMAT == kFp8) {
#pragma unroll
        for (int o = kFp8Group / 16; o > 0; o >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const uint32_t byte = fp8_scale_byte(most);
        const float m = fp8_scale_inverse(byte);
        if (in) {
          static_cast<uint2 *>(p.out)[row * nvec + vi] =
              make_uint2(fp8_pack4(v[0] * m, v[1] * m, v[2] * m, v[3] * m),
                         fp8_pack4(v[4] * m, v[5] * m, v[6] * m, v[7] * m));
          if ((lane & 15) == 0)
            static_cast<uint8_t *>(p.scale)[row * ((nvec + 15) >> 4) + (vi >> 4)] =
                static_cast<uint8_t>(byte);
        }
      } else if (FORMAT == kValues) {
        uint4 o;
        __half2 *a = reinterpret_cast<__half2 *>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        if (in) static_cast<uint4 *>(p.out)[row * nvec + vi] = o;
      } else {
        if (width != 0) {
          for (int o = width >> 1; o > 0; o >>= 1)
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          s = __fdiv_rn(most, 127.f);
          rcp = s == 0.f ? 0.f : __frcp_rn(s);
          if (in && (lane & (width - 1)) == 0)
            static_cast<float *>(p.scale)[row * (p.K / p.gs) + (vi << 3) / p.gs] = s;
        }
        float q[8];
        quant8(v, s, rcp, q);
        if (in) {
          if (FORMAT == kHalf)
            static_cast<uint4 *>(p.out)[row * nvec + vi] = pack_h8(q);
          else
            static_cast<uint2 *>(p.out)[row * nvec + vi] = pack_i8x8(q);
        }
      }
    }
  }
}

template <int FORMAT, bool NORM, bool RES, bool EARLY, int V>
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
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, norm_kernel<FORMAT, NORM, RES, EARLY, V>,
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
  if (cudaLaunchKernelEx(&cfg, norm_kernel<FORMAT, NORM, RES, EARLY, V>, p) != cudaSuccess) {
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
    case 1: return launch_v<FORMAT, NORM, RES, EARLY, 1>(p, T, s);
    case 2: return launch_v<FORMAT, NORM, RES, EARLY, 2>(p, T, s);
    case 4: return launch_v<FORMAT, NORM, RES, EARLY, 4>(p, T, s);
    case 8: return launch_v<FORMAT, NORM, RES, EARLY, 8>(p, T, s);
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
  return p.r != nullptr ? launch_f<FORMAT, true, true, true>(p, s)
                        : launch_f<FORMAT, true, false, true>(p, s);
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

int launch_quant_fp8(const __half *x, long rows, int K, bool weights, uint8_t *q, uint8_t *scale,
                     cudaStream_t s) {
  const NormParams p = params(x, nullptr, nullptr, rows, K, 0.f, 0, nullptr, q, scale);
  return weights ? launch_f<kFp8, false, false, false>(p, s) : launch_f<kFp8, false, false, true>(p, s);
}

}  // namespace w8a8
