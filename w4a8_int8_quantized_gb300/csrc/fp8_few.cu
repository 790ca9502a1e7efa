// Products of a few rows of 8-bit floats with a weight matrix: the layer's and
// the gated pair's form for single tokens and small batches, bound by the
// weights' bytes.
//
//   y[m, n] = fp16(sum_g 2^(ea[m,g] + ew[n,g]) sum_{k in g} a[m,k] w[n,k])
//   h[m, f] = act(x . Wg[f]) (x . Wu[f]), as fp16 or as e4m3 codes with scales
//
// mma.sync m16n8k16 with 16 weight rows as M and 8 tokens as N: one token
// wastes only multiplications, which cost nothing beside the bytes.  e4m3
// codes become fp16 exactly, products and sums of a group are fp32 in the
// tensor core, and each group's sum is scaled and added in fp32.  Which
// elements of K share an instruction is free as long as both operands agree,
// so a lane takes 16 consecutive bytes of its row (four of 64 consecutive
// bytes per row and load) and feeds four instructions with them.
//
// Eight warps a block: KW of them share the same 16 weight rows and take its
// groups in turn, the other 8 / KW are further rows.  Their sums are joined in
// shared memory in a fixed order.  A group's weights are requested one group
// ahead, the first ones before the previous kernel on the stream has finished.
//
// Codes out: a group of 128 outputs is a cluster of KW blocks, which exchange
// their tokens' maxima through distributed shared memory.
#include <cooperative_groups.h>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8_kernels.cuh"

namespace cg = cooperative_groups;

namespace w8a8 {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// four e4m3 codes as two pairs of fp16 values, exactly
__device__ __forceinline__ void to_half4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n.reg .b16 a, b;\n"
      "mov.b32 {a, b}, %2;\n"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// What a lane holds of one group: two rows (16 of the tile: lane / 4 and + 8)
// of each weight matrix, its token's codes, and the scales.
template <int MATS, int NT>
struct Slice {
  uint4 w[MATS][2][2];  // [matrix][row][half of the group]
  uint32_t sw[MATS][2];
  uint4 x[NT][2];
  uint32_t sx[NT][2];   // tokens 2 (lane % 4), + 1
};

template <int MATS, int NT, int KW, bool CODES, bool GELU>
__global__ void __launch_bounds__(kWarps * 32, 2) few_kernel(const Fp8Params p) {
  constexpr int RT = kWarps / KW;  // 16-row tiles of a block
  __shared__ float red[kWarps][MATS][NT * 4][32];
  __shared__ uint32_t tops[NT * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int kw = warp % KW, rw = warp / KW;
  const long n0 = (static_cast<long>(blockIdx.x) * RT + rw) * 16;
  const long m0 = static_cast<long>(blockIdx.y) * (NT * 8);
  const int K = p.K, G = p.G;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  auto weights = [&](int g, Slice<MATS, NT> &s) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const long n = n0 + gid + 8 * r;
        const bool in = n < p.N && g < G;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = g * kFp8Group + h * 64 + tig * 16;
          s.w[a][r][h] = in && k < K
                             ? __ldcs(reinterpret_cast<const uint4 *>(p.w[a] + n * K + k))
                             : zero;
        }
        s.sw[a][r] = in ? __ldg(p.sw[a] + n * G + g) : 127u;
      }
  };
  auto tokens = [&](int g, Slice<MATS, NT> &s) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const long m = m0 + t * 8 + gid;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = g * kFp8Group + h * 64 + tig * 16;
        s.x[t][h] = m < p.M && g < G && k < K
                        ? *reinterpret_cast<const uint4 *>(p.x + m * K + k)
                        : zero;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const long ms = m0 + t * 8 + 2 * tig + e;
        s.sx[t][e] = ms < p.M && g < G ? p.sx[ms * G + g] : 127u;
      }
    }
  };

  float acc[MATS][NT][4];
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][t][i] = 0.f;

  Slice<MATS, NT> cur, next;
  weights(kw, cur);
  // the codes of the tokens come from the previous kernel, the weights do not
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tokens(kw, cur);
#pragma unroll 1
  for (int g = kw; g < G; g += KW) {
    weights(g + KW, next);
    tokens(g + KW, next);
    float part[MATS][NT][4];
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[a][t][i] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t b[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) to_half4(word_of(cur.x[t][h], i), b[t][0], b[t][1]);
#pragma unroll
        for (int a = 0; a < MATS; ++a) {
          uint32_t f[4];
          to_half4(word_of(cur.w[a][0][h], i), f[0], f[2]);
          to_half4(word_of(cur.w[a][1][h], i), f[1], f[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(part[a][t], f, b[t][0], b[t][1]);
        }
      }
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[a][t][i] = fmaf(part[a][t][i] * fp8_scale(cur.sw[a][i >> 1]),
                              fp8_scale(cur.sx[t][i & 1]), acc[a][t][i]);
    cur = next;
  }

#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][a][t * 4 + i][lane] = acc[a][t][i];
  if (CODES && threadIdx.x < NT * 8) tops[threadIdx.x] = 0;
  __syncthreads();

  // one output each: token e / (16 RT), row e % (16 RT)
  constexpr int OUTS = NT * 8 * 16 * RT, EACH = (OUTS + kWarps * 32 - 1) / (kWarps * 32);
  float value[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int e = threadIdx.x + j * kWarps * 32;
    value[j] = 0.f;
    if (e >= OUTS) continue;
    const int row = e % (16 * RT), tok = e / (16 * RT);
    const int i = (tok >> 3) * 4 + ((row >> 3) & 1) * 2 + (tok & 1);
    const int from = (row & 7) * 4 + ((tok & 7) >> 1);
    float sum[MATS];
#pragma unroll
    for (int a = 0; a < MATS; ++a) {
      sum[a] = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) sum[a] += red[(row >> 4) * KW + k][a][i][from];
    }
    value[j] = MATS == 2 ? gated<GELU>(sum[0], sum[MATS - 1]) : sum[0];
    const long n = static_cast<long>(blockIdx.x) * (16 * RT) + row, m = m0 + tok;
    if (!CODES) {
      if (n < p.N && m < p.M) p.y[m * p.N + n] = __float2half_rn(value[j]);
    } else if (n < p.N) {
      atomicMax(&tops[tok], __float_as_uint(fabsf(value[j])));
    }
  }
  if (CODES) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int e = threadIdx.x + j * kWarps * 32;
      if (e >= OUTS) continue;
      const int row = e % (16 * RT), tok = e / (16 * RT);
      uint32_t top = 0;
#pragma unroll
      for (int b = 0; b < KW; ++b) top = max(top, *cluster.map_shared_rank(&tops[tok], b));
      const uint32_t byte = fp8_scale_byte(__uint_as_float(top));
      const long n = static_cast<long>(blockIdx.x) * (16 * RT) + row, m = m0 + tok;
      if (n < p.N && m < p.M) {
        p.codes[m * p.N + n] =
            static_cast<uint8_t>(fp8_pack4(value[j] * fp8_scale_inverse(byte), 0.f, 0.f, 0.f));
        if ((n & (kFp8Group - 1)) == 0)
          p.scales[m * fp8_groups_of(p.N) + n / kFp8Group] = static_cast<uint8_t>(byte);
      }
    }
    cluster.sync();  // the others may still read this block's maxima
  }
}

template <int MATS, int NT, int KW, bool CODES, bool GELU>
int launch_t(const Fp8Params &p, cudaStream_t s) {
  constexpr int rows = 16 * (kWarps / KW);
  long blocks = (p.N + rows - 1) / rows;
  if (CODES) blocks = (blocks + KW - 1) / KW * KW;
  const long tiles = (p.M + NT * 8 - 1) / (NT * 8);
  if (blocks > 0x7fffffffL || tiles > 65535) return W8A8_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(tiles));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = KW;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CODES ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, few_kernel<MATS, NT, KW, CODES, GELU>, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  return launch_status();
}

template <int MATS, bool CODES, bool GELU>
int launch_n(const Fp8Params &p, cudaStream_t s) {
  // eight warps on a row's groups where it has 32 or more, so that every warp
  // still has four; else four
  const bool wide = p.G >= 32;
  if (p.M <= 8) return wide ? launch_t<MATS, 1, 8, CODES, GELU>(p, s) : launch_t<MATS, 1, 4, CODES, GELU>(p, s);
  return wide ? launch_t<MATS, 2, 8, CODES, GELU>(p, s) : launch_t<MATS, 2, 4, CODES, GELU>(p, s);
}

}  // namespace

int launch_fp8_few(const Fp8Params &p, cudaStream_t s) {
  if (p.w[1] == nullptr) return launch_n<1, false, false>(p, s);
  if (p.codes != nullptr) return p.gelu ? launch_n<2, true, true>(p, s) : launch_n<2, true, false>(p, s);
  return p.gelu ? launch_n<2, false, true>(p, s) : launch_n<2, false, false>(p, s);
}

}  // namespace w8a8
