// The 8-bit float products' launchers, shared by their translation units.
#pragma once

#include "common.cuh"

namespace w8a8 {

// y = x w[0]^T, or act(x w[0]^T) (x w[1]^T) where w[1] is given, as fp16 (y) or
// as e4m3 codes with scales (codes, scales).
struct Fp8Params {
  const uint8_t *x, *sx;        // e4m3 [M, K], e8m0 [M, G]
  const __half *xh;             // or fp16 [M, K], quantized by the product (fp8_mid_quantizes())
  const uint8_t *w[2], *sw[2];  // e4m3 [N, K], e8m0 [N, G]
  int M, N, K, G;
  bool gelu;
  bool early;                   // the next kernel may start at once: not before a caller's codes (see norm.cu)
  __half *y;                    // fp16 [M, N]
  uint8_t *codes, *scales;      // e4m3 [M, N], e8m0 [M, ceil(N / 128)]
};

__host__ __device__ __forceinline__ int fp8_groups_of(int K) { return (K + 127) / 128; }

// How fp8_mid.cu works on a product: CTAs that share a tile, tokens of each and
// columns of the tile, parts of K, tiles that share a group of codes; and about how long it takes, in microseconds.
struct Fp8Plan {
  int cg, mr, bn, split, nx;
  float us;
};

// Tiles of up to 128 x 128, K divided (fp8_mid.cu), and pairs of CTAs on tiles of
// 256 x 256 (fp8_tc.cu), which is for undivided K alone.
Fp8Plan plan_fp8_mid(const Fp8Params &p);
bool fp8_mid_quantizes(const Fp8Params &p, const Fp8Plan &plan);  // a few fp16 rows: xh
int launch_fp8_mid(const Fp8Params &p, const Fp8Plan &plan, cudaStream_t s);
float estimate_fp8_tc(const Fp8Params &p);
int launch_fp8_tc(const Fp8Params &p, cudaStream_t s);

// early: the next kernel may start at once (see norm.cu): for codes that only this library reads
int launch_quant_fp8(const __half *x, long rows, int K, bool early, uint8_t *q, uint8_t *scale,
                     cudaStream_t s);
int launch_rms_norm(const __half *x, const __half *r, const __half *w, int M, int K, float eps,
                    __half *h, __half *y, cudaStream_t s);
int launch_rms_norm_quant(const __half *x, const __half *r, const __half *w, int M, int K,
                          float eps, int format, int group_size, __half *h, void *q, void *scale,
                          cudaStream_t s);

}  // namespace w8a8
