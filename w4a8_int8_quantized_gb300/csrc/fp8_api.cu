// The C ABI of the norm and of the 8-bit float layers: host-side argument
// checks, then the launches on the caller's stream.  See include/w8a8.h for the
// contract of each call.
#include <math.h>

#include "common.cuh"
#include "fp8_kernels.cuh"

namespace w8a8 {
namespace {

#define W8A8_TRY(expr)              \
  do {                              \
    int _st = (expr);               \
    if (_st != W8A8_OK) return _st; \
  } while (0)

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int check_row(int K) {
  if (K <= 0 || K > kMaxK) return W8A8_ERR_INVALID_ARG;
  return K % 16 == 0 ? W8A8_OK : W8A8_ERR_MISALIGNED;
}

int check_ptrs(std::initializer_list<const void *> ps, unsigned align) {
  for (const void *p : ps)
    if (p == nullptr) return W8A8_ERR_INVALID_ARG;
  for (const void *p : ps)
    if ((reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0) return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  return ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need
             ? W8A8_ERR_WORKSPACE
             : W8A8_OK;
}

cudaStream_t as_stream(w8a8_stream_t s) { return static_cast<cudaStream_t>(s); }
const __half *as_half(const w8a8_half *p) { return reinterpret_cast<const __half *>(p); }
__half *as_half(w8a8_half *p) { return reinterpret_cast<__half *>(p); }

// bytes of e4m3 rows, and of them with their scales, each region rounded up
size_t code_bytes(int M, int K) { return round256(static_cast<size_t>(M) * K); }
size_t held_bytes(int M, int K) {
  return code_bytes(M, K) + round256(static_cast<size_t>(M) * fp8_groups_of(K));
}

Fp8Params product(const uint8_t *x, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, int M,
                  int N, int K) {
  Fp8Params p = {};
  p.x = x;
  p.sx = sx;
  p.w[0] = w;
  p.sw[0] = sw;
  p.M = M;
  p.N = N;
  p.K = K;
  p.G = fp8_groups_of(K);
  p.early = true;
  return p;
}

// The product of p.x, p.sx, or of fp16 rows x: quantized into the room at p.x, p.sx
// before it, or, if they are few, by the product itself.
int launch_product(Fp8Params &p, cudaStream_t s, const __half *x = nullptr) {
  // The small tiles are for up to about a thousand rows, or for few columns; beyond
  // 8192 rows they are not considered, nor is K divided (8192 x 64 x 14336 takes 27
  // us, 8193 rows 38).
  bool small = p.M <= 8192;
  Fp8Plan plan = {};
  if (small) {
    plan = plan_fp8_mid(p);
    small = p.M <= 128 || plan.split > 1 || plan.us <= estimate_fp8_tc(p);
  }
  if (x != nullptr) {
    if (small && fp8_mid_quantizes(p, plan))
      p.xh = x;
    else
      W8A8_TRY(launch_quant_fp8(x, p.M, p.K, true, const_cast<uint8_t *>(p.x), const_cast<uint8_t *>(p.sx), s));
  }
  return small ? launch_fp8_mid(p, plan, s) : launch_fp8_tc(p, s);
}

// x, r, w, h of the norm; the outputs are the callers' to check
int check_norm(const w8a8_half *x, const w8a8_half *residual, const w8a8_half *weight, int M, int K,
               float eps, const w8a8_half *residual_out) {
  if (M < 0 || !isfinite(eps) || eps < 0.f) return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  if ((residual == nullptr) != (residual_out == nullptr)) return W8A8_ERR_INVALID_ARG;
  if (M == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({x, weight}, 16));
  if (residual != nullptr) W8A8_TRY(check_ptrs({residual, residual_out}, 16));
  return W8A8_OK;
}

}  // namespace
}  // namespace w8a8

using namespace w8a8;

extern "C" {

int rms_norm(const w8a8_half *x, const w8a8_half *residual, const w8a8_half *weight, int M, int K,
             float eps, w8a8_half *residual_out, w8a8_half *y, w8a8_stream_t stream) {
  W8A8_TRY(check_norm(x, residual, weight, M, K, eps, residual_out));
  if (M == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({y}, 16));
  W8A8_TRY(check_device());
  return launch_rms_norm(as_half(x), as_half(residual), as_half(weight), M, K, eps,
                         as_half(residual_out), as_half(y), as_stream(stream));
}

int rms_norm_quantize(const w8a8_half *x, const w8a8_half *residual, const w8a8_half *weight, int M,
                      int K, float eps, int format, int group_size, w8a8_half *residual_out, void *q,
                      void *scale, w8a8_stream_t stream) {
  if (format != W8A8_CODES_INT8 && format != W8A8_CODES_HALF && format != W8A8_CODES_FP8)
    return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_norm(x, residual, weight, M, K, eps, residual_out));
  if (format == W8A8_CODES_FP8 ? group_size != 128 : !valid_group_size(K, group_size))
    return W8A8_ERR_INVALID_ARG;
  if (M == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({q}, 16));
  W8A8_TRY(check_ptrs({scale}, format == W8A8_CODES_FP8 ? 1 : 4));
  W8A8_TRY(check_device());
  return launch_rms_norm_quant(as_half(x), as_half(residual), as_half(weight), M, K, eps, format,
                               group_size, as_half(residual_out), q, scale, as_stream(stream));
}

static int quantize_fp8(const w8a8_half *x, int rows, int K, uint8_t *q, uint8_t *scale,
                        w8a8_stream_t stream) {
  if (rows < 0) return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  if (rows == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({x, q}, 16));
  W8A8_TRY(check_ptrs({scale}, 1));
  W8A8_TRY(check_device());
  return launch_quant_fp8(as_half(x), rows, K, false, q, scale, as_stream(stream));
}

int quantize_weight_fp8(const w8a8_half *W, int N, int K, uint8_t *Wq, uint8_t *scale_w,
                        w8a8_stream_t stream) {
  return quantize_fp8(W, N, K, Wq, scale_w, stream);
}

int quantize_act_fp8(const w8a8_half *x, int M, int K, uint8_t *xq, uint8_t *scale_a,
                     w8a8_stream_t stream) {
  return quantize_fp8(x, M, K, xq, scale_a, stream);
}

int fp8_gemm(const uint8_t *xq, const uint8_t *scale_a, const uint8_t *Wq, const uint8_t *scale_w,
             int M, int N, int K, w8a8_half *y, w8a8_stream_t stream) {
  if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  if (M == 0 || N == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({xq, Wq, y}, 16));
  W8A8_TRY(check_ptrs({scale_a, scale_w}, 1));
  W8A8_TRY(check_device());
  Fp8Params p = product(xq, scale_a, Wq, scale_w, M, N, K);
  p.y = as_half(y);
  return launch_product(p, as_stream(stream));
}

int fp8_gated_gemm(const uint8_t *xq, const uint8_t *scale_a, const uint8_t *Wg,
                   const uint8_t *scale_g, const uint8_t *Wu, const uint8_t *scale_u, int M, int F,
                   int K, int activation, w8a8_half *h, uint8_t *hq, uint8_t *scale_h,
                   w8a8_stream_t stream) {
  if (M < 0 || F < 0 || (activation != W8A8_GATE_SILU && activation != W8A8_GATE_GELU))
    return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  // one form of output, and codes are rows of a product to come
  if (h != nullptr && (hq != nullptr || scale_h != nullptr)) return W8A8_ERR_INVALID_ARG;
  if (h == nullptr && F > 0) W8A8_TRY(check_row(F));
  if (M == 0 || F == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({xq, Wg, Wu}, 16));
  W8A8_TRY(check_ptrs({scale_a, scale_g, scale_u}, 1));
  if (h != nullptr) {
    W8A8_TRY(check_ptrs({h}, 16));
  } else {
    W8A8_TRY(check_ptrs({hq}, 16));
    W8A8_TRY(check_ptrs({scale_h}, 1));
  }
  W8A8_TRY(check_device());
  Fp8Params p = product(xq, scale_a, Wg, scale_g, M, F, K);
  p.w[1] = Wu;
  p.sw[1] = scale_u;
  p.gelu = activation == W8A8_GATE_GELU;
  p.y = as_half(h);
  p.codes = hq;
  p.scales = scale_h;
  p.early = h != nullptr;
  return launch_product(p, as_stream(stream));
}

size_t fp8_linear_workspace_bytes(int M, int K) {
  return M < 0 || check_row(K) != W8A8_OK ? 0 : held_bytes(M, K);
}

int fp8_linear(const w8a8_half *x, const uint8_t *Wq, const uint8_t *scale_w, int M, int N, int K,
               void *workspace, size_t ws_bytes, w8a8_half *y, w8a8_stream_t stream) {
  if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  if (M == 0 || N == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({x, Wq, y}, 16));
  W8A8_TRY(check_ptrs({scale_w}, 1));
  W8A8_TRY(check_workspace(workspace, ws_bytes, held_bytes(M, K)));
  W8A8_TRY(check_device());
  uint8_t *xq = static_cast<uint8_t *>(workspace), *sx = xq + code_bytes(M, K);
  Fp8Params p = product(xq, sx, Wq, scale_w, M, N, K);
  p.y = as_half(y);
  return launch_product(p, as_stream(stream), as_half(x));
}

size_t fp8_feed_forward_workspace_bytes(int M, int K, int F) {
  return M < 0 || check_row(K) != W8A8_OK || check_row(F) != W8A8_OK
             ? 0
             : held_bytes(M, K) + held_bytes(M, F);
}

int fp8_feed_forward(const w8a8_half *x, const uint8_t *Wg, const uint8_t *scale_g,
                     const uint8_t *Wu, const uint8_t *scale_u, const uint8_t *Wd,
                     const uint8_t *scale_d, int M, int K, int F, int N, int activation,
                     void *workspace, size_t ws_bytes, w8a8_half *y, w8a8_stream_t stream) {
  if (M < 0 || N < 0 || (activation != W8A8_GATE_SILU && activation != W8A8_GATE_GELU))
    return W8A8_ERR_INVALID_ARG;
  W8A8_TRY(check_row(K));
  W8A8_TRY(check_row(F));
  if (M == 0 || N == 0) return W8A8_OK;
  W8A8_TRY(check_ptrs({x, Wg, Wu, Wd, y}, 16));
  W8A8_TRY(check_ptrs({scale_g, scale_u, scale_d}, 1));
  W8A8_TRY(check_workspace(workspace, ws_bytes, fp8_feed_forward_workspace_bytes(M, K, F)));
  W8A8_TRY(check_device());
  const cudaStream_t s = as_stream(stream);
  uint8_t *xq = static_cast<uint8_t *>(workspace), *sx = xq + code_bytes(M, K);
  uint8_t *hq = xq + held_bytes(M, K), *sh = hq + code_bytes(M, F);
  Fp8Params up = product(xq, sx, Wg, scale_g, M, F, K);
  up.w[1] = Wu;
  up.sw[1] = scale_u;
  up.gelu = activation == W8A8_GATE_GELU;
  up.codes = hq;
  up.scales = sh;
  W8A8_TRY(launch_product(up, s, as_half(x)));
  Fp8Params down = product(hq, sh, Wd, scale_d, M, N, F);
  down.y = as_half(y);
  return launch_product(down, s);
}

}  // extern "C"
