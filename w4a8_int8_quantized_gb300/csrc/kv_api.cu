// The C ABI of the key/value cache: host-side argument checks, then the
// launches on the caller's stream.  See include/w8a8.h for the contract.
#include <math.h>

#include "common.cuh"
#include "kv_attn.cuh"
#include "kv_common.cuh"

namespace w8a8 {

int launch_kv_write(const KvView &kv, int bits, int D, const __half *k, long long k_ts,
                    long long k_hs, const __half *v, long long v_ts, long long v_hs,
                    const long long *slots, int T, cudaStream_t s);
int launch_kv_read(const KvView &kv, int bits, int D, const long long *slots, int T, __half *k,
                   __half *v, cudaStream_t s);
namespace {

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Shape of a cache, without its pointers: W8A8_OK or the error.
int check_cache_shape(const w8a8_kv_cache *c) {
  if (c == nullptr) return W8A8_ERR_INVALID_ARG;
  if (c->bits != 4 && c->bits != 8) return W8A8_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return W8A8_ERR_INVALID_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 1024) return W8A8_ERR_INVALID_ARG;
  if (c->page_size < kMinPage || c->page_size > kMaxPage ||
      (c->page_size & (c->page_size - 1)) != 0)
    return W8A8_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->num_pages > 0x7fffffffLL) return W8A8_ERR_INVALID_ARG;
  return W8A8_OK;
}

int check_cache(const w8a8_kv_cache *c) {
  const int st = check_cache_shape(c);
  if (st != W8A8_OK) return st;
  if (c->k_codes == nullptr || c->v_codes == nullptr || c->k_scale == nullptr ||
      c->v_scale == nullptr)
    return W8A8_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

KvView view_of(const w8a8_kv_cache *c) {
  KvView v;
  v.kc = static_cast<uint8_t *>(c->k_codes);
  v.vc = static_cast<uint8_t *>(c->v_codes);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.pages = c->num_pages;
  v.heads = c->kv_heads;
  v.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
  v.err = nullptr;
  return v;
}

// fp16 rows addressed by strides: 16-byte vectors
int check_rows(const void *x, long long ts, long long hs) {
  if (x == nullptr || ts < 0 || hs < 0) return W8A8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || ts % 8 != 0 || hs % 8 != 0) return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

#define W8A8_TRY(expr)              \
  do {                              \
    int _st = (expr);               \
    if (_st != W8A8_OK) return _st; \
  } while (0)

}  // namespace
}  // namespace w8a8

using namespace w8a8;

extern "C" {

int kv_cache_write(const w8a8_half *k, long long k_token_stride, long long k_head_stride,
                   const w8a8_half *v, long long v_token_stride, long long v_head_stride,
                   const int64_t *slots, int T, const w8a8_kv_cache *cache,
                   w8a8_stream_t stream) {
  W8A8_TRY(check_cache_shape(cache));
  if (T < 0) return W8A8_ERR_INVALID_ARG;
  if (T == 0) return W8A8_OK;
  W8A8_TRY(check_cache(cache));
  W8A8_TRY(check_rows(k, k_token_stride, k_head_stride));
  W8A8_TRY(check_rows(v, v_token_stride, v_head_stride));
  if (slots == nullptr) return W8A8_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return W8A8_ERR_MISALIGNED;
  W8A8_TRY(check_device());
  KvView kv = view_of(cache);
  if ((kv.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  return launch_kv_write(kv, cache->bits, cache->head_dim, reinterpret_cast<const __half *>(k),
                         k_token_stride, k_head_stride, reinterpret_cast<const __half *>(v),
                         v_token_stride, v_head_stride,
                         reinterpret_cast<const long long *>(slots), T,
                         static_cast<cudaStream_t>(stream));
}

int kv_cache_read(const int64_t *slots, int T, const w8a8_kv_cache *cache, w8a8_half *k,
                  w8a8_half *v, w8a8_stream_t stream) {
  W8A8_TRY(check_cache_shape(cache));
  if (T < 0) return W8A8_ERR_INVALID_ARG;
  if (T == 0) return W8A8_OK;
  W8A8_TRY(check_cache(cache));
  if (slots == nullptr || k == nullptr || v == nullptr) return W8A8_ERR_INVALID_ARG;
  if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return W8A8_ERR_MISALIGNED;
  W8A8_TRY(check_device());
  KvView kv = view_of(cache);
  if ((kv.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  return launch_kv_read(kv, cache->bits, cache->head_dim,
                        reinterpret_cast<const long long *>(slots), T,
                        reinterpret_cast<__half *>(k), reinterpret_cast<__half *>(v),
                        static_cast<cudaStream_t>(stream));
}

size_t kv_cache_attention_workspace_bytes(int T, int q_heads, int B, int max_q, int table_width,
                                          const w8a8_kv_cache *cache) {
  if (check_cache_shape(cache) != W8A8_OK || T < 0 || q_heads < 1 || B < 0 || max_q < 1 ||
      table_width < 0 || q_heads % cache->kv_heads != 0)
    return 0;
  if (T == 0 || B == 0) return 0;
  const long long rows = static_cast<long long>(max_q < T ? max_q : T) * (q_heads / cache->kv_heads);
  return rows <= few_rows(cache->bits, cache->head_dim) ? kv_decode_workspace(cache->head_dim, rows)
                                                              : kv_prefill_workspace(cache->head_dim);
}

int kv_cache_attention(const w8a8_half *q, long long q_token_stride, long long q_head_stride,
                       int T, int q_heads, const int32_t *q_offsets, int B, int max_q,
                       const int32_t *block_table, int table_width, const int32_t *seq_lens,
                       const w8a8_kv_cache *cache, float softmax_scale, int causal, int window,
                       void *workspace, size_t ws_bytes, w8a8_half *out, float *lse,
                       w8a8_stream_t stream) {
  W8A8_TRY(check_cache_shape(cache));
  if (T < 0 || B < 0 || q_heads < 1 || q_heads % cache->kv_heads != 0 || max_q < 1 ||
      table_width < 0 || window < 0 || (causal != 0 && causal != 1) || (window > 0 && !causal) ||
      !isfinite(softmax_scale))
    return W8A8_ERR_INVALID_ARG;
  if (q_offsets == nullptr && T != B) return W8A8_ERR_INVALID_ARG;
  if (static_cast<long long>(table_width) * cache->page_size > kMaxTokens)
    return W8A8_ERR_INVALID_ARG;
  if (T == 0) return W8A8_OK;
  if (B == 0) {  // no sequence owns a row
    if (out == nullptr) return W8A8_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4)) return W8A8_ERR_MISALIGNED;
    W8A8_TRY(check_device());
    return launch_kv_blank(reinterpret_cast<__half *>(out), lse, static_cast<long long>(T) * q_heads,
                           cache->head_dim, static_cast<cudaStream_t>(stream));
  }
  W8A8_TRY(check_cache(cache));
  W8A8_TRY(check_rows(q, q_token_stride, q_head_stride));
  if (out == nullptr || seq_lens == nullptr || (block_table == nullptr && table_width > 0))
    return W8A8_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q_offsets, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(lse, 4))
    return W8A8_ERR_MISALIGNED;
  if (q_offsets == nullptr) max_q = 1;
  if (max_q > T) max_q = T;
  const size_t need = kv_cache_attention_workspace_bytes(T, q_heads, B, max_q, table_width, cache);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < need))
    return W8A8_ERR_WORKSPACE;
  W8A8_TRY(check_device());
  KvAttnParams p;
  p.kv = view_of(cache);
  if ((p.kv.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  p.q = reinterpret_cast<const __half *>(q);
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.T = T;
  p.Hq = q_heads;
  p.group = q_heads / cache->kv_heads;
  p.B = B;
  p.max_q = max_q;
  p.q_offsets = q_offsets;
  p.table = block_table;
  p.table_w = table_width;
  p.lens = seq_lens;
  p.scale = softmax_scale;
  p.causal = causal;
  p.window = window;
  p.out = reinterpret_cast<__half *>(out);
  p.lse = lse;
  p.ws = static_cast<float *>(workspace);
  p.wait_limit = role_wait_limit();
  p.skip_first_copy = skip_first_copy();
  const bool few = static_cast<long long>(max_q) * p.group <= few_rows(cache->bits, cache->head_dim);
  return (few ? launch_kv_decode : launch_kv_prefill)(p, cache->bits, cache->head_dim,
                                                      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
