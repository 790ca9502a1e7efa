// What the key/value cache kernels share: the cache as the kernels see it and
// the exact conversion of its codes.
#pragma once

#include "common.cuh"

namespace w8a8 {

// A paged cache.  Token row (page, head, offset) of K and of V is row
// ((page * heads + head) << page_shift) + offset of codes [rows, D bits / 8]
// and scales [rows]; every row index is 64-bit (a cache of one layer may pass
// 4 GB).
struct KvView {
  uint8_t *kc, *vc;
  float *ks, *vs;
  long long pages;
  int heads, page_shift;
  unsigned int *err;

  __device__ __forceinline__ long long row(long long page, int h) const {
    return (page * heads + h) << page_shift;
  }
};

constexpr int kMinPage = 16, kMaxPage = 1024;

// Tokens that a table may hold.  Token positions are 32-bit numbers, also those of the
// last unit of work that lie past a sequence's end (fewer than 1024): they must not wrap,
// or they would pass as positions before it, and the table be read before its start.
constexpr long long kMaxTokens = 0x80000000LL - 65536;

struct KvAttnParams {
  KvView kv;
  const __half *q;
  long long q_ts, q_hs;  // strides of q in elements: token, head
  int T, Hq, group, B, max_q;
  const int *q_offsets;  // [B + 1], or null: one query per sequence
  const int *table;      // [B, table_w]
  int table_w;
  const int *lens;       // [B]
  float scale;           // of the scores
  int causal, window;
  __half *out;           // [T, Hq, D]
  float *lse;            // [T, Hq] or null
  float *ws;
  long long wait_limit;  // of the kernels' waits, in cycles
  int skip_first_copy;   // test only: each block's first copy or hand-over is left out
};

// Queries [q0, q0 + nq) and length of sequence b.  Offsets outside [0, T] or
// out of order and lengths outside [0, table_w * page] are clamped, so that
// no index taken from them leaves its buffer, and reported.
__device__ __forceinline__ void seq_of(const KvAttnParams &p, int b, int &q0, int &nq, int &len) {
  int bad = 0;
  if (p.q_offsets != nullptr) {
    const int a = __ldg(p.q_offsets + b), e = __ldg(p.q_offsets + b + 1);
    q0 = min(max(a, 0), p.T);
    const int q1 = min(max(e, q0), p.T);
    nq = q1 - q0;
    bad = (q0 != a) | (q1 != e) | (nq > p.max_q);
    nq = min(nq, p.max_q);
  } else {
    q0 = b;
    nq = 1;
  }
  const int n = __ldg(p.lens + b);
  const long long cap = static_cast<long long>(p.table_w) << p.kv.page_shift;
  len = static_cast<int>(min(static_cast<long long>(max(n, 0)), cap));
  bad |= len != n;
  if (bad) report_index(p.kv.err);
}

// Keys that the query at position pos of a sequence of len tokens sees:
// [lo, hi).  pos may be negative (more queries than tokens): nothing.  (The window is
// not taken from a position before its end: for a window near 2^31 that wraps.)
__device__ __forceinline__ void visible(const KvAttnParams &p, int pos, int len, int &lo, int &hi) {
  hi = p.causal ? min(pos + 1, len) : len;
  lo = p.window > 0 && pos >= p.window ? pos + 1 - p.window : 0;
}

__device__ __forceinline__ int entry_of(const KvAttnParams &p, int b, int i) {
  return __ldg(p.table + static_cast<long long>(b) * p.table_w + i);
}

// Page of a table entry; an entry outside the cache reads as -1 (its tokens
// are left out) and is reported.
__device__ __forceinline__ int checked_page(const KvAttnParams &p, int e) {
  if (static_cast<unsigned>(e) < static_cast<unsigned long long>(p.kv.pages)) return e;
  report_index(p.kv.err);
  return -1;
}
__device__ __forceinline__ int page_of(const KvAttnParams &p, int b, int i) {
  return checked_page(p, entry_of(p, b, i));
}

// ---- exact conversion of codes to fp16 --------------------------------------

// 0x6400 | u is the fp16 value 1024 + u for u < 1024
__device__ __forceinline__ uint32_t h2_add(uint32_t a, float c) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&a), __float2half2_rn(c));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, float m, float c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), __float2half2_rn(m), __float2half2_rn(c));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// (w & MASK) ^ magic in one instruction.  One operand may be an immediate, so
// the magic has to sit in a register: opaque() keeps the compiler from folding
// it back, which would take two instructions (measured: a quarter of the
// few-row attention kernel's integer work).
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(w), "n"(MASK), "r"(magic));
  return d;
}
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  uint32_t d;
  asm volatile("mov.b32 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// Two's-complement nibbles k and k + 4 of a word, k = 0 .. 3, as the fp16 pairs
// o[k] = (nibble k, nibble k + 4): the nibble with its sign bit flipped (v + 8)
// lands in the low bits of 1024 + (v + 8), or of 1024 + 16 (v + 8), which
// one multiply-add brings back; every step is exact.
struct Nibbles {
  uint32_t lo, hi;  // the magics
  __device__ __forceinline__ Nibbles() : lo(opaque(0x64086408u)), hi(opaque(0x64806480u)) {}
  __device__ __forceinline__ void to_h(uint32_t w, uint32_t (&o)[4]) const {
    const uint32_t x = w >> 8;
    o[0] = h2_add(and_xor<0x000f000fu>(w, lo), -1032.f);
    o[1] = h2_fma(and_xor<0x00f000f0u>(w, hi), 0.0625f, -72.f);
    o[2] = h2_add(and_xor<0x000f000fu>(x, lo), -1032.f);
    o[3] = h2_fma(and_xor<0x00f000f0u>(x, hi), 0.0625f, -72.f);
  }
};

// Bytes 0, 1 and 2, 3 (two's complement) of a word as two fp16 pairs.
__device__ __forceinline__ void bytes_to_h(uint32_t w, uint32_t &h01, uint32_t &h23) {
  const uint32_t x = w ^ 0x80808080u;
  h01 = h2_add(__byte_perm(x, 0x64646464u, 0x5140), -1152.f);
  h23 = h2_add(__byte_perm(x, 0x64646464u, 0x7362), -1152.f);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The running reference M of a row's exponents.  Weights are 2^(u - M); M is the
// largest u seen when it was set and moves only when some u passes it by kRoom,
// so a weight is below 2^kRoom (fp16 holds 2^15.99) and the largest one at least 1:
// what fp16 cannot hold, under 2^-25, is under 2^-25 of it.  That is a key's share: n keys
// just under it, behind a dominant one, hold up to n 2^-25 together (0.4 % at 131072),
// which the row's sum counts and the output does not.  (Set 7 below that u,
// weights above 2^-21 stayed normal numbers, but M moved more often: a prompt took
// 201 us against 180.)  A row starts at kNoRef, under every u but the very last that
// 32 bits hold.
constexpr float kRoom = 15.f, kNoRef = -3e38f;

// What stands for s_v where it is 0.  All codes are 0 there, so the products do not
// need it, but u and with it M do: it lies below every scale that is ever stored (the
// smallest is 2^-24 / 127), so that a token without a value never takes M above what
// the tokens with one weigh.  (As 1, a leading key of this kind took the others'
// weights out of fp16's range: with values of 0.05 they lost a tenth.)
constexpr float kZeroScale = 0x1p-32f;

}  // namespace w8a8
