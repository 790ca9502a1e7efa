// Attention of a few query rows per sequence over the quantized cache (one
// token a step, or a handful for draft verification).
//
// Rows of one kv head share its keys, so an item is (sequence, kv head, block
// of 8 NT rows = queries x heads of the group), and the cache is read once per
// item.  Bound by that read: at 4 bits, D = 128, 136 bytes a token and kv head
// against 4 D multiply-adds per row, far too many for scalar arithmetic at
// the rate the bytes arrive (4 rows: 64 us of fused multiply-adds for 46 us of
// bytes), so both products run on mma.sync.m16n8k16 with the tokens (then the
// head dimension) as the 16 rows and the query rows as the 8 columns.  A warp converts
// codes straight into its operand registers that way; tcgen05, whose rows the tokens
// could fill just as well, takes them from shared or tensor memory, where every code
// would have to be written as fp16 first.
//
// Measured (8 kv heads of 4 rows, D = 128, 4 bits): 64 sequences of 512..8192 tokens 80 us,
// one of 131072 35.5, against 44.9 and 21.1 of bytes.  Nothing is saturated (53 % issue,
// 52 % ALU, 51 % DRAM): what is left is the latency of one dependent chain a warp.
//
// The contraction index of either product may be permuted freely as long as
// both operands agree, which removes every shuffle between memory and the
// tensor cores (lane = 4 g + t throughout):
//   S^T = K Q^T   the lane reads 16 bytes (4 bits, D = 128) of the rows of two
//                 tokens per tile of 16; its codes are the operand of D / 16
//                 products once converted, and Q is laid out to match once per
//                 item;
//   O^T = V^T P^T the lane reads its D / 8 values of the tokens of its columns;
//                 tokens are merged into operand registers by byte permutes.
// Codes arrive in a ring of shared-memory stages per warp, by bulk copies that
// the warp itself issues two steps ahead, page by page.
//
// Softmax: u = S * scale * log2e * s_k + log2 s_v, weight p = 2^(u - M), so the
// weight carries the value's scale: O = sum p code_v with exact codes, and the
// row's sum is sum p / s_v.  M is the lazy reference of kv_common.cuh: while no
// weight passes 2^15 (one vote per step) nothing is rescaled or exchanged.
// s_v = 0 (all codes 0) counts as kZeroScale.
//
// Split: the units (4 warps x one step of tokens) of all items form one line,
// cut into equal ranges, one per resident block, so ragged lengths balance to
// one unit.  An item inside one range is finished there; an item cut by
// ranges leaves one partial (M, sum, O) per block, which a second kernel joins
// in ascending order (the result does not depend on timing).
#include <math_constants.h>

#include <mutex>

#include "common.cuh"
#include "kv_attn.cuh"
#include "kv_common.cuh"

namespace w8a8 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// BITS, D: the cache; NT: column tiles of 8 rows in an item.
template <int BITS, int D, int NT>
struct Plan {
  static constexpr int ROW = D * BITS / 8;           // bytes of a token's codes
  // 16-token tiles per step: 4 KB of K (2 KB for two column tiles, whose sums
  // take the registers; 64 tokens at most).  Half as much cost a tenth more time
  // (64 sequences of 512..8192 tokens: 87 us against 81): the step's fixed work.
  static constexpr int MT = NT == 2 ? 16 / BITS * 64 / D : BITS == 4 && D == 64 ? 4 : 32 / BITS * 64 / D;
  static constexpr int STEP = 16 * MT;               // tokens of a warp's step
  static constexpr int UNIT = kWarps * STEP;         // tokens of a block's step
  static constexpr int KW = ROW / 16;                // K words per token and lane
  static constexpr int VW = ROW / 32;                // V words per token and lane
  static constexpr int MMAS = D / 16;                // 16-row tiles of D
  static constexpr int COLS = 8 * NT;  // rows of an item
  static constexpr int PAD = D + 4;                  // floats of a staged row
  static constexpr int BLOCKS = 3;                   // resident per SM
  // a stage of a warp's ring: one step's K codes, V codes, K scales, V scales
  static constexpr int OFF_V = STEP * ROW, OFF_KS = 2 * STEP * ROW, OFF_VS = OFF_KS + STEP * 4;
  static constexpr int STAGE = OFF_VS + STEP * 4;
  static constexpr int TILE_BYTES = 2 * 16 * ROW + 2 * 16 * 4;  // of one 16-token tile
  static constexpr int STAGES = NT == 2 ? 4 : 2;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int JOIN = kWarps * COLS * PAD * 4;  // the warps' results, over the drained ring
  static constexpr int OFF_SCALES = RING > JOIN ? RING : JOIN;  // a warp's step: 16 bytes a token
  static constexpr int OFF_BAR = OFF_SCALES + kWarps * STEP * 16;
  static constexpr int SMEM = OFF_BAR + kWarps * STAGES * 8;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Waits for a phase of an mbarrier, the whole warp together; false if it gave up
// after `limit` cycles.
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, long long limit) {
  uint32_t ok;
  long long t0 = 0;
  for (int i = 0;; ++i) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "vote.sync.all.pred p, p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (i == 64) t0 = clock64();
    if (i > 64 && __any_sync(0xffffffffu, clock64() - t0 > limit)) return false;
  }
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, int bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// W words from shared memory
template <int W>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *o) {
  static_assert(W == 1 || W == 2 || W == 4, "");
  if (W == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(o[0]) : "r"(a));
  else if (W == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(o[0]), "=r"(o[1]) : "r"(a));
  else
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
                 : "r"(a));
}

// W words from p, as the widest loads
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *o) {
  static_assert(W == 1 || W == 2 || W == 4, "");
  if (W == 1) {
    o[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
  } else if (W == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    o[0] = v.x;
    o[1] = v.y;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
    o[0] = v.x;
    o[1] = v.y;
    o[2] = v.z;
    o[3] = v.w;
  }
}

// What a warp knows of its item: which keys its rows see.
struct Item {
  int b, h, rb, R;             // sequence, kv head, row block, its rows
  int q0, nq, len;             // queries, tokens of the sequence
  int lo_max, hi_min;          // keys [lo_max, hi_min) are seen by all rows,
  int lo_min, hi_max;          // those outside [lo_min, hi_max) by none
  bool bad;                    // a page outside the cache was met

  // output row of row c
  __device__ __forceinline__ long long row(const KvAttnParams &p, int c, int cols) const {
    const int ri = rb * cols + c;
    return (static_cast<long long>(q0) + ri / p.group) * p.Hq + h * p.group + ri % p.group;
  }
  // its query
  __device__ __forceinline__ const __half *query(const KvAttnParams &p, int c, int cols) const {
    const int ri = rb * cols + c;
    return p.q + (q0 + ri / p.group) * p.q_ts + static_cast<long long>(h * p.group + ri % p.group) * p.q_hs;
  }
  __device__ __forceinline__ void limits(const KvAttnParams &p, int c, int cols, int &lo, int &hi) const {
    lo = hi = 0;
    if (c < R) visible(p, len - nq + (rb * cols + c) / p.group, len, lo, hi);
  }
  // token a belongs to a page outside the cache
  __device__ __forceinline__ bool gone(const KvAttnParams &p, int a) const {
    return bad && a < hi_max && page_of(p, b, a >> p.kv.page_shift) < 0;
  }
};

// A token's scales from a stage: s_k times `f`, log2 s_v and 1 / s_v.
__device__ __forceinline__ void token_scales(uint32_t ks_at, uint32_t vs_at, float f, float &sk,
                                             float &lv, float &rv) {
  uint32_t x, y;
  lds_words<1>(ks_at, &x);
  lds_words<1>(vs_at, &y);
  sk = __uint_as_float(x) * f;
  const float sv = y == 0 ? kZeroScale : __uint_as_float(y);
  lv = log2_fast(sv);
  rv = rcp_fast(sv);
}

template <int BITS, int D, int NT>
struct Math {
  using PL = Plan<BITS, D, NT>;
  static constexpr int MT = PL::MT, MMAS = PL::MMAS, ROW = PL::ROW, COLS = PL::COLS;
  const KvAttnParams &p;
  const int g, t;
  const Nibbles nib;
  const float f;
  const uint32_t scales;  // the step's (s_k f, log2 s_v, 1 / s_v) per token, in shared memory
  uint32_t k_at, v_at, v_row[2], s_at;
  int tokg;
  uint32_t qf[NT][MMAS][2];  // Q: column g of each n
  float o[NT][MMAS][4];
  float m[NT][2], l[NT][2];
  int lo[NT][2], hi[NT][2];

  __device__ __forceinline__ Math(const KvAttnParams &p, int lane, uint32_t scales)
      : p(p), g(lane >> 2), t(lane & 3), f(p.scale * kLog2e), scales(scales) {
    // Row r of a 16-token product stands for token tok(r) (+ 8 for the second
    // half): rows 2t and 2t + 1 are tokens t and 4 + (t ^ 1), so that the lanes
    // of a value load (rows 2t of four t) and of a key load (rows g, g + 1) read
    // rows of both parities of 64 bytes, half of the bank conflicts of tokens
    // in their own order.
    tokg = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;
    k_at = tokg * ROW + t * (PL::KW >= 4 ? 16 : PL::KW * 4);
    v_at = PL::OFF_V + g * (PL::VW * 4);
    v_row[0] = t * ROW;
    v_row[1] = (4 + (t ^ 1)) * ROW;
    s_at = scales + 16 * tokg;
  }

  __device__ __forceinline__ void begin(const Item &it) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = n * 8 + g;
      const bool on = c < it.R;
      const __half *qp = it.query(p, on ? c : 0, COLS);
#pragma unroll
      for (int w = 0; w < PL::KW; ++w) {
        uint32_t x[4] = {0, 0, 0, 0};
        if (BITS == 4) {
          // word w holds d = 8 (t KW + w) .. + 7, in pairs (k, k + 4)
          if (on) load_words<4>(reinterpret_cast<const uint8_t *>(qp + 8 * (t * PL::KW + w)), x);
          qf[n][2 * w][0] = __byte_perm(x[0], x[2], 0x5410);
          qf[n][2 * w][1] = __byte_perm(x[0], x[2], 0x7632);
          qf[n][2 * w + 1][0] = __byte_perm(x[1], x[3], 0x5410);
          qf[n][2 * w + 1][1] = __byte_perm(x[1], x[3], 0x7632);
        } else {
          // words 0-3: d = 16 t + 4 w .. + 3, words 4-7: 64 further on
          const int d = (w & 4) * 16 + 16 * t + 4 * (w & 3);
          if (on) load_words<2>(reinterpret_cast<const uint8_t *>(qp + d), x);
          qf[n][w][0] = x[0];
          qf[n][w][1] = x[1];
        }
      }
#pragma unroll
      for (int i = 0; i < MMAS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = kNoRef;
        l[n][e] = 0.f;
        it.limits(p, n * 8 + 2 * t + e, COLS, lo[n][e], hi[n][e]);
      }
    }
  }

  // The step whose codes are at `stage` and whose first token is j; `ends`:
  // not every row sees every token.
  __device__ __forceinline__ void step(const Item &it, uint32_t stage, int j, bool ends) {
    // scales, once per token
#pragma unroll
    for (int k = 0; k < PL::STEP; k += 32) {
      const int tok = k + 4 * g + t;
      if (PL::STEP >= 32 || tok < PL::STEP) {
        float sk, lv, rv;
        token_scales(stage + PL::OFF_KS + 4 * tok, stage + PL::OFF_VS + 4 * tok, f, sk, lv, rv);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %3};" ::"r"(scales + 16 * tok), "f"(sk), "f"(lv), "f"(rv) : "memory");
      }
    }
    __syncwarp();
    float s[NT][MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t kraw[2][PL::KW];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t a = stage + k_at + (16 * i + 8 * r) * ROW;
        lds_words<(PL::KW < 4 ? PL::KW : 4)>(a, kraw[r]);
        if (PL::KW == 8) lds_words<4>(a + 64, &kraw[r][PL::KW - 4]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][i][0] = s[n][i][1] = s[n][i][2] = s[n][i][3] = 0.f;
#pragma unroll
      for (int w = 0; w < PL::KW; ++w) {
        if (BITS == 4) {
          uint32_t a[4], c[4];
          nib.to_h(kraw[0][w], a);
          nib.to_h(kraw[1][w], c);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(s[n][i], a[0], c[0], a[1], c[1], qf[n][2 * w][0], qf[n][2 * w][1]);
            mma16816(s[n][i], a[2], c[2], a[3], c[3], qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
          }
        } else {
          uint32_t a0, a1, a2, a3;
          bytes_to_h(kraw[0][w], a0, a2);
          bytes_to_h(kraw[1][w], a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(s[n][i], a0, a1, a2, a3, qf[n][w][0], qf[n][w][1]);
        }
      }
    }
    // exponents
    float rv[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t x[4];
        lds_words<4>(s_at + 16 * (16 * i + 8 * r), x);
        const float sk = __uint_as_float(x[0]), lv = __uint_as_float(x[1]);
        rv[i][r] = __uint_as_float(x[2]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[n][i][2 * r + e] = fmaf(s[n][i][2 * r + e], sk, lv);
      }
    if (ends) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int a = j + 16 * i + 8 * r + tokg;
          // from hi_max on nothing was copied: the stage holds an older step's scales;
          // before lo_min, in the 16 that hold the window's first key, any slot's
          const bool out = a < it.lo_min || a >= it.hi_max || it.gone(p, a);
          if (out) rv[i][r] = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (out || a < lo[n][e] || a >= hi[n][e]) s[n][i][2 * r + e] = -CUDART_INF_F;
        }
    }
    // reference
    bool over = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[n][e] = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < MT; ++i) top[n][e] = fmaxf(top[n][e], fmaxf(s[n][i][e], s[n][i][2 + e]));
        over |= top[n][e] > m[n][e] + kRoom;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[n][e];
#pragma unroll
          for (int q = 4; q < 32; q <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, q));
          const float nm = x > m[n][e] + kRoom ? x : m[n][e];
          const float a = exp2_fast(m[n][e] - nm);
          m[n][e] = nm;
          l[n][e] *= a;
#pragma unroll
          for (int i = 0; i < MMAS; ++i) {
            o[n][i][e] *= a;
            o[n][i][2 + e] *= a;
          }
        }
    }
    // weights
    uint32_t pf[NT][MT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w0 = exp2_fast(s[n][i][2 * r] - m[n][0]);
          const float w1 = exp2_fast(s[n][i][2 * r + 1] - m[n][1]);
          l[n][0] = fmaf(w0, rv[i][r], l[n][0]);
          l[n][1] = fmaf(w1, rv[i][r], l[n][1]);
          pf[n][i][r] = transpose8x8(pack_h2(w0, w1));
        }
    // values
    uint32_t vraw[MT][4][PL::VW];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        lds_words<PL::VW>(stage + v_at + v_row[r & 1] + (16 * i + (r & 2) * 4) * ROW, vraw[i][r]);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int w = 0; w < PL::VW; ++w) {
        const uint32_t x0 = vraw[i][0][w], x1 = vraw[i][1][w];
        const uint32_t x2 = vraw[i][2][w], x3 = vraw[i][3][w];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (BITS == 4) {
            const int sel = half ? 0x7632 : 0x5410;
            uint32_t a[4], c[4];
            nib.to_h(__byte_perm(x0, x1, sel), a);
            nib.to_h(__byte_perm(x2, x3, sel), c);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(o[n][4 * w + 2 * half], a[0], a[1], c[0], c[1], pf[n][i][0], pf[n][i][1]);
              mma16816(o[n][4 * w + 2 * half + 1], a[2], a[3], c[2], c[3], pf[n][i][0], pf[n][i][1]);
            }
          } else {
            const int sel = half ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            bytes_to_h(__byte_perm(x0, x1, sel), a0, a1);
            bytes_to_h(__byte_perm(x2, x3, sel), a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[n][2 * w + half], a0, a1, a2, a3, pf[n][i][0], pf[n][i][1]);
          }
        }
      }
  }

  // This warp's sums of the item: o_sm [COLS][PAD], references and sums of weights.
  __device__ __forceinline__ void finish(float (*o_sm)[PL::PAD], float *m_sm, float *l_sm) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = n * 8 + 2 * t + e;
        float x = l[n][e];
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) x += __shfl_xor_sync(0xffffffffu, x, q);
        if (g == 0) {
          m_sm[c] = m[n][e];
          l_sm[c] = x;
        }
        // this lane's d: MMAS pairs (2 i, 2 i + 1) from 2 MMAS g on
        float *dst = &o_sm[c][2 * MMAS * g];
#pragma unroll
        for (int i = 0; i < MMAS; i += 2)
          *reinterpret_cast<float4 *>(dst + 2 * i) =
              make_float4(o[n][i][e], o[n][i][2 + e], o[n][i + 1][e], o[n][i + 1][2 + e]);
      }
  }
};

// Keys that any query of sequence b sees: units of UNIT tokens from `first`
// (a multiple of 16), at least one unit when there is a query to answer.
template <int UNIT>
__device__ __forceinline__ int units_of(const KvAttnParams &p, int nq, int len, int &first) {
  int lo, hi, lo2, hi2;
  visible(p, len - nq, len, lo, hi);
  visible(p, len - 1, len, lo2, hi2);
  first = min(lo, len) & ~15;
  return max((hi2 - first + UNIT - 1) / UNIT, 1);
}

// The joined partials of a row: block c's range ends in an item whose first
// unit it holds; later blocks hold the rest, up to `last`.
struct Desc {
  int b, h, rb, last;
};

template <int BITS, int D, int NT>
__global__ void __launch_bounds__(kThreads, Plan<BITS, D, NT>::BLOCKS)
    kv_decode_kernel(const KvAttnParams p) {
  using PL = Plan<BITS, D, NT>;
  constexpr int MT = PL::MT, COLS = PL::COLS, ROW = PL::ROW;
  extern __shared__ __align__(128) uint8_t dyn[];
  float(*o_sm)[COLS][PL::PAD] = reinterpret_cast<float(*)[COLS][PL::PAD]>(dyn);
  __shared__ float m_sm[kWarps][COLS], l_sm[kWarps][COLS];
  __shared__ long long sums[kThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The next kernel is not let in early: the join's blocks would take their places on the
  // SMs that finish first (64 sequences 80.2 us against 79.3).
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // -- this block's range of units -------------------------------------------
  auto work_of = [&](int b, int &q0, int &nq, int &len, int &first, int &nu, int &nrb) {
    seq_of(p, b, q0, nq, len);
    nu = units_of<PL::UNIT>(p, nq, len, first);
    nrb = (nq * p.group + COLS - 1) / COLS;
    return static_cast<long long>(nu) * nrb * p.kv.heads;
  };
  auto inclusive = [&](long long x) {  // over the warp's lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  // The sequence in which this block's range starts, its first unit, and the range:
  // prefix sums over the sequences, a lane each while they fit a warp (every
  // warp for itself), else `chunk` of them a thread.
  int b;
  long long start, per, c0, c1;
  auto range = [&](long long total) {
    per = total < 0x7fffffff ? (static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x
                             : (total + gridDim.x - 1) / gridDim.x;
    c0 = blockIdx.x * per;
    c1 = min(c0 + per, total);
  };
  if (p.B <= 32) {
    int q0, nq, len, first, nu, nrb;
    const long long mine = lane < p.B ? work_of(lane, q0, nq, len, first, nu, nrb) : 0;
    const long long x = inclusive(mine);
    range(__shfl_sync(0xffffffffu, x, 31));
    b = __popc(__ballot_sync(0xffffffffu, x <= c0));  // sequences that end before c0
    start = __shfl_sync(0xffffffffu, x - mine, b & 31);
  } else {
    const int chunk = (p.B + kThreads - 1) / kThreads;
    long long x = 0;
    for (int i = 0; i < chunk; ++i) {
      const int e = threadIdx.x * chunk + i;
      int q0, nq, len, first, nu, nrb;
      if (e < p.B) x += work_of(e, q0, nq, len, first, nu, nrb);
    }
    x = inclusive(x);
    sums[threadIdx.x] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += sums[w * 32 + 31];
    __syncthreads();
    sums[threadIdx.x] = x;
    __syncthreads();
    range(sums[kThreads - 1]);
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] > c0) hi = mid; else lo = mid + 1;
    }
    b = lo * chunk;
    start = lo > 0 ? sums[lo - 1] : 0;
  }
  Desc *descs = reinterpret_cast<Desc *>(p.ws);
  float *parts = reinterpret_cast<float *>(descs + gridDim.x);
  if (threadIdx.x == 0) descs[blockIdx.x].last = -1;
  if (__any_sync(0xffffffffu, some_unowned(p))) blank_unowned<D>(p.out, p.lse, p.q_offsets, p.T, p.Hq, p.B, p.max_q);
  if (c0 >= c1) return;

  int q0, nq, len, first, nu, nrb;
  long long work = work_of(b, q0, nq, len, first, nu, nrb);
  while (start + work <= c0) {
    start += work;
    work = work_of(++b, q0, nq, len, first, nu, nrb);
  }

  // the warp's ring, and its barriers (one arrival a phase: lane 0)
  constexpr int S = PL::STAGES;
  const uint32_t ring = smem_u32(dyn) + warp * (S * PL::STAGE);
  const uint32_t bars = smem_u32(dyn) + PL::OFF_BAR + warp * (S * 8);
  if (lane < S) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * lane));
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  uint32_t phases = 0;  // bit s: parity of the next wait on stage s
  Math<BITS, D, NT> math(p, lane, smem_u32(dyn) + PL::OFF_SCALES + warp * PL::STEP * 16);

  // copies: lane i < 4 MT brings array i % 4 (K, V, K scales, V scales) of tile
  // i / 4; `page_bytes` from one page to the next
  const int ctile = 16 * (lane >> 2), carr = lane & 3;
  const bool copier = lane < 4 * MT;
  const uint8_t *csrc = carr == 0 ? p.kv.kc : carr == 1 ? p.kv.vc
                        : reinterpret_cast<const uint8_t *>(carr == 2 ? p.kv.ks : p.kv.vs);
  const uint32_t cbytes = carr < 2 ? ROW : 4;  // per token
  const uint32_t page_bytes = (static_cast<uint32_t>(p.kv.heads) << p.kv.page_shift) * cbytes;
  const uint32_t cdst = ring + ctile * cbytes +
                        (carr == 0 ? 0 : carr == 1 ? PL::OFF_V : carr == 2 ? PL::OFF_KS : PL::OFF_VS);
  const int pmask = (1 << p.kv.page_shift) - 1;
  const int run_tokens = min(pmask + 1, PL::STEP);

  for (long long at = c0; at < c1;) {
    while (at >= start + work) {
      start += work;
      work = work_of(++b, q0, nq, len, first, nu, nrb);
    }
    // item: units [istart, istart + nu) of the line
    const int item = at - start < 0x7fffffff ? static_cast<int>(at - start) / nu
                                             : static_cast<int>((at - start) / nu);
    const long long istart = start + static_cast<long long>(item) * nu;
    const int u0 = static_cast<int>(at - istart);
    const int u1 = static_cast<int>(min(static_cast<long long>(nu), c1 - istart));
    at = istart + u1;
    Item it;
    it.b = b;
    it.h = item / nrb;
    it.rb = item % nrb;
    it.R = min(nq * p.group - it.rb * COLS, COLS);
    it.q0 = q0;
    it.nq = nq;
    it.len = len;
    it.bad = false;
    {
      visible(p, len - nq + it.rb * COLS / p.group, len, it.lo_min, it.hi_min);
      visible(p, len - nq + (it.rb * COLS + it.R - 1) / p.group, len, it.lo_max, it.hi_max);
    }

    // -- steps: this warp's tokens are j .. j + STEP - 1 of each unit ----------
    // Page of the copier's tile of the step at token j (-1: past the last key,
    // -2: outside the cache); fetched a step before the copies that use it.
    const uint8_t *hsrc = csrc + (static_cast<size_t>(it.h) << p.kv.page_shift) * cbytes;
    auto page_at = [&](int j) {
      const int a = j + ctile;
      if (!copier || a >= it.hi_max) return -1;
      const int e = page_of(p, b, a >> p.kv.page_shift);
      return e < 0 ? -2 : e;
    };
    auto issue = [&](int page, int j, int st, bool lost = false) {
      if (__any_sync(0xffffffffu, page == -2)) it.bad = true;
      // tiles that follow one another in a page come in one copy
      const int run = (j & (run_tokens - 1)) == 0 ? run_tokens : 16;
      const bool copies = page >= 0 && (ctile & (run - 1)) == 0;
      const uint32_t there = __ballot_sync(0xffffffffu, copies);
      const uint32_t bar = bars + 8 * st;
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                     "r"(__popc(there) / 4 * (run >> 4) * PL::TILE_BYTES)
                     : "memory");
      __syncwarp();
      if (copies && !lost)
        bulk_copy(cdst + st * PL::STAGE,
                  hsrc + static_cast<size_t>(page) * page_bytes + ((j + ctile) & pmask) * cbytes,
                  run * cbytes, bar);
    };
    int j = first + u0 * PL::UNIT + warp * PL::STEP;
    int page[S + 1];  // pages of the first steps; the last one: of the next to be issued
#pragma unroll
    for (int i = 0; i <= S; ++i) page[i] = u0 + i < u1 ? page_at(j + i * PL::UNIT) : -1;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (u0 + i < u1)
        issue(page[i], j + i * PL::UNIT, i, i == 0 && warp == 0 && p.skip_first_copy && istart + u0 == c0);
    int next = page[S];
    int st = 0;
    math.begin(it);

    int u = u0;
    for (; u < u1; ++u, j += PL::UNIT) {
      if (!wait_stage(bars + 8 * st, (phases >> st) & 1u, p.wait_limit)) break;
      phases ^= 1u << st;
      math.step(it, ring + st * PL::STAGE, j, j < it.lo_max || j + PL::STEP > it.hi_min || it.bad);
      // refill the stage: every lane has its registers
      __syncwarp();
      if (u + S < u1) {
        issue(next, j + S * PL::UNIT, st);
        next = u + S + 1 < u1 ? page_at(j + (S + 1) * PL::UNIT) : -1;
      }
      st = st + 1 == S ? 0 : st + 1;
    }

    if (u < u1) {
      // a copy did not land: report it, and let those of the steps u .. u + S - 1,
      // which are all that this warp has in flight, land (bounded)
      if (lane == 0) atomicCAS(p.kv.err, 0u, static_cast<unsigned>(kDevErrCacheCopy));
      for (int i = u; i < u1 && i < u + S; ++i) {
        wait_stage(bars + 8 * st, (phases >> st) & 1u, kTimeoutCycles);
        st = st + 1 == S ? 0 : st + 1;
      }
    }

    // -- join the warps -----------------------------------------------------------
    // Every ring is drained.  After a wait that gave up no barrier is armed again: the
    // block ends.
    if (__syncthreads_or(u < u1)) return;
    math.finish(o_sm[warp], m_sm[warp], l_sm[warp]);
    __syncthreads();
    const bool whole = u0 == 0 && u1 == nu;
    // a block's first piece may go on from the block before: slot 0, else 1
    const int slot = u0 == 0 ? 1 : 0;
    float *part = parts + (static_cast<long long>(blockIdx.x) * 2 + slot) * COLS * (D + 2);
    for (int i = threadIdx.x; i < it.R * (D / 4); i += kThreads) {
      const int c = i / (D / 4), d = i % (D / 4) * 4;
      float mm = m_sm[0][c];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, m_sm[w][c]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = exp2_fast(m_sm[w][c] - mm);
        const float4 y = *reinterpret_cast<const float4 *>(&o_sm[w][c][d]);
        x.x = fmaf(a, y.x, x.x);
        x.y = fmaf(a, y.y, x.y);
        x.z = fmaf(a, y.z, x.z);
        x.w = fmaf(a, y.w, x.w);
        sum = fmaf(a, l_sm[w][c], sum);
      }
      if (whole) {
        const long long row = it.row(p, c, COLS);
        store_row4<D>(p, row, d, x, mm, sum);
      } else {
        *reinterpret_cast<float4 *>(part + c * D + d) = x;
        if (d == 0) {
          part[COLS * D + 2 * c] = mm;
          part[COLS * D + 2 * c + 1] = sum;
        }
      }
    }
    if (!whole && u0 == 0 && threadIdx.x == 0)
      descs[blockIdx.x] = Desc{b, it.h, it.rb, static_cast<int>((istart + nu - 1) / per)};
    // the next copies (another proxy) write where the results were
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

// Joins the partials of the items cut by the ranges: block (c, r) takes row r of
// the item that starts in range c and ends in a later one; warp w takes every
// W-th piece from the w-th on, and the warps are added in order.
template <int D, int NT, int W>
__global__ void __launch_bounds__(32 * W) kv_decode_join_kernel(const KvAttnParams p, int ranges) {
  constexpr int COLS = 8 * NT;
  __shared__ float4 o_sm[W][32];
  __shared__ float2 s_sm[W];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Desc de = reinterpret_cast<const Desc *>(p.ws)[blockIdx.x];
  if (de.last < 0) return;
  int q0, nq, len;
  seq_of(p, de.b, q0, nq, len);
  const int r = blockIdx.y, ri = de.rb * COLS + r;
  if (ri >= nq * p.group) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Partials<D, COLS> ps{reinterpret_cast<const float *>(reinterpret_cast<const Desc *>(p.ws) + ranges),
                             static_cast<int>(blockIdx.x)};
  JoinedRow<1> mine;
  for (int i = blockIdx.x + warp; i <= de.last; i += 8 * W)
    join_pieces<8>(ps, r, lane * 4 < D ? r * D + lane * 4 : -1, 0, i, W, de.last, mine);
  float4 o = mine.o[0];
  float m = mine.m, l = mine.l;
  o_sm[warp][lane] = o;
  if (lane == 0) s_sm[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0 || lane * 4 >= D) return;
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, s_sm[w].x);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float a = exp2_fast(s_sm[w].x - m);
    const float4 x = o_sm[w][lane];
    l = fmaf(a, s_sm[w].y, l);
    o.x = fmaf(a, x.x, o.x);
    o.y = fmaf(a, x.y, o.y);
    o.z = fmaf(a, x.z, o.z);
    o.w = fmaf(a, x.w, o.w);
  }
  const long long row = (static_cast<long long>(q0) + ri / p.group) * p.Hq + de.h * p.group + ri % p.group;
  store_row4<D>(p, row, lane * 4, o, m, l);
}

template <int BITS, int D, int NT>
long long most_units(const KvAttnParams &p) {
  using PL = Plan<BITS, D, NT>;
  const long long tokens = static_cast<long long>(p.table_w) << p.kv.page_shift;
  const long long rb = (static_cast<long long>(p.max_q) * p.group + PL::COLS - 1) / PL::COLS;
  // + 15: the first unit starts on a multiple of 16 before the first key
  const long long units = tokens > 0 ? (tokens + 15 + PL::UNIT - 1) / PL::UNIT : 1;
  return static_cast<long long>(p.B) * p.kv.heads * rb * units;
}

// The kernel's shared memory, allowed once per device.
template <int BITS, int D, int NT>
bool allow_smem() {
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev])
    done[dev] = cudaFuncSetAttribute(kv_decode_kernel<BITS, D, NT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Plan<BITS, D, NT>::SMEM) == cudaSuccess;
  return done[dev];
}

template <int BITS, int D, int NT>
int launch_t(const KvAttnParams &p, cudaStream_t s) {
  using PL = Plan<BITS, D, NT>;
  const long long units = most_units<BITS, D, NT>(p);
  const long long room = kNumSMsGB300 * PL::BLOCKS;
  const int grid = static_cast<int>(units < room ? units : room);
  if (!allow_smem<BITS, D, NT>()) return W8A8_ERR_CUDA;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = PL::SMEM;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_decode_kernel<BITS, D, NT>, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  // no item can be cut when none has more than one unit
  if ((static_cast<long long>(p.table_w) << p.kv.page_shift) + 15 > PL::UNIT) {
    const long long most = static_cast<long long>(p.max_q) * p.group;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(most < PL::COLS ? most : PL::COLS));
    // items of many pieces: more warps fetch them (131072 tokens, 57 pieces: 4 warps
    // 40 us in all, 8 warps 38; 64 sequences, 2 pieces: 82 and 84)
    const bool many = grid / (static_cast<long long>(p.B) * p.kv.heads) >= 32;
    cfg.blockDim = dim3(many ? 256 : 128);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, many ? kv_decode_join_kernel<D, NT, 8> : kv_decode_join_kernel<D, NT, 4>,
                           p, grid) != cudaSuccess) {
      cudaGetLastError();
      return W8A8_ERR_CUDA;
    }
  }
  return launch_status();
}

}  // namespace

// Rows that a sequence's queries make per kv head: blocks of 8 or 16.
static int column_tiles(long long rows) { return rows <= 8 ? 1 : 2; }

size_t kv_decode_workspace(int D, long long rows) {
  const int nt = column_tiles(rows);
  const size_t cols = 8 * nt, grid = kNumSMsGB300 * 3;
  return grid * (sizeof(Desc) + 2 * sizeof(float) * cols * (D + 2));
}

int launch_kv_decode(const KvAttnParams &p, int bits, int D, cudaStream_t s) {
  const int nt = column_tiles(static_cast<long long>(p.max_q) * p.group);
  if (bits == 4) {
    if (D == 64)
      return nt == 1 ? launch_t<4, 64, 1>(p, s) : launch_t<4, 64, 2>(p, s);
    return nt == 1 ? launch_t<4, 128, 1>(p, s) : launch_t<4, 128, 2>(p, s);
  }
  if (D == 64) return nt == 1 ? launch_t<8, 64, 1>(p, s) : launch_t<8, 64, 2>(p, s);
  return nt == 1 ? launch_t<8, 128, 1>(p, s) : launch_t<8, 128, 2>(p, s);
}

}  // namespace w8a8
