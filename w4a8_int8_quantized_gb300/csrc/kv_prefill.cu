// Attention of many query rows (prompts, chunks) over the quantized cache, on
// the 5th-generation tensor cores.
//
// Rows of one kv head share its keys: row r of a sequence is query r / group,
// head r % group of the group, and an item is (sequence, 256 rows, kv head).
// Per 128 keys an item needs S = Q K^T and O += P V, 4 * 256 * 128 * D flops
// (2048 cycles of the tensor pipe at D = 128) against 17 KB of cache, so it is
// bound by the tensor pipe, with the softmax (32768 exponentials) close behind.
//
// One CTA of 16 warps per SM:
//   warps 0-3, 4-7   softmax of rows 0-127 and 128-255, 32 rows a warp: scores
//                    from TMEM, weights P back over them as fp16;
//   warps 8-11       converters: a thread owns a token; codes to fp16 (exact)
//                    into 128-byte-swizzled stages, and the token's scales;
//   warp 12          issues the MMAs: once the weights of 64 keys are there, their
//                    P V, then the scores of the next tile into the same buffer,
//                    while the softmax works on the other buffer;
//   warps 13, 14     bring the next item's Q rows while the current one finishes;
//   warp 15          walks this block's range of work and publishes its pieces.
// TMEM: S_0, S_1 (two buffers of 64 keys each, P in the first half of its buffer's
// columns), O_0, O_1 (D columns).
//
// Operands: Q and K are K-major.  V keeps its token rows and is read as the
// MN-major operand, so nothing is transposed.  At 4 bits the converter's pairs
// (d, d + 4) permute the d of each 8 of V; the output undoes it.
//
// Softmax, with the codes exact and both scales in fp32: u = S (scale log2e s_k)
// + log2 s_v, p = 2^(u - M), O = sum p code_v, l = sum p / s_v.  M is the lazy
// reference of kv_common.cuh, a row's own: O is rescaled (TMEM to TMEM) only when
// some row of the warp passes it.  Tokens that no row of the item sees get s_k = 0,
// log2 s_v = -inf, 1 / s_v = 0, so only tiles at a row's causal end or window
// start test single keys.
//
// Split: as in the few-row kernel, the 128-key tiles of all items form one line
// cut into equal ranges, one per SM, whatever the lengths, the causal triangle
// and the number of items; an item cut by ranges leaves fp32 partials that a
// second kernel joins in order.
//
// Measured (8 kv heads of 4 rows, D = 128, 4 bits): 512 tokens behind 32256 215 us,
// 1.27 PFLOP/s, 0.67 of a measured dense product; a prompt of 4516 tokens 165 us, 1.01.
// A tile takes about 3700 cycles: shared memory is busy for 3300 of them (see the
// softmax), the tensor pipe for 2048.  An item's start and end add about 9000.
#include <math_constants.h>

#include <mutex>

#include "common.cuh"
#include "kv_attn.cuh"
#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace w8a8 {
namespace {

constexpr int kSoftWarps = 8, kWarps = kSoftWarps + 8, kThreads = 32 * kWarps;
constexpr int kRows = 256;  // of an item
constexpr int kKeys = 128;  // of a tile
constexpr int kRing = 4;    // published pieces
// An item's start and end, in tiles, for the split (a prompt of 4516 tokens and six
// ragged ones: 3 167 and 122 us, 4 170 and 124, 5 171 and 127).
constexpr int kItemCost = 3;

// A piece of an item: its tiles t0 .. t1 - 1 of nt.
struct Piece {
  int b, h, qt, R;     // R: rows of the item; 0: no more pieces
  int q0, nq, len;     // of the sequence
  int first;           // token of tile 0
  int lo_min, hi_max;  // keys outside [lo_min, hi_max) are seen by no row
  int t0, t1, nt;
  int last;            // range that holds the item's last tile
};

// An item cut by ranges, for the join: its first query, kv head, row block, rows and
// the range of its last tile.
struct alignas(16) Desc {
  int q0, h, qt, R, last;
};

template <int D>
struct Plan {
  static constexpr int SUBS = D / 64;                  // 64-wide sub-tiles of 128-byte rows
  static constexpr int SUB = 128 * 128;                // bytes of one
  static constexpr int TILE = SUBS * SUB;              // a Q, K or V tile
  static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE, OFF_S = 6 * TILE;
  static constexpr int SLOTS = 3;                      // of token scales (see the converters)
  static constexpr int OFF_BAR = OFF_S + SLOTS * 3 * kKeys * 4;
  static constexpr int BARS = 24 + 2 * kRing + 1;
  static constexpr int OFF_PIECE = OFF_BAR + BARS * 8;
  static constexpr int OFF_MISC = OFF_PIECE + kRing * static_cast<int>(sizeof(Piece));
  static constexpr int OFF_LIM = OFF_MISC + 16;        // keys each row sees
  static constexpr int SMEM = OFF_LIM + kRows * 8 + 1024;  // 1024: aligned by hand
  static_assert(OFF_LIM % 8 == 0, "row limits are pairs");
  static constexpr uint32_t COL_S = 0, COL_O = 256;    // S_w at 128 w + 64 c, O_w at 256 + 128 w
};
static_assert(Plan<128>::SMEM <= 232448, "shared memory plan too large");

// D fp32, A and B fp16, M = 128; S: N = 64, both K-major; PV: N = D, B MN-major
constexpr uint32_t kIdescS = (1u << 4) | (64u >> 3 << 17) | (128u >> 4 << 24);
template <int D>
__host__ __device__ constexpr uint32_t idesc_pv() {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D) >> 3 << 17) | (128u >> 4 << 24);
}

// V as MN-major operand, 128-byte swizzle: 64 d of 8 tokens per 1 KB atom, the
// next 8 tokens 1 KB on (stride offset), the next 64 d a sub-tile on (leading offset)
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3ffff) >> 4);
  d |= static_cast<uint64_t>((128 * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Whether a phase is over, asked by the whole warp together: no branch of single
// lanes (a finished phase costs 76 cycles to pass this way, 152 with a loop per
// lane, 270 with one lane polling for the others).
__device__ __forceinline__ bool try_all(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "vote.sync.all.pred p, p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The wait itself, bounded: false if the block is aborting, or if this wait
// gave up (which is recorded and aborts the block).
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                      unsigned int *err, long long limit) {
  const long long t0 = clock64();
  while (!try_all(bar, parity)) {
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
      atomicCAS(err, 0u, static_cast<unsigned>(kDevErrCacheCopy));
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// MMAs and commits of one elected lane, as predicated instructions of a warp
// that runs in step: the descriptors then stay in uniform registers.  (From
// inside a one-lane branch a K = 16, N = 128 MMA took 96 to 108 cycles to
// issue, this way 65 to 71; it executes in 64.)
__device__ __forceinline__ uint32_t elect() {
  uint32_t on;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(on));
  return on;
}
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum), "r"(on));
}
// A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accum), "r"(on));
}
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(on)
      : "memory");
}

// 16 TMEM lanes x 64 columns as fragments: register 4 n + e of lane 4 g + t is TMEM
// lane g + 8 (e / 2), column 8 n + 2 t + (e & 1).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// the same for 32 columns
__device__ __forceinline__ void tmem_ld_frag4(uint32_t taddr, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag4(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 lanes x 32 columns: register 2 n + e is TMEM lane g + 8 e, column 4 n + t.
__device__ __forceinline__ void tmem_st_half_frag(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// waits for this thread's TMEM loads; the registers pass through
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// paired fp32 arithmetic: each half an IEEE operation
__device__ __forceinline__ void fma2(float &a, float &b, float x0, float x1, float y0, float y1,
                                     float z0, float z1) {
  asm("{\n.reg .b64 x, y, z, d;\n"
      "mov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 d, x, y, z;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(a), "=f"(b)
      : "f"(x0), "f"(x1), "f"(y0), "f"(y1), "f"(z0), "f"(z1));
}
__device__ __forceinline__ void add2(float &a, float &b, float x0, float x1, float y) {
  asm("{\n.reg .b64 x, y, d;\n"
      "mov.b64 x, {%2, %3};\nmov.b64 y, {%4, %4};\n"
      "add.rn.f32x2 d, x, y;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(a), "=f"(b)
      : "f"(x0), "f"(x1), "f"(y));
}

__device__ __forceinline__ void sts4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void sts1(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Counts of units are 64 bits wide but rarely that large, and a 64-bit division takes
// hundreds of cycles of a call's start.
__device__ __forceinline__ long long div_units(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Rows and tiles of entity e = sequence * nqt + row block; 0 tiles: no rows.
struct Entity {
  int b, qt, R, q0, nq, len, first, lo_min, hi_max, nt;
  // units of the line that one of its items takes: kItemCost, then its tiles
  __device__ __forceinline__ long long cost() const { return nt > 0 ? nt + kItemCost : 0; }
};
__device__ __forceinline__ Entity entity_of(const KvAttnParams &p, int nqt, int e) {
  Entity x;
  x.b = e / nqt;
  x.qt = e - x.b * nqt;
  seq_of(p, x.b, x.q0, x.nq, x.len);
  const long long left = static_cast<long long>(x.nq) * p.group - static_cast<long long>(x.qt) * kRows;
  x.R = static_cast<int>(min(left, static_cast<long long>(kRows)));
  x.nt = 0;
  x.first = x.lo_min = x.hi_max = 0;
  if (x.R > 0) {
    int hi, lo2;
    visible(p, x.len - x.nq + (x.qt * kRows) / p.group, x.len, x.lo_min, hi);
    visible(p, x.len - x.nq + (x.qt * kRows + x.R - 1) / p.group, x.len, lo2, x.hi_max);
    x.hi_max = max(x.hi_max, 0);
    x.first = min(x.lo_min, x.hi_max) & ~15;
    x.nt = max((x.hi_max - x.first + kKeys - 1) / kKeys, 1);
  }
  return x;
}

// Token row i of a tile: byte offset of its 16-byte chunk c (8 d) in a swizzled tile
__device__ __forceinline__ uint32_t chunk_at(int i, int c) {
  return (c >> 3) * (128 * 128) + (i >> 3) * 1024 + (i & 7) * 128 + (((c & 7) ^ (i & 7)) << 4);
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const KvAttnParams p) {
  using PL = Plan<D>;
  extern __shared__ uint8_t raw[];
  __shared__ long long sums[kWarps], first_at;  // of the warps; units before the first entity
  __shared__ int first_e;                       // the entity of this block's first unit, or one before
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The next kernel is not let in early: the join's blocks would all take their places on
  // the SMs that finish first (prompt 211 us against 202, chunk 255 against 240).
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // -- this block's range of tiles --------------------------------------------
  const int nqt = static_cast<int>((static_cast<long long>(p.max_q) * p.group + kRows - 1) / kRows);
  const int entities = p.B * nqt, per_thread = (entities + kThreads - 1) / kThreads;
  long long mine = 0, upto = 0;  // units of this thread's entities, and of all up to them
  for (int i = 0; i < per_thread; ++i) {
    const int e = threadIdx.x * per_thread + i;
    if (e < entities) mine += entity_of(p, nqt, e).cost() * p.kv.heads;
  }
  upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) upto += total;
    total += sums[w];
  }
  const long long per = div_units(total + gridDim.x - 1, gridDim.x);
  const long long c0 = blockIdx.x * per, c1 = min(c0 + per, total);
  Desc *descs = reinterpret_cast<Desc *>(p.ws);
  float *parts = reinterpret_cast<float *>(descs + gridDim.x);
  if (threadIdx.x == 0) descs[blockIdx.x].last = -1;
  if (__any_sync(0xffffffffu, some_unowned(p))) blank_unowned<D>(p.out, p.lse, p.q_offsets, p.T, p.Hq, p.B, p.max_q);
  if (c0 >= c1) return;
  if (upto - mine <= c0 && c0 < upto) {
    first_e = threadIdx.x * per_thread;
    first_at = upto - mine;
  }

  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *sm = raw + (base - smem_u32(raw));
  const uint32_t bar0 = base + PL::OFF_BAR;
  auto q_full = [&](int w) { return bar0 + 8u * w; };
  auto q_empty = [&](int w) { return bar0 + 8u * (2 + w); };
  auto k_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto k_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (8 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (10 + s); };
  // per row half w and key half c of a tile: scores there, weights there, products done
  auto s_full = [&](int w, int c) { return bar0 + 8u * (12 + 2 * w + c); };
  auto p_full = [&](int w, int c) { return bar0 + 8u * (16 + 2 * w + c); };
  auto o_done = [&](int w, int c) { return bar0 + 8u * (20 + 2 * w + c); };
  auto piece_full = [&](int i) { return bar0 + 8u * (24 + i); };
  auto piece_empty = [&](int i) { return bar0 + 8u * (24 + kRing + i); };
  const uint32_t drain = bar0 + 8u * (PL::BARS - 1);
  Piece *pieces = reinterpret_cast<Piece *>(sm + PL::OFF_PIECE);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + PL::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
      mbar_init(k_full(i), 4);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 4);
      mbar_init(v_empty(i), 1);
      for (int c = 0; c < 2; ++c) {
        mbar_init(s_full(i, c), 1);
        mbar_init(p_full(i, c), kSoftWarps / 2);
        mbar_init(o_done(i, c), 1);
      }
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(piece_full(i), 1);
      mbar_init(piece_empty(i), kSoftWarps + 4 + 1 + 2);  // softmax, converter, MMA and Q warps
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoftWarps + 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // 0: all 512 columns are this block's
  unsigned int *err = p.kv.err;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return try_all(bar, parity) || wait_all(bar, parity, abort_flag, err, p.wait_limit);
  };
  // a warp's view of the published pieces
  struct Reader {
    int i = 0;
    uint32_t phase = 0;
  };
  auto done_piece = [&](Reader &r) {
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty(r.i));
    if (++r.i == kRing) {
      r.i = 0;
      r.phase ^= 1u;
    }
  };
  auto next_piece = [&](Reader &r, Piece &x) {
    if (!wait(piece_full(r.i), r.phase)) return false;
    x = pieces[r.i];
    done_piece(r);
    return x.R > 0;
  };
  Reader reader;

  // Registers per warpgroup, together the launch's share of 4 * 128 (allow_smem checks
  // that the kernel was built with 128).  The converters hold a K and a V row each, which
  // at 8 bits does not fit in 80 (ragged prompts 177 us against 128).
  constexpr int kSoftRegs = 168, kConvRegs = 96, kRestRegs = 80;
  static_assert(2 * kSoftRegs + kConvRegs + kRestRegs == 4 * 128, "register shares");
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax ----
    // Scores come as fragments: a thread (lane 4 g + t) holds rows g + 8 y of its
    // warp's 32 and two of every 8 columns, so a token's scales, read from shared
    // memory, serve four rows.  Shared memory is the tightest resource here: per
    // tile the MMAs read 256 KB of operands (2048 cycles), the converters write 64
    // and these reads take 96; two rows a thread on twice the warps doubles them
    // (512 tokens behind 32256: 283 us against 263 when it was tried), one row a
    // thread with 16-byte broadcasts quadruples them.
    constexpr int Y = 4;  // rows of a thread: g + 8 y
    const int w = warp >> 2, g = lane >> 2, t = lane & 3;
    const int r0 = w * 128 + (warp & 3) * 32;  // the warp's first row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr uint32_t kLane16 = 16u << 16;
    const uint32_t col_s = lanes + PL::COL_S + 128 * w, col_o = lanes + PL::COL_O + 128 * w;
    int2 *limit = reinterpret_cast<int2 *>(sm + PL::OFF_LIM) + r0;
    uint32_t s_phase = 0;  // of the tile's barriers
    uint32_t tiles = 0;  // so far
    bool ok = true;
    while (ok && wait(piece_full(reader.i), reader.phase)) {
      // the piece stays in shared memory until its end (registers are short)
      const Piece &x = pieces[reader.i];
      if (x.R == 0) break;
      if (x.R <= w * 128) {  // this half has no rows; keep up with the scales' slots
        tiles += x.t1 - x.t0;
        done_piece(reader);
        continue;
      }
      // keys that row r0 + lane sees (rows past the item's: all), for whoever holds it
      int lo = 0, hi = 0x7fffffff;
      if (r0 + lane < x.R) visible(p, x.len - x.nq + (x.qt * kRows + r0 + lane) / p.group, x.len, lo, hi);
      limit[lane] = make_int2(lo, max(hi, 0));
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      __syncwarp();
      float m[Y], l[Y][2];
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        m[y] = kNoRef;
        l[y][0] = l[y][1] = 0.f;
      }
      int j = x.first + x.t0 * kKeys;
      const int j_end = x.first + x.t1 * kKeys;
      bool fresh = true;
      for (; j < j_end; j += kKeys) {
        const uint32_t slot = tiles % PL::SLOTS;
        ++tiles;
        const float2 *sc = reinterpret_cast<const float2 *>(sm + PL::OFF_S + slot * (3 * kKeys * 4)) + t;
        // 64 keys at a time, each half of the tile with its own columns of TMEM: while
        // one half's weights are made, the other half's products and the scores of
        // the next tile run
#pragma unroll 1
        for (int c = 0; c < 2; ++c, sc += kKeys / 4) {
          // the token scales are there too: they precede K's arrival, which these
          // scores waited for (a barrier of their own cost 1 %)
          ok = wait(s_full(w, c), s_phase);
          if (!ok) break;
          tc_fence_after();
          // u[32 (y / 2) + 4 n + 2 (y % 2) + e]: row y, column 64 c + 8 n + 2 t + e
          uint32_t s[64];
#pragma unroll
          for (int z = 0; z < 2; ++z) tmem_ld_frag(col_s + 64 * c + z * kLane16, s + 32 * z);
          tmem_wait_ld<64>(s);
          float *u = reinterpret_cast<float *>(s);
          auto at = [&](int y, int n) { return u + 32 * (y >> 1) + 4 * n + 2 * (y & 1); };
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float2 k = sc[4 * n], z = sc[kKeys / 2 + 4 * n];
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              float *d = at(y, n);
              fma2(d[0], d[1], d[0], d[1], k.x, k.y, z.x, z.y);
            }
          }
          const int jc = j + 64 * c;
          if (hi_min < jc + 64) {
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              const int end = limit[8 * y + g].y - jc - 2 * t;
#pragma unroll
              for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * n + e >= end) at(y, n)[e] = -CUDART_INF_F;
            }
          }
          if (lo_max > jc) {
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              const int begin = limit[8 * y + g].x - jc - 2 * t;
#pragma unroll
              for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * n + e < begin) at(y, n)[e] = -CUDART_INF_F;
            }
          }
          float top[Y];
          bool over = false;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            top[y] = fmaxf(at(y, 0)[0], at(y, 0)[1]);
#pragma unroll
            for (int n = 1; n < 8; ++n) top[y] = max3(top[y], at(y, n)[0], at(y, n)[1]);
            over |= top[y] > m[y] + kRoom;
          }
          if (__any_sync(0xffffffffu, over)) {
            float a[Y];
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 1));
              top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 2));
              const float nm = top[y] > m[y] + kRoom ? top[y] : m[y];
              a[y] = exp2_fast(m[y] - nm);
              m[y] = nm;
              l[y][0] *= a[y];
              l[y][1] *= a[y];
            }
            // O is this warp's to change once the products of the 64 keys before are in
            if (!fresh || c == 1) {
              ok = wait(o_done(w, c ^ 1), c == 1 ? s_phase : s_phase ^ 1u);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                  uint32_t v[16];
                  tmem_ld_frag4(col_o + 32 * q + z * kLane16, v);
                  tmem_wait_ld<16>(v);
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    v[e] = __float_as_uint(__uint_as_float(v[e]) * a[2 * z + ((e >> 1) & 1)]);
                  tmem_st_frag4(col_o + 32 * q + z * kLane16, v);
                }
            }
          }
          // 8 scores become 4 columns of fp16 pairs
          uint32_t v[32];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float2 rv = sc[kKeys + 4 * n];
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              float *d = at(y, n);
              add2(d[0], d[1], d[0], d[1], -m[y]);
              const float w0 = exp2_fast(d[0]), w1 = exp2_fast(d[1]);
              fma2(l[y][0], l[y][1], w0, w1, rv.x, rv.y, l[y][0], l[y][1]);
              const __half2 h = __floats2half2_rn(w0, w1);
              v[16 * (y >> 1) + 2 * n + (y & 1)] = *reinterpret_cast<const uint32_t *>(&h);
            }
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) tmem_st_half_frag(col_s + 64 * c + z * kLane16, v + 16 * z);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w, c));
        }
        if (!ok) break;
        fresh = false;
        s_phase ^= 1u;
      }
      if (!ok) break;
      // -- the item's (or piece's) end: lane 8 y + g takes the row that lanes 4 g .. + 3
      // summed as their y, so that a lane's columns are consecutive and the code is
      // short (it is fetched anew every time: exchanging the fragments' pairs among four
      // lanes took 16000 cycles a piece)
      float ms = 0.f, zs = 0.f;
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        float z = l[y][0] + l[y][1];
        z += __shfl_xor_sync(0xffffffffu, z, 1);
        z += __shfl_xor_sync(0xffffffffu, z, 2);
        z = __shfl_sync(0xffffffffu, z, 4 * (lane & 7));
        const float my = __shfl_sync(0xffffffffu, m[y], 4 * (lane & 7));
        if (lane >> 3 == y) {
          zs = z;
          ms = my;
        }
      }
      const int r = r0 + lane, ri = x.qt * kRows + r;
      const bool in = r < x.R, whole = x.t0 == 0 && x.t1 == x.nt;
      const long long row = (static_cast<long long>(x.q0) + ri / p.group) * p.Hq + x.h * p.group + ri % p.group;
      const long long part = static_cast<long long>(blockIdx.x) * 2 + (x.t0 == 0 ? 1 : 0);
      float *part_at = parts + part * kRows * (D + 2);
      const float inv = zs == 0.f ? 0.f : 1.f / zs;
      if (!whole) {
        if (in) *reinterpret_cast<float2 *>(part_at + kRows * D + 2 * r) = make_float2(ms, zs);
        if (x.t0 == 0 && threadIdx.x == 0) descs[blockIdx.x] = Desc{x.q0, x.h, x.qt, x.R, x.last};
      } else if (in && p.lse != nullptr) {
        p.lse[row] = zs == 0.f ? -CUDART_INF_F : (ms + log2f(zs)) * kLn2;
      }
      ok = wait(o_done(w, 1), s_phase ^ 1u);
      if (!ok) break;
      __syncwarp();  // lanes without a row skipped the stores above
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t v[32];
        tmem_ld32(col_o + 32 * q, v);
        tmem_wait_ld<32>(v);
        if (in && !whole) {
          // four columns of every row, then the next four: the lanes' stores are
          // consecutive.  (The columns' order stays; the join knows it.)
          float4 *dst = reinterpret_cast<float4 *>(part_at) + 8 * q * kRows + r;
#pragma unroll
          for (int n = 0; n < 8; ++n)
            dst[n * kRows] = make_float4(__uint_as_float(v[4 * n]), __uint_as_float(v[4 * n + 1]),
                                 __uint_as_float(v[4 * n + 2]), __uint_as_float(v[4 * n + 3]));
        } else if (in) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * D + 32 * q);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            // at 4 bits columns 2 s, 2 s + 1 of an 8 are d = s and s + 4
            auto pair = [&](int i) {
              const int c0 = BITS == 4 ? (i < 2 ? 4 * i : 4 * i - 7) : 2 * i, c1 = BITS == 4 ? c0 + 2 : c0 + 1;
              return output2(__uint_as_float(v[8 * n + c0]) * inv, __uint_as_float(v[8 * n + c1]) * inv);
            };
            dst[n] = make_uint4(pair(0), pair(1), pair(2), pair(3));
          }
        }
        __syncwarp();  // lanes without a row rejoin: the next TMEM load is the whole warp's
      }
      tc_fence_before();
      done_piece(reader);
    }
  } else if (warp < kSoftWarps + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // --------------------------------------------------------- converters ----
    // The scales have a third slot: a tile's are read until both halves' weights
    // are written, and slot s is refilled for tile i + 3 only once the K stage
    // of tile i + 1 is free, whose scores are issued after those weights.
    // A lane owns a token's scales; the codes of a warp's 32 tokens lie in two runs of
    // 16 (a page holds a multiple of 16), read 512 consecutive bytes at a time.  Which
    // 16 of them a lane takes is chosen so that 8 lanes' stores of one chunk each, of
    // 8 / VPS rows, fall into different banks.  (With a token a lane, whose loads touch
    // 32 lines each, ragged prompts at 8 bits took 149 us against 128.)
    constexpr int ROW = D * BITS / 8, NV = ROW / 16;  // bytes of a token; a lane's vectors
    constexpr int VPS = BITS / 2, RP = 8 / VPS;       // vectors of 64 d; rows of 8 lanes
    constexpr int RL = 512 / ROW, CPV = 16 / BITS;    // rows of a load; chunks of a vector
    const int cw = warp - kSoftWarps, tok = cw * 32 + lane;
    const int vrow = (lane >> 3) / PL::SUBS * RP + lane / VPS % RP;
    const int vk = (lane >> 3) % PL::SUBS * VPS + lane % VPS;
    const uint32_t lane_at = chunk_at(cw * 32 + vrow, CPV * vk);
    const int lane_from = vrow * ROW + vk * 16;
    const Nibbles nib;
    int st = 0, slot = 0;
    uint32_t phase = 1;  // the first wait on an empty stage passes
    const int pmask = (1 << p.kv.page_shift) - 1;
    bool ok = true;
    // The nibble trick gives pairs (d, d + 4).  K's are put in order, since permuting Q
    // instead delays an item's start; V's stay, and the output undoes them.
    auto convert = [&](const uint4 (&v)[NV], uint32_t stage, bool order) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t y[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        // token 16 (i / (NV / 2)) + RL (i % (NV / 2)) + vrow of the warp's
        const int t0 = 16 * (i / (NV / 2)) + RL * (i % (NV / 2));
        const uint32_t at = (stage + lane_at) ^ ((t0 & 7) << 4);
        if (BITS == 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t o[4];
            nib.to_h(y[e], o);
            if (order) {
              const uint32_t z[4] = {__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                                     __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632)};
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = z[i];
            }
            sts4((at ^ (e << 4)) + 128 * t0, make_uint4(o[0], o[1], o[2], o[3]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 o;
            bytes_to_h(y[2 * e], o.x, o.y);
            bytes_to_h(y[2 * e + 1], o.z, o.w);
            sts4((at ^ (e << 4)) + 128 * t0, o);
          }
        }
      }
    };
    // The codes of the next K are fetched when this tile's are converted, those of
    // the next V likewise, so that memory's latency lies under the other's work.
    // The tile to fetch: its sequence, head, this lane's token, where the keys
    // begin and end, and the piece's tiles after it; and the table's entry of the token's
    // page, itself fetched a tile ahead.
    int tb = 0, th = 0, ta = 0, tlo = 0, tend = 0, left = 0, entry = 0;
    auto advance = [&]() {
      if (left > 0) {
        ta += kKeys;
        --left;
      } else {
        Piece x;
        if (!next_piece(reader, x)) return false;
        tb = x.b;
        ta = x.first + x.t0 * kKeys + tok;
        th = x.h;
        tlo = x.lo_min;
        tend = min(x.hi_max, x.len);
        left = x.t1 - x.t0 - 1;
      }
      if (ta < tend) entry = entry_of(p, tb, ta >> p.kv.page_shift);
      return true;
    };
    uint4 kv[NV] = {}, vv[NV] = {};
    // the token's scales; kNone for s_v: left out.  (A bit pattern that no arithmetic
    // makes: the row itself, kept for this, spilled at 8 bits.)
    constexpr int kNone = -1;
    float ks = 0.f, vs = 0.f;
    long long run[2] = {-1, -1};     // rows in the cache of the warp's tokens 0 and 16
    // Codes of tokens that are left out are any: they are finite, and weigh nothing
    auto load = [&](const uint8_t *codes, uint4 (&v)[NV]) {
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (run[e / (NV / 2)] >= 0)
          v[e] = __ldg(reinterpret_cast<const uint4 *>(codes + run[e / (NV / 2)] * ROW + lane_from + 512 * (e % (NV / 2))));
    };
    bool ahead = advance();  // whether that tile is there
    auto load_k = [&]() {
      const int page = ta < tend ? checked_page(p, entry) : -1;
      const long long row = page < 0 ? -1 : p.kv.row(page, th) + (ta & pmask);
      run[0] = __shfl_sync(0xffffffffu, row, 0);
      run[1] = __shfl_sync(0xffffffffu, row, 16);
      load(p.kv.kc, kv);
      vs = __int_as_float(kNone);
      if (row >= 0 && ta >= tlo) {  // a slot that nobody sees may hold any scale
        ks = __ldg(p.kv.ks + row);
        vs = __ldg(p.kv.vs + row);
      }
      ahead = advance();
    };
    bool have = ahead;
    if (have) {
      load_k();
      load(p.kv.vc, vv);
    }
    bool lost = p.skip_first_copy && cw == 0;  // test only: the first hand-over
    while (ok && have) {
      ok = wait(k_empty(st), phase);
      if (!ok) break;
      convert(kv, base + PL::OFF_K + st * PL::TILE, true);
      const uint32_t sc = base + PL::OFF_S + slot * (3 * kKeys * 4) + tok * 4;
      const float sv = vs == 0.f ? kZeroScale : vs;
      const bool none = __float_as_int(vs) == kNone;
      sts1(sc, none ? 0.f : ks * (p.scale * kLog2e));
      sts1(sc + kKeys * 4, none ? -CUDART_INF_F : log2_fast(sv));
      sts1(sc + 2 * kKeys * 4, none ? 0.f : 1.f / sv);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && !lost) mbar_arrive(k_full(st));
      lost = false;
      have = ahead;
      if (have) load_k();
      ok = wait(v_empty(st), phase);
      if (!ok) break;
      convert(vv, base + PL::OFF_V + st * PL::TILE, false);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
      if (have) load(p.kv.vc, vv);
      slot = slot + 1 == PL::SLOTS ? 0 : slot + 1;
      st ^= 1;
      if (st == 0) phase ^= 1u;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == kSoftWarps + 4) {
      // ------------------------------------------------------------- MMAs ----
      const uint32_t on = elect();
      int ks = 0, vs = 0;  // stages, and their phases
      uint32_t kph = 0, vph = 0, qph[2] = {0, 0}, pph[2] = {0, 0};
      const uint64_t q_desc = sw128_desc(base + PL::OFF_Q), k_desc = sw128_desc(base + PL::OFF_K);
      const uint64_t v_desc0 = v_desc(base + PL::OFF_V);
      // S_w of keys 64 c .. + 63 of the open K stage
      auto scores = [&](int w, int c) {
        tc_fence_after();
        const uint64_t a = q_desc + w * (PL::TILE >> 4), b = k_desc + ks * (PL::TILE >> 4) + c * (64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = ((k >> 2) * PL::SUB + (k & 3) * 32) >> 4;
          mma_ss(on, PL::COL_S + 128 * w + 64 * c, a + at, b + at, kIdescS, k > 0);
        }
        commit_if(on, s_full(w, c));
      };
      // O_w += P V over keys 64 c .. + 63
      auto values = [&](int w, int c, bool fresh) {
        tc_fence_after();
        const uint64_t b = v_desc0 + vs * (PL::TILE >> 4) + c * (64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(on, PL::COL_O + 128 * w, PL::COL_S + 128 * w + 64 * c + 8 * k, b + k * (2048 >> 4),
                 idesc_pv<D>(), !(fresh && k == 0));
        commit_if(on, o_done(w, c));
      };
      // the K stage whose scores are next: waited for once, released after the last half
      auto open_k = [&]() { return wait(k_full(ks), kph); };
      auto close_k = [&]() {
        commit_if(on, k_empty(ks));
        ks ^= 1;
        if (ks == 0) kph ^= 1u;
      };
      Piece x;
      // the first scores of a piece
      auto start = [&](const Piece &z) {
        if (!open_k()) return false;
        for (int c = 0; c < 2; ++c)
          for (int w = 0; w < 2 && z.R > 128 * w; ++w) {
            if (c == 0) {
              if (!wait(q_full(w), qph[w])) return false;
              qph[w] ^= 1u;
            }
            scores(w, c);
            if (c == 1 && z.t1 - z.t0 == 1) commit_if(on, q_empty(w));
          }
        close_k();
        return true;
      };
      bool ok = true, have = next_piece(reader, x);
      if (have) ok = start(x);
      while (ok && have) {
        Piece y;
        bool more = false;
        for (int i = x.t0; i < x.t1 && ok; ++i) {
          const bool last = i + 1 == x.t1;
          if (last) {
            more = next_piece(reader, y);
            ok = !__any_sync(0xffffffffu, *abort_flag != 0);
            if (!ok) break;
          }
          ok = wait(v_full(vs), vph);
          if (!ok) break;
          if (!last) ok = open_k();
          for (int c = 0; c < 2 && ok; ++c)
            for (int w = 0; w < 2 && x.R > 128 * w; ++w) {
              ok = wait(p_full(w, c), pph[w]);
              if (!ok) break;
              values(w, c, i == x.t0 && c == 0);
              if (!last) {
                // into the buffer whose weights have just been used
                scores(w, c);
                // the item's last scores: its Q rows may be replaced
                if (c == 1 && i + 2 == x.t1) commit_if(on, q_empty(w));
              }
            }
          if (!ok) break;
          pph[0] ^= 1u;
          if (x.R > 128) pph[1] ^= 1u;
          commit_if(on, v_empty(vs));
          if (!last) {
            close_k();
          } else if (more) {  // nothing of this item waits for the next one's rows
            ok = start(y);
            if (!ok) break;
          }
          vs ^= 1;
          if (vs == 0) vph ^= 1u;
        }
        x = y;
        have = more;
      }
      // every MMA has landed before TMEM is freed
      commit_if(on, drain);
      wait_bar_teardown(drain, 0);
      __syncwarp();
    } else if (warp < kSoftWarps + 7) {
      // ---------------------------------------------------------- Q rows ----
      const int w = warp - (kSoftWarps + 5);
      uint32_t phase = 1;
      Piece x;
      while (next_piece(reader, x)) {
        if (x.R <= w * 128) continue;
        // where the half's rows lane, lane + 32, ... are (in elements; -1: beyond the
        // item's, zero): found before Q is free, since from there on every cycle delays
        // the item's first scores
        long long from[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = w * 128 + 32 * k + lane, ri = x.qt * kRows + r;
          from[k] = r < x.R ? (x.q0 + ri / p.group) * p.q_ts +
                                  static_cast<long long>(x.h * p.group + ri % p.group) * p.q_hs
                            : -1;
        }
        if (!wait(q_empty(w), phase)) break;
        phase ^= 1u;
        // all rows in flight at once (by way of registers it took 8 round trips); a lane
        // takes chunk lane % C of every row.  (With the addresses worked out at each step
        // the issue alone took 8000 to 13000 cycles;
        // four steps at a time instead of all, a prompt takes 168 us against 165.)
        constexpr int C = D / 8, RPS = 32 / C;  // chunks of a row; rows per step of the warp
        const int c = lane % C;
        const uint32_t dst = base + PL::OFF_Q + w * PL::TILE;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 32; i += RPS) {
            const long long f = __shfl_sync(0xffffffffu, from[k], i + lane / C);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + chunk_at(32 * k + i + lane / C, c)),
                         "l"(p.q + (f < 0 ? 0 : f + 8 * c)), "r"(f < 0 ? 0 : 16)
                         : "memory");
          }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(w));
      }
    } else {
      // ---------------------------------------------------------- the walk ----
      int e = first_e;
      long long start = first_at;  // first unit of entity e
      Entity en = entity_of(p, nqt, e);
      Reader slot;
      uint32_t phase = 1;
      bool ok = true;
      for (long long at = c0; ok;) {
        // the next piece that has a tile in the range
        int t0 = 0, t1 = 0, h = 0;
        long long istart = 0;
        while (at < c1 && t0 == t1) {
          while (at >= start + en.cost() * p.kv.heads) {
            start += en.cost() * p.kv.heads;
            en = entity_of(p, nqt, ++e);
          }
          h = static_cast<int>(div_units(at - start, en.cost()));
          istart = start + h * en.cost();
          t0 = static_cast<int>(max(at - istart - kItemCost, 0LL));
          t1 = static_cast<int>(max(min(en.cost(), c1 - istart) - kItemCost, 0LL));
          at = istart + kItemCost + t1;
        }
        const bool end = t0 == t1;
        ok = wait(piece_empty(slot.i), phase);
        if (!ok) break;
        if (end) {
          if (lane == 0) pieces[slot.i].R = 0;
        } else {
          if (lane == 0)
            pieces[slot.i] = Piece{en.b, h, en.qt, en.R, en.q0, en.nq, en.len, en.first, en.lo_min, en.hi_max,
                                   t0, t1, en.nt, static_cast<int>(div_units(istart + en.cost() - 1, per))};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_full(slot.i));
        if (++slot.i == kRing) {
          slot.i = 0;
          phase ^= 1u;
        }
        if (end) break;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftWarps + 4)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the partials of the items cut by the ranges: block (c, y) takes rows
// kJoinRows y .. of the item that starts in range c and ends in a later one, a
// thread eight columns of a row.  Most items have two pieces, one for each side of
// a cut; the few of a short call with long keys have one for every range.  (A warp a
// row and four pieces at a time, whether there or not, was bound by its
// instructions and took 15 us of a prompt; 9 now.)
constexpr int kJoinRows = 16;

template <int BITS, int D>
__global__ void __launch_bounds__(kJoinRows * D / 8) kv_prefill_join_kernel(const KvAttnParams p, int ranges) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x;
  const Desc de = reinterpret_cast<const Desc *>(p.ws)[first];
  const int r = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows;
  const int c = threadIdx.x / kJoinRows;  // of 8 columns
  const Partials<D, kRows> ps{reinterpret_cast<const float *>(reinterpret_cast<const Desc *>(p.ws) + ranges), first};
  JoinedRow<2> x;
  const int at = (2 * c * kRows + r) * 4;
  // where the first two pieces would be is known before the item is
  join_pieces<2>(ps, r, at, 4 * kRows, first, 1, min(first + 1, ranges - 1), x);
  if (de.last < 0 || r >= de.R) return;
  for (int i = first + 2; i <= de.last; i += 4) join_pieces<4>(ps, r, at, 4 * kRows, i, 1, de.last, x);
  const int ri = de.qt * kRows + r;
  const long long row = (static_cast<long long>(de.q0) + ri / p.group) * p.Hq + de.h * p.group + ri % p.group;
  float4 a = x.o[0], b = x.o[1];
  if (BITS == 4) {  // columns 2 s, 2 s + 1 are d = s and s + 4
    a = make_float4(x.o[0].x, x.o[0].z, x.o[1].x, x.o[1].z);
    b = make_float4(x.o[0].y, x.o[0].w, x.o[1].y, x.o[1].w);
  }
  store_row4<D>(p, row, 8 * c, a, x.m, x.l);
  store_row4<D>(p, row, 8 * c + 4, b, x.m, x.l);
}

template <int BITS, int D>
bool allow_smem() {
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    // the warpgroups' register shares add up to what a launch with 128 brings
    cudaFuncAttributes a;
    done[dev] = cudaFuncSetAttribute(kv_prefill_kernel<BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Plan<D>::SMEM) == cudaSuccess &&
                cudaFuncGetAttributes(&a, kv_prefill_kernel<BITS, D>) == cudaSuccess && a.numRegs == 128;
  }
  return done[dev];
}

template <int BITS, int D>
int launch_t(const KvAttnParams &p, cudaStream_t s) {
  if (!allow_smem<BITS, D>()) return W8A8_ERR_CUDA;
  const long long nqt = (static_cast<long long>(p.max_q) * p.group + kRows - 1) / kRows;
  if (nqt * p.B > 0x3fffffffLL) return W8A8_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(p.table_w) << p.kv.page_shift;
  // + 15: the first tile starts on a multiple of 16 before the first key
  const long long tiles = tokens > 0 ? (tokens + 15 + kKeys - 1) / kKeys : 1;
  const long long most = nqt * p.B * p.kv.heads * (tiles + kItemCost);
  const int grid = static_cast<int>(most < kNumSMsGB300 ? most : kNumSMsGB300);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Plan<D>::SMEM;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_prefill_kernel<BITS, D>, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  if (tiles > 1) {  // else no item can be cut
    cfg.gridDim = dim3(static_cast<unsigned>(grid), kRows / kJoinRows);
    cfg.blockDim = dim3(kJoinRows * D / 8);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, kv_prefill_join_kernel<BITS, D>, p, grid) != cudaSuccess) {
      cudaGetLastError();
      return W8A8_ERR_CUDA;
    }
  }
  return launch_status();
}

// Every row: a call with queries and no sequence.
__global__ void __launch_bounds__(256) kv_blank_kernel(uint4 *out, long long vectors, float *lse, long long rows) {
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<long long>(gridDim.x) * 256;
  for (long long i = at; i < vectors; i += step) out[i] = make_uint4(0, 0, 0, 0);
  if (lse != nullptr)
    for (long long i = at; i < rows; i += step) lse[i] = -CUDART_INF_F;
}

}  // namespace

int launch_kv_blank(__half *out, float *lse, long long rows, int D, cudaStream_t s) {
  const long long vectors = rows * D / 8, want = (vectors + 255) / 256;
  kv_blank_kernel<<<static_cast<int>(want < kNumSMsGB300 * 8 ? want : kNumSMsGB300 * 8), 256, 0, s>>>(
      reinterpret_cast<uint4 *>(out), vectors, lse, rows);
  return launch_status();
}

size_t kv_prefill_workspace(int D) {
  return kNumSMsGB300 * (sizeof(Desc) + 2 * sizeof(float) * kRows * (D + 2));
}

int launch_kv_prefill(const KvAttnParams &p, int bits, int D, cudaStream_t s) {
  if (bits == 4) return D == 64 ? launch_t<4, 64>(p, s) : launch_t<4, 128>(p, s);
  return D == 64 ? launch_t<8, 64>(p, s) : launch_t<8, 128>(p, s);
}

}  // namespace w8a8
