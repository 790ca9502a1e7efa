// Products of 8-bit float rows on the 5th-generation tensor cores, the scales
// applied by the tensor core itself.
//
//   y[m, n] = fp16(sum_g 2^(ea[m,g] + ew[n,g]) sum_{k in g} a[m,k] w[n,k])
//   h[m, f] = act(x . Wg[f]) (x . Wu[f]), as fp16 or as e4m3 codes with scales
//
// tcgen05.mma kind::mxf8f6f4 multiplies e4m3 operands by a power of two per row
// and 32 elements of K.  A scale of this library covers 128 elements, so four
// consecutive instructions use the same scale byte, and a word of four bytes,
// one per lane and 32 rows of a tile in tensor memory, serves K = 512: the
// instruction's descriptor says which byte.  Sums stay in fp32 in tensor memory
// from the first group to the last; there is no rescaling pass.
//
// Roles: the tokens are the MMA's A operand (tensor-memory lanes), the weights
// its B operand (columns), so that a thread of the epilogue owns a token's row
// of 128 outputs: a group of codes needs no exchange between threads.
//
// Tiles: a pair of CTAs (cta_group::2) works on 256 tokens x 256 columns, each
// CTA fetching 128 rows of either operand, half of what two CTAs on their own
// would; the gated form takes the first CTA's rows from Wg and the second's
// from Wu, so a tile is 128 columns of both.  Few tokens (up to 128): one CTA,
// 128 tokens x 64 columns (gated: 128 x 128 of both), to have more CTAs that
// stream weights.
//
// Warps of a CTA: 0 copies the codes (TMA), 1 issues the MMAs (in the pair's
// first CTA; the second's passes on that its scales are there), 2 and 3 gather the scale bytes into the layout that tcgen05.cp
// takes, 4 - 7 are the epilogue.  Persistent, static tiles.
//
// Tensor memory: two accumulators of 256 columns and two sets of scales (12
// columns each) are 536 of 512 columns.  So the accumulators overlap by 24
// columns: the epilogue reads the shared ones first, and the next tile's MMAs
// wait for that alone.
//
// Every wait is bounded as in the GEMM; a CTA of a pair leaves only after both
// are done (cluster barrier), since either one's copies and MMAs reach into the
// other.
#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8_kernels.cuh"
#include "tc_ptx.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;     // tokens of a CTA's tile
constexpr int kBlock = 128;    // K of a stage
constexpr int kScaleBlocks = 4;  // stages of a set of scales
constexpr int kScaleSets = 4;    // sets in shared memory (two of them in tensor memory)

enum Mode { kLinear = 0, kGatedHalf = 1, kGatedCodes = 2 };

// CG: CTAs that share a tile; BN: columns of the tile's accumulator
template <int CG, int BN>
struct Plan {
  static constexpr int BROWS = BN / CG;  // weight rows that a CTA fetches
  static constexpr int A_BYTES = kRows * kBlock, B_BYTES = BROWS * kBlock;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int S = CG == 2 ? 6 : BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int SFB = BN == 256 ? 2 : 1;  // 128-row sets of weight scales
  static constexpr int SF_BYTES = 512 * (1 + SFB);
  static constexpr int OFF_OUT = S * STAGE;      // 4 warps x 32 rows x 128 bytes
  static constexpr int OFF_SF = OFF_OUT + 4 * 4096;
  static constexpr int OFF_BAR = OFF_SF + kScaleSets * SF_BYTES;
  static constexpr int NUM_BARS = 2 * S + 2 * kScaleSets + 2 + 2 + 1;
  static constexpr int SMEM_BYTES = OFF_BAR + NUM_BARS * 8 + 16 + 1024;  // + alignment by hand
  static constexpr bool OVERLAP = BN == 256;
  static constexpr uint32_t SF_COLS = 4 * (1 + SFB);
  static constexpr uint32_t TMEM_COLS = BN == 64 ? 256 : 512;
  static constexpr uint32_t ACC1 = OVERLAP ? 512 - 2 * SF_COLS - BN : BN;  // second accumulator
  static constexpr uint32_t SF0 = ACC1 + BN;
  static_assert(SF0 + 2 * SF_COLS <= TMEM_COLS, "tensor memory");
  static_assert(!OVERLAP || ACC1 + 32 >= BN, "the shared columns are within one 32-column read");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  static_assert(STAGE % 1024 == 0 && OFF_OUT % 1024 == 0, "swizzled tiles start at 1 KB");
};

struct TcParams {
  const uint8_t *sx, *sw[2];
  int M, N, G, nkb, ntiles, mtiles, ntn;  // N: columns of the output
  int m_first;      // tiles walk the tokens first
  int access[3];    // bytes that a load of sx, sw[0], sw[1] may take at once: 16, 4 or 1
  bool gelu;
  __half *y;        // stored directly (no map) where the rows are not 16-byte multiples
  uint8_t *scales;
  unsigned int *err;
  long long wait_limit;
  int skip_first_copy;
};

// MMAs, scale copies and commits are predicated instructions of a converged
// warp (`on`: the elected lane), so that descriptors stay in uniform registers.
__device__ __forceinline__ uint32_t elect() {
  uint32_t on;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(on));
  return on;
}

template <int CG>
__device__ __forceinline__ void mma_scaled(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accum) {
  if (CG == 2)
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(on));
  else
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(on));
}

// 32 rows x 16 bytes from shared memory to 4 columns, the same in every
// quarter of the lanes (with a pair: in either CTA, from its own memory)
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t on, uint32_t tmem, uint32_t smem) {
  // no swizzle, 8-row groups 128 bytes apart, descriptor version 1
  const uint64_t desc = static_cast<uint64_t>((smem & 0x3ffff) >> 4) | (uint64_t(8) << 16) |
                        (uint64_t(8) << 32) | (uint64_t(1) << 46);
  if (CG == 2)
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n"
                 "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(tmem), "l"(desc), "r"(on));
  else
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n"
                 "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(tmem), "l"(desc), "r"(on));
}

// All MMAs issued so far arrive on this barrier when they are done, in both
// CTAs of a pair.
template <int CG>
__device__ __forceinline__ void commit(uint32_t on, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
        "%1;\n}\n" ::"r"(bar), "h"(static_cast<uint16_t>(3)), "r"(on) : "memory");
  else
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
                 "r"(on)
                 : "memory");
}

// this address in the pair's first CTA
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The same for reads of tensor memory that have completed (tcgen05.wait::ld and
// the fence before it order them): nothing else to release.
__device__ __forceinline__ void arrive_read(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int CG>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    tma_load_2d(dst, map, bar, x, y);
}

__device__ __forceinline__ void store_tile(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The shared memory that this thread's stores read may be written again.
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(100)
      : "memory");
  return ok != 0;
}

struct Waits {
  volatile int *abort_flag;
  unsigned int *err;
  long long limit;
  __device__ bool operator()(uint32_t bar, uint32_t parity, unsigned code) const {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (clock64() - t0 > limit) {
        if (err != nullptr) atomicCAS(err, 0u, code);
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Tile {
  int m, n;  // tile indexes
};

__device__ __forceinline__ Tile tile_at(const TcParams &p, int t) {
  return p.m_first ? Tile{t % p.mtiles, t / p.mtiles} : Tile{t / p.ntn, t % p.ntn};
}

// The word at `at`; of one that is only partly within [first, end), the bytes
// that are, and 1.0 for the others.
__device__ __forceinline__ uint32_t word_within(uintptr_t at, uintptr_t first, uintptr_t end) {
  if (at >= first && at + 4 <= end) return *reinterpret_cast<const uint32_t *>(at);
  uint32_t w = 0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i)
    w |= (at + i >= first && at + i < end ? static_cast<uint32_t>(*reinterpret_cast<const uint8_t *>(at + i)) : 0x7fu)
         << (8 * i);
  return w;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Writes 32 rows x 64 columns of fp16, staged in `buf` (row = lane, 16-byte
// chunks exchanged as the 128-byte swizzle does), to y.
__device__ __forceinline__ void put_half(const TcParams &p, const CUtensorMap *map, uint8_t *buf, int lane,
                                         long row0, long col0) {
  if (row0 >= p.M || col0 >= p.N) return;
  if (p.y == nullptr) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) store_tile(map, smem_u32(buf), static_cast<int>(col0), static_cast<int>(row0));
    return;
  }
  __syncwarp();
  const int rows = static_cast<int>(min(32L, p.M - row0));
  for (int r = 0; r < rows; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                                           (lane & 3) * 4);
    const long c = col0 + 2 * lane;
    __half *at = p.y + (row0 + r) * p.N + c;
    if (c < p.N) at[0] = __ushort_as_half(static_cast<unsigned short>(w));
    if (c + 1 < p.N) at[1] = __ushort_as_half(static_cast<unsigned short>(w >> 16));
  }
}

template <int CG, int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w0,
                  const __grid_constant__ CUtensorMap map_w1, const __grid_constant__ CUtensorMap map_out,
                  const TcParams p) {
  using PL = Plan<CG, BN>;
  constexpr int S = PL::S;
  constexpr int COLS = MODE == kLinear ? BN : BN / 2;  // output columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank = 0;
  if (CG == 2) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  const uint32_t bar0 = base + PL::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto sf_full = [&](int i) { return bar0 + 8u * (2 * S + i); };
  auto sf_empty = [&](int i) { return bar0 + 8u * (2 * S + kScaleSets + i); };
  auto acc_full = [&](int r) { return bar0 + 8u * (2 * (S + kScaleSets) + r); };
  auto acc_free = [&](int r) { return bar0 + 8u * (2 * (S + kScaleSets) + 2 + r); };
  const uint32_t drain = bar0 + 8u * (2 * (S + kScaleSets) + 4);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + PL::OFF_BAR + PL::NUM_BARS * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const Waits wait{abort_flag, p.err, p.wait_limit};
  auto all_wait = [&](uint32_t bar, uint32_t parity, unsigned code) {
    return __all_sync(0xffffffffu, wait(bar, parity, code)) != 0;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < kScaleSets; ++i) {
      mbar_init(sf_full(i), CG == 2 && rank == 0 ? 3 : 2);  // the scale warps; in the pair's first CTA, the second's sets too
      mbar_init(sf_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), 4 * CG);  // the epilogue warps of each CTA
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)), "r"(PL::TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)), "r"(PL::TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  const int nkb = p.nkb, nsets = (nkb + kScaleBlocks - 1) / kScaleBlocks;
  bool ok = true;

  if (warp == 0) {
    // -------------------------------------------------------- code copies --
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, pend = 0, pph = 0;
      for (int t = first; t < p.ntiles && ok; t += step) {
        const Tile tl = tile_at(p, t);
        const int row = tl.m * (kRows * CG) + static_cast<int>(rank) * kRows;
        const int col = tl.n * COLS;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!(ok = wait(empty(s), ph ^ 1u, kDevErrEmptyBarrier))) break;
          // (test only) the first stage left unissued: the MMAs' wait for it gives up
          if (!(p.skip_first_copy && t == first && kb == 0)) {
            const uint32_t bar = CG == 2 ? in_leader(full(s)) : full(s);
            if (rank == 0) {
              mbar_arrive_expect_tx(full(s), CG * PL::STAGE);
              pend |= 1u << s;
              pph = (pph & ~(1u << s)) | (ph << s);
            }
            const uint32_t a = base + s * PL::STAGE, b = a + PL::A_BYTES;
            load_tile<CG>(a, &map_x, bar, kb * kBlock, row);
            if (MODE == kLinear) {
              load_tile<CG>(b, &map_w0, bar, kb * kBlock, col + static_cast<int>(rank) * PL::BROWS);
            } else if (CG == 2) {
              load_tile<CG>(b, rank == 0 ? &map_w0 : &map_w1, bar, kb * kBlock, col);
            } else {
              load_tile<CG>(b, &map_w0, bar, kb * kBlock, col);
              load_tile<CG>(b + PL::B_BYTES / 2, &map_w1, bar, kb * kBlock, col);
            }
          }
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // Every copy has landed before the CTAs can leave: the first CTA's
      // barriers count those of both.  After a wait that gave up a stage may
      // be half issued, which no barrier tells: copies land within
      // microseconds, so wait a while.
      if (ok) {
        for (int i = 0; i < S; ++i)
          if ((pend >> i) & 1u) wait_bar_teardown(full(i), (pph >> i) & 1u);
      }
      if (!ok || p.skip_first_copy) {
        const long long t0 = clock64();
        while (clock64() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMAs ----
    if (rank == 0) {
      const uint32_t on = elect();
      constexpr uint32_t idesc = (1u << 23) | (static_cast<uint32_t>(BN >> 3) << 17) |
                                 (static_cast<uint32_t>(kRows * CG >> 4) << 24);
      const uint64_t desc0 = sw128_desc(base);
      int s = 0, sets = 0, done = 0;
      uint32_t ph = 0;
      for (int t = first; t < p.ntiles && ok; t += step, ++done) {
        const uint32_t r = done & 1;
        if (PL::OVERLAP) {
          if (done > 0) ok = all_wait(acc_free(0), (done - 1) & 1u, kDevErrTmemEmpty);
        } else {
          ok = all_wait(acc_free(r), ((done >> 1) & 1u) ^ 1u, kDevErrTmemEmpty);
        }
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (r ? PL::ACC1 : 0);
        uint32_t sfa = 0;
        for (int kb = 0; kb < nkb; ++kb) {
          const int id = kb % kScaleBlocks, set = sets % kScaleSets;
          if (id == 0) {
            // the tensor memory of the set before last is written again
            if (sets >= 2 && !(ok = all_wait(sf_empty((sets - 2) % kScaleSets),
                                             ((sets - 2) / kScaleSets) & 1u, kDevErrEmptyBarrier)))
              break;
            if (!(ok = all_wait(sf_full(set), (sets / kScaleSets) & 1u, kDevErrFullBarrier))) break;
            sfa = tmem + PL::SF0 + (sets & 1) * PL::SF_COLS;
            const uint32_t from = base + PL::OFF_SF + set * PL::SF_BYTES;
#pragma unroll
            for (int i = 0; i < 1 + PL::SFB; ++i) copy_scales<CG>(on, sfa + 4 * i, from + 512 * i);
          }
          if (!(ok = all_wait(full(s), ph, kDevErrFullBarrier))) break;
          tc_fence_after();
          const uint64_t a = desc0 + s * (PL::STAGE >> 4), b = a + (PL::A_BYTES >> 4);
          const uint32_t with_id = idesc | (static_cast<uint32_t>(id) << 29) | (static_cast<uint32_t>(id) << 4);
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k)
            mma_scaled<CG>(on, d, a + k * 2, b + k * 2, with_id, sfa, sfa + 4,
                           kb > 0 || k > 0);
          commit<CG>(on, empty(s));
          if (id == kScaleBlocks - 1 || kb == nkb - 1) {
            commit<CG>(on, sf_empty(set));
            ++sets;
          }
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        commit<CG>(on, acc_full(r));
      }
      // every MMA has landed before tensor memory is freed
      commit<CG>(on, drain);
      wait_bar_teardown(drain, 0);
      __syncwarp();
    } else {
      // The second CTA passes on that its scales are there.  Not the scale
      // warps themselves: a release to the cluster waits for all that its
      // thread has requested, and theirs have loads under way (the MMAs waited
      // for scales a third of the time).
      int sets = 0;
      for (int t = first; t < p.ntiles && ok; t += step)
        for (int q = 0; q < nsets; ++q, ++sets) {
          const int set = sets % kScaleSets;
          if (!(ok = all_wait(sf_full(set), (sets / kScaleSets) & 1u, kDevErrFullBarrier))) break;
          if (lane == 0) arrive_cluster(in_leader(sf_full(set)));
          __syncwarp();
        }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales ----
    // Set of 128 rows x 4 blocks: row r's word at (r % 32) 16 + (r / 32) 4, so
    // lane l gathers rows l, l + 32, l + 64, l + 96.  Warp 2 takes the tokens'
    // set and the second set of weights, warp 3 the first one.
    //
    // A load queues behind the stages that this SM has requested, up to 192 KB,
    // and touches 32 lines, of which few fit beside the stages: so up to four
    // sets of a tile are requested at once (a line is fetched once for them),
    // a batch ahead.  What does not exist is 1.0; behind a row's last block
    // comes the next row's, which no MMA uses.
    constexpr int BATCH = 4, PARTS = PL::SFB;
    const bool two = warp == 2 && PARTS == 2;
    const uint8_t *const from[2] = {warp == 2 ? p.sx : p.sw[0], MODE == kLinear ? p.sw[0] : p.sw[1]};
    const int rows[2] = {warp == 2 ? p.M : p.N, p.N};
    const int access[2] = {warp == 2 ? p.access[0] : p.access[1], MODE == kLinear ? p.access[1] : p.access[2]};
    typedef uint32_t Batch[PARTS][4][BATCH];
    int nt = first, nq = 0;  // the next batch to request
    auto request = [&](Batch &w) {
      if (nt >= p.ntiles) return;
      const Tile tl = tile_at(p, nt);
      const int col = tl.n * COLS, row = tl.m * (kRows * CG) + static_cast<int>(rank) * kRows;
      const int r0[2] = {lane + (warp == 2 ? row : col), lane + (MODE == kLinear ? col + 128 : col)};
#pragma unroll
      for (int e = 0; e < PARTS; ++e) {
        if (e == 1 && !two) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0[e] + 32 * i;
          const uint8_t *at = from[e] + static_cast<long>(r) * p.G + 4 * nq;
          if (r >= rows[e]) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j) w[e][i][j] = 0x7f7f7f7fu;
          } else if (access[e] == 16) {  // then the sets of a tile are a multiple of BATCH
            const uint4 v = *reinterpret_cast<const uint4 *>(at);
            w[e][i][0] = v.x;
            w[e][i][1] = v.y;
            w[e][i][2] = v.z;
            w[e][i][3] = v.w;
          } else if (access[e] == 4) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
              if (nq + j < nsets) w[e][i][j] = *reinterpret_cast<const uint32_t *>(at + 4 * j);
          } else {
            // any address: the words around it, shifted
            const uintptr_t lo = reinterpret_cast<uintptr_t>(from[e]), end = lo + static_cast<long>(rows[e]) * p.G;
            const uintptr_t word = reinterpret_cast<uintptr_t>(at) & ~static_cast<uintptr_t>(3);
            const uint32_t shift = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 3u) * 8u;
            uint32_t v[BATCH + 1];
#pragma unroll
            for (int j = 0; j <= BATCH; ++j) v[j] = word_within(word + 4 * j, lo, end);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) w[e][i][j] = __funnelshift_r(v[j], v[j + 1], shift);
          }
        }
      }
      if ((nq += BATCH) >= nsets) {
        nq = 0;
        nt += step;
      }
    };
    int sets = 0;
    auto hand_over = [&](const Batch &w, int count) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (j >= count || !ok) break;
        const int set = sets % kScaleSets;
        if (!(ok = all_wait(sf_empty(set), ((sets / kScaleSets) & 1u) ^ 1u, kDevErrEmptyBarrier))) break;
        uint8_t *to = sm + PL::OFF_SF + set * PL::SF_BYTES + lane * 16;
        *reinterpret_cast<uint4 *>(to + (warp == 2 ? 0 : 512)) = make_uint4(w[0][0][j], w[0][1][j], w[0][2][j], w[0][3][j]);
        if (two)
          *reinterpret_cast<uint4 *>(to + 1024) =
              make_uint4(w[PARTS - 1][0][j], w[PARTS - 1][1][j], w[PARTS - 1][2][j], w[PARTS - 1][3][j]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full(set));
        ++sets;
      }
    };
    Batch w0, w1;
    request(w0);
    for (int t = first, q = 0; t < p.ntiles && ok;) {
      auto turn = [&](Batch &now, Batch &next) {
        request(next);
        hand_over(now, min(BATCH, nsets - q));
        if ((q += BATCH) >= nsets) {
          q = 0;
          t += step;
        }
      };
      turn(w0, w1);
      if (t >= p.ntiles || !ok) break;
      turn(w1, w0);
    }
  } else {
    // ---------------------------------------------------------- epilogue ----
    const int q = warp & 3;
    uint8_t *buf = sm + PL::OFF_OUT + q * 4096, *mine = buf + lane * 128;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    auto put = [&](int chunk, uint4 v) {
      *reinterpret_cast<uint4 *>(mine + ((chunk ^ (lane & 7)) << 4)) = v;
    };
    int done = 0;
    for (int t = first; t < p.ntiles; t += step, ++done) {
      const Tile tl = tile_at(p, t);
      const uint32_t r = done & 1;
      const long row0 = static_cast<long>(tl.m) * (kRows * CG) + rank * kRows + q * 32;
      const long col0 = static_cast<long>(tl.n) * COLS;
      if (!__all_sync(0xffffffffu, wait(acc_full(r), (done >> 1) & 1u, kDevErrAccumBarrier))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (r ? PL::ACC1 : 0) + lanes;
      // this warp has read what the next tile (overlapping accumulators), or
      // the one after it, writes over
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = acc_free(PL::OVERLAP ? 0 : r);
          if (CG == 2)
            arrive_read(in_leader(bar));
          else
            mbar_arrive(bar);
        }
      };
      if (MODE == kLinear) {
#pragma unroll 1
        for (int i = 0; i < BN / 64; ++i) {
          // the shared columns first: the end of the first accumulator, the
          // start of the second
          const int j = PL::OVERLAP && r == 0 ? BN / 64 - 1 - i : i;
          uint32_t v[32], w[32];
          tmem_ld32(acc + j * 64, v);
          tmem_ld32(acc + j * 64 + 32, w);
          tmem_wait_ld32(v);
          tmem_wait_ld32(w);
          if (i == (PL::OVERLAP ? 0 : BN / 64 - 1)) release();
          if (lane == 0) stores_read();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            auto f = [](uint32_t x) { return __uint_as_float(x); };
            put(c, make_uint4(half2_bits(f(v[8 * c]), f(v[8 * c + 1])), half2_bits(f(v[8 * c + 2]), f(v[8 * c + 3])),
                              half2_bits(f(v[8 * c + 4]), f(v[8 * c + 5])),
                              half2_bits(f(v[8 * c + 6]), f(v[8 * c + 7]))));
            put(4 + c, make_uint4(half2_bits(f(w[8 * c]), f(w[8 * c + 1])), half2_bits(f(w[8 * c + 2]), f(w[8 * c + 3])),
                                  half2_bits(f(w[8 * c + 4]), f(w[8 * c + 5])),
                                  half2_bits(f(w[8 * c + 6]), f(w[8 * c + 7]))));
          }
          put_half(p, &map_out, buf, lane, row0, col0 + j * 64);
          __syncwarp();
        }
      } else {
        float h[MODE == kGatedCodes ? 128 : 32];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = r == 0 ? 3 - i : i;  // 32 columns of both halves, the shared ones first
          uint32_t g[32], u[32];
          tmem_ld32(acc + 32 * c, g);
          tmem_ld32(acc + 128 + 32 * c, u);
          tmem_wait_ld32(g);
          tmem_wait_ld32(u);
          if (i == 0) release();
          float *hi = h + (MODE == kGatedCodes ? 32 * i : 0);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float a = __uint_as_float(g[e]), b = __uint_as_float(u[e]);
            hi[e] = p.gelu ? gated<true>(a, b) : gated<false>(a, b);
            if (MODE == kGatedCodes) top = fmaxf(top, fabsf(hi[e]));
          }
          if (MODE == kGatedHalf) {
            if ((i & 1) == 0) {
              if (lane == 0) stores_read();
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              put(4 * (c & 1) + e,
                  make_uint4(half2_bits(hi[8 * e], hi[8 * e + 1]), half2_bits(hi[8 * e + 2], hi[8 * e + 3]),
                             half2_bits(hi[8 * e + 4], hi[8 * e + 5]), half2_bits(hi[8 * e + 6], hi[8 * e + 7])));
            if ((i & 1) == 1) {
              put_half(p, &map_out, buf, lane, row0, col0 + 64 * (c >> 1));
              __syncwarp();
            }
          }
        }
        if (MODE == kGatedCodes) {
          const uint32_t byte = fp8_scale_byte(top);
          const float m = fp8_scale_inverse(byte);
          if (row0 + lane < p.M)
            p.scales[(row0 + lane) * fp8_groups_of(p.N) + tl.n] = static_cast<uint8_t>(byte);
          if (lane == 0) stores_read();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = r == 0 ? 3 - i : i;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float *v = h + 32 * i + 16 * e + 4 * k;
                w[k] = fp8_pack4(v[0] * m, v[1] * m, v[2] * m, v[3] * m);
              }
              put(2 * c + e, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          if (row0 < p.M) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) store_tile(&map_out, smem_u32(buf), static_cast<int>(col0), static_cast<int>(row0));
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) stores_read();
    tc_fence_before();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    if (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(PL::TMEM_COLS));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(PL::TMEM_COLS));
  }
}

// ------------------------------------------------------------ host side --

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (fn == nullptr) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess || q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

// Row-major [rows, cols], boxes of box_rows rows of 128 bytes with the 128-byte
// swizzle; elements outside read 0 and are not written.
bool make_map(CUtensorMap *map, const void *ptr, long rows, long cols, int elem_bytes, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem_bytes};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem_bytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
             const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int BN, int MODE>
int launch_t(const Fp8Params &f, cudaStream_t s) {
  using PL = Plan<CG, BN>;
  static int ctas[64] = {};  // resident CTAs, per device
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W8A8_ERR_CUDA;
  int most = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ctas[dev] == 0) {
      int sms = 0;
      if (cudaFuncSetAttribute(fp8_tc_kernel<CG, BN, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               PL::SMEM_BYTES) != cudaSuccess ||
          cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return W8A8_ERR_CUDA;
      ctas[dev] = sms / CG * CG;
    }
    most = ctas[dev];
  }
  TcParams p = {};
  p.sx = f.sx;
  p.sw[0] = f.sw[0];
  p.sw[1] = f.sw[1];
  p.M = f.M;
  p.N = f.N;
  p.G = f.G;
  p.nkb = f.G;
  constexpr int COLS = MODE == kLinear ? BN : BN / 2;
  const long mt = (static_cast<long>(f.M) + kRows * CG - 1) / (kRows * CG);
  const long nt = (static_cast<long>(f.N) + COLS - 1) / COLS;
  if (mt * nt > 0x3fffffffL) return W8A8_ERR_INVALID_ARG;
  p.mtiles = static_cast<int>(mt);
  p.ntn = static_cast<int>(nt);
  p.ntiles = static_cast<int>(mt * nt);
  // the operand that is walked first is read again and again: the smaller one
  p.m_first = f.M <= f.N;
  auto access = [&](const uint8_t *at) {
    const uintptr_t low = reinterpret_cast<uintptr_t>(at) | static_cast<uintptr_t>(f.G);
    return low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 1;
  };
  p.access[0] = access(f.sx);
  p.access[1] = access(f.sw[0]);
  p.access[2] = access(f.sw[1]);
  p.gelu = f.gelu;
  p.scales = f.scales;
  if ((p.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  p.wait_limit = role_wait_limit();
  p.skip_first_copy = skip_first_copy();

  CUtensorMap mx, mw0, mw1, mo;
  const int wrows = MODE == kLinear ? PL::BROWS : BN / 2;
  if (!make_map(&mx, f.x, f.M, f.K, 1, kRows) || !make_map(&mw0, f.w[0], f.N, f.K, 1, wrows)) return W8A8_ERR_CUDA;
  mw1 = mw0;
  mo = mx;
  if (MODE != kLinear && !make_map(&mw1, f.w[1], f.N, f.K, 1, wrows)) return W8A8_ERR_CUDA;
  if (MODE == kGatedCodes) {
    if (!make_map(&mo, f.codes, f.M, f.N, 1, 32)) return W8A8_ERR_CUDA;
  } else if (f.N % 8 == 0) {  // rows of y are 16-byte multiples
    if (!make_map(&mo, f.y, f.M, f.N, 2, 32)) return W8A8_ERR_CUDA;
  } else {
    p.y = f.y;
  }

  cudaLaunchConfig_t cfg = {};
  const long need = static_cast<long>(p.ntiles) * CG;
  cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = PL::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fp8_tc_kernel<CG, BN, MODE>, mx, mw0, mw1, mo, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

int launch_fp8_tc(const Fp8Params &f, cudaStream_t s) {
  const bool pair = f.M > kRows;
  if (f.w[1] == nullptr) return pair ? launch_t<2, 256, kLinear>(f, s) : launch_t<1, 64, kLinear>(f, s);
  if (f.codes != nullptr) return pair ? launch_t<2, 256, kGatedCodes>(f, s) : launch_t<1, 256, kGatedCodes>(f, s);
  return pair ? launch_t<2, 256, kGatedHalf>(f, s) : launch_t<1, 256, kGatedHalf>(f, s);
}

}  // namespace w8a8
