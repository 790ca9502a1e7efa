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
// from Wu, so a tile is 128 columns of both.  (Few rows or few tiles: fp8_mid.cu.)
//
// Warps of a CTA: 0 copies the codes (TMA), 1 issues the MMAs (in the pair's
// first CTA; the second's passes on that its scales are there), 2 and 3 gather
// the scale bytes into the layout that tcgen05.cp takes, 4 - 7 are the
// epilogue.  Persistent, static tiles.
//
// Tensor memory: two accumulators of 256 columns and two sets of scales (12
// columns each) are 536 of 512 columns.  So the accumulators overlap by 24
// columns: the epilogue reads the shared ones first, and the next tile's MMAs
// wait for that alone.
//
// Every wait is bounded as in the GEMM; a CTA of a pair leaves only after both
// are done (cluster barrier), since either one's copies and MMAs reach into the
// other.
#include <mutex>

#include "fp8.cuh"
#include "fp8_kernels.cuh"
#include "fp8_mma.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;      // tokens of a CTA's part of a tile
constexpr int kScaleSets = 8;   // sets in shared memory (two of them in tensor memory)
constexpr int kScaleLag = 4;    // sets whose copies are under way

enum Mode { kLinear = 0, kGatedHalf = 1, kGatedCodes = 2 };

constexpr int kCols = 256;      // columns of a tile's accumulator
constexpr int kTileRows = 2 * kRows;
constexpr int kTileBytes = kRows * kBlock;  // what a CTA fetches of either operand: 128 rows
constexpr int kStage = 2 * kTileBytes;
constexpr int kStages = 5;
constexpr int kSetBytes = 3 * 512;          // scales of 128 tokens and of 256 columns
constexpr int kOffOut = kStages * kStage;   // 4 warps x 2 x 32 rows x 128 bytes
constexpr int kOffScales = kOffOut + 4 * 8192;
constexpr int kOffBars = kOffScales + kScaleSets * kSetBytes;
constexpr int kBars = 2 * (kStages + kScaleSets) + 2 + 1 + 1;
constexpr int kSmemBytes = kOffBars + kBars * 8 + 16 + 1024;  // + alignment by hand
constexpr uint32_t kTmemCols = 512, kSetCols = 12;
constexpr uint32_t kScaleCol = kTmemCols - 2 * kSetCols, kAcc1 = kScaleCol - kCols;  // the second accumulator
static_assert(kAcc1 + 32 >= kCols, "the shared columns are within one 32-column read");
static_assert(kSmemBytes <= 232448, "shared memory");

struct TcParams {
  const uint8_t *sx, *sw[2];
  int M, N, G, nkb, ntiles, mtiles, ntn;  // N: columns of the output
  int m_first;      // tiles walk the tokens first
  int access[3];    // bytes that a load of sx, sw[0], sw[1] may take at once: 16, 4 or 1
  bool gelu, early;
  __half *y;        // stored directly (no map) where the rows are not 16-byte multiples
  uint8_t *scales;
  unsigned int *err;
  long long wait_limit;
  int skip_first_copy;
};

__device__ __forceinline__ void store_tile(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The shared memory that this thread's stores but the last MOST read may be
// written again.
template <int MOST>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(MOST) : "memory");
}

struct Tile {
  int m, n;  // tile indexes
};

__device__ __forceinline__ Tile tile_at(const TcParams &p, int t) {
  return p.m_first ? Tile{t % p.mtiles, t / p.mtiles} : Tile{t / p.ntn, t % p.ntn};
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
  // Rows that do not start at 16 bytes.  The epilogue has one warp a scheduler, so
  // what counts is instructions a row: whole tiles have paths without branches.
  const uint8_t *const from = buf + (lane & 3) * 4;
  auto word = [&](int r) { return *reinterpret_cast<const uint32_t *>(from + r * 128 + (((lane >> 2) ^ (r & 7)) << 4)); };
  uint16_t *to = reinterpret_cast<uint16_t *>(p.y + row0 * p.N + col0) + 2 * lane;
  if (row0 + 32 <= p.M && col0 + 64 <= p.N) {
    if ((p.N & 1) == 0) {  // every row starts at a word
#pragma unroll 8
      for (int r = 0; r < 32; ++r, to += p.N) *reinterpret_cast<uint32_t *>(to) = word(r);
      return;
    }
    // The first row starts at a word (y is 16-byte aligned, row0 and col0 are even),
    // every other one between two words: halves there.  (Words that straddle two
    // lanes' halves took 181 us for 12703 x 7009 x 512, halves throughout 79.)
#pragma unroll 4
    for (int k = 0; k < 16; ++k, to += 2 * static_cast<long>(p.N)) {
      const uint32_t a = word(2 * k), b = word(2 * k + 1);
      uint16_t *const next = to + p.N;
      *reinterpret_cast<uint32_t *>(to) = a;
      next[0] = static_cast<uint16_t>(b);
      next[1] = static_cast<uint16_t>(b >> 16);
    }
    return;
  }
  const int rows = static_cast<int>(min(32L, p.M - row0)), left = static_cast<int>(min(64L, p.N - col0));
  for (int r = 0; r < rows; ++r, to += p.N) {
    const uint32_t w = word(r);
    if (2 * lane < left) to[0] = static_cast<uint16_t>(w);
    if (2 * lane + 1 < left) to[1] = static_cast<uint16_t>(w >> 16);
  }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w0,
                  const __grid_constant__ CUtensorMap map_w1, const __grid_constant__ CUtensorMap map_out,
                  const TcParams p) {
  constexpr int S = kStages, COLS = MODE == kLinear ? kCols : kCols / 2;  // output columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  const uint32_t bar0 = base + kOffBars;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto sf_full = [&](int i) { return bar0 + 8u * (2 * S + i); };
  auto sf_empty = [&](int i) { return bar0 + 8u * (2 * S + kScaleSets + i); };
  auto acc_full = [&](int r) { return bar0 + 8u * (2 * (S + kScaleSets) + r); };
  const uint32_t acc_free = bar0 + 8u * (2 * (S + kScaleSets) + 2), drain = acc_free + 8u;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBars + kBars * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const Waits wait{abort_flag, p.err, p.wait_limit};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < kScaleSets; ++i) {
      mbar_init(sf_full(i), rank == 0 ? 3 : 2);  // the scale warps; in the pair's first CTA, the second's sets too
      mbar_init(sf_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(acc_full(i), 1);
    mbar_init(acc_free, 8);  // the epilogue warps of both CTAs
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();  // whole warps again: what follows is for all lanes at once (.aligned)
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // not before the tensor memory is ours: a CTA of the next kernel that got it
  // first would wait for this one
  if (p.early) asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int nkb = p.nkb, nsets = (nkb + kScaleBlocks - 1) / kScaleBlocks;
  bool ok = true;

  if (warp == 0) {
    // -------------------------------------------------------- code copies --
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, pend = 0, pph = 0;
      for (int t = first; t < p.ntiles && ok; t += step) {
        const Tile tl = tile_at(p, t);
        const int row = tl.m * (kTileRows) + static_cast<int>(rank) * kRows;
        const int col = tl.n * COLS;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!(ok = wait(empty(s), ph ^ 1u, kDevErrEmptyBarrier))) break;
          // (test only) the first stage left unissued: the MMAs' wait for it gives up
          if (!(p.skip_first_copy && t == first && kb == 0)) {
            const uint32_t bar = in_leader(full(s));
            if (rank == 0) {
              mbar_arrive_expect_tx(full(s), 2 * kStage);
              pend |= 1u << s;
              pph = (pph & ~(1u << s)) | (ph << s);
            }
            const uint32_t a = base + s * kStage, b = a + kTileBytes;
            load_tile(a, &map_x, bar, kb * kBlock, row);
            if (MODE == kLinear)
              load_tile(b, &map_w0, bar, kb * kBlock, col + static_cast<int>(rank) * kRows);
            else
              load_tile(b, rank == 0 ? &map_w0 : &map_w1, bar, kb * kBlock, col);
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
      constexpr uint32_t idesc = (1u << 23) | (static_cast<uint32_t>(kCols >> 3) << 17) |
                                 (static_cast<uint32_t>(kTileRows >> 4) << 24);
      const uint64_t desc0 = sw128_desc(base);
      int s = 0, sets = 0, done = 0;
      uint32_t ph = 0;
      for (int t = first; t < p.ntiles && ok; t += step, ++done) {
        const uint32_t r = done & 1;
        if (done > 0) ok = wait.warp(acc_free, (done - 1) & 1u, kDevErrTmemEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (r ? kAcc1 : 0);
        uint32_t sfa = 0;
        for (int kb = 0; kb < nkb; ++kb) {
          const int id = kb % kScaleBlocks, set = sets % kScaleSets;
          if (id == 0) {
            // the tensor memory of the set before last is written again
            if (sets >= 2 && !(ok = wait.warp(sf_empty((sets - 2) % kScaleSets),
                                             ((sets - 2) / kScaleSets) & 1u, kDevErrEmptyBarrier)))
              break;
            if (!(ok = wait.warp(sf_full(set), (sets / kScaleSets) & 1u, kDevErrFullBarrier))) break;
            sfa = tmem + kScaleCol + (sets & 1) * kSetCols;
            const uint32_t from = base + kOffScales + set * kSetBytes;
#pragma unroll
            for (int i = 0; i < 3; ++i) copy_scales<2>(on, sfa + 4 * i, from + 512 * i);
          }
          if (!(ok = wait.warp(full(s), ph, kDevErrFullBarrier))) break;
          tc_fence_after();
          const uint64_t a = desc0 + s * (kStage >> 4), b = a + (kTileBytes >> 4);
          const uint32_t with_id = idesc | (static_cast<uint32_t>(id) << 29) | (static_cast<uint32_t>(id) << 4);
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k)
            mma_scaled<2>(on, d, a + k * 2, b + k * 2, with_id, sfa, sfa + 4,
                           kb > 0 || k > 0);
          commit<2>(on, empty(s));
          if (id == kScaleBlocks - 1 || kb == nkb - 1) {
            commit<2>(on, sf_empty(set));
            ++sets;
          }
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        commit<2>(on, acc_full(r));
      }
      // every MMA has landed before tensor memory is freed
      commit<2>(on, drain);
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
          if (!(ok = wait.warp(sf_full(set), (sets / kScaleSets) & 1u, kDevErrFullBarrier))) break;
          if (lane == 0) arrive_cluster(in_leader(sf_full(set)));
          __syncwarp();
        }
      // the first CTA's last commit arrives here too, before this CTA may leave
      wait_bar_teardown(drain, 0);
      __syncwarp();
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales ----
    // Set of 128 rows x 4 blocks: row r's word at (r % 32) 16 + (r / 32) 4, so
    // lane l gathers rows l, l + 32, l + 64, l + 96.  Warp 2 takes the tokens'
    // set and the second set of weights, warp 3 the first one.
    //
    // What is requested queues behind the stages that this SM has requested, up to
    // 160 KB.  So rows of whole words go by asynchronous copies, four sets ahead
    // (4000 x 8192 x 512: 20 us, 3000 x 4096 x 2048: 21.6; by registers, a batch of up
    // to four sets of a tile ahead, 28.5 and 24.5, and no better two batches ahead).
    // Rows at any address go by registers.  What does not exist is 1.0; behind a
    // row's last block comes the next row's, which no MMA uses.
    constexpr int BATCH = kScaleBatch, PARTS = 2;
    const bool two = warp == 2;
    const uint8_t *const from[2] = {warp == 2 ? p.sx : p.sw[0], MODE == kLinear ? p.sw[0] : p.sw[1]};
    const int rows[2] = {warp == 2 ? p.M : p.N, p.N};
    const int access[2] = {warp == 2 ? p.access[0] : p.access[1], MODE == kLinear ? p.access[1] : p.access[2]};
    if (access[0] >= 4 && (!two || access[1] >= 4)) {
      int sets = 0;
      auto hand_over = [&](int n) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full(n % kScaleSets));
      };
      for (int t = first; t < p.ntiles && ok; t += step) {
        const Tile tl = tile_at(p, t);
        const int col = tl.n * COLS, row = tl.m * kTileRows + static_cast<int>(rank) * kRows;
        const int r0[2] = {lane + (warp == 2 ? row : col), lane + (MODE == kLinear ? col + 128 : col)};
        const uint8_t *at[PARTS][4];
#pragma unroll
        for (int e = 0; e < PARTS; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0[e] + 32 * i;
            at[e][i] = (e == 0 || two) && r < rows[e] ? from[e] + static_cast<long>(r) * p.G : nullptr;
          }
        for (int q = 0; q < nsets; ++q, ++sets) {
          const int set = sets % kScaleSets;
          if (!(ok = wait.warp(sf_empty(set), ((sets / kScaleSets) & 1u) ^ 1u, kDevErrEmptyBarrier))) break;
          uint8_t *to = sm + kOffScales + set * kSetBytes + lane * 16;
#pragma unroll
          for (int e = 0; e < PARTS; ++e) {
            if (e == 1 && !two) continue;
            uint8_t *const place = to + (e == 1 ? 1024 : warp == 2 ? 0 : 512);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (at[e][i] != nullptr)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(place + 4 * i)),
                             "l"(at[e][i] + 4 * q)
                             : "memory");
              else
                *reinterpret_cast<uint32_t *>(place + 4 * i) = 0x7f7f7f7fu;
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (sets >= kScaleLag) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kScaleLag) : "memory");
            hand_over(sets - kScaleLag);
          }
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (ok)
        for (int n = max(0, sets - kScaleLag); n < sets; ++n) hand_over(n);
    } else {
      typedef ScaleRow Batch[PARTS][4];
      int nt = first, nq = 0;  // the next batch to request
      auto request = [&](Batch &w) {
        if (nt >= p.ntiles) return;
        const Tile tl = tile_at(p, nt);
        const int col = tl.n * COLS, row = tl.m * (kTileRows) + static_cast<int>(rank) * kRows;
        const int r0[2] = {lane + (warp == 2 ? row : col), lane + (MODE == kLinear ? col + 128 : col)};
#pragma unroll
        for (int e = 0; e < PARTS; ++e) {
          if (e == 1 && !two) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0[e] + 32 * i;
            const uint8_t *at = r < rows[e] ? from[e] + static_cast<long>(r) * p.G + 4 * nq : nullptr;
            w[e][i].request(at, nsets - nq, access[e], from[e], static_cast<long>(rows[e]) * p.G);
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
          if (!(ok = wait.warp(sf_empty(set), ((sets / kScaleSets) & 1u) ^ 1u, kDevErrEmptyBarrier))) break;
          uint8_t *to = sm + kOffScales + set * kSetBytes + lane * 16;
          *reinterpret_cast<uint4 *>(to + (warp == 2 ? 0 : 512)) = make_uint4(w[0][0].get(j), w[0][1].get(j), w[0][2].get(j), w[0][3].get(j));
          if (two)
            *reinterpret_cast<uint4 *>(to + 1024) =
                make_uint4(w[PARTS - 1][0].get(j), w[PARTS - 1][1].get(j), w[PARTS - 1][2].get(j), w[PARTS - 1][3].get(j));
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
    }
  } else {
    // ---------------------------------------------------------- epilogue ----
    const int q = warp & 3;
    // two buffers in turn: a store reads its own for several hundred cycles
    uint8_t *buf = sm + kOffOut + q * 8192, *mine = buf + lane * 128;
    int turn = 0;
    auto next_buffer = [&]() {
      if (lane == 0) stores_read<1>();
      __syncwarp();
      turn ^= 1;
      buf = sm + kOffOut + q * 8192 + turn * 4096;
      mine = buf + lane * 128;
    };
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    auto put = [&](int chunk, uint4 v) {
      *reinterpret_cast<uint4 *>(mine + ((chunk ^ (lane & 7)) << 4)) = v;
    };
    int done = 0;
    for (int t = first; t < p.ntiles; t += step, ++done) {
      const Tile tl = tile_at(p, t);
      const uint32_t r = done & 1;
      const long row0 = static_cast<long>(tl.m) * (kTileRows) + rank * kRows + q * 32;
      const long col0 = static_cast<long>(tl.n) * COLS;
      if (!wait.warp(acc_full(r), (done >> 1) & 1u, kDevErrAccumBarrier)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (r ? kAcc1 : 0) + lanes;
      // this warp has read what the next tile (overlapping accumulators), or
      // the one after it, writes over
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_read(in_leader(acc_free));
        __syncwarp();  // the next load from tensor memory is the whole warp's
      };
      if (MODE == kLinear) {
#pragma unroll 1
        for (int i = 0; i < kCols / 64; ++i) {
          // the shared columns first: the end of the first accumulator, the
          // start of the second
          const int j = r == 0 ? kCols / 64 - 1 - i : i;
          uint32_t v[32], w[32];
          tmem_ld32(acc + j * 64, v);
          tmem_ld32(acc + j * 64 + 32, w);
          tmem_wait_ld32(v);
          tmem_wait_ld32(w);
          if (i == 0) release();
          next_buffer();
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
          float a[32], b[32], o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            a[e] = __uint_as_float(g[e]);
            b[e] = __uint_as_float(u[e]);
          }
          gate_all<32>(p.gelu, a, b, o);
          float *hi = h + (MODE == kGatedCodes ? 32 * i : 0);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            hi[e] = o[e];
            if (MODE == kGatedCodes) top = fmaxf(top, fabsf(o[e]));
          }
          if (MODE == kGatedHalf) {
            if ((i & 1) == 0) next_buffer();
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
          next_buffer();
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
    if (lane == 0) stores_read<0>();
    tc_fence_before();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// ------------------------------------------------------------ host side --

template <int MODE>
int launch_t(const Fp8Params &f, cudaStream_t s) {
  static int ctas[64] = {};  // resident CTAs, per device
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W8A8_ERR_CUDA;
  int most = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ctas[dev] == 0) {
      int sms = 0;
      if (cudaFuncSetAttribute(fp8_tc_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmemBytes) != cudaSuccess ||
          cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return W8A8_ERR_CUDA;
      ctas[dev] = sms / 2 * 2;
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
  constexpr int COLS = MODE == kLinear ? kCols : kCols / 2;
  const long mt = (static_cast<long>(f.M) + kTileRows - 1) / (kTileRows);
  const long nt = (static_cast<long>(f.N) + COLS - 1) / COLS;
  if (mt * nt > 0x3fffffffL || nt * COLS > 0x7fffffffL || mt * kTileRows > 0x7fffffffL) return W8A8_ERR_INVALID_ARG;
  p.mtiles = static_cast<int>(mt);
  p.ntn = static_cast<int>(nt);
  p.ntiles = static_cast<int>(mt * nt);
  // the operand that is walked first is read again and again: the smaller one
  p.m_first = f.M <= f.N;
  p.access[0] = scale_access(f.sx, f.G);
  p.access[1] = scale_access(f.sw[0], f.G);
  p.access[2] = scale_access(f.sw[1], f.G);
  p.gelu = f.gelu;
  p.early = f.early;
  p.scales = f.scales;
  if ((p.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  p.wait_limit = role_wait_limit();
  p.skip_first_copy = skip_first_copy();

  CUtensorMap mx, mw0, mw1, mo;
  if (!make_map(&mx, f.x, f.M, f.K, 1, kRows) || !make_map(&mw0, f.w[0], f.N, f.K, 1, kRows)) return W8A8_ERR_CUDA;
  mw1 = mw0;
  mo = mx;
  if (MODE != kLinear && !make_map(&mw1, f.w[1], f.N, f.K, 1, kRows)) return W8A8_ERR_CUDA;
  if (MODE == kGatedCodes) {
    if (!make_map(&mo, f.codes, f.M, f.N, 1, 32)) return W8A8_ERR_CUDA;
  } else if (f.N % 8 == 0) {  // rows of y are 16-byte multiples
    if (!make_map(&mo, f.y, f.M, f.N, 2, 32)) return W8A8_ERR_CUDA;
  } else {
    p.y = f.y;
  }

  cudaLaunchConfig_t cfg = {};
  const long need = static_cast<long>(p.ntiles) * 2;
  cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, fp8_tc_kernel<MODE>, mx, mw0, mw1, mo, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

// A K block of a tile takes about 0.32 us, a tile 1.5 more, a call 6.5 (fitted to
// 131 to 1500 rows on twelve shapes of weights).
float estimate_fp8_tc(const Fp8Params &f) {
  const int cols = f.w[1] == nullptr ? 256 : 128;
  const long tiles = static_cast<long>(ceil_div(f.M, 256)) * ceil_div(f.N, cols);
  const float rounds = static_cast<float>((tiles + kNumSMsGB300 / 2 - 1) / (kNumSMsGB300 / 2));
  return 6.5f + rounds * (f.G * 0.32f + 1.5f);
}

int launch_fp8_tc(const Fp8Params &f, cudaStream_t s) {
  if (f.w[1] == nullptr) return launch_t<kLinear>(f, s);
  return f.codes != nullptr ? launch_t<kGatedCodes>(f, s) : launch_t<kGatedHalf>(f, s);
}

}  // namespace w8a8
