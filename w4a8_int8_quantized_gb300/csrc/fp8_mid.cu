// Products of 8-bit float rows that are bound by the weights' bytes or by few
// tiles: up to about a thousand rows, and up to 8192 where the columns are few.
// The arithmetic of fp8_tc.cu (block-scaled tcgen05 MMAs, sums in fp32 from the
// first group to the last), in tiles of up to 128 tokens x 128 columns, one tile a
// CTA, two CTAs an SM, and K divided among the CTAs of a cluster where the tiles
// alone are too few.
//
// Above 128 rows a tile may be a pair's (cta_group::2): 256 tokens x up to 160
// columns, each CTA fetching its own tokens and half of the weights.  What an SM
// takes in is the limit there: 512 rows of 10240 x 2560 take 22.9 us in single CTAs
// and 15.9 in pairs, 131 rows 10.1 and 11.6 (a cluster more to start), so the
// estimate decides.
//
// The stages (a ring in half an SM's shared memory) hold only the rows that
// there are: with 40 tokens a stage is 5 KB of tokens and up to 16 KB of
// weights.  The MMA takes 128 rows all the same; what the others hold reaches
// only lanes that nobody reads.
//
// The weights do not come from the previous kernel: the first stages of them
// are requested before it has finished, into the half of the SM that its CTAs
// leave.
//
// Epilogue: a CTA writes its sums as fp32 over its stages; then all threads of
// the cluster add the parts in ascending order of K, apply the gate and write
// 8 columns each: 16 lanes have the 128 columns of a group of codes.
#include <algorithm>
#include <mutex>

#include "fp8.cuh"
#include "fp8_kernels.cuh"
#include "fp8_mma.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStages = 12;
constexpr int kScaleSets = 8;       // sets of scales in shared memory, and in tensor memory
// half of an SM's 228 KB, less 1 KB that the system keeps for each CTA
constexpr int kSmemBytes = 228 * 1024 / 2 - 1024;
constexpr int kBars = 2 * (kMaxStages + kScaleSets) + 2;
constexpr uint32_t kTmemCols = 256;

// CG: CTAs that share a tile.  Columns up to kMostCols, of which 128 and 32 (pairs)
// in sets of scales of their own; behind them the scales in tensor memory.
template <int CG>
struct Room {
  static constexpr int MOST_COLS = CG == 2 ? 160 : 128, SFB = CG == 2 ? 2 : 1;
  static constexpr int SET_BYTES = 512 * (1 + SFB), SET_COLS = 4 * (1 + SFB);
  static constexpr int TAIL = kScaleSets * SET_BYTES + kBars * 8 + 16;
  static constexpr int REGION = (kSmemBytes - 1024 - TAIL) / 1024 * 1024;  // stages; 1 KB for alignment by hand
  static_assert(MOST_COLS + kScaleSets * SET_COLS <= kTmemCols, "tensor memory");
};


enum Mode { kLinear = 0, kGatedHalf = 1, kGatedCodes = 2 };

struct MidParams {
  const __half *x;   // QUANT: the tokens themselves
  const uint8_t *sx, *sw[2];
  int M, N, K, G;
  int mr, bn;        // rows and columns (of both matrices, if gated) of a tile
  int split, nx;     // CTAs of a cluster: parts of K, tiles of a group of codes
  int stages, token_bytes;
  int access[3];     // see scale_access()
  bool gelu, early;
  __half *y;
  uint8_t *codes, *scales;
  unsigned int *err;
  long long wait_limit;
  int skip_first_copy;
};

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void take(float (&to)[8], const float4 &lo, const float4 &hi) {
  to[0] += lo.x;
  to[1] += lo.y;
  to[2] += lo.z;
  to[3] += lo.w;
  to[4] += hi.x;
  to[5] += hi.y;
  to[6] += hi.z;
  to[7] += hi.w;
}

template <int CG, int MODE, bool QUANT>
__global__ void __launch_bounds__(kThreads, 2)
    fp8_mid_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w0,
                   const __grid_constant__ CUtensorMap map_w1, const MidParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRegion = Room<CG>::REGION, kSetBytes = Room<CG>::SET_BYTES, SFB = Room<CG>::SFB;
  constexpr uint32_t kScaleCol = Room<CG>::MOST_COLS;
  // QUANT: the tokens of all K blocks first, then the stages, of weights alone
  const int S = p.stages, a_bytes = p.mr * kBlock, stage = (QUANT ? 0 : a_bytes) + p.bn / CG * kBlock;
  const int cols = MODE == kLinear ? p.bn : p.bn / 2;
  // a cluster: parts of K, each of nx tiles, each of one CTA or a pair
  // (32-bit divisions: 64-bit ones took a third of the start)
  const int team = p.split * p.nx * CG, cluster = static_cast<int>(blockIdx.x / static_cast<unsigned>(team));
  const int rank = static_cast<int>(blockIdx.x) - cluster * team;
  const int half = CG == 2 ? rank & 1 : 0, leader = rank - half;
  const int part = rank / (p.nx * CG), xi = rank / CG - part * p.nx, tile_n = cluster * p.nx + xi;
  const int col0 = tile_n * cols, row0 = (static_cast<int>(blockIdx.y) * CG + half) * p.mr;
  // K blocks of this part; its sets of scales are those of the whole row
  const int kb0 = p.G * part / p.split, nkb = p.G * (part + 1) / p.split - kb0;
  const int set0 = kb0 / kScaleBlocks, nsets = (kb0 + nkb + kScaleBlocks - 1) / kScaleBlocks - set0;
  const uint32_t a_base = base, b_base = base + (QUANT ? p.token_bytes : a_bytes);

  const uint32_t sf = base + kRegion, bar0 = sf + kScaleSets * kSetBytes;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto sf_full = [&](int i) { return bar0 + 8u * (2 * kMaxStages + i); };
  auto sf_empty = [&](int i) { return bar0 + 8u * (2 * kMaxStages + kScaleSets + i); };
  const uint32_t acc_full = bar0 + 8u * (2 * (kMaxStages + kScaleSets)), drain = acc_full + 8u;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kRegion + kScaleSets * kSetBytes + kBars * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const Waits wait{abort_flag, p.err, p.wait_limit};

  // a thread a barrier: full, empty, the scales' full and empty, the sums, the drain
  if (threadIdx.x < kBars) {
    const int i = static_cast<int>(threadIdx.x) - 2 * kMaxStages;
    mbar_init(bar0 + 8u * threadIdx.x, i >= 0 && i < kScaleSets ? (QUANT ? 5 : CG == 2 && half == 0 ? 3 : 2) : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (threadIdx.x == kThreads - 1) {
    prefetch_map(&map_w0);
    if (MODE != kLinear) prefetch_map(&map_w1);
    if (!QUANT) prefetch_map(&map_x);
    *abort_flag = 0;
  }
  __syncwarp();  // whole warps again: what follows is for all lanes at once (.aligned)
  if (warp == 1) {
    if (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "n"(kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "n"(kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tc_fence_before();
  if (CG == 2)
    cluster_sync();  // the other half's barriers are ready
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Not before the tensor memory is ours: a CTA of the next kernel that got it
  // first would wait for this one.
  if (p.early) asm volatile("griddepcontrol.launch_dependents;");
  bool ok = true;

  if (warp == 0) {
    // -------------------------------------------------------- code copies --
    if (lane == 0) {
      auto weights = [&](int s, int kb) {
        const uint32_t b = b_base + s * stage;
        const int k = (kb0 + kb) * kBlock;
        if (CG == 2) {
          // all of a pair's bytes count in its first CTA
          if (half == 0) mbar_arrive_expect_tx(full(s), 2 * stage);
          const uint32_t bar = in_leader(full(s), leader);
          if (MODE == kLinear)
            load_tile(b, &map_w0, bar, k, col0 + half * (p.bn / 2));
          else
            load_tile(b, half == 0 ? &map_w0 : &map_w1, bar, k, col0);
        } else {
          mbar_arrive_expect_tx(full(s), stage);
          tma_load_2d(b, &map_w0, full(s), k, col0);
          if (MODE != kLinear) tma_load_2d(b + cols * kBlock, &map_w1, full(s), k, col0);
        }
      };
      auto tokens = [&](int s, int kb) {
        if (QUANT) return;
        if (CG == 2)
          load_tile(a_base + s * stage, &map_x, in_leader(full(s), leader), (kb0 + kb) * kBlock, row0);
        else
          tma_load_2d(a_base + s * stage, &map_x, full(s), (kb0 + kb) * kBlock, row0);
      };
      // (test only) the first stage left unissued: the MMAs' wait for it gives up
      const int from = p.skip_first_copy ? 1 : 0, ahead = min(S, nkb);
      for (int kb = from; kb < ahead; ++kb) weights(kb, kb);
      if (!QUANT) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int kb = from; kb < ahead; ++kb) tokens(kb, kb);
      int s = ahead == S ? 0 : ahead, kb = ahead;
      uint32_t ph = 0;  // of the stage's last use
      for (; kb < nkb; ++kb) {
        if (!(ok = wait(empty(s), ph, kDevErrEmptyBarrier))) break;
        weights(s, kb);
        tokens(s, kb);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      // every copy has landed before the CTA can leave: a pair's at the first's barriers
      if (half == 0)
        for (int i = max(from, kb - S); i < kb; ++i) wait_bar_teardown(full(i % S), (i / S) & 1);
      if (CG == 2 && (!ok || p.skip_first_copy)) {
        // of a stage that only one of them issued no barrier tells: copies land
        // within microseconds
        const long long t0 = clock64();
        while (clock64() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMAs ----
    if (CG == 2 && half == 1) {
      // passes on that its scales are there (as in fp8_tc.cu)
      for (int q = 0; q < nsets && ok; ++q) {
        if (!(ok = wait.warp(sf_full(q % kScaleSets), (q / kScaleSets) & 1u, kDevErrFullBarrier))) break;
        if (lane == 0) arrive_cluster(in_leader(sf_full(q % kScaleSets), leader));
        __syncwarp();
      }
      // the first CTA's last commit arrives here too, before this CTA may leave
      wait_bar_teardown(drain, 0);
      __syncwarp();
    } else {
    const uint32_t on = elect();
    const uint32_t idesc = (1u << 23) | (static_cast<uint32_t>(p.bn >> 3) << 17) | (static_cast<uint32_t>(8 * CG) << 24);
    const uint64_t a0 = sw128_desc(a_base), b0 = sw128_desc(b_base);
    int s = 0;
    uint32_t ph = 0, sfa = 0;
    // the barriers of a step are looked at under the step before it
    bool staged = false, scaled = false;
    for (int kb = 0; kb < nkb; ++kb) {
      const int id = (kb0 + kb) % kScaleBlocks, at = (kb0 + kb) / kScaleBlocks - set0, set = at % kScaleSets;
      if (id == 0 || kb == 0) {
        // a set that is there has its place in tensor memory free too: the
        // places are as many, and its own in shared memory was
        if (!__all_sync(0xffffffffu, scaled) &&
            !(ok = wait.warp(sf_full(set), (at / kScaleSets) & 1u, kDevErrFullBarrier)))
          break;
        sfa = tmem + kScaleCol + set * Room<CG>::SET_COLS;
#pragma unroll
        for (int i = 0; i < 1 + SFB; ++i) copy_scales<CG>(on, sfa + 4 * i, sf + set * kSetBytes + 512 * i);
      }
      if (!__all_sync(0xffffffffu, staged) && !(ok = wait.warp(full(s), ph, kDevErrFullBarrier))) break;
      tc_fence_after();
      const uint64_t a = a0 + (((QUANT ? kb * a_bytes : s * stage)) >> 4), b = b0 + ((s * stage) >> 4);
      const uint32_t with_id = idesc | (static_cast<uint32_t>(id) << 29) | (static_cast<uint32_t>(id) << 4);
      const uint32_t freed = empty(s);
      if (++s == S) {
        s = 0;
        ph ^= 1u;
      }
      staged = is_over(full(s), ph);
      if (id == kScaleBlocks - 1) scaled = is_over(sf_full((at + 1) % kScaleSets), ((at + 1) / kScaleSets) & 1u);
#pragma unroll
      for (int k = 0; k < kBlock / 32; ++k)
        mma_scaled<CG>(on, tmem, a + k * 2, b + k * 2, with_id, sfa, sfa + 4, kb > 0 || k > 0);
      if (kb + S < nkb) commit<CG>(on, freed, leader);  // else it is not filled again
      if (id == kScaleBlocks - 1 && at + kScaleSets < nsets) commit<CG>(on, sf_empty(set), leader);
    }
    if (ok) commit<CG>(on, acc_full, leader);
    // every MMA has landed before tensor memory is freed
    commit<CG>(on, drain, leader);
    wait_bar_teardown(drain, 0);
    __syncwarp();
    }
  } else if (warp == 3 || (warp == 2 && !QUANT)) {
    // ------------------------------------------------------------ scales ----
    // Set of 128 rows x 4 blocks: row r's word at (r % 32) 16 + (r / 32) 4.  Warp 2
    // gathers the tokens' rows, warp 3 the weights', of which the gate's come
    // first (a pair's columns from 128 on in a second set).
    const bool mine = warp == 2;  // the tokens' rows
    if (mine) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int all_sets = (p.G + kScaleBlocks - 1) / kScaleBlocks;
    constexpr int R = 3 + SFB;  // rows of a lane
    const uint8_t *at[R], *first[R];
    int access[R];
    long bytes[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = lane + 32 * i, which = mine ? 0 : MODE != kLinear && r >= cols ? 2 : 1;
      const int row = mine ? row0 + r : col0 + (which == 2 ? r - cols : r);
      const bool there = row < (mine ? p.M : p.N) && r < (mine ? p.mr : p.bn);
      first[i] = mine ? p.sx : which == 2 ? p.sw[1] : p.sw[0];
      access[i] = mine ? p.access[0] : which == 2 ? p.access[2] : p.access[1];
      if (set0 % 4 != 0 && access[i] == 16) access[i] = 4;
      bytes[i] = static_cast<long>(mine ? p.M : p.N) * p.G;
      at[i] = there ? first[i] + static_cast<long>(row) * p.G + set0 * kScaleBlocks : nullptr;
    }
    const int left = all_sets - set0;
    auto request = [&](ScaleRow (&w)[R], int q) {
      if (q >= nsets) return;
#pragma unroll
      for (int i = 0; i < R; ++i)
        w[i].request(at[i] == nullptr ? nullptr : at[i] + 4 * q, left - q, access[i], first[i], bytes[i]);
    };
    auto hand_over = [&](const ScaleRow (&w)[R], int q) {
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        if (q + j >= nsets || !ok) break;
        const int set = (q + j) % kScaleSets;
        if (!(ok = wait.warp(sf_empty(set), (((q + j) / kScaleSets) & 1u) ^ 1u, kDevErrEmptyBarrier))) break;
        uint8_t *to = sm + kRegion + set * kSetBytes + (mine ? 0 : 512) + lane * 16;
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0].get(j), w[1].get(j), w[2].get(j), w[3].get(j));
        if (R == 5 && !mine) *reinterpret_cast<uint32_t *>(to + 512) = w[R - 1].get(j);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full(set));
      }
    };
    ScaleRow w0[R], w1[R];
    request(w0, 0);
    for (int q = 0; q < nsets && ok; q += 2 * kScaleBatch) {
      request(w1, q + kScaleBatch);
      hand_over(w0, q);
      request(w0, q + 2 * kScaleBatch);
      hand_over(w1, q + kScaleBatch);
    }
  } else if (warp >= 4) {
    if (QUANT) {
      // ------------------------------------------- quantizing the tokens ----
      // Half a warp a token and K block, as the quantizer's kernel does it: 8
      // elements a lane; codes at their place in the swizzled tile, the scale
      // at its own among the set's bytes.
      asm volatile("griddepcontrol.wait;" ::: "memory");
      constexpr int AHEAD = 8, TEAMS = 8;
      const int units = p.M * nkb, l = lane & 15;
      for (int u0 = (warp - 4) * 2 + (lane >> 4); (u0 & ~1) < units; u0 += AHEAD * TEAMS) {
        uint4 x[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int u = u0 + j * TEAMS, kb = u / p.M, k = (kb0 + kb) * kBlock + l * 8;
          x[j] = make_uint4(0, 0, 0, 0);
          if (u < units && k < p.K) x[j] = *reinterpret_cast<const uint4 *>(p.x + static_cast<long>(u - kb * p.M) * p.K + k);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int u = u0 + j * TEAMS, kb = u / p.M, row = u - kb * p.M;
          if ((u & ~1) >= units) break;
          const __half2 *h = reinterpret_cast<const __half2 *>(&x[j]);
          float v[8], top = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(h[e]);
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const uint32_t byte = fp8_scale_byte(top);
          const float m = fp8_scale_inverse(byte);
          if (u < units) {
            *reinterpret_cast<uint2 *>(sm + kb * a_bytes + row * 128 + (((l >> 1) ^ (row & 7)) << 4) + (l & 1) * 8) =
                make_uint2(fp8_pack4(v[0] * m, v[1] * m, v[2] * m, v[3] * m),
                           fp8_pack4(v[4] * m, v[5] * m, v[6] * m, v[7] * m));
            const int gb = kb0 + kb;
            if (l == 0)
              sm[kRegion + (gb / kScaleBlocks - set0) * kSetBytes + row * 16 + gb % kScaleBlocks] =
                  static_cast<uint8_t>(byte);
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane < nsets) mbar_arrive(sf_full(lane));  // no more sets than places
      __syncwarp();
    }
    // ----------------------------------------- sums to shared memory --------
    // Rows of bn + 4 floats: eight rows' 16-byte pieces fill all banks.
    if ((warp & 3) * 32 < p.mr && wait.warp(acc_full, 0, kDevErrAccumBarrier)) {
      tc_fence_after();
      const int row = (warp & 3) * 32 + lane;
      const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      float *to = reinterpret_cast<float *>(sm) + row * (p.bn + 4);
      // behind bn: columns of this CTA's own tensor memory, not kept
      auto keep = [&](const uint32_t (&v)[32], int c) {
        if (row < p.mr) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + 4 * e < p.bn)
              *reinterpret_cast<uint4 *>(to + c + 4 * e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
      };
      for (int c = 0; c < p.bn; c += 64) {
        uint32_t v[32], w[32];
        tmem_ld32(from + c, v);
        if (c + 32 < p.bn) tmem_ld32(from + c + 32, w);
        tmem_wait_ld32(v);
        tmem_wait_ld32(w);
        keep(v, c);
        if (c + 32 < p.bn) keep(w, c + 32);
      }
      tc_fence_before();
    }
  }

  __syncwarp();
  tc_fence_before();
  const int out_team = p.split * p.nx, out_rank = rank / CG;  // who writes together
  if (out_team > 1) {
    cluster_sync();
  } else {
    __syncthreads();
    if (CG == 2) {  // both are done with the tensor memory; nothing is handed over
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
  }
  tc_fence_after();
  if (warp == 1) {
    if (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------------------------------------- outputs ----
  {
    const int rows = min(p.mr, p.M - row0), per_tile = cols / 8, per_row = p.nx * per_tile;
    const int group0 = cluster * p.nx * cols;  // first column of the cluster
    const int items = rows * per_row, stride = out_team * kThreads, pitch = (p.bn + 4) * 4;
    int i = out_rank * kThreads + static_cast<int>(threadIdx.x);
    int row = i / per_row, ch = i - row * per_row;
    const int rows_on = stride / per_row, ch_on = stride - rows_on * per_row;
    // whole warps: the lanes of a group of codes exchange their maxima
    for (; (i & ~31) < items; i += stride, row += rows_on, ch += ch_on) {
      if (ch >= per_row) {
        ch -= per_row;
        ++row;
      }
      const bool in = i < items;
      const int x = ch >= per_tile ? 1 : 0;
      const uint32_t at = (in ? row : 0) * pitch + (ch - x * per_tile) * 32;
      float v[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.f;
      if (out_team == 1) {
        take(v, reinterpret_cast<const float4 *>(sm + at)[0], reinterpret_cast<const float4 *>(sm + at)[1]);
        if (MODE != kLinear)
          take(u, reinterpret_cast<const float4 *>(sm + at + cols * 4)[0], reinterpret_cast<const float4 *>(sm + at + cols * 4)[1]);
      } else {
        // parts of K in ascending order, two of them on their way at a time
        for (int k = 0; k < p.split; k += 2) {
          float4 w[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (k + e >= p.split) break;
            uint32_t a;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(base + at), "r"(((k + e) * p.nx + x) * CG + half));
            w[e][0] = load_cluster(a);
            w[e][1] = load_cluster(a + 16);
            if (MODE != kLinear) {
              w[e][2] = load_cluster(a + cols * 4);
              w[e][3] = load_cluster(a + cols * 4 + 16);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (k + e >= p.split) break;
            take(v, w[e][0], w[e][1]);
            if (MODE != kLinear) take(u, w[e][2], w[e][3]);
          }
        }
      }
      if (MODE != kLinear) {
        gate_all<8>(p.gelu, v, u, v);
      }
      const long m = row0 + row, n = group0 + ch * 8;
      if (MODE == kGatedCodes) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t byte = fp8_scale_byte(top);
        const float s = fp8_scale_inverse(byte);
        if (in && n < p.N) {  // N is a multiple of 16
          *reinterpret_cast<uint2 *>(p.codes + m * p.N + n) =
              make_uint2(fp8_pack4(v[0] * s, v[1] * s, v[2] * s, v[3] * s), fp8_pack4(v[4] * s, v[5] * s, v[6] * s, v[7] * s));
          if (ch == 0) p.scales[m * ((p.N + 127) >> 7) + (n >> 7)] = static_cast<uint8_t>(byte);
        }
      } else if (in && n < p.N) {
        // as wide as the address allows: rows may start at any half
        __half *to = p.y + m * p.N + n;
        const uint32_t w[4] = {half2_bits(v[0], v[1]), half2_bits(v[2], v[3]), half2_bits(v[4], v[5]), half2_bits(v[6], v[7])};
        const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to)) & 15u;
        if (n + 8 > p.N) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < p.N) to[e] = __float2half_rn(v[e]);
        } else if (low == 0) {
          *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if ((low & 7u) == 0) {
          reinterpret_cast<uint2 *>(to)[0] = make_uint2(w[0], w[1]);
          reinterpret_cast<uint2 *>(to)[1] = make_uint2(w[2], w[3]);
        } else if ((low & 3u) == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) reinterpret_cast<uint32_t *>(to)[e] = w[e];
        } else {
          to[0] = __float2half_rn(v[0]);
#pragma unroll
          for (int e = 0; e < 3; ++e)
            *reinterpret_cast<uint32_t *>(to + 1 + 2 * e) = __funnelshift_r(w[e], w[e + 1], 16);
          to[7] = __float2half_rn(v[7]);
        }
      }
    }
  }
  __syncwarp();
  if (team > 1) {  // the others may still read this CTA's sums; nothing is handed over
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
}

// ------------------------------------------------------------ host side --

// CTAs of this kernel that run at once, by the cluster's size: two an SM, less what
// clusters leave of the processor clusters (from cudaOccupancyMaxActiveClusters, which
// counts one an SM for a kernel with tcgen05 instructions; two were seen to run).
constexpr int kResident[9] = {0, 304, 304, 276, 288, 280, 276, 210, 240};

// Microseconds of a call by a model fitted to 11600 timings (1 to 1000 rows, twelve
// shapes of weights, all tiles and parts, single CTAs and pairs): its choice takes on
// average 2 % and at most 27 % longer than the best one.  A CTA takes 77 GB/s, or
// 0.27 us a K block (one thread issues its MMAs; a pair a little more), an SM 137
// GB/s; HBM gives 6200 GB/s to all; the epilogue and the joining of parts go with the
// tile's size.
float estimate(const Fp8Params &f, int cg, int mr, int bn, int split, int nx) {
  const int blocks = ceil_div(f.G, split), cols = f.w[1] == nullptr ? bn : bn / 2, team = split * nx * cg;
  const long groups = (static_cast<long>(f.N) + cols * nx - 1) / (cols * nx);
  const long ctas = groups * team * ceil_div(f.M, 128 * cg);
  const float waves = static_cast<float>((ctas + kResident[team] - 1) / kResident[team]);
  const float bytes = (mr + bn / cg) * (kBlock * 1e-3f);  // of a stage, in KB
  const float block = std::max((ctas <= kNumSMsGB300 ? 0.27f : 0.32f) * (cg == 2 ? 1.18f : 1.f), bytes / 77.f);
  const float sm = static_cast<float>(ctas) * blocks * bytes / (kNumSMsGB300 * 137.f);
  const float hbm = static_cast<float>(f.N) * (f.w[1] == nullptr ? 1 : 2) * f.G * kBlock / 6.2e6f;
  const float tile = mr * bn / 16384.f;
  const float join = team == 1 ? 0.f : 0.24f + 0.06f * team + 2.2f * (split - 1) * tile;
  return 2.5f + std::max(std::max(waves * blocks * block, hbm), sm) + (waves - 1.f) * 3.6f + join +
         (cg == 2 ? 2.9f : 2.2f) * waves * tile;
}

template <int CG, int MODE, bool QUANT>
int launch_t(const Fp8Params &f, const Fp8Plan &plan, cudaStream_t s) {
  static bool ready[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W8A8_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(fp8_mid_kernel<CG, MODE, QUANT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
              cudaSuccess ||
          cudaFuncSetAttribute(fp8_mid_kernel<CG, MODE, QUANT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return W8A8_ERR_CUDA;
      ready[dev] = true;
    }
  }
  const int mt = ceil_div(f.M, plan.mr * CG);
  constexpr int kRegion = Room<CG>::REGION;
  MidParams p = {};
  p.sx = f.sx;
  p.sw[0] = f.sw[0];
  p.sw[1] = f.sw[1];
  p.M = f.M;
  p.N = f.N;
  p.K = f.K;
  p.G = f.G;
  p.mr = plan.mr;
  p.bn = plan.bn;
  p.split = plan.split;
  p.nx = plan.nx;
  if (QUANT) {
    p.x = f.xh;
    p.token_bytes = ceil_div(f.G, p.split) * p.mr * kBlock;
    p.stages = (kRegion - p.token_bytes) / (p.bn * kBlock);
  } else {
    // the last stage's MMAs read 128 rows from its start
    const int rows = p.mr + p.bn / CG, spare = (128 - rows) * kBlock;
    p.stages = (kRegion - (spare > 0 ? spare : 0)) / (rows * kBlock);
  }
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.access[0] = scale_access(f.sx, f.G);
  p.access[1] = scale_access(f.sw[0], f.G);
  p.access[2] = scale_access(f.sw[1], f.G);
  p.gelu = f.gelu;
  p.early = f.early;
  p.y = f.y;
  p.codes = f.codes;
  p.scales = f.scales;
  if ((p.err = device_error_word()) == nullptr) return W8A8_ERR_CUDA;
  p.wait_limit = role_wait_limit();
  p.skip_first_copy = skip_first_copy();

  const int cols = MODE == kLinear ? p.bn : p.bn / 2, team = p.split * p.nx * CG, wrows = MODE == kLinear ? p.bn / CG : cols;
  const long groups = (static_cast<long>(f.N) + cols * p.nx - 1) / (cols * p.nx);
  if (groups * cols * p.nx > 0x7fffffffL || groups * team > 0x7fffffffL) return W8A8_ERR_INVALID_ARG;
  CUtensorMap mx, mw0, mw1;
  if (!make_map(&mw0, f.w[0], f.N, f.K, 1, wrows)) return W8A8_ERR_CUDA;
  mx = mw1 = mw0;
  if (!QUANT && !make_map(&mx, f.x, f.M, f.K, 1, p.mr)) return W8A8_ERR_CUDA;
  if (MODE != kLinear && !make_map(&mw1, f.w[1], f.N, f.K, 1, wrows)) return W8A8_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * team), static_cast<unsigned>(mt));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(team);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = team > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fp8_mid_kernel<CG, MODE, QUANT>, mx, mw0, mw1, p) != cudaSuccess) {
    cudaGetLastError();
    return W8A8_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

namespace {

// The best tile for these parts of K.
Fp8Plan best_tile(const Fp8Params &f, int split) {
  Fp8Plan best = {};
  const int nx = f.codes != nullptr ? 2 : 1;
  for (int cg = 1; cg <= (f.M > 128 ? 2 : 1); ++cg) {
    if (split * nx * cg > 8) break;
    const int tiles_m = ceil_div(f.M, 128 * cg), mr = (ceil_div(f.M, tiles_m * cg) + 7) & ~7;
    const int most = nx == 2 ? 128 : cg == 2 ? Room<2>::MOST_COLS : Room<1>::MOST_COLS;
    for (int bn = nx == 2 ? 128 : f.w[1] == nullptr ? 32 : 48; bn <= most; bn += 16) {
      const float t = estimate(f, cg, mr, bn, split, nx);
      if (best.us == 0.f || t < best.us) best = {cg, mr, bn, split, nx, t};
    }
  }
  return best;
}

Fp8Plan find_plan(const Fp8Params &f) {
  // The parts of K decide the order of a sum, so they are the same for a class of
  // batches, whose result for a row then does not depend on the others: those that
  // suit the class's largest (up to 1000 rows 2 % slower on average than each batch's
  // own, at most 25 %; not compared above, where the model is not fitted either).
  // Undivided, both kernels give the same sums.
  Fp8Params typical = f;
  typical.M = f.M <= 16 ? 16 : f.M <= 64 ? 64 : f.M <= 128 ? 128 : f.M <= 384 ? 384 : f.M <= 1024 ? 1024 : f.M <= 2560 ? 2560 : 8192;
  const int most = f.M > 8192 ? 1 : std::min(f.codes != nullptr ? 4 : 8, f.G);
  Fp8Plan best = {};
  if (typical.M > 128) best.us = estimate_fp8_tc(typical), best.split = 1;
  for (int split = 1; split <= most; ++split) {
    const Fp8Plan plan = best_tile(typical, split);
    if (best.us == 0.f || plan.us < best.us) best = plan;
  }
  return best_tile(f, best.split);
}

}  // namespace

Fp8Plan plan_fp8_mid(const Fp8Params &f) {
  // by sizes alone; looking for it takes 0.6 us of a call
  struct Known {
    int M, N, G, form;
    Fp8Plan plan;
  };
  static thread_local Known known[64] = {};
  const int form = f.w[1] == nullptr ? 1 : f.codes == nullptr ? 2 : 3;
  const unsigned at = (static_cast<unsigned>(f.M) * 31u + static_cast<unsigned>(f.N) * 17u + static_cast<unsigned>(f.G) * 7u + form) % 64u;
  Known &k = known[at];
  if (k.M != f.M || k.N != f.N || k.G != f.G || k.form != form) k = {f.M, f.N, f.G, form, find_plan(f)};
  return k.plan;
}

bool fp8_mid_quantizes(const Fp8Params &f, const Fp8Plan &plan) {
  // every part's sets have places of their own, and a thread's share of the work
  // is two rounds of requests
  const int blocks = ceil_div(f.G, plan.split);
  return f.M <= 32 && f.M * blocks <= 128 && (blocks + 2 * kScaleBlocks - 2) / kScaleBlocks <= kScaleSets;
}

int launch_fp8_mid(const Fp8Params &f, const Fp8Plan &plan, cudaStream_t s) {
  const bool pair = plan.cg == 2;
  if (f.w[1] == nullptr) {
    if (f.xh != nullptr) return launch_t<1, kLinear, true>(f, plan, s);
    return pair ? launch_t<2, kLinear, false>(f, plan, s) : launch_t<1, kLinear, false>(f, plan, s);
  }
  if (f.codes == nullptr) return pair ? launch_t<2, kGatedHalf, false>(f, plan, s) : launch_t<1, kGatedHalf, false>(f, plan, s);
  if (f.xh != nullptr) return launch_t<1, kGatedCodes, true>(f, plan, s);
  return pair ? launch_t<2, kGatedCodes, false>(f, plan, s) : launch_t<1, kGatedCodes, false>(f, plan, s);
}

}  // namespace w8a8
