// What the 8-bit float tensor-core kernels share: block-scaled MMAs, the scales'
// way from their rows to tensor memory, bounded waits, tensor maps.
#pragma once

#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace w8a8 {

constexpr int kBlock = 128;      // K of a stage
constexpr int kScaleBlocks = 4;  // stages of a set of scales: the bytes of a word
constexpr int kScaleBatch = 4;   // sets requested at once

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

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// All MMAs issued so far arrive on this barrier when they are done, in both
// CTAs of a pair.
template <int CG>
__device__ __forceinline__ void commit(uint32_t on, uint32_t bar, uint32_t leader = 0) {
  if (CG == 2)
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
        "%1;\n}\n" ::"r"(bar), "h"(static_cast<uint16_t>(3u << leader)), "r"(on) : "memory");
  else
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
                 "r"(on)
                 : "memory");
}

// this address in the pair's first CTA (by its rank in the cluster)
__device__ __forceinline__ uint32_t in_leader(uint32_t addr, uint32_t leader = 0) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(leader));
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

// A tile whose bytes count at a barrier of the pair's first CTA
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
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

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool is_over(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Waits {
  volatile int *abort_flag;
  unsigned int *err;
  long long limit;
  // one thread
  __device__ bool operator()(uint32_t bar, uint32_t parity, unsigned code) const {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (clock64() - t0 > limit) return give_up(code);
    }
    return true;
  }
  // a whole warp, by a vote: a phase that is over costs 76 cycles, against 152
  // with a loop per lane
  __device__ bool warp(uint32_t bar, uint32_t parity, unsigned code) const {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, try_wait(bar, parity))) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
      if (__any_sync(0xffffffffu, clock64() - t0 > limit)) return give_up(code);
    }
    return true;
  }
  __device__ bool give_up(unsigned code) const {
    if (err != nullptr) atomicCAS(err, 0u, code);
    *abort_flag = 1;
    return false;
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// Four words of a row of scales, requested and taken apart, so that the loads can
// be under way.  Rows may start at any address: five words around them, shifted.
struct ScaleRow {
  uint32_t w[kScaleBatch + 1], shift;
  // from `at` (nullptr: no such row, 1.0), as far as the row has them (`left`
  // words).  `access`: see scale_access(); all rows are [first, first + bytes).
  // Behind a row's last byte come the next row's, which no MMA uses.
  __device__ __forceinline__ void request(const uint8_t *at, int left, int access, const uint8_t *first, long bytes) {
    shift = 0;
    if (at == nullptr) {
#pragma unroll
      for (int j = 0; j <= kScaleBatch; ++j) w[j] = 0x7f7f7f7fu;
    } else if (access == 16 && left >= kScaleBatch) {
      const uint4 v = *reinterpret_cast<const uint4 *>(at);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if (access >= 4) {
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j)
        if (j < left) w[j] = *reinterpret_cast<const uint32_t *>(at + 4 * j);
    } else {
      const uintptr_t a = reinterpret_cast<uintptr_t>(at), lo = reinterpret_cast<uintptr_t>(first), end = lo + bytes;
      const uintptr_t word = a & ~static_cast<uintptr_t>(3);
      shift = (static_cast<uint32_t>(a) & 3u) * 8u;
      if (word >= lo && word + 4 * (kScaleBatch + 1) <= end) {
#pragma unroll
        for (int j = 0; j <= kScaleBatch; ++j) w[j] = *reinterpret_cast<const uint32_t *>(word + 4 * j);
      } else {
#pragma unroll
        for (int j = 0; j <= kScaleBatch; ++j) w[j] = j <= left ? word_within(word + 4 * j, lo, end) : 0x7f7f7f7fu;
      }
    }
  }
  __device__ __forceinline__ uint32_t get(int j) const { return __funnelshift_r(w[j], w[j + 1], shift); }
};

// Bytes that a load of rows of G scales may take at once: 16, 4 or 1.
inline int scale_access(const uint8_t *at, int G) {
  const uintptr_t low = reinterpret_cast<uintptr_t>(at) | static_cast<uintptr_t>(G);
  return low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 1;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// ------------------------------------------------------------ host side --

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
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
inline bool make_map(CUtensorMap *map, const void *ptr, long rows, long cols, int elem_bytes, int box_rows) {
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

}  // namespace w8a8
