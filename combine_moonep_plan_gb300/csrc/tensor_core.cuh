// What the tensor-core kernels share: CTA pairs, barriers with bounded waits,
// TMA and tcgen05 instructions, and tiles handed out by a warp of the CTA.
//
// A kernel's Shared has `dead` (a warp gave up), `tile` (two batches of 32) and
// the barriers tile_full and tile_empty.
#pragma once

#include <cuda.h>

#include "moonep_internal.cuh"

namespace moonep {

constexpr long long kLimitNs = 1000000000LL;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The same shared address in the pair's first CTA.
__device__ __forceinline__ uint32_t in_leader(uint32_t a) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ long long now_ns() {
  long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// A whole warp waits for a phase, at most a second; false for every lane (and
// the CTA marked dead) after that, or once another warp has given up.
template <typename Shared>
__device__ __noinline__ bool wait_long(Shared *sh, uint32_t bar, uint32_t parity, int32_t *status) {
  const long long t0 = now_ns();
  while (!__all_sync(0xffffffffu, try_wait(bar, parity))) {
    const bool late = now_ns() - t0 > kLimitNs;
    if (late) {
      *(volatile int32_t *)&sh->dead = 1;
      set_status(status, MOONEP_ERR_TIMEOUT);
    }
    if (__any_sync(0xffffffffu, late || *(volatile int32_t *)&sh->dead)) return false;
  }
  return true;
}
template <typename Shared>
__device__ __forceinline__ bool wait(Shared *sh, const void *bar, uint32_t parity,
                                     int32_t *status) {
  if (__all_sync(0xffffffffu, try_wait(smem_addr(bar), parity))) return true;
  return __all_sync(0xffffffffu, wait_long(sh, smem_addr(bar), parity, status));
}
// A value that every lane holds alike, in a uniform register: what comes from
// shared memory, a call or mapa is not known to be one, nor is anything that
// depends on it, and every tensor-core or TMA operand would move first (2.5 to
// 3 % of the kernel's time).
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}
// One lane of the warp, the same each time.  The tensor-core and TMA
// instructions take uniform operands: under this condition, in code that the
// whole warp walks, they issue directly, where a test of the lane number made
// the compiler move every operand for each of them (150 cycles per product).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}
// Without a cluster-scope release: that waits for every load in flight, 1 us
// per stage.  What the arrivals announce is read by the tensor cores alone,
// scales (behind a proxy fence) and accumulator columns (behind a tcgen05
// fence), not by threads of the other CTA.
__device__ __forceinline__ void arrive_leader(const void *bar, uint32_t to_leader) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(smem_addr(bar) + to_leader)
               : "memory");
}
__device__ __forceinline__ void arrive(const void *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void commit(const void *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The i-th tile of this CTA, for a whole warp that reads them in order.
template <typename Shared>
__device__ __forceinline__ bool next_tile(Shared *sh, int i, int32_t *status, int4 *tile) {
  if ((i & 31) == 0 && !wait(sh, &sh->tile_full[(i >> 5) & 1], (i >> 6) & 1, status)) return false;
  const int4 t = sh->tile[(i >> 5) & 1][i & 31];
  *tile = make_int4(uniform(t.x), uniform(t.y), uniform(t.z), uniform(t.w));
  if ((i & 31) == 31) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(&sh->tile_empty[(i >> 5) & 1]);
  }
  return true;
}

// 32 accumulator columns of this warp's 32 lanes; valid after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t v[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
// All loads so far; the registers pass through so that no use moves ahead.
__device__ __forceinline__ void tmem_wait(uint32_t v[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
inline EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return (EncodeFn)p;
  }();
  return fn;
}

}  // namespace moonep
