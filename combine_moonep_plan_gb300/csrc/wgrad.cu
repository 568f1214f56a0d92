// The experts' weight gradients: for every segment of the dispatched layout
//
//   G[g][n, k] (+)= sum over the segment's rows of D[row, n] X[row, k]
// g the segment's weight row: home expert e's gradient is grad[e], slot (j, b)'s
// is slots[j, b], the two sides that the gradient reduction adds up.
//
// The rows are the products' depth, so both operands lie the wrong way round for
// a row-by-row dot product: 64 columns by 8 rows of a swizzled tile, which the
// tensor cores take as they are (both operands "MN-major").  A pair of SMs holds
// a 256 x 256 tile of G in TMEM, twice, 64 rows per stage and five stages.
//
// A segment may end anywhere.  The tensor cores take 16 rows at a time, so the
// last step may hold up to 15 rows of the next segment (or of another rank):
// these are set to zero in shared memory, in both operands, between their
// arrival and the product.  Steps past them are left out.  What lies past a
// matrix's columns arrives as zeros.
//
// One persistent pair of CTAs (cluster of two) per pair of SMs; warps:
//   0      TMA: 64 rows per stage, 128 columns of D and of X per CTA
//   1      products, one thread of the pair's first CTA, four steps per stage
//   2      clears the rows past a segment's end (only where its rows are no
//          multiple of 16): the stage arrives on the CTA's own barrier first
//   3      schedule: the CTA's next 32 tiles at a time
//   4-11   epilogue: accumulator (lane = n, TMEM column = k) through swizzled
//          shared memory, 32 x 32 values per TMA store, or per TMA reduction
//          where the gradients are added to (one addition per element, so the
//          order of nothing changes a result).  The tensor cores' own sums drop
//          bits at every addition, 2e-6 of the result over 2000 rows, so they
//          end after 512 rows and the epilogue adds the parts up in registers
// Where the gradients are so few that their tiles leave SMs idle, the segments' rows
// are split over tiles in a workspace, which join_kernel adds up in order.
// Home experts without rows get zeros unless gradients are added to; slots
// without rows are not touched.  Every wait has a limit of one second, after
// which the kernel latches MOONEP_ERR_TIMEOUT, drains and returns; every warp
// reaches the cluster barrier before the CTAs leave, on every path.
//
// Measured (the kernel alone, 16 experts of 2048 x 7168): 2048 rows each 553 us,
// 1.74 PFLOP/s, 0.90 of the library's burst rate for a plain product; 4096 rows
// 1.03 ms, 1.87; 512 rows 222 us and 128 rows 165 us, 5.7 TB/s, where the outputs'
// bytes bound it (a plain kernel writes such a tensor at 6.4 TB/s).  In a long run
// the power limit takes the clock from 2.07 to 1.5 GHz and a fifth of the rate.
// Between the two bounds the loads of the operands (a pair's 256 x 256 tile asks
// every SM for 64 bytes a cycle of L2) and the stores slow each other down: 512
// rows take 142 us without the stores, and as long with all loads from L2.  What
// the stages hold counts most: five of 64 rows beat four with two store buffers
// per warp (549 against 606 us for 2048 rows) and shorter stages.  Stores of the
// registers themselves, 32 bytes per lane, took 284 us for 512 rows, through
// shared memory by the threads 346; twice the epilogue warps, stores that L2 drops
// first and the next tile's operands prefetched to L2 gained nothing.  Prefetching
// the gradients that are added to took 256 rows of 7168 x 2048 from 388 to 331 us.
#include "moonep_internal.cuh"
#include "tensor_core.cuh"

namespace moonep {
namespace {

constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr int kSide = 256;                 // both sides of a pair's tile
constexpr int kDeep = 64;                  // rows of a stage
constexpr int kChunkBytes = kDeep * 128;   // 64 columns of a stage
constexpr int kSideBytes = 2 * kChunkBytes;
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kPart = 8;                   // stages summed in TMEM at a time
constexpr int kEpilogueWarps = 8;
constexpr int kTileReaders = 2 + kEpilogueWarps;  // and the leader's product warp
constexpr int kEntries = 1024;

struct __align__(1024) Shared {
  uint8_t stage[kStages][kStageBytes];
  uint8_t out[kEpilogueWarps][4096];
  int32_t last[kEntries];   // tiles up to and including the entry's groups
  int32_t start[kEntries];  // first row (rank-local) of the entry's one group
  int32_t rows[kEntries];
  int32_t wsum[8];
  int4 tile[2][32];  // group, tile of n and of k, first row, rows
  uint64_t full[kStages], empty[kStages], tail[kStages], acc_full[2], acc_empty[2];
  uint64_t tile_full[2], tile_empty[2];
  uint32_t tmem;
  int32_t dead;
};

struct GradArgs {
  const int32_t *cu;  // [R, EB]
  int E, B, L, EB, NvS, N, Kd, nb, kb;  // nb, kb: tiles of n and of k
  // Shares: a segment's rows are split into so many (whole stages each), which
  // fill tiles of their own in a workspace [shares, E + R*B, N, Kd] where there are
  // several.  A group below is a share of one: weight row * shares + share.
  int shares;
  int groups, per;    // groups, groups per table entry
  int add;
  int whole_d, whole_x;  // columns in whole blocks of 64
  int32_t *status;
};

// Both operands: rows of 128 bytes (64 columns) with the 128-byte swizzle,
// eight-row groups 1 KB apart, the next 64 columns kChunkBytes further.
__device__ __forceinline__ uint64_t columns_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(kChunkBytes >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Arrival at the pair's first CTA that also passes on this warp's writes.
__device__ __forceinline__ void release_leader(const void *bar, uint32_t to_leader) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   smem_addr(bar) + to_leader)
               : "memory");
}
// fp32 out, bf16 both sides, both with their columns contiguous, 256 x 256
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            ((uint32_t)(kSide >> 3) << 17) | ((uint32_t)(kSide >> 4) << 24);

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdesc), "r"((uint32_t)add)
      : "memory");
}

// Rows [start, start + rows) of weight row w's segment in its rank's window; offsets
// outside the window are reported and the segment treated as empty.
__device__ __forceinline__ bool segment_of(const GradArgs &a, int w, int *start, int *rows) {
  const int j = w < a.E ? w / a.L : (w - a.E) / a.B;
  const int x = w < a.E ? w : a.E + (w - a.E) % a.B;
  const int32_t *cu = a.cu + (int64_t)j * a.EB;
  const int lo = x ? cu[x - 1] : 0, hi = cu[x];
  const bool bad = lo < 0 || hi < lo || hi > a.NvS;
  *start = bad ? 0 : lo;
  *rows = bad ? 0 : hi - lo;
  return !bad;
}
// Rows of a share of a segment, the last ones have fewer or none.
__device__ __forceinline__ int share_rows(int rows, int shares) {
  return ((rows + shares - 1) / shares + kDeep - 1) / kDeep * kDeep;
}
// The same of group g.
__device__ __forceinline__ bool segment(const GradArgs &a, int g, int *start, int *rows) {
  const bool ok = segment_of(a, g / a.shares, start, rows);
  if (a.shares > 1) {
    const int each = share_rows(*rows, a.shares), from = min(g % a.shares * each, *rows);
    *start += from;
    *rows = min(each, *rows - from);
  }
  return ok;
}

__device__ __forceinline__ int tiles_of(const GradArgs &a, int g, int rows) {
  // home experts without rows are zeros, that the kernel after this one writes
  // where there are shares
  return rows > 0 || (g < a.E && !a.add && a.shares == 1) ? a.nb * a.kb : 0;
}

// Tile t: its group and place in the group's gradient, tiles of n fastest within
// bands of eight, so that what all pairs work on at a time is about as high as it
// is wide (7168 x 2048, 1024 rows, added to: 994 us for 48 gradients, 1049 with all
// 28 tiles of n in a row).
__device__ int4 tile_of(const GradArgs &a, const Shared *sh, int t) {
  int lo = 0, hi = (a.groups + a.per - 1) / a.per - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sh->last[mid] > t) hi = mid; else lo = mid + 1;
  }
  int rest = t - (lo ? sh->last[lo - 1] : 0);
  int g = lo * a.per, start = sh->start[lo], rows = sh->rows[lo];
  if (a.per > 1)
    for (;; g++) {
      segment(a, g, &start, &rows);
      const int n = tiles_of(a, g, rows);
      if (rest < n) break;
      rest -= n;
    }
  const int band = rest / (8 * a.kb), left = rest - band * 8 * a.kb;
  const int wide = min(8, a.nb - band * 8), kt = left / wide, nt = band * 8 + left - kt * wide;
  const int w = g / a.shares, j = w < a.E ? w / a.L : (w - a.E) / a.B;
  return make_int4(g, nt | kt << 16, j * a.NvS + start, rows);
}

// The table of tiles; every thread of the CTA takes part.  Returns the count.
__device__ __noinline__ int build_table(const GradArgs &a, Shared *sh) {
  const int entries = (a.groups + a.per - 1) / a.per;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kEntries; i += kThreads) {
    int n = 0, start = 0, rows = 0;
    if (i < entries)
      for (int g = i * a.per; g < min(a.groups, (i + 1) * a.per); g++) {
        if (!segment(a, g, &start, &rows) && blockIdx.x == 0)
          set_status(a.status, MOONEP_ERR_PLAN);
        n += tiles_of(a, g, rows);
      }
    sh->last[i] = n;
    sh->start[i] = start;
    sh->rows[i] = rows;
  }
  __syncthreads();
  // eight warps scan 128 entries each, four per lane
  int4 v = make_int4(0, 0, 0, 0);
  int sum = 0;
  if (warp < 8) {
    v = ((const int4 *)sh->last)[tid];
    v.y += v.x;
    v.z += v.y;
    v.w += v.z;
    sum = v.w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) sh->wsum[warp] = sum;
  }
  __syncthreads();
  if (warp < 8) {
    int base = sum - v.w;
    for (int i = 0; i < warp; i++) base += sh->wsum[i];
    ((int4 *)sh->last)[tid] = make_int4(v.x + base, v.y + base, v.z + base, v.w + base);
  }
  __syncthreads();
  return sh->last[kEntries - 1];
}

// 128 columns from column c on of a stage's rows; whole: in one box, of a map
// that has the columns as blocks of 64.
__device__ __forceinline__ void load_side(uint32_t dst, const CUtensorMap *map, int c, int row,
                                          uint32_t bar, int whole) {
  if (whole) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(c >> 6), "r"(bar)
        : "memory");
  } else {
    tma_load(dst, map, c, row, bar);
    tma_load(dst + kChunkBytes, map, c + 64, row, bar);
  }
}

// 32 x 32 values of shared memory to a gradient, or added to it.
__device__ __forceinline__ void tma_out(const CUtensorMap *map, uint32_t src, int x, int y, int z,
                                        bool add) {
  if (add)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group "
        "[%0, {%1, %2, %3}], [%4];" ::"l"(map),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            map),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap map_d,
                 const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_home,
                 const __grid_constant__ CUtensorMap map_slots, const GradArgs a) {
  extern __shared__ uint8_t raw[];
  Shared *sh = (Shared *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = uniform(cluster_rank());
  // from a shared address to the same one in the pair's first CTA
  const uint32_t to_leader = uniform(in_leader(smem_addr(sh)) - smem_addr(sh));
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  if (tid == 0) {
    sh->dead = 0;
    auto init = [](void *bar, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(n));
    };
    for (int s = 0; s < kStages; s++) {
      init(&sh->full[s], 2);  // both CTAs' loads, or their cleared rows
      init(&sh->empty[s], 1);
      init(&sh->tail[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      init(&sh->tile_full[b], 1);
      init(&sh->tile_empty[b], kTileReaders + (rank == 0));
      init(&sh->acc_full[b], 1);
      init(&sh->acc_empty[b], 2 * kEpilogueWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sh->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  pdl_wait();
  pdl_launch_dependents();
  const int tiles = (int)uniform(build_table(a, sh));
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = uniform(*(volatile uint32_t *)&sh->tmem);
  const int mine = tiles > first ? (tiles - first + step - 1) / step : 0;  // tiles of this pair

  if (warp == 0) {
    uint32_t s = 0, phase = 0, pending = 0, tails = 0, tail_use = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; i++) {
      int4 tile;
      if (!(ok = next_tile(sh, i, a.status, &tile))) break;
      const int stages = (tile.w + kDeep - 1) / kDeep;
      const int n0 = (tile.y & 0xffff) * kSide + (int)rank * 128;
      const int k0 = (tile.y >> 16) * kSide + (int)rank * 128;
      for (int k = 0; k < stages; k++) {
        if (!(ok = wait(sh, &sh->empty[s], phase ^ 1, a.status))) break;
        const uint32_t base = smem_addr(sh->stage[s]);
        const uint32_t full = smem_addr(&sh->full[s]), tail = smem_addr(&sh->tail[s]);
        const bool ragged = k == stages - 1 && (tile.w & 15);
        const uint32_t bar = ragged ? tail : full + to_leader;
        const int row = tile.z + k * kDeep;
        if (elect()) {
          if (ragged)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tail),
                         "r"(kStageBytes)
                         : "memory");
          else if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                         "r"(2 * kStageBytes)
                         : "memory");
          else
            arrive_leader(&sh->full[s], to_leader);
          load_side(base, &map_d, n0, row, bar, a.whole_d);
          load_side(base + kSideBytes, &map_x, k0, row, bar, a.whole_x);
        }
        pending |= 1u << s;
        tails = ragged ? tails | 1u << s : tails & ~(1u << s);
        if (ragged) tail_use ^= 1u << s;
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // the last products release their stages in both CTAs, some time after the
    // accumulator is announced: a CTA does not leave before its own are
    for (int q = 0; q < kStages && ok; q++)
      ok = wait(sh, &sh->empty[q], (uint32_t)q < s ? phase : phase ^ 1, a.status);
    // given up: the copies in flight end before the CTA does
    if (!ok)
      for (int q = 0; q < kStages; q++) {
        const long long t0 = now_ns();
        const bool own = (tails >> q) & 1;
        const uint32_t ph = own ? ((tail_use >> q) & 1) ^ 1 : ((uint32_t)q < s ? phase : phase ^ 1);
        const uint32_t bar = smem_addr(own ? &sh->tail[q] : &sh->full[q]);
        if ((pending & (1u << q)) && (own || rank == 0))
          while (!try_wait(bar, ph) && now_ns() - t0 < kLimitNs / 4) {
          }
      }
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t s = 0, phase = 0;
      int acc = 0;
      bool ok = true;
      const uint32_t stage0 = smem_addr(sh->stage[0]);
      for (int i = 0; i < mine && ok; i++) {
        int4 tile;
        if (!(ok = next_tile(sh, i, a.status, &tile))) break;
        const int stages = (tile.w + kDeep - 1) / kDeep;
        uint32_t d = 0;
        for (int k = 0; k < stages; k++) {
          const int at = k % kPart;
          if (at == 0) {
            d = tmem + (acc & 1) * kSide;
            if (!(ok = wait(sh, &sh->acc_empty[acc & 1], ((acc >> 1) & 1) ^ 1, a.status))) break;
          }
          if (!(ok = wait(sh, &sh->full[s], phase, a.status))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t base = stage0 + s * kStageBytes;
          const uint64_t da = columns_desc(base), db = columns_desc(base + kSideBytes);
          const int steps = min(kDeep / 16, (tile.w - k * kDeep + 15) >> 4);
          if (elect()) {
#pragma unroll
            for (int q = 0; q < kDeep / 16; q++)
              // 16 rows: two groups of eight, 2 KB
              if (q < steps) mma(d, da + 128 * q, db + 128 * q, at + q > 0);
            commit(&sh->empty[s]);
            if (at == kPart - 1 || k == stages - 1) commit(&sh->acc_full[acc & 1]);
          }
          if (at == kPart - 1 || k == stages - 1) acc++;
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 2) {
    uint32_t s = 0, use = 0;  // use: each tail barrier's phase
    for (int i = 0; i < mine; i++) {
      int4 tile;
      if (!next_tile(sh, i, a.status, &tile)) break;
      const int stages = (tile.w + kDeep - 1) / kDeep;
      s = (s + stages) % kStages;
      if (!(tile.w & 15)) continue;
      const uint32_t q = (s + kStages - 1) % kStages;  // the tile's last stage
      if (!wait(sh, &sh->tail[q], (use >> q) & 1, a.status)) break;
      use ^= 1u << q;
      const int from = tile.w - (stages - 1) * kDeep, to = (from + 15) & ~15;
      // a row's lines of the four blocks of 64 columns
      for (int v = lane; v < (to - from) * 32; v += 32) {
        const uint32_t p = smem_addr(sh->stage[q]) + (lane >> 3) * kChunkBytes +
                           (from + (v >> 5)) * 128 + (lane & 7) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
      }
      // the tensor cores read these lines through the async proxy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) release_leader(&sh->full[q], to_leader);
    }
  } else if (warp == 3) {
    // 32 tiles at a time, two such batches
    for (int i = 0; i < mine; i += 32) {
      const int b = (i >> 5) & 1;
      if (!wait(sh, &sh->tile_empty[b], ((i >> 6) & 1) ^ 1, a.status)) break;
      if (i + lane < mine) sh->tile[b][lane] = tile_of(a, sh, first + (i + lane) * step);
      __syncwarp();
      if (lane == 0) arrive(&sh->tile_full[b]);
    }
  } else {
    // epilogue: lane = n, accumulator columns = k
    const int q = warp & 3, half = (warp >> 2) & 1;
    const uint32_t buf = smem_addr(sh->out[warp - 4]);
    int acc = 0;
    for (int i = 0; i < mine; i++) {
      int4 tile;
      if (!next_tile(sh, i, a.status, &tile)) break;
      const int parts = (tile.w + kPart * kDeep - 1) / (kPart * kDeep);
      const int n = (tile.y & 0xffff) * kSide + (int)rank * 128 + q * 32;
      const int k0 = (tile.y >> 16) * kSide + half * 128;
      const bool home = tile.x < a.E || a.shares > 1;
      const CUtensorMap *map = home ? &map_home : &map_slots;
      // the workspace's tensors are share by share
      const int z = a.shares > 1 ? tile.x % a.shares * (a.groups / a.shares) + tile.x / a.shares
                                 : home ? tile.x : tile.x - a.E;
      // gradients that are added to, on their way to L2 while the products run
      if (a.add && n < a.N && elect())
#pragma unroll
        for (int c = 0; c < 4; c++)
          if (k0 + c * 32 < a.Kd)
            asm volatile(
                "cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map),
                "r"(k0 + c * 32), "r"(n), "r"(z)
                : "memory");
      float sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; c++)
#pragma unroll
        for (int k = 0; k < 32; k++) sum[c][k] = 0.0f;
      bool ok = true;
      // the last part's columns go out as they come, so that stores are under
      // way while the next ones are read
      for (int p = 0; p < max(parts, 1); p++) {
        const bool some = parts > 0, end = p >= parts - 1;
        if (some && !(ok = wait(sh, &sh->acc_full[acc & 1], (acc >> 1) & 1, a.status))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + (acc & 1) * kSide + half * 128 + ((uint32_t)(q * 32) << 16);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          if (some) {
            uint32_t v[32];
            tmem_load(v, d + c * 32);
            tmem_wait(v);
#pragma unroll
            for (int k = 0; k < 32; k++) sum[c][k] += __uint_as_float(v[k]);
            if (c == 3) {
              asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
              __syncwarp();
              if (lane == 0) arrive_leader(&sh->acc_empty[acc & 1], to_leader);
              acc++;
            }
          }
          if (!end || n >= a.N || k0 + c * 32 >= a.Kd) continue;
          // the buffer's last store has read it
          if (elect()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; k++)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             buf + lane * 128 + ((k ^ (lane & 7)) * 16)),
                         "f"(sum[c][4 * k]), "f"(sum[c][4 * k + 1]), "f"(sum[c][4 * k + 2]),
                         "f"(sum[c][4 * k + 3])
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (elect()) tma_out(map, buf, k0 + c * 32, n, z, a.add);
        }
      }
      if (!ok) break;
    }
    if (elect()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  // both CTAs are done with each other's memory and with TMEM
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Adds up the shares of every gradient, in order.
__global__ void __launch_bounds__(256)
    join_kernel(const GradArgs a, const float4 *work, float4 *grad, float4 *slots, int add) {
  pdl_wait();
  pdl_launch_dependents();
  const int weights = a.groups / a.shares;
  const int64_t size = (int64_t)a.N * a.Kd / 4, whole = weights * size;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < whole;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int w = (int)(i / size);
    int start, rows;
    segment_of(a, w, &start, &rows);
    const bool home = w < a.E;
    if (rows == 0 && (add || !home)) continue;
    float4 *to = home ? grad + i : slots + (i - (int64_t)a.E * size);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int each = share_rows(rows, a.shares);
    for (int s = 0; s * each < rows; s++) {
      const float4 p = __ldcs(work + s * whole + i);
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    if (add) {
      const float4 o = *to;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *to = v;
  }
}

constexpr size_t kSmem = sizeof(Shared) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

// bf16 rows `pitch` bytes apart, in boxes of kDeep rows x 64 columns, or where
// the columns are whole blocks of 64 (the third dimension) x two of these.
bool rows_map(CUtensorMap *m, const void *p, int cols, int64_t rows, int64_t pitch) {
  const bool whole = cols % 64 == 0;
  const cuuint64_t dims[3] = {(cuuint64_t)(whole ? 64 : cols), (cuuint64_t)rows,
                              (cuuint64_t)(cols / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, 128};
  const cuuint32_t box[3] = {64, kDeep, 2}, one[3] = {1, 1, 1};
  return encoder() &&
         encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, whole ? 3 : 2, (void *)p, dims, strides,
                   box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Gradients [count, N, Kd] fp32 in boxes of 32 x 32.
bool grad_map(CUtensorMap *m, float *p, int64_t count, int N, int Kd) {
  const cuuint64_t dims[3] = {(cuuint64_t)Kd, (cuuint64_t)N, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)Kd * 4, (cuuint64_t)Kd * 4 * N};
  const cuuint32_t box[3] = {32, 32, 1}, one[3] = {1, 1, 1};
  return encoder() &&
         encoder()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int wgrad_clusters(int sms) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sms / 2 > 0 ? sms / 2 : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute((const void *)wgrad_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, (const void *)wgrad_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n < sms / 2 ? n : (sms / 2 > 0 ? sms / 2 : 1);
}

// Shares of a segment's rows: as many as the pairs of SMs can take at once beside
// each other, of 1024 rows or more if each rank's rows are spread evenly over its
// experts.  (Two experts of 256 x 512, 65536 rows each: 51 us in 19 shares, 69 in
// 38, 284 in one; eight of 512 x 512 with 8192 rows: 43 us in two, 48 in one; eight
// of 256 x 256 with 1024 rows: 16 in two, 13 in one.)
int wgrad_shares(const moonep_ctx *ctx, int N, int Kd) {
  const int64_t tiles = (int64_t)ctx->cfg.E * ((N + kSide - 1) / kSide) * ((Kd + kSide - 1) / kSide);
  const int64_t want = (int64_t)ctx->wgrad_clusters / tiles;
  const int64_t most = (int64_t)ctx->NvS / ctx->L / (2 * kPart * kDeep);
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n > 64 ? 64 : n);
}

int launch_wgrad(moonep_ctx *ctx, const int32_t *cu, const uint16_t *x, int64_t x_pitch,
                 const uint16_t *d, int64_t d_pitch, int N, int Kd, int add, float *grad,
                 float *slots, float *work, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  if (ctx->wgrad_clusters <= 0) return MOONEP_ERR_CUDA;
  const int64_t rows = (int64_t)c.R * ctx->NvS, extra = (int64_t)c.R * c.B;
  const int shares = wgrad_shares(ctx, N, Kd);
  CUtensorMap md, mx, mh, ms;
  if (!rows_map(&md, d, N, rows, d_pitch) || !rows_map(&mx, x, Kd, rows, x_pitch) ||
      !(shares > 1 ? grad_map(&mh, work, shares * (c.E + extra), N, Kd)
                   : grad_map(&mh, grad, c.E, N, Kd)))
    return MOONEP_ERR_CUDA;
  if (extra == 0 || shares > 1)
    ms = mh;  // no group reads it
  else if (!grad_map(&ms, slots, extra, N, Kd))
    return MOONEP_ERR_CUDA;
  GradArgs a{};
  a.cu = cu;
  a.E = c.E;
  a.B = c.B;
  a.L = ctx->L;
  a.EB = ctx->EB;
  a.NvS = ctx->NvS;
  a.N = N;
  a.Kd = Kd;
  a.nb = (N + kSide - 1) / kSide;
  a.kb = (Kd + kSide - 1) / kSide;
  a.shares = shares;
  a.groups = (int)(c.E + extra) * shares;
  a.per = (a.groups + kEntries - 1) / kEntries;
  a.add = add && shares == 1;
  a.whole_d = N % 64 == 0;
  a.whole_x = Kd % 64 == 0;
  a.status = ctx->d_status;
  cudaError_t e = launch_pdl(wgrad_kernel, dim3(2 * ctx->wgrad_clusters), dim3(kThreads), kSmem, st,
                             false, md, mx, mh, ms, a);
  if (e == cudaSuccess && shares > 1) {
    const int64_t need = ((c.E + extra) * N * Kd / 4 + 255) / 256, most = (int64_t)ctx->sms * 8;
    e = launch_pdl(join_kernel, dim3((unsigned)(need < most ? need : most)), dim3(256), 0, st,
                   false, a, (const float4 *)work, (float4 *)grad, (float4 *)slots, add);
  }
  return cuda_status(e);
}

}  // namespace moonep
