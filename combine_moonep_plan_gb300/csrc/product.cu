// The experts' grouped product: every segment's rows times its expert's
// weights, both microscaled 4-bit, on the block-scaled tensor cores.
//
//   out[row, n] = sum_k A[row, k] W[g, n, k]
// Group g is a weight row of the [E + R*B, N, Kd] tensor: home expert e holds
// segment e of rank e / (E/R), slot (j, b) is row E + j*B + b and segment E+b
// of rank j, so groups and segments that can hold rows pair up one to one.
//
// The weights are the tensor cores' M side (256 of the N outputs per tile, a
// pair of SMs with 128 each) and the segment's rows the N side, which comes in
// steps of 16: segments are ragged and often short (a decode step has a few
// rows per expert), so the side with the fine step wastes the least.  A
// segment is cut into equal pieces of at most 192 rows.
//
// One persistent pair of CTAs (cluster of two) per pair of SMs; warps:
//   0      TMA: 256 values of k per stage, 128 weight rows and half the
//          piece's rows per CTA
//   1-6    scales: plain [rows, Kd/32] tensors (as prefetch and dispatch move
//          them) rearranged to the tensor cores' 128 x 4 blocks on the way to
//          shared memory; each lane loads 16 scales of four rows 32 apart and
//          so holds whole 16-byte lines of four such blocks.  Two sets of
//          three warps take turns: one set needed 600 cycles per stage, twice
//          the products' time
//   7      MMA, one thread of the pair's first CTA: scales to TMEM, then four
//          64-deep products per stage
//   8-15   epilogue: accumulator (lane = output column, TMEM column = row) to
//          global memory, two neighbouring columns per store; the two groups
//          of four warps take alternate 32 rows
//   16     schedule: the CTA's next 32 tiles at a time, one per lane, to shared
//          memory (every warp working its tiles out itself cost 4000 cycles
//          per tile)
// Accumulators are double-buffered in TMEM (2 x 192 columns); each of the five
// shared-memory stages has its own 24 columns of scales, so a stage's scales
// are only overwritten once its products are done (the stage's barrier).
// Every wait has a limit of one second, after which the kernel latches
// MOONEP_ERR_TIMEOUT, drains and returns; every warp reaches the cluster
// barrier before the CTAs leave, on every path.
//
// A wait by parity must not come a whole use of its barrier early, and nothing
// promises that the releases of two stages arrive in their order.  The load
// warp waits for every release and passes it on (`passed`); the scale warps,
// which skip the other set's stages, wait for that: arrivals of one thread in
// their own CTA are seen in order, a warp's waits are at most three stages apart
// and a stage is used again after five, so the one that it saw last implies the
// use before.  (Waiting for the releases themselves, every one of them, held a
// scale warp to three stages ahead: 1.43 ms for the largest case below.)
//
// Measured (the kernel alone): 128 experts with 9536 rows, N = 4096, Kd =
// 1536: 106 us, 6.5 TB/s, 0.96 of the copy rate, bound by the weights' bytes.
// 256 experts with 283520 rows, N = 2048, Kd = 7168: 1358 us, 6.13 PFLOP/s,
// the tensor pipe busy 67 % of the time (352 cycles a stage for 176 rows, some
// 520 needed); after a few runs in a row the power limit adds 3 to 5 %.
// More stages, longer stages, scales written to TMEM by the warps, a thread of
// its own for the scale copies, L2 prefetch, and clusters of two pairs sharing
// the rows took 1320 to 1630 us, and what gained in this shape lost in
// another.  Without its loads the kernel took 1228 us, without scales too
// 1059: the rest is the ring of barriers between the warps and what the loads
// add to it.
#include <cuda.h>

#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kThreads = 544;
constexpr int kStages = 5;
constexpr int kScaleSets = 2;             // sets of scale warps that take turns,
constexpr int kScaleWarps = 3;            // warps of a set,
constexpr int kChunkStages = 2;           // and stages of a turn (512 values of k)
constexpr int kTileBatch = 32;            // tiles that the schedule warp hands out at a time
// Arrivals: a stage is full with the leader's expect_tx and one set of scale
// warps of each CTA; an accumulator is free with the epilogue warps of both
// CTAs; a batch of tiles is read by a CTA's load, scale and epilogue warps, and
// by the leader's product warp.
constexpr int kFullArrivals = 1 + 2 * kScaleWarps;
constexpr int kAccReaders = 16;
constexpr int kTileReaders = 1 + kScaleSets * kScaleWarps + kAccReaders / 2;
constexpr int kMaxCols = 192;             // rows of a piece (MMA N)
constexpr int kTileN = 256;               // outputs per tile (MMA M of the pair)
constexpr int kStageK = 256;              // values of k per stage (128 bytes)
constexpr int kBoxRows = 32;              // rows per TMA box of the row side,
constexpr int kWideRows = kMaxCols / 2;   // or all of half a piece in one
constexpr int kABytes = 128 * 128;
constexpr int kBBytes = 96 * 128;         // half a piece
constexpr int kSfBytes = 2 * 512 + 4 * 512;  // two weight blocks, four row blocks
constexpr int kStageBytes = kABytes + kBBytes + kSfBytes;
constexpr int kSfCols = 24;               // TMEM columns of one stage's scales
constexpr int kSfBase = 2 * kMaxCols;
constexpr int kEntries = 1024;            // tile table entries
constexpr long long kLimitNs = 1000000000LL;
static_assert(kSfBase + kStages * kSfCols <= 512, "TMEM columns");
static_assert(kStageBytes % 1024 == 0, "operand tiles start on 1 KB");
static_assert(kChunkStages * (kScaleSets - 1) + 1 <= kStages,
              "a scale warp's waits lie at most one use of a stage apart");
static_assert(kThreads == 32 * (1 + kScaleSets * kScaleWarps + 1 + kAccReaders / 2 + 1), "warps");

struct __align__(1024) Shared {
  uint8_t stage[kStages][kStageBytes];
  int32_t last[kEntries];   // tiles up to and including the entry's groups
  int32_t start[kEntries];  // first row (rank-local) of the entry's one group
  int32_t rows[kEntries];
  int32_t wsum[8];
  int4 tile[2][32];  // the CTA's tiles: group, first output, first row, rows
  uint64_t full[kStages], empty[kStages], passed[kStages], acc_full[2], acc_empty[2];
  uint64_t tile_full[2], tile_empty[2];
  uint32_t tmem;
  int32_t dead;
};

struct ProductArgs {
  const uint8_t *as, *ws;  // scales: rows (pitch lds), weights [G, N, Kd/32]
  const int32_t *cu;       // [R, EB]
  void *out;               // [R*NvS, N]
  int64_t lds;
  int R, E, B, L, EB, NvS, N, Kd;
  int groups, per;  // groups, groups per table entry
  int as16, ws16;   // scale rows are whole aligned 16-byte vectors
  int32_t *status;
};

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
// Operand descriptors: rows of 128 bytes, 128-byte swizzle, eight-row groups
// 1 KB apart; scale blocks of 32 lines of 16 bytes, unswizzled, eight-line
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void scales_to_tmem(uint32_t col, uint32_t addr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(col), "l"(scale_desc(addr))
               : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t sfa, uint32_t sfb, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
      : "memory");
}

// Rows [start, start + rows) of group g in its rank's window; offsets outside
// the window are reported and the segment treated as empty.
__device__ __forceinline__ bool segment(const ProductArgs &a, int g, int *start, int *rows) {
  const int j = g < a.E ? g / a.L : (g - a.E) / a.B;
  const int x = g < a.E ? g : a.E + (g - a.E) % a.B;
  const int32_t *cu = a.cu + (int64_t)j * a.EB;
  const int lo = x ? cu[x - 1] : 0, hi = cu[x];
  const bool bad = lo < 0 || hi < lo || hi > a.NvS;
  *start = bad ? 0 : lo;
  *rows = bad ? 0 : hi - lo;
  return !bad;
}

__device__ __forceinline__ int pieces(int rows) { return (rows + kMaxCols - 1) / kMaxCols; }

// Tile t: the piece of a segment and 256 outputs, outputs fastest.
__device__ int4 tile_of(const ProductArgs &a, const Shared *sh, int t) {
  const int nb = (a.N + kTileN - 1) / kTileN;
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
      const int n = pieces(rows) * nb;
      if (rest < n) break;
      rest -= n;
    }
  const int p = pieces(rows), m = rest / nb;
  const int each = ((rows + p - 1) / p + 15) & ~15;
  const int j = g < a.E ? g / a.L : (g - a.E) / a.B;
  return make_int4(g, (rest - m * nb) * kTileN, j * a.NvS + start + m * each,
                   min(each, rows - m * each));
}

// The table of tiles; every thread of the CTA takes part.  Returns the count.
__device__ __noinline__ int build_table(const ProductArgs &a, Shared *sh) {
  const int nb = (a.N + kTileN - 1) / kTileN;
  const int entries = (a.groups + a.per - 1) / a.per;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kEntries; i += kThreads) {
    int n = 0, start = 0, rows = 0;
    if (i < entries)
      for (int g = i * a.per; g < min(a.groups, (i + 1) * a.per); g++) {
        if (!segment(a, g, &start, &rows) && blockIdx.x == 0)
          set_status(a.status, MOONEP_ERR_PLAN);
        n += pieces(rows) * nb;
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

// Sixteen scale bytes at p, the first `need` of them wanted and 1.0 in place of
// the others, from the aligned words around them; bytes outside [base, end)
// are never touched.  Out of line: inlined for every row of every scale warp
// it made the kernel 150 KB of code, which no instruction cache holds.
__device__ __noinline__ uint4 load_bytes(const uint8_t *base, const uint8_t *end, const uint8_t *p,
                                         int need) {
  const uint32_t shift = (uint32_t)((uintptr_t)p & 3) * 8;
  const uint8_t *w0 = p - ((uintptr_t)p & 3);
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; i++) {
    const uint8_t *q = w0 + 4 * i;
    w[i] = 0;
    if (q < p + need && q >= base && q + 4 <= end) w[i] = __ldg((const uint32_t *)q);
  }
  if (w0 < base || w0 + 20 > end) {
    // the tensor's first or last word: what of it lies inside
    for (int i = 0; i < 20; i++) {
      const uint8_t *q = w0 + i, *v = w0 + (i & ~3);
      if (q >= base && q < end && !(v >= base && v + 4 <= end)) {
        const uint32_t x = (uint32_t)__ldg(q) << (8 * (i & 3));
#pragma unroll
        for (int j = 0; j < 5; j++)
          if (j == i >> 2) w[j] |= x;
      }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int have = need - 4 * i;
    const uint32_t keep = have >= 4 ? 0xffffffffu : have <= 0 ? 0u : (1u << (8 * have)) - 1;
    o[i] = (__funnelshift_r(w[i], w[i + 1], shift) & keep) | (0x7f7f7f7fu & ~keep);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sixteen scales of one row from column c on, 1.0 past the row's end or for a
// row that is not there.  `vec`: rows of whole aligned vectors.
__device__ __forceinline__ uint4 load_scales(const uint8_t *base, int64_t total, int64_t row,
                                             int64_t pitch, int c, int n, bool vec, bool there) {
  const uint32_t one = 0x7f7f7f7fu;
  if (!there || c >= n) return make_uint4(one, one, one, one);
  const uint8_t *p = base + row * pitch + c;
  if (vec) return __ldg((const uint4 *)p);
  return load_bytes(base, base + total, p, min(16, n - c));
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Two rows of one output column (this lane's) and the neighbouring lane's same
// rows become both columns of one row, the even lane's first row or the odd
// lane's second.
__device__ __forceinline__ void store_pair(float *p, uint32_t lo, uint32_t hi, bool odd, uint32_t) {
  const uint32_t mine = odd ? hi : lo, got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
  if (p) *(uint2 *)p = odd ? make_uint2(got, mine) : make_uint2(mine, got);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, uint32_t lo, uint32_t hi, bool,
                                           uint32_t pick) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
      : "=r"(w)
      : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  const uint32_t got = __shfl_xor_sync(0xffffffffu, w, 1);
  if (p) *(uint32_t *)p = __byte_perm(w, got, pick);
}

// The i-th tile of this CTA, for a whole warp that reads them in order.
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

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_wide, const ProductArgs a) {
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
    for (int s = 0; s < kStages; s++) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&sh->full[s])),
                   "r"(kFullArrivals));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&sh->empty[s])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&sh->passed[s])));
    }
    for (int b = 0; b < 2; b++) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&sh->tile_full[b])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&sh->tile_empty[b])),
                   "r"(kTileReaders + (rank == 0)));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&sh->acc_full[b])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&sh->acc_empty[b])),
                   "r"(kAccReaders));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 7) {
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
  const int stages = (a.Kd + kStageK - 1) / kStageK;  // per tile
  const int mine = tiles > first ? (tiles - first + step - 1) / step : 0;  // tiles of this pair

  if (warp == 0) {
    uint32_t s = 0, phase = 0, pending = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; i++) {
      int4 tile;
      if (!(ok = next_tile(sh, i, a.status, &tile))) break;
      const int half = ((tile.w + 15) & ~15) >> 1;
      const bool wide = half > 2 * kBoxRows;
      const int boxes = (half + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = 2u * (kABytes + (wide ? kWideRows : boxes * kBoxRows) * 128);
      const int wrow = tile.x * a.N + tile.y + (int)rank * 128;
      const int arow = tile.z + (int)rank * half;
      for (int k = 0; k < stages; k++) {
        if (!(ok = wait(sh, &sh->empty[s], phase ^ 1, a.status))) break;
        if (lane == 0) arrive(&sh->passed[s]);
        const uint32_t base = smem_addr(sh->stage[s]);
        const uint32_t full = smem_addr(&sh->full[s]), bar = full + to_leader;
        if (elect()) {
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                         "r"(bytes)
                         : "memory");
          tma_load(base, &map_w, k * 128, wrow, bar);
          if (wide) {
            tma_load(base + kABytes, &map_wide, k * 128, arow, bar);
          } else {
            tma_load(base + kABytes, &map_a, k * 128, arow, bar);
            if (boxes > 1)
              tma_load(base + kABytes + kBoxRows * 128, &map_a, k * 128, arow + kBoxRows, bar);
          }
        }
        pending |= 1u << s;
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
    if (!ok && rank == 0)
      for (int q = 0; q < kStages; q++) {
        const long long t0 = now_ns();
        const uint32_t ph = (uint32_t)q < s ? phase : phase ^ 1;
        if (pending & (1u << q))
          while (!try_wait(smem_addr(&sh->full[q]), ph) && now_ns() - t0 < kLimitNs / 4) {
          }
      }
  } else if (warp < 7) {
    // role 0: the CTA's 128 weight rows; 1, 2: the piece's rows 0-127, 128-191.
    // A warp takes every second chunk (512 values of k, two stages) of the
    // CTA's sequence of tiles, two of its chunks' loads in flight.
    const int role = (warp - 1) % kScaleWarps, turn = (warp - 1) / kScaleWarps;
    const int nsc = a.Kd / 32, chunks = (a.Kd + 511) / 512;
    const bool vec = role ? a.as16 : a.ws16;
    const uint8_t *base = role ? a.as : a.ws;
    const int64_t pitch = role ? a.lds : nsc;
    const int64_t total = role ? ((int64_t)a.R * a.NvS - 1) * a.lds + nsc
                               : (int64_t)a.groups * a.N * nsc;
    const uint32_t at = kABytes + kBBytes + (role ? 1024 + (role - 1) * 512 : 0) + lane * 16;
    uint32_t s = 0, phase = 0;
    bool ok = true;
    int li = 0, lc = turn, have = -1;  // tile and chunk to load next; tile in `tile`
    int4 tile = make_int4(0, 0, 0, 0);
    auto load = [&](uint4 v[4]) {
      for (; lc >= chunks; lc -= chunks) li++;
      if (!ok) return;
      for (; have < li && have < mine - 1; have++)
        if (!(ok = next_tile(sh, have + 1, a.status, &tile))) return;
      if (li >= mine) return;
      const int lim = role ? tile.w - (role - 1) * 128 : a.N - tile.y - (int)rank * 128;
      const int64_t row0 = role ? (int64_t)tile.z + (role - 1) * 128
                                : (int64_t)tile.x * a.N + tile.y + rank * 128;
#pragma unroll
      for (int i = 0; i < 4; i++)
        v[i] = load_scales(base, total, row0 + lane + 32 * i, pitch, lc * 16, nsc, vec,
                           lane + 32 * i < lim);
      lc += 2;
    };
    // moves the stage on by n, at most kStages
    auto skip = [&](int n) {
      s += n;
      if (s >= kStages) {
        s -= kStages;
        phase ^= 1;
      }
    };
    // writes a chunk's scales into its one or two stages
    auto fill = [&](const uint4 v[4], int c) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (c * 2 + h >= stages) break;
        if (!wait(sh, &sh->passed[s], phase, a.status)) return false;
        const uint32_t p = smem_addr(sh->stage[s]) + at;
#pragma unroll
        for (int i = 0; i < 2; i++)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           p + i * (role ? 1024 : 512)),
                       "r"(word(v[0], 2 * h + i)), "r"(word(v[1], 2 * h + i)),
                       "r"(word(v[2], 2 * h + i)), "r"(word(v[3], 2 * h + i))
                       : "memory");
        // the tensor cores read these lines through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_leader(&sh->full[s], to_leader);
        skip(1);
      }
      return true;
    };
    uint4 buf[2][4];
    load(buf[0]);
    load(buf[1]);
    int t = 0, c = 0;  // tile and chunk to fill next
    auto move = [&] {
      if (++c == chunks) {
        c = 0;
        t++;
      }
    };
    // past the other set's chunk
    auto pass = [&] {
      skip(min(2, stages - 2 * c));
      move();
    };
    if (turn) pass();
    while (t < mine && ok) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if (t >= mine || !ok) break;
        if (!(ok = fill(buf[i], c))) break;
        load(buf[i]);
        move();
        if (t < mine) pass();
      }
    }
  } else if (warp == 7) {
    if (rank == 0) {
      uint32_t s = 0, phase = 0;
      int it = 0;
      bool ok = true;
      const uint32_t stage0 = smem_addr(sh->stage[0]);
      for (; it < mine && ok; it++) {
        int4 tile;
        if (!(ok = next_tile(sh, it, a.status, &tile))) break;
        const int cols = (tile.w + 15) & ~15;
        const uint32_t d = tmem + (it & 1) * kMaxCols;
        if (!(ok = wait(sh, &sh->acc_empty[it & 1], ((it >> 1) & 1) ^ 1, a.status))) break;
        // E2M1 both sides, E8M0 scales, M = 256, N = cols
        const uint32_t idesc = (1u << 7) | (1u << 10) | (1u << 23) | ((uint32_t)(cols >> 3) << 17) |
                               (16u << 24);
        const bool wide = cols > 128;
        for (int k = 0; k < stages; k++) {
          if (!(ok = wait(sh, &sh->full[s], phase, a.status))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t base = stage0 + s * kStageBytes;
          const uint32_t sf = base + kABytes + kBBytes;
          const uint32_t ca = tmem + kSfBase + s * kSfCols, cb = ca + 8;
          const int deep = (a.Kd - k * kStageK + 63) >> 6;
          const uint64_t da = operand_desc(base), db = operand_desc(base + kABytes);
          if (elect()) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
              scales_to_tmem(ca + i * 4, sf + i * 512);
              scales_to_tmem(cb + i * 8, sf + 1024 + i * 1024);
              if (wide) scales_to_tmem(cb + i * 8 + 4, sf + 1024 + i * 1024 + 512);
            }
#pragma unroll
            for (int q = 0; q < 4; q++)
              if (q < deep)
                mma(d, da + 2 * q, db + 2 * q,
                    idesc | ((uint32_t)(q & 1) << 5) | ((uint32_t)(q & 1) << 30),
                    ca + (q >> 1) * 4, cb + (q >> 1) * 8, k + q > 0);
            commit(&sh->empty[s]);
            if (k == stages - 1) commit(&sh->acc_full[it & 1]);
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp < 16) {
    // epilogue: lane = output n, accumulator columns = rows
    const int q = warp & 3, group = (warp >> 2) & 1;
    const bool odd = lane & 1;
    // bytes of a row's two columns in (own two rows, neighbour's two rows)
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    for (int it = 0; it < mine; it++) {
      int4 tile;
      if (!next_tile(sh, it, a.status, &tile)) break;
      if (!wait(sh, &sh->acc_full[it & 1], (it >> 1) & 1, a.status)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + (it & 1) * kMaxCols + ((uint32_t)(q * 32) << 16);
      const int n = tile.y + (int)rank * 128 + q * 32 + (lane & ~1);
      const int rows = n < a.N ? tile.w - odd : 0;
      T *out = (T *)a.out + ((int64_t)tile.z + odd) * a.N + n;
      // columns past the piece's rows hold an earlier piece's: read, not stored
      auto store = [&](const uint32_t v[32], int c) {
        T *p = out + (int64_t)c * a.N;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          store_pair(c + i < rows ? p : (T *)nullptr, v[i], v[i + 1], odd, pick);
          p += 2 * a.N;
        }
      };
      for (int c = group * 32; c < tile.w; c += 64) {
        uint32_t v[32];
        tmem_load(v, d + c);
        tmem_wait(v);
        store(v, c);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_leader(&sh->acc_empty[it & 1], to_leader);
    }
  } else {
    // 32 tiles at a time, two such batches
    for (int i = 0; i < mine; i += 32) {
      const int b = (i >> 5) & 1;
      if (!wait(sh, &sh->tile_empty[b], ((i >> 6) & 1) ^ 1, a.status)) break;
      if (i + lane < mine) sh->tile[b][lane] = tile_of(a, sh, first + (i + lane) * step);
      __syncwarp();
      if (lane == 0) arrive(&sh->tile_full[b]);
    }
  }
  __syncwarp();
  // both CTAs are done with each other's memory and with TMEM
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 7)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// A product over no terms: zeros in every segment's rows.
template <typename T>
__global__ void __launch_bounds__(256) zero_rows_kernel(const int32_t *cu, T *out, int R, int EB,
                                                        int NvS, int N) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < (int64_t)R * NvS; row += gridDim.x) {
    const int j = (int)(row / NvS);
    if (row - (int64_t)j * NvS >= used_rows(cu, j, EB, NvS)) continue;
    for (int n = threadIdx.x; n < N; n += blockDim.x) out[row * N + n] = T(0.0f);
  }
}

constexpr size_t kSmem = sizeof(Shared) + 1024;

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeFn encoder() {
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

// Rows of `bytes` packed bytes, `pitch` apart, in boxes of `box` rows x 128
// bytes.
bool make_map(CUtensorMap *m, const void *p, int64_t bytes, int64_t rows, int64_t pitch, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, one[2] = {1, 1};
  return encoder() &&
         encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)p, dims, strides, boxes, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int product_clusters(int sms) {
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
  for (auto fn : {(const void *)product_kernel<float>, (const void *)product_kernel<__nv_bfloat16>})
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  return n < sms / 2 ? n : (sms / 2 > 0 ? sms / 2 : 1);
}

int launch_product(moonep_ctx *ctx, const int32_t *cu, const uint8_t *rows, int64_t lda,
                   const uint8_t *row_scales, int64_t lds, const uint8_t *w,
                   const uint8_t *w_scales, int N, int Kd, void *out, int fp32, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  if (Kd == 0) {
    if (fp32)
      return cuda_status(launch_pdl(zero_rows_kernel<float>, dim3(ctx->sms * 4), dim3(256), 0, st,
                                    false, cu, (float *)out, c.R, ctx->EB, ctx->NvS, N));
    return cuda_status(launch_pdl(zero_rows_kernel<__nv_bfloat16>, dim3(ctx->sms * 4), dim3(256),
                                  0, st, false, cu, (__nv_bfloat16 *)out, c.R, ctx->EB, ctx->NvS,
                                  N));
  }
  if (ctx->product_clusters <= 0) return MOONEP_ERR_CUDA;
  const int64_t groups = (int64_t)c.E + (int64_t)c.R * c.B;
  CUtensorMap mw, ma, mwide;
  if (!make_map(&mw, w, Kd / 2, groups * N, Kd / 2, 128) ||
      !make_map(&ma, rows, Kd / 2, (int64_t)c.R * ctx->NvS, lda, kBoxRows) ||
      !make_map(&mwide, rows, Kd / 2, (int64_t)c.R * ctx->NvS, lda, kWideRows))
    return MOONEP_ERR_CUDA;
  ProductArgs a{};
  a.as = row_scales;
  a.ws = w_scales;
  a.cu = cu;
  a.out = out;
  a.lds = lds;
  a.R = c.R;
  a.E = c.E;
  a.B = c.B;
  a.L = ctx->L;
  a.EB = ctx->EB;
  a.NvS = ctx->NvS;
  a.N = N;
  a.Kd = Kd;
  a.groups = (int)groups;
  a.per = (int)((groups + kEntries - 1) / kEntries);
  a.as16 = Kd % 512 == 0 && lds % 16 == 0 && aligned16(row_scales);
  a.ws16 = Kd % 512 == 0 && aligned16(w_scales);
  a.status = ctx->d_status;
  auto kern = fp32 ? product_kernel<float> : product_kernel<__nv_bfloat16>;
  return cuda_status(launch_pdl(kern, dim3(2 * ctx->product_clusters), dim3(kThreads), kSmem, st,
                                false, mw, ma, mwide, a));
}

}  // namespace moonep
