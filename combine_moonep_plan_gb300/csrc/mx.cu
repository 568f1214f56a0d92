// Microscaled 4-bit quantisation (E2M1 elements, one E8M0 scale per 32) and
// its read-back.  Both move memory: 2.53 bytes per bf16 value each way.
//
// Four lanes hold a block, eight values each: one or two 16-byte loads, the
// block's largest magnitude by two exchanges, one 4-byte store of eight
// codes, and one lane's scale byte.
#include "copy_common.cuh"
#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kThreads = 256;

// Units (eight values) per thread whose loads are in flight together.  65536
// x 7168 bf16 took 270, 198 and 189 us with 2, 4 and 8 to quantise, and 173 us
// with 4 to read back (8: 184); small tensors want blocks more than batches
// (1024 x 4096: 3.4 us with 4, 3.8 with 8).
constexpr int kBatch = 4, kLongBatch = 8;

struct MxArgs {
  const void *x;        // [rows, cols] bf16 or fp32
  uint8_t *packed;      // [rows, cols / 2]
  uint8_t *scales;      // [rows, cols / 32]
  const int32_t *cu;    // [R, EB] or null: every row
  int64_t units;        // all units (no cu), or of one rank's window
  int cols8, EB, NvS;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *x, int64_t u, uint4 v[1]) {
  v[0] = ld_stream((const uint4 *)x + u);
}
__device__ __forceinline__ void load8(const float *x, int64_t u, uint4 v[2]) {
  v[0] = ld_stream((const uint4 *)x + 2 * u);
  v[1] = ld_stream((const uint4 *)x + 2 * u + 1);
}
__device__ __forceinline__ void values8(const __nv_bfloat16 *, const uint4 v[1], float f[8]) {
  bf16x8(v[0], f);
}
__device__ __forceinline__ void values8(const float *, const uint4 v[2], float f[8]) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = __uint_as_float(w[i]);
}

// blockIdx.y: rank (0 without cu).  A rank's used rows are one span of memory
// from its window's start, walked without regard to rows.
template <typename T, int BATCH>
__global__ void __launch_bounds__(kThreads) quantize_kernel(MxArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int j = blockIdx.y;
  const int64_t n = a.cu ? (int64_t)used_rows(a.cu, j, a.EB, a.NvS) * a.cols8 : a.units;
  const int64_t first = j * a.units;
  const T *x = (const T *)a.x + first * 8;
  uint32_t *packed = (uint32_t *)a.packed + first;
  uint8_t *scales = a.scales + first / 4;
  // the four lanes of a block are inside or outside together (n is a multiple
  // of 4); lanes outside take part in the exchanges
  for (int64_t u0 = (int64_t)blockIdx.x * (kThreads * BATCH) + threadIdx.x;
       u0 - threadIdx.x < n; u0 += (int64_t)gridDim.x * (kThreads * BATCH)) {
    uint4 v[BATCH][sizeof(T) / 2] = {};
#pragma unroll
    for (int b = 0; b < BATCH; b++)
      if (u0 + b * kThreads < n) load8(x, u0 + b * kThreads, v[b]);
#pragma unroll
    for (int b = 0; b < BATCH; b++) {
      const int64_t u = u0 + b * kThreads;
      float f[8];
      values8(x, v[b], f);
      const uint32_t s = mx_scale<2>(mx_amax(f));
      if (u >= n) continue;
      const float inv = mx_inverse(s);
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] *= inv;
      packed[u] = s == 255u ? 0u : mx_pack_e2m1(f);
      if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)s;
    }
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *y, int64_t u, const float f[8]) {
  st_global((uint4 *)y + u, to_bf16x8(f));
}
__device__ __forceinline__ void store8(float *y, int64_t u, const float f[8]) {
  st_global_f4((float4 *)y + 2 * u, make_float4(f[0], f[1], f[2], f[3]));
  st_global_f4((float4 *)y + 2 * u + 1, make_float4(f[4], f[5], f[6], f[7]));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *packed,
                                                              const uint8_t *scales, T *y,
                                                              int64_t units) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t u0 = (int64_t)blockIdx.x * (kThreads * kBatch) + threadIdx.x; u0 < units;
       u0 += (int64_t)gridDim.x * (kThreads * kBatch)) {
    uint32_t w[kBatch] = {}, s[kBatch] = {};
#pragma unroll
    for (int b = 0; b < kBatch; b++)
      if (u0 + b * kThreads < units) {
        w[b] = __ldg((const uint32_t *)packed + u0 + b * kThreads);
        s[b] = __ldg(scales + ((u0 + b * kThreads) >> 2));
      }
#pragma unroll
    for (int b = 0; b < kBatch; b++) {
      if (u0 + b * kThreads >= units) break;
      const float v = mx_value(s[b]);
      float f[8];
      mx_e2m1x8(w[b], f);
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] *= v;
      store8(y, u0 + b * kThreads, f);
    }
  }
}

// One block for every `batch` units per thread, in each of `spans` equal
// spans (a capped grid that walks its span was 3 to 18 % slower); the loops
// serve tensors whose blocks would not fit in a grid, or in num_sms SMs (`cap`
// blocks, at least one per span).
dim3 grid_for(int64_t units, int spans, int batch, int64_t cap) {
  const int64_t need = (units + (int64_t)kThreads * batch - 1) / ((int64_t)kThreads * batch);
  const int64_t most = cap / spans > 0 ? cap / spans : 1;
  return dim3((unsigned)(need < most ? need : most), spans);
}

}  // namespace

int launch_quantize_mx(moonep_ctx *ctx, const void *x, int fp32, int64_t rows, int64_t cols,
                       const int32_t *cu, uint8_t *packed, uint8_t *scales, cudaStream_t st) {
  const int spans = cu ? ctx->cfg.R : 1;
  MxArgs a{x, packed, scales, cu, rows / spans * (cols / 8), (int)(cols / 8), ctx->EB, ctx->NvS};
  const bool lng = a.units * spans >= (int64_t)ctx->sms * 8 * kThreads * kLongBatch;
  auto kern = lng ? (fp32 ? quantize_kernel<float, kLongBatch>
                          : quantize_kernel<__nv_bfloat16, kLongBatch>)
                  : (fp32 ? quantize_kernel<float, kBatch> : quantize_kernel<__nv_bfloat16, kBatch>);
  const dim3 grid = grid_for(a.units, spans, lng ? kLongBatch : kBatch,
                             blocks_in_cap(ctx, kern, kThreads, 0));
  return cuda_status(launch_pdl(kern, grid, dim3(kThreads), 0, st, false, a));
}

int launch_dequantize_mx(moonep_ctx *ctx, const uint8_t *packed, const uint8_t *scales, int fp32,
                         int64_t rows, int64_t cols, void *y, cudaStream_t st) {
  const int64_t units = rows * (cols / 8);
  auto grid = [&](auto kern) {
    return grid_for(units, 1, kBatch, blocks_in_cap(ctx, kern, kThreads, 0));
  };
  if (fp32)
    return cuda_status(launch_pdl(dequantize_kernel<float>, grid(dequantize_kernel<float>),
                                  dim3(kThreads), 0, st, false, packed, scales, (float *)y, units));
  return cuda_status(launch_pdl(dequantize_kernel<__nv_bfloat16>,
                                grid(dequantize_kernel<__nv_bfloat16>), dim3(kThreads), 0, st,
                                false, packed, scales, (__nv_bfloat16 *)y, units));
}

}  // namespace moonep
