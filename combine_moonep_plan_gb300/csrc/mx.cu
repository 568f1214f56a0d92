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

struct MxArgs {
  const void *x;        // [rows, cols] bf16 or fp32
  uint8_t *packed;      // [rows, cols / 2]
  uint8_t *scales;      // [rows, cols / 32]
  const int32_t *cu;    // [R, EB] or null: every row
  int64_t units;        // rows * cols / 8
  int cols8, EB, NvS;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *x, int64_t u, float f[8]) {
  bf16x8(ld_stream((const uint4 *)x + u), f);
}
__device__ __forceinline__ void load8(const float *x, int64_t u, float f[8]) {
  const uint4 a = ld_stream((const uint4 *)x + 2 * u), b = ld_stream((const uint4 *)x + 2 * u + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = __uint_as_float(w[i]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(MxArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * kThreads;
  // the four lanes of a block enter and leave together: units is a multiple
  // of 4 and so is the step; lanes past the end take part in the exchanges
  for (int64_t u0 = (int64_t)blockIdx.x * kThreads; u0 < a.units; u0 += step) {
    const int64_t u = u0 + threadIdx.x;
    bool on = u < a.units;
    if (on && a.cu) {
      const int64_t row = u / a.cols8;
      const int j = (int)(row / a.NvS);
      on = row - (int64_t)j * a.NvS < used_rows(a.cu, j, a.EB, a.NvS);
    }
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) load8((const T *)a.x, u, f);
    const uint32_t s = mx_scale<2>(mx_amax(f));
    if (!on) continue;
    const float inv = mx_inverse(s);
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = s == 255u ? 0.0f : f[i] * inv;
    ((uint32_t *)a.packed)[u] = mx_pack_e2m1(f);
    if ((threadIdx.x & 3) == 0) a.scales[u >> 2] = (uint8_t)s;
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
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units;
       u += (int64_t)gridDim.x * kThreads) {
    const uint32_t w = ((const uint32_t *)packed)[u];
    const float s = mx_value(scales[u >> 2]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = mx_e2m1((w >> (4 * i)) & 15u) * s;
    store8(y, u, f);
  }
}

unsigned grid_for(const moonep_ctx *ctx, int64_t units) {
  const int64_t need = (units + kThreads - 1) / kThreads, cap = (int64_t)ctx->sms * 8;
  return (unsigned)(need < cap ? need : cap);
}

}  // namespace

int launch_quantize_mx(moonep_ctx *ctx, const void *x, int fp32, int64_t rows, int64_t cols,
                       const int32_t *cu, uint8_t *packed, uint8_t *scales, cudaStream_t st) {
  MxArgs a{x, packed, scales, cu, rows * (cols / 8), (int)(cols / 8), ctx->EB, ctx->NvS};
  auto kern = fp32 ? quantize_kernel<float> : quantize_kernel<__nv_bfloat16>;
  return cuda_status(
      launch_pdl(kern, dim3(grid_for(ctx, a.units)), dim3(kThreads), 0, st, false, a));
}

int launch_dequantize_mx(moonep_ctx *ctx, const uint8_t *packed, const uint8_t *scales, int fp32,
                         int64_t rows, int64_t cols, void *y, cudaStream_t st) {
  const int64_t units = rows * (cols / 8);
  const dim3 grid(grid_for(ctx, units));
  if (fp32)
    return cuda_status(launch_pdl(dequantize_kernel<float>, grid, dim3(kThreads), 0, st, false,
                                  packed, scales, (float *)y, units));
  return cuda_status(launch_pdl(dequantize_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st,
                                false, packed, scales, (__nv_bfloat16 *)y, units));
}

}  // namespace moonep
