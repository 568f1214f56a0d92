// The experts' gated activation over the dispatched rows, times the route
// weight (combine sums unweighted), with an 8-bit checkpoint for its backward
// pass.
//
//   s = 1 / (1 + exp(-g)),  h = g s u,  a = w h
// The checkpoint holds g and u as E4M3 with one E8M0 scale per 32 columns
// (2.06 bytes per column instead of 4).  The backward pass takes the
// formula's gradient at the values that the checkpoint stands for:
//   d_up = w d g s,   d_gate = w d u s (1 + g (1 - s)),   d_w = sum d h
// Sums and products are fp32; each output is rounded to bf16 once.
// Memory-bound: 6 bytes per value forward (8.06 with a checkpoint), 8.06
// backward.  Rows after a rank's last segment are neither read nor written.
#include "copy_common.cuh"
#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kThreads = 256;

struct GatedArgs {
  const uint16_t *gate, *up, *d_act;  // [R*NvS, F] bf16
  const float *w;                     // [R*NvS] or null
  uint16_t *act;                      // [R*NvS, F] bf16
  uint8_t *g8, *u8;                   // [R*NvS, F] E4M3
  uint8_t *gs, *us;                   // [R*NvS, F/32] E8M0
  uint16_t *d_gate, *d_up;            // [R*NvS, F] bf16
  float *d_w;                         // [R*NvS] or null
  const int32_t *cu;                  // [R, EB]
  int R, EB, NvS, F8;
};

// Through exp(-|g|), which cannot overflow: below -88 the result is a small
// number, not zero.  The denominator is in [1, 2].
__device__ __forceinline__ float sigmoid(float g) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g < 0.0f ? e : 1.0f, 1.0f + e);
}

// Eight values to E4M3 codes at their block's scale; lane 0 of the block's
// four writes the scale byte.
__device__ __forceinline__ void checkpoint8(const float f[8], uint8_t *codes, uint8_t *scales,
                                            int64_t u, bool on) {
  const uint32_t s = mx_scale<8>(mx_amax(f));
  if (!on) return;
  const float inv = mx_inverse(s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i++) q[i] = s == 255u ? 0.0f : f[i] * inv;
  ((uint2 *)codes)[u] = make_uint2(mx_pack_e4m3(q[0], q[1], q[2], q[3]),
                                   mx_pack_e4m3(q[4], q[5], q[6], q[7]));
  if ((u & 3) == 0) scales[u >> 2] = (uint8_t)s;
}

// One warp per row.
template <bool CKPT>
__global__ void __launch_bounds__(kThreads) gated_kernel(GatedArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.R * a.NvS;
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
       row += (int64_t)gridDim.x * (kThreads / 32)) {
    const int j = (int)(row / a.NvS);
    if (row - (int64_t)j * a.NvS >= used_rows(a.cu, j, a.EB, a.NvS)) continue;
    const float w = a.w ? a.w[row] : 1.0f;
    for (int c0 = 0; c0 < a.F8; c0 += 32) {
      const int c = c0 + lane;
      const bool on = c < a.F8;
      const int64_t u = row * a.F8 + c;
      float g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (on) {
        bf16x8(ld_stream((const uint4 *)a.gate + u), g);
        bf16x8(ld_stream((const uint4 *)a.up + u), v);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = w * (g[i] * sigmoid(g[i]) * v[i]);
        st_global((uint4 *)a.act + u, to_bf16x8(o));
      }
      if (CKPT) {
        checkpoint8(g, a.g8, a.gs, u, on);
        checkpoint8(v, a.u8, a.us, u, on);
      }
    }
  }
}

__device__ __forceinline__ void read8(const uint8_t *codes, const uint8_t *scales, int64_t u,
                                      float f[8]) {
  const uint2 c = ((const uint2 *)codes)[u];
  const float s = mx_value(scales[u >> 2]);
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 p = mx_e4m3x2(w[i >> 1] >> (16 * (i & 1)));
    f[2 * i] = p.x * s;
    f[2 * i + 1] = p.y * s;
  }
}

__global__ void __launch_bounds__(kThreads) gated_backward_kernel(GatedArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.R * a.NvS;
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
       row += (int64_t)gridDim.x * (kThreads / 32)) {
    const int j = (int)(row / a.NvS);
    if (row - (int64_t)j * a.NvS >= used_rows(a.cu, j, a.EB, a.NvS)) continue;
    const float w = a.w ? a.w[row] : 1.0f;
    float sum = 0.0f;
    for (int c = lane; c < a.F8; c += 32) {
      const int64_t u = row * a.F8 + c;
      float d[8], g[8], v[8], dg[8], du[8];
      bf16x8(ld_stream((const uint4 *)a.d_act + u), d);
      read8(a.g8, a.gs, u, g);
      read8(a.u8, a.us, u, v);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float s = sigmoid(g[i]), gsd = d[i] * (g[i] * s);
        sum += gsd * v[i];
        du[i] = w * gsd;
        dg[i] = w * (d[i] * v[i] * (s * (1.0f + g[i] * (1.0f - s))));
      }
      st_global((uint4 *)a.d_gate + u, to_bf16x8(dg));
      st_global((uint4 *)a.d_up + u, to_bf16x8(du));
    }
    if (a.d_w) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) a.d_w[row] = sum;
    }
  }
}

GatedArgs args_of(const moonep_ctx *ctx, const int32_t *cu, int F) {
  GatedArgs a{};
  a.cu = cu;
  a.R = ctx->cfg.R;
  a.EB = ctx->EB;
  a.NvS = ctx->NvS;
  a.F8 = F / 8;
  return a;
}

dim3 grid_for(const moonep_ctx *ctx) {
  const int64_t need = ((int64_t)ctx->cfg.R * ctx->NvS + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = (int64_t)ctx->sms * 8;
  return dim3((unsigned)(need < cap ? need : cap));
}

}  // namespace

int launch_gated(moonep_ctx *ctx, const int32_t *cu, const uint16_t *gate, const uint16_t *up,
                 const float *w, int F, uint16_t *act, uint8_t *g8, uint8_t *u8, uint8_t *gs,
                 uint8_t *us, cudaStream_t st) {
  GatedArgs a = args_of(ctx, cu, F);
  a.gate = gate;
  a.up = up;
  a.w = w;
  a.act = act;
  a.g8 = g8;
  a.u8 = u8;
  a.gs = gs;
  a.us = us;
  auto kern = g8 ? gated_kernel<true> : gated_kernel<false>;
  return cuda_status(launch_pdl(kern, grid_for(ctx), dim3(kThreads), 0, st, false, a));
}

int launch_gated_backward(moonep_ctx *ctx, const int32_t *cu, const uint8_t *g8, const uint8_t *u8,
                          const uint8_t *gs, const uint8_t *us, const uint16_t *d_act,
                          const float *w, int F, uint16_t *d_gate, uint16_t *d_up, float *d_w,
                          cudaStream_t st) {
  GatedArgs a = args_of(ctx, cu, F);
  a.g8 = (uint8_t *)g8;
  a.u8 = (uint8_t *)u8;
  a.gs = (uint8_t *)gs;
  a.us = (uint8_t *)us;
  a.d_act = d_act;
  a.w = w;
  a.d_gate = d_gate;
  a.d_up = d_up;
  a.d_w = d_w;
  return cuda_status(
      launch_pdl(gated_backward_kernel, grid_for(ctx), dim3(kThreads), 0, st, false, a));
}

}  // namespace moonep
