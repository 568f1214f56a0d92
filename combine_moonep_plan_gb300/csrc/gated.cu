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

// Through exp(-|g|), which cannot overflow; for g below -87 it is a subnormal,
// and zero from about -104 on.  The denominator is in [1, 2].
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

// Rows of rank blockIdx.y, WPR warps to a row, two units (eight columns) per
// lane at a time with their loads in flight together.
template <bool CKPT, int WPR>
__global__ void __launch_bounds__(kThreads) gated_kernel(GatedArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRows = kThreads / 32 / WPR, kLanes = WPR * 32;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int used = used_rows(a.cu, blockIdx.y, a.EB, a.NvS);
  for (int64_t r = (int64_t)blockIdx.x * kRows + sub; r < used; r += (int64_t)gridDim.x * kRows) {
    const int64_t row = (int64_t)blockIdx.y * a.NvS + r;
    const float w = a.w ? a.w[row] : 1.0f;
    for (int c0 = 0; c0 < a.F8; c0 += kLanes * 2) {
      uint4 gv[2] = {}, uv[2] = {};
#pragma unroll
      for (int b = 0; b < 2; b++) {
        const int c = c0 + b * kLanes + lane;
        if (c < a.F8) {
          gv[b] = ld_stream((const uint4 *)a.gate + row * a.F8 + c);
          uv[b] = ld_stream((const uint4 *)a.up + row * a.F8 + c);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; b++) {
        const int c = c0 + b * kLanes + lane;
        const bool on = c < a.F8;
        const int64_t u = row * a.F8 + c;
        float g[8], v[8];
        bf16x8(gv[b], g);
        bf16x8(uv[b], v);
        if (on) {
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
}

// Eight checkpointed values from their codes and scale byte.
__device__ __forceinline__ void read8(uint2 c, uint32_t scale, float f[8]) {
  const float s = mx_value(scale);
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 p = mx_e4m3x2(w[i >> 1] >> (16 * (i & 1)));
    f[2 * i] = p.x * s;
    f[2 * i + 1] = p.y * s;
  }
}

template <int WPR>
__global__ void __launch_bounds__(kThreads) gated_backward_kernel(GatedArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRows = kThreads / 32 / WPR, kLanes = WPR * 32;
  __shared__ float part[WPR];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int used = used_rows(a.cu, blockIdx.y, a.EB, a.NvS);
  for (int64_t r = (int64_t)blockIdx.x * kRows + sub; r < used; r += (int64_t)gridDim.x * kRows) {
    const int64_t row = (int64_t)blockIdx.y * a.NvS + r;
    const float w = a.w ? a.w[row] : 1.0f;
    float sum = 0.0f;
    for (int c0 = 0; c0 < a.F8; c0 += kLanes * 2) {
      uint4 dv[2];
      uint2 gv[2], uv[2];
      uint32_t gs[2], us[2];
#pragma unroll
      for (int b = 0; b < 2; b++) {
        const int c = c0 + b * kLanes + lane;
        if (c < a.F8) {
          const int64_t u = row * a.F8 + c;
          dv[b] = ld_stream((const uint4 *)a.d_act + u);
          gv[b] = ((const uint2 *)a.g8)[u];
          uv[b] = ((const uint2 *)a.u8)[u];
          gs[b] = a.gs[u >> 2];
          us[b] = a.us[u >> 2];
        }
      }
#pragma unroll
      for (int b = 0; b < 2; b++) {
        const int c = c0 + b * kLanes + lane;
        if (c >= a.F8) break;
        const int64_t u = row * a.F8 + c;
        float d[8], g[8], v[8], dg[8], du[8];
        bf16x8(dv[b], d);
        read8(gv[b], gs[b], g);
        read8(uv[b], us[b], v);
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
    }
    if (a.d_w) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (WPR > 1) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int i = 0; i < WPR; i++) sum += part[i];
      }
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

// A whole block to a row where one warp to a row would leave SMs without
// work; otherwise a warp.
bool few_rows(const moonep_ctx *ctx) {
  return (int64_t)ctx->cfg.R * ctx->NvS <= (int64_t)ctx->sms * 4;
}

// Blocks over a rank's rows, at most `per_sm` per SM over all ranks (0: one
// for every rows_per_block rows), and no more than num_sms SMs hold (`cap`, at
// least one per rank).  At 327168 x 2048 the forward pass took 604, 511 and
// 495 us with 8, 16 and no limit, the backward pass 706, 696 and 711.
dim3 grid_for(const moonep_ctx *ctx, int rows_per_block, int per_sm, int64_t cap) {
  const int R = ctx->cfg.R;
  int64_t blocks = ((int64_t)ctx->NvS + rows_per_block - 1) / rows_per_block;
  const int64_t most = ((int64_t)ctx->sms * per_sm + R - 1) / R;
  if (per_sm && blocks > most) blocks = most;
  if (blocks > cap / R) blocks = cap / R > 0 ? cap / R : 1;
  return dim3((unsigned)blocks, R);
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
  const bool few = few_rows(ctx);
  auto kern = few ? (g8 ? gated_kernel<true, 8> : gated_kernel<false, 8>)
                  : (g8 ? gated_kernel<true, 1> : gated_kernel<false, 1>);
  const dim3 grid = grid_for(ctx, few ? 1 : 8, 0, blocks_in_cap(ctx, kern, kThreads, 0));
  return cuda_status(launch_pdl(kern, grid, dim3(kThreads), 0, st, false, a));
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
  const bool few = few_rows(ctx);
  auto kern = few ? gated_backward_kernel<8> : gated_backward_kernel<1>;
  const dim3 grid = grid_for(ctx, few ? 1 : 8, 16, blocks_in_cap(ctx, kern, kThreads, 0));
  return cuda_status(launch_pdl(kern, grid, dim3(kThreads), 0, st, false, a));
}

}  // namespace moonep
