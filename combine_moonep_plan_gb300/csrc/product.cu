// The experts' grouped product: every segment's rows times its expert's
// weights, both microscaled 4-bit.
//
//   out[row, n] = sum_k A[row, k] * W[g, n, k]
// Group g is a weight row of the [E + R*B, N, Kd] tensor: home expert e holds
// segment e of rank e / (E/R), slot (j, b) is row E + j*B + b and segment E+b
// of rank j, so groups and segments that can hold rows pair up one to one.
#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kTileRows = 64, kTileCols = 64, kStep = 32;

struct ProductArgs {
  const uint8_t *a, *as;  // rows: [.., Kd/2] pitch lda, scales pitch lds
  const uint8_t *w, *ws;  // [G, N, Kd/2], [G, N, Kd/32]
  const int32_t *cu;      // [R, EB]
  void *out;              // [R*NvS, N]
  int64_t lda, lds;
  int R, E, B, L, EB, NvS, N, Kd;
  int32_t *status;
};

// Rows [first, last) of group g in the whole buffer; an offset outside the
// rank's window is reported and the segment treated as empty.
__device__ __forceinline__ bool segment(const ProductArgs &a, int g, int64_t *first, int *rows) {
  const int j = g < a.E ? g / a.L : (g - a.E) / a.B;
  const int x = g < a.E ? g : a.E + (g - a.E) % a.B;
  const int32_t *cu = a.cu + (int64_t)j * a.EB;
  const int lo = x ? cu[x - 1] : 0, hi = cu[x];
  const bool bad = lo < 0 || hi < lo || hi > a.NvS;
  *first = (int64_t)j * a.NvS + lo;
  *rows = bad ? 0 : hi - lo;
  return !bad;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One block per (64 columns, group): 64-row tiles, fp32 accumulation.
template <typename T>
__global__ void __launch_bounds__(256) product_kernel(ProductArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float sa[kStep][kTileRows + 4], sb[kStep][kTileCols + 4];
  const int g = blockIdx.y, n0 = blockIdx.x * kTileCols, tid = threadIdx.x;
  int64_t first;
  int rows;
  if (!segment(a, g, &first, &rows)) {
    if (blockIdx.x == 0 && tid == 0) set_status(a.status, MOONEP_ERR_PLAN);
    return;
  }
  const int tx = tid & 15, ty = tid >> 4;
  for (int m0 = 0; m0 < rows; m0 += kTileRows) {
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.Kd; k0 += kStep) {
      // one block of 32 values per row: four threads take eight values each
      const int r = tid >> 2, c = (tid & 3) * 8;
      const bool va = m0 + r < rows, vb = n0 + r < a.N;
      const int64_t ra = first + m0 + r, rb = (int64_t)g * a.N + n0 + r;
      const uint32_t pa = va ? *(const uint32_t *)(a.a + ra * a.lda + (k0 + c) / 2) : 0u;
      const uint32_t pb = vb ? *(const uint32_t *)(a.w + (rb * a.Kd + k0 + c) / 2) : 0u;
      const float fa = va ? mx_value(a.as[ra * a.lds + k0 / 32]) : 0.0f;
      const float fb = vb ? mx_value(a.ws[(rb * a.Kd + k0) / 32]) : 0.0f;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; i++) {
        sa[c + i][r] = mx_e2m1((pa >> (4 * i)) & 15u) * fa;
        sb[c + i][r] = mx_e2m1((pb >> (4 * i)) & 15u) * fb;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; k++) {
        const float4 x = *(const float4 *)&sa[k][ty * 4], y = *(const float4 *)&sb[k][tx * 4];
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int q = 0; q < 4; q++) acc[i][q] += xs[i] * ys[q];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int q = 0; q < 4; q++)
        if (m0 + ty * 4 + i < rows && n0 + tx * 4 + q < a.N)
          put((T *)a.out + (first + m0 + ty * 4 + i) * a.N + n0 + tx * 4 + q, acc[i][q]);
  }
}

}  // namespace

int launch_product(moonep_ctx *ctx, const int32_t *cu, const uint8_t *rows, int64_t lda,
                   const uint8_t *row_scales, int64_t lds, const uint8_t *w,
                   const uint8_t *w_scales, int N, int Kd, void *out, int fp32, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  ProductArgs a{rows, row_scales, w, w_scales, cu, out, lda, lds, c.R, c.E, c.B, ctx->L,
                ctx->EB, ctx->NvS, N, Kd, ctx->d_status};
  const dim3 grid((N + kTileCols - 1) / kTileCols, c.E + c.R * c.B);
  auto kern = fp32 ? product_kernel<float> : product_kernel<__nv_bfloat16>;
  return cuda_status(launch_pdl(kern, grid, dim3(256), 0, st, false, a));
}

}  // namespace moonep
