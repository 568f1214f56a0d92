// The router: top-K picks, normalised route weights, per-expert counts and
// the balance loss, with the gradient of the logits.
//
// Row of logits z[E] of a valid token, scoring:
//   softmax  s_e = exp(z_e - max z);   sigmoid  s_e = 1 / (1 + exp(-z_e))
//   p_e = s_e / sum_j s_j     picks = the K largest z (equal: lowest index)
//   w_k = p_k / sum_picks p
// Balance loss, c[r, e] the picks of expert e among rank r's n_r valid tokens,
// P[r, e] = sum over them of p_e:
//   rank scope    L = a/R' sum_r sum_e (E c[r,e] / (K n_r)) (P[r,e] / n_r)
//                 (R' = ranks that hold a token)
//   global scope  L = a sum_e (E sum_r c[r,e] / (K T)) (sum_r P[r,e] / T)
// Both are sum_{r,e} coef[r,e] P[r,e] with coef constant under the gradient
// (counts have none), so the backward pass needs coef alone:
//   g_e  = dL p_e (coef_e - sum_j p_j coef_j)  + [e picked] w_e (dw_e - sum_k w_k dw_k)
//   dz_e = g_e (softmax),  g_e (1 - s_e) (sigmoid)
// A row whose scores sum to zero (every logit -inf) has p = w = 0 and no
// gradient; its picks are the lowest indices.  A NaN logit ranks first and
// makes its row's weights NaN; the ids stay in [0, E).
#include <cuda_bf16.h>

#include "moonep_internal.cuh"

namespace moonep {
namespace {

constexpr int kWarps = 8;

struct RouteArgs {
  const void *logits;  // [R, S, E] fp32 or bf16
  int32_t *topk;       // [R, S, K]
  float *w;            // [R, S, K]
  float *part_p;       // [R, bpr, E] sums of p of one block's tokens, or null
  int32_t *part_c;     // [R, bpr, E] picks of one block's tokens
  int R, S, E, K, bpr, sigmoid;
  int32_t ntok[kMaxRanks];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Order-preserving bits: a larger logit has a larger key, -0 equals +0, NaN
// is largest; 0 is below every logit.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Score of one logit; m is the row's maximum (softmax).
__device__ __forceinline__ float score(float z, float m, bool sigmoid) {
  if (sigmoid) return 1.0f / (1.0f + expf(-z));
  return m == -INFINITY ? 0.0f : expf(z - m);
}

// One warp per token, any E: the row in shared memory.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float sh[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *row = sh + (size_t)warp * a.E;                       // this token's logits
  float *acc = sh + (size_t)(warps + warp) * a.E;             // this warp's sums of p
  int32_t *cnt = (int32_t *)(sh + (size_t)2 * warps * a.E);   // this block's picks
  const int r = blockIdx.y;
  const int n = a.ntok[r];
  for (int e = lane; e < a.E; e += 32) acc[e] = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  for (int s = blockIdx.x * warps + warp; s < a.S; s += gridDim.x * warps) {
    const int64_t t = (int64_t)r * a.S + s;
    if (s >= n) {
      if (lane < a.K) {
        a.topk[t * a.K + lane] = 0;
        a.w[t * a.K + lane] = 0.0f;
      }
      continue;
    }
    const T *z = (const T *)a.logits + t * a.E;
    for (int e = lane; e < a.E; e += 32) row[e] = to_f(z[e]);
    __syncwarp();
    uint32_t taken = 0;  // keys at or above (taken, at) in the order are gone
    int at = -1, my = 0;
    float m = 0.0f, zk = 0.0f;
    for (int k = 0; k < a.K; k++) {
      uint32_t best = 0;
      int bi = 0x7fffffff;
      for (int e = lane; e < a.E; e += 32) {
        const uint32_t q = order_key(row[e]);
        const bool gone = k && (q > taken || (q == taken && e <= at));
        if (!gone && q > best) {
          best = q;
          bi = e;
        }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      at = (int)__reduce_min_sync(0xffffffffu, best == top ? (unsigned)bi : 0x7fffffffu);
      taken = top;
      if (k == 0) m = row[at];
      if (lane == k) {
        my = at;
        zk = row[at];
      }
      if (lane == 0) atomicAdd(&cnt[at], 1);
    }
    float sk = lane < a.K ? score(zk, m, a.sigmoid) : 0.0f;
    const float Zk = warp_sum(sk);
    if (lane < a.K) {
      a.topk[t * a.K + lane] = my;
      a.w[t * a.K + lane] = Zk == 0.0f ? 0.0f : sk / Zk;
    }
    if (a.part_p) {
      float Z = 0.0f;
      for (int e = lane; e < a.E; e += 32) Z += score(row[e], m, a.sigmoid);
      Z = warp_sum(Z);
      const float inv = Z == 0.0f ? 0.0f : 1.0f / Z;
      for (int e = lane; e < a.E; e += 32) acc[e] += score(row[e], m, a.sigmoid) * inv;
    }
    __syncwarp();
  }
  __syncthreads();
  const int64_t o = ((int64_t)r * gridDim.x + blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    a.part_c[o + e] = cnt[e];
    if (a.part_p) {
      float v = 0.0f;
      for (int i = 0; i < warps; i++) v += sh[(size_t)(warps + i) * a.E + e];
      a.part_p[o + e] = v;
    }
  }
}

struct FinishArgs {
  const float *part_p;
  const int32_t *part_c;
  int32_t *tpe;  // [R, E]
  float *coef;   // [R, E] or null
  float *loss;   // [1] or null
  float alpha;
  int R, S, E, K, bpr, global;
  int32_t ntok[kMaxRanks];
};

// Sums the blocks' partials in block order: counts, coefficients, loss.
__global__ void __launch_bounds__(1024) route_finish_kernel(FinishArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[32];
  int64_t total = 0;
  int busy = 0;
  for (int r = 0; r < a.R; r++) {
    total += a.ntok[r];
    busy += a.ntok[r] > 0;
  }
  float loss = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    int64_t call = 0;
    float pall = 0.0f;
    for (int r = 0; r < a.R; r++) {
      int c = 0;
      float p = 0.0f;
      for (int b = 0; b < a.bpr; b++) {
        const int64_t o = ((int64_t)r * a.bpr + b) * a.E + e;
        c += a.part_c[o];
        if (a.loss) p += a.part_p[o];
      }
      const int n = a.ntok[r];
      a.tpe[(int64_t)r * a.E + e] = c + (e == 0 ? (a.S - n) * a.K : 0);
      if (!a.loss) continue;
      if (a.global) {
        call += c;
        pall += p;
      } else {
        const float t = (float)(n > 0 ? n : 1);
        const float q = a.alpha * (float)a.E * (float)c / ((float)a.K * t * t * (float)(busy > 0 ? busy : 1));
        a.coef[(int64_t)r * a.E + e] = q;
        loss += q * p;
      }
    }
    if (a.loss && a.global) {
      const float t = (float)(total > 0 ? total : 1);
      const float q = a.alpha * (float)a.E * (float)call / ((float)a.K * t * t);
      for (int r = 0; r < a.R; r++) a.coef[(int64_t)r * a.E + e] = q;
      loss += q * pall;
    }
  }
  if (!a.loss) return;
  loss = warp_sum(loss);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = loss;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float v = warp_sum(red[threadIdx.x]);
    if (threadIdx.x == 0) *a.loss = v;
  }
}

struct RouteBwdArgs {
  const void *logits;
  const int32_t *topk;
  const float *w;
  const float *dw;     // [R, S, K] or null
  const float *coef;   // [R, E] or null
  const float *dloss;  // [1] or null (1)
  void *dz;            // [R, S, E] in the logits' type
  int R, S, E, K, sigmoid;
  int32_t ntok[kMaxRanks];
};

// 1 - sigmoid(z), without cancellation.
__device__ __forceinline__ float one_minus_sigmoid(float z) { return 1.0f / (1.0f + expf(z)); }

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteBwdArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tokens = (int64_t)a.R * a.S;
  const float dl = a.dloss ? *a.dloss : 1.0f;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < tokens; t += (int64_t)gridDim.x * kWarps) {
    const int r = (int)(t / a.S);
    T *out = (T *)a.dz + t * a.E;
    if (t - (int64_t)r * a.S >= a.ntok[r]) {
      for (int e = lane; e < a.E; e += 32) put(out + e, 0.0f);
      continue;
    }
    const T *z = (const T *)a.logits + t * a.E;
    const float *cf = a.coef ? a.coef + (int64_t)r * a.E : nullptr;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f(z[e]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float Z = 0.0f, pc = 0.0f;
    if (cf) {
      for (int e = lane; e < a.E; e += 32) {
        const float s = score(to_f(z[e]), m, a.sigmoid);
        Z += s;
        pc += s * cf[e];
      }
      Z = warp_sum(Z);
      pc = warp_sum(pc);
    }
    const float inv = Z == 0.0f ? 0.0f : 1.0f / Z;
    pc *= inv;
    float wk = 0.0f, dk = 0.0f;
    int id = -1;
    if (lane < a.K) {
      id = a.topk[t * a.K + lane];
      wk = a.w[t * a.K + lane];
      dk = a.dw ? a.dw[t * a.K + lane] : 0.0f;
      if (id < 0 || id >= a.E) id = -1;
    }
    const float wd = warp_sum(wk * dk);
    for (int e = lane; e < a.E; e += 32) {
      const float x = to_f(z[e]);
      float g = 0.0f;
      if (cf) g = dl * score(x, m, a.sigmoid) * inv * (cf[e] - pc);
      if (a.sigmoid) g *= one_minus_sigmoid(x);
      put(out + e, g);
    }
    __syncwarp();
    if (id >= 0) {
      const float x = to_f(z[id]);
      float g = wk * (dk - wd);
      if (cf) g += dl * score(x, m, a.sigmoid) * inv * (cf[id] - pc);
      if (a.sigmoid) g *= one_minus_sigmoid(x);
      put(out + id, g);
    }
  }
}

// Blocks per rank of the forward pass: as many as fill the SMs once, no more
// than the rank's tokens need.
int blocks_per_rank(int R, int S, int sms) {
  const int need = (S + kWarps - 1) / kWarps;
  const int fill = (sms + R - 1) / R;
  return need < fill ? (need > 0 ? need : 1) : fill;
}

// Warps of a forward block: fewer where a row of all experts per warp would
// not fit in shared memory.
int warps_of(int E) { return E <= 1024 ? kWarps : 4; }

}  // namespace

int64_t route_scratch_words(int R, int E, int sms) {
  return (int64_t)2 * R * ((sms + R - 1) / R) * E;
}

int launch_route(moonep_ctx *ctx, const void *logits, int bf16, int scoring, float alpha, int global,
                 const int32_t *num_tokens, int32_t *topk, float *w, int32_t *tpe, float *coef,
                 float *loss, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  RouteArgs a{};
  FinishArgs f{};
  a.R = f.R = c.R;
  a.S = f.S = c.S;
  a.E = f.E = c.E;
  a.K = f.K = c.K;
  a.bpr = f.bpr = blocks_per_rank(c.R, c.S, ctx->sms);
  a.logits = logits;
  a.topk = topk;
  a.w = w;
  a.sigmoid = scoring;
  const int64_t half = (int64_t)c.R * a.bpr * c.E;
  a.part_c = ctx->d_route;
  a.part_p = loss ? (float *)(ctx->d_route + half) : nullptr;
  f.part_c = a.part_c;
  f.part_p = a.part_p;
  f.tpe = tpe;
  f.coef = coef;
  f.loss = loss;
  f.alpha = alpha;
  f.global = global;
  for (int r = 0; r < c.R; r++) a.ntok[r] = f.ntok[r] = num_tokens ? num_tokens[r] : c.S;
  const int warps = warps_of(c.E);
  const size_t smem = (size_t)(2 * warps + 1) * c.E * sizeof(float);
  auto kern = bf16 ? route_kernel<__nv_bfloat16> : route_kernel<float>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = launch_pdl(kern, dim3(a.bpr, c.R), dim3(warps * 32), smem, st, false, a);
  if (e == cudaSuccess) e = launch_pdl(route_finish_kernel, dim3(1), dim3(1024), 0, st, false, f);
  return cuda_status(e);
}

int launch_route_backward(moonep_ctx *ctx, const void *logits, int bf16, int scoring,
                          const int32_t *num_tokens, const int32_t *topk, const float *w,
                          const float *dw, const float *coef, const float *dloss, void *dz,
                          cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  RouteBwdArgs a{};
  a.logits = logits;
  a.topk = topk;
  a.w = w;
  a.dw = dw;
  a.coef = coef;
  a.dloss = dloss;
  a.dz = dz;
  a.R = c.R;
  a.S = c.S;
  a.E = c.E;
  a.K = c.K;
  a.sigmoid = scoring;
  for (int r = 0; r < c.R; r++) a.ntok[r] = num_tokens ? num_tokens[r] : c.S;
  const int64_t need = ((int64_t)c.R * c.S + kWarps - 1) / kWarps;
  const int64_t cap = (int64_t)ctx->sms * 8;
  auto kern = bf16 ? route_backward_kernel<__nv_bfloat16> : route_backward_kernel<float>;
  return cuda_status(launch_pdl(kern, dim3((unsigned)(need < cap ? need : cap)), dim3(kWarps * 32),
                                0, st, false, a));
}

}  // namespace moonep
