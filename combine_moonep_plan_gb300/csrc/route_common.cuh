// What the router's kernels share: the order of logits, scores, rows of logits
// in registers, and the sums that a cluster of blocks adds up.
#pragma once

#include <cuda_bf16.h>

#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {

constexpr int kRouteWarps = 8;
constexpr int kCluster = 8;  // blocks that add up their sums before they leave

struct RouteArgs {
  const void *logits;  // [R, S, E] fp32 or bf16
  int32_t *topk;       // [R, S, K]
  float *w;            // [R, S, K]
  float *part_p;       // [R, parts, E] sums of p of one cluster's tokens, or null
  int32_t *part_c;     // [R, parts, E] picks of one cluster's tokens
  int32_t *tpe;        // [R, E], written here when a rank has one cluster and no loss
  int R, S, E, K, sigmoid, cluster;
  int32_t ntok[kMaxRanks];
};

// Order-preserving bits: a larger logit has a larger key, -0 equals +0 and NaN
// is largest (adding +0 turns -0 into +0 and every NaN into 0x7fffffff); 0 is
// below every logit.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The logit of a key (NaN for the NaN key).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the LP lanes that share a token.
template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// exp(x) as a power of two: two parts in 2^23, and the rounding of x log2(e)
// (|x| parts in 2^24); below 2^-126 zero.  1/x within an ulp.
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Score of one logit; m is the row's maximum (softmax).  exp(-z) may be
// infinite, its inverse is then zero.
__device__ __forceinline__ float score(float z, float m, bool sigmoid) {
  if (sigmoid) return inverse(1.0f + exp_fast(-z));
  return m == -INFINITY ? 0.0f : exp_fast(z - m);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// V logits of a row from column c on; -inf past the row's end.  `vec`: rows
// are whole aligned vectors.
template <int V>
__device__ __forceinline__ void load_row(const float *z, int c, int E, bool vec, float f[V]) {
  if (V % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = c + i < E ? *(const float4 *)(z + c + i)
                                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      f[i] = v.x;
      f[i + 1] = v.y;
      f[i + 2] = v.z;
      f[i + 3] = v.w;
    }
    return;
  }
  if (V == 2 && vec) {
    const float2 v = c < E ? *(const float2 *)(z + c) : make_float2(-INFINITY, -INFINITY);
    f[0] = v.x;
    f[V - 1] = v.y;
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++) f[i] = c + i < E ? z[c + i] : -INFINITY;
}
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *z, int c, int E, bool vec,
                                         float f[V]) {
  if (V % 8 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      if (c + i < E) {
        bf16x8(*(const uint4 *)(z + c + i), f + i);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) f[i + j] = -INFINITY;
      }
    }
    return;
  }
  if (V % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint2 v = c + i < E ? *(const uint2 *)(z + c + i)
                                : make_uint2(0xff80ff80u, 0xff80ff80u);
      f[i] = __uint_as_float(v.x << 16);
      f[i + 1] = __uint_as_float(v.x & 0xffff0000u);
      f[i + 2] = __uint_as_float(v.y << 16);
      f[i + 3] = __uint_as_float(v.y & 0xffff0000u);
    }
    return;
  }
  if (V == 2 && vec) {
    const uint32_t v = c < E ? *(const uint32_t *)(z + c) : 0xff80ff80u;
    f[0] = __uint_as_float(v << 16);
    f[V - 1] = __uint_as_float(v & 0xffff0000u);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++) f[i] = c + i < E ? to_f(z[c + i]) : -INFINITY;
}

template <int V>
__device__ __forceinline__ void store_row(float *z, int c, int E, bool vec, const float f[V]) {
  if (V % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      if (c + i < E) *(float4 *)(z + c + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    return;
  }
  if (V == 2 && vec) {
    if (c < E) *(float2 *)(z + c) = make_float2(f[0], f[V - 1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++)
    if (c + i < E) z[c + i] = f[i];
}
template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16 *z, int c, int E, bool vec,
                                          const float f[V]) {
  if (V % 8 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 8)
      if (c + i < E) *(uint4 *)(z + c + i) = to_bf16x8(f + i);
    return;
  }
  if (V % 2 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      if (c + i < E) *(__nv_bfloat162 *)(z + c + i) = __floats2bfloat162_rn(f[i], f[i + 1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++)
    if (c + i < E) z[c + i] = __float2bfloat16_rn(f[i]);
}

// Adds up the blocks' sums cnt[E] and acc[E] (acc: `warps` rows of E, one per
// warp) over the cluster, in a fixed order, and writes them.
__device__ __forceinline__ void finish_block(const RouteArgs &a, int32_t *cnt, float *acc, int warps) {
  const int r = blockIdx.y;
  __syncthreads();
  if (a.part_p) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
      float v = acc[e];
      for (int i = 1; i < warps; i++) v += acc[(size_t)i * a.E + e];
      acc[e] = v;
    }
  }
  const int n = a.cluster, me = blockIdx.x % n, parts = gridDim.x / n;
  const int64_t o = ((int64_t)r * parts + blockIdx.x / n) * a.E;
  if (n > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
  else
    __syncthreads();
  const uint32_t c0 = (uint32_t)__cvta_generic_to_shared(cnt);
  const uint32_t a0 = (uint32_t)__cvta_generic_to_shared(acc);
  for (int e = me * blockDim.x + threadIdx.x; e < a.E; e += n * blockDim.x) {
    int c = 0;
    float p = 0.0f;
    for (int b = 0; b < n; b++) {
      uint32_t ca, pa;
      int cv;
      float pv;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ca) : "r"(c0 + 4 * e), "r"(b));
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(cv) : "r"(ca) : "memory");
      c += cv;
      if (!a.part_p) continue;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(pa) : "r"(a0 + 4 * e), "r"(b));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pv) : "r"(pa) : "memory");
      p += pv;
    }
    if (a.tpe) {
      a.tpe[(int64_t)r * a.E + e] = c + (e == 0 ? (a.S - a.ntok[r]) * a.K : 0);
    } else {
      a.part_c[o + e] = c;
      if (a.part_p) a.part_p[o + e] = p;
    }
  }
  // no block leaves before the others have read its sums
  if (n > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}

// The K largest of a warp's keys (V per lane, index col + i), in order, into
// stage[0..K): the K-th largest of the lanes' maxima is at most the K-th
// largest key, so the few keys at or above it (usually K to K + 4 of 256)
// move to one per lane, through buf, and the rounds work on a single register:
// 170 instructions for K = 8, V = 8, against 400 over all keys.  False, with
// nothing written, when more than a warp's worth of keys qualify (equal
// logits).
template <int V>
__device__ __forceinline__ bool pick_few(const uint32_t key[V], int col, int K, int lane,
                                         uint2 *buf, uint2 *stage) {
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < V; i++) best = max(best, key[i]);
  uint32_t least = 0;
  for (int k = 0; k < K; k++) {
    least = __reduce_max_sync(0xffffffffu, best);
    if (best == least) best = 0;  // equal maxima together: only more keys qualify
  }
  if (least == 0) least = 1;  // fewer lanes than picks hold logits
  int n = 0;
  unsigned in[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    in[i] = __ballot_sync(0xffffffffu, key[i] >= least);
    n += __popc(in[i]);
  }
  if (n > 32) return false;
  const unsigned before = (1u << lane) - 1;
  int at = 0;
#pragma unroll
  for (int i = 0; i < V; i++) {
    if (key[i] >= least) buf[at + __popc(in[i] & before)] = make_uint2(key[i], col + i);
    at += __popc(in[i]);
  }
  __syncwarp();
  uint2 c = lane < n ? buf[lane] : make_uint2(0u, 0xffffffffu);
  for (int k = 0; k < K; k++) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, c.x);
    const uint32_t id = __reduce_min_sync(0xffffffffu, c.x == top ? c.y : 0xffffffffu);
    if (c.y == id) {
      stage[k] = c;
      c.x = 0;
    }
  }
  return true;
}

struct FinishArgs {
  float *part_p;
  const int32_t *part_c;
  int32_t *tpe;  // [R, E]
  float *coef;   // [R, E] or null
  float *loss;   // [1] or null
  float alpha;
  int R, S, E, K, parts, global;
  int32_t ntok[kMaxRanks];
};

// Sums the route kernel's partials into counts, coefficients and the loss.
cudaError_t launch_route_finish(const FinishArgs &f, cudaStream_t st);

}  // namespace moonep
