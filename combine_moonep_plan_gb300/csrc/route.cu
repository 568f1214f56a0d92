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
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kWarps = 8;
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
      const float4 v = c + i < E ? __ldg((const float4 *)(z + c + i))
                                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      f[i] = v.x;
      f[i + 1] = v.y;
      f[i + 2] = v.z;
      f[i + 3] = v.w;
    }
    return;
  }
  if (V == 2 && vec) {
    const float2 v = c < E ? __ldg((const float2 *)(z + c)) : make_float2(-INFINITY, -INFINITY);
    f[0] = v.x;
    f[V - 1] = v.y;
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i++) f[i] = c + i < E ? __ldg(z + c + i) : -INFINITY;
}
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *z, int c, int E, bool vec,
                                         float f[V]) {
  if (V % 8 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      if (c + i < E) {
        bf16x8(__ldg((const uint4 *)(z + c + i)), f + i);
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
      const uint2 v = c + i < E ? __ldg((const uint2 *)(z + c + i))
                                : make_uint2(0xff80ff80u, 0xff80ff80u);
      f[i] = __uint_as_float(v.x << 16);
      f[i + 1] = __uint_as_float(v.x & 0xffff0000u);
      f[i + 2] = __uint_as_float(v.y << 16);
      f[i + 3] = __uint_as_float(v.y & 0xffff0000u);
    }
    return;
  }
  if (V == 2 && vec) {
    const uint32_t v = c < E ? __ldg((const uint32_t *)(z + c)) : 0xff80ff80u;
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
__device__ void finish_block(const RouteArgs &a, int32_t *cnt, float *acc, int warps) {
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

// Rows of at most LP * V logits in registers, LP lanes to a token, lane l
// holding columns l*V .. l*V + V - 1 (so the lowest lane and the lowest of its
// values is the lowest index).  A round finds the largest key that is left:
// a warp to a token by one integer reduction and a vote, a few lanes by
// exchanges of (key, index).
template <typename T, int LP, int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTok = 32 / LP;  // tokens of a warp at a time
  extern __shared__ float sh[];
  float *acc = sh;                                             // [kWarps, E]
  int32_t *cnt = (int32_t *)(sh + (size_t)kWarps * a.E);       // [E]
  uint2 *stage = (uint2 *)(cnt + ((a.E + 1) & ~1));            // [tokens, K] (key, index)
  uint2 *few = stage + (size_t)kWarps * kTok * a.K + (threadIdx.x >> 5) * 32;  // LP == 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LP, col = (lane % LP) * V;
  const int r = blockIdx.y, n = a.ntok[r];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; i++) sum[i] = 0.0f;
  stage += (size_t)(warp * kTok + sub) * a.K;
  for (int s0 = (blockIdx.x * kWarps + warp) * kTok; s0 < a.S; s0 += gridDim.x * kWarps * kTok) {
    const int s = s0 + sub;
    const int64_t t = (int64_t)r * a.S + s;
    const bool on = s < n;  // a token; else padding, or past the batch
    float z[V];
#pragma unroll
    for (int i = 0; i < V; i++) z[i] = -INFINITY;
    if (on) load_row<V>((const T *)a.logits + t * a.E, col, a.E, vec, z);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = col + i < a.E ? order_key(z[i]) : 0u;
    const bool done = LP == 32 && V >= 4 && pick_few<V>(key, col, a.K, lane, few, stage);
    for (int k = 0; k < a.K && !done; k++) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; i++) best = max(best, key[i]);
      uint32_t top;
      int id = 0;
      bool win;
      if (LP == 32) {
        top = __reduce_max_sync(0xffffffffu, best);
        const int src = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        win = lane == src;
      } else {
        // this lane's lowest index of its best value, then the group's
#pragma unroll
        for (int i = V - 1; i >= 0; i--)
          if (key[i] == best) id = col + i;
        top = best;
        int tid = id;
#pragma unroll
        for (int o = LP / 2; o; o >>= 1) {
          const uint32_t q = __shfl_xor_sync(0xffffffffu, top, o);
          const int qi = __shfl_xor_sync(0xffffffffu, tid, o);
          if (q > top || (q == top && qi < tid)) {
            top = q;
            tid = qi;
          }
        }
        win = tid == id;
      }
      // the winner notes its pick and drops it
      bool look = win;
#pragma unroll
      for (int i = 0; i < V; i++)
        if (look && key[i] == top) {
          key[i] = 0;
          id = col + i;
          look = false;
        }
      if (win) stage[k] = make_uint2(top, id);
    }
    __syncwarp();
    const float m = key_value(stage[0].x);
    // weights: the group's lanes share the picks
    float Zk = 0.0f;
    for (int k = lane % LP; k < a.K; k += LP) Zk += score(key_value(stage[k].x), m, a.sigmoid);
    Zk = group_sum<LP>(Zk);
    for (int k = lane % LP; k < a.K; k += LP) {
      const uint2 q = stage[k];
      const float v = score(key_value(q.x), m, a.sigmoid);
      if (s < a.S) {
        a.topk[t * a.K + k] = on ? (int)q.y : 0;
        a.w[t * a.K + k] = !on || Zk == 0.0f ? 0.0f : v / Zk;
      }
      if (on) atomicAdd(&cnt[q.y], 1);
    }
    if (a.part_p) {
      float Z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) {
        z[i] = score(z[i], m, a.sigmoid);  // -inf past the row's end: 0
        Z += z[i];
      }
      Z = group_sum<LP>(Z);
      const float inv = !on || Z == 0.0f ? 0.0f : 1.0f / Z;
#pragma unroll
      for (int i = 0; i < V; i++) sum[i] += on ? z[i] * inv : 0.0f;
    }
    __syncwarp();
  }
  if (a.part_p) {
#pragma unroll
    for (int i = 0; i < V; i++) {
#pragma unroll
      for (int o = LP; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      if (sub == 0 && col + i < a.E) acc[(size_t)warp * a.E + col + i] = sum[i];
    }
  }
  finish_block(a, cnt, acc, kWarps);
}

// Any E: one warp per token, the row in shared memory.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_long_kernel(RouteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float sh[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *acc = sh + (size_t)warp * a.E;                       // this warp's sums of p
  float *row = sh + (size_t)(warps + warp) * a.E;             // this token's logits
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
    const float sk = lane < a.K ? score(zk, m, a.sigmoid) : 0.0f;
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
  finish_block(a, cnt, sh, warps);
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

constexpr int kFinishBlocks = 8;

__device__ __forceinline__ void finish_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void finish_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums the route kernel's partials in order: counts, coefficients, loss.  One
// cluster; block b takes ranks b, b + 8, ... and, in global scope, a share of
// the experts once every rank is summed.  Every block meets the others once
// before its part of the loss goes to block 0's shared memory, which is there
// only from block 0's start on: in rank scope the arrival is the first thing
// done, so the wait costs nothing.
__global__ void __cluster_dims__(kFinishBlocks, 1, 1) __launch_bounds__(256)
    route_finish_kernel(FinishArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[8];
  __shared__ float share[kFinishBlocks];  // block 0's: the blocks' parts of the loss
  const int b = blockIdx.x;
  if (a.loss && !a.global) finish_arrive();
  int64_t total = 0;
  int busy = 0;
  for (int r = 0; r < a.R; r++) {
    total += a.ntok[r];
    busy += a.ntok[r] > 0;
  }
  const float groups = (float)(busy > 0 ? busy : 1);
  float loss = 0.0f;
  for (int r = b; r < a.R; r += kFinishBlocks) {
    const int n = a.ntok[r];
    const float t = (float)(n > 0 ? n : 1);
    const float q0 = a.alpha * (float)a.E / ((float)a.K * t * t * groups);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
      const int64_t o = (int64_t)r * a.parts * a.E + e;
      int c = 0;
      float p = 0.0f;
#pragma unroll 8
      for (int i = 0; i < a.parts; i++) {
        c += a.part_c[o + (int64_t)i * a.E];
        if (a.loss) p += a.part_p[o + (int64_t)i * a.E];
      }
      a.tpe[(int64_t)r * a.E + e] = c + (e == 0 ? (a.S - n) * a.K : 0);
      if (!a.loss) continue;
      if (a.global) {
        a.part_p[o] = p;  // read again below, by another block
      } else {
        a.coef[(int64_t)r * a.E + e] = q0 * (float)c;
        loss += q0 * (float)c * p;
      }
    }
  }
  if (!a.loss) return;
  if (a.global) finish_arrive();
  finish_wait();
  if (a.global) {
    const float t = (float)(total > 0 ? total : 1);
    const float q0 = a.alpha * (float)a.E / ((float)a.K * t * t);
    for (int e = b * blockDim.x + threadIdx.x; e < a.E; e += kFinishBlocks * blockDim.x) {
      int64_t c = 0;
      float p = 0.0f;
#pragma unroll 8
      for (int r = 0; r < a.R; r++) {
        c += a.tpe[(int64_t)r * a.E + e] - (e == 0 ? (a.S - a.ntok[r]) * a.K : 0);
        p += a.part_p[(int64_t)r * a.parts * a.E + e];
      }
      for (int r = 0; r < a.R; r++) a.coef[(int64_t)r * a.E + e] = q0 * (float)c;
      loss += q0 * (float)c * p;
    }
  }
  loss = warp_sum(loss);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int i = 0; i < (int)(blockDim.x >> 5); i++) v += red[i];
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                 : "=r"(to)
                 : "r"((uint32_t)__cvta_generic_to_shared(share + b)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
  }
  __syncwarp();
  finish_arrive();
  finish_wait();
  if (b == 0 && threadIdx.x == 0) {
    float v = 0.0f;
    for (int i = 0; i < kFinishBlocks; i++) v += share[i];
    *a.loss = v;
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
__device__ __forceinline__ float one_minus_sigmoid(float z) { return inverse(1.0f + exp_fast(z)); }

// Coefficients are held times 2^40: their products with scores near 2^-126 are
// then ordinary numbers, as the shares that they stand for are.
constexpr float kCoefScale = 0x1p40f, kCoefUnscale = 0x1p-40f;

// The same layout of rows in registers; blockIdx.y is the rank, whose
// coefficients stay in registers too.  A pick's term reaches the lane of its
// column through a zeroed row of shared memory.
template <typename T, int LP, int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteBwdArgs a, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTok = 32 / LP, kRow = LP * V;
  __shared__ __align__(16) float term[kWarps * kTok * kRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LP, col = (lane % LP) * V;
  const int r = blockIdx.y, n = a.ntok[r];
  const float dl = a.dloss ? *a.dloss : 1.0f;
  float *row = term + (warp * kTok + sub) * kRow;
  float cf[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    cf[i] = a.coef && col + i < a.E
                ? __ldg(a.coef + (int64_t)r * a.E + col + i) * kCoefScale : 0.0f;
    row[col + i] = 0.0f;
  }
  __syncwarp();
  // a row and its picks, loaded while the row before is worked on; a warp to a
  // token holds one pick per lane
  constexpr int kPicks = LP == 32 ? 1 : 8;  // K is at most LP * V, and at most 32
  const int stride = gridDim.x * kWarps * kTok;
  float ahead[V], pw[kPicks], pd[kPicks];
  int pid[kPicks];
  auto fetch = [&](int s) {
    const int64_t t = (int64_t)r * a.S + s;
#pragma unroll
    for (int i = 0; i < V; i++) ahead[i] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPicks; i++) {
      pid[i] = -1;
      pw[i] = pd[i] = 0.0f;
    }
    if (s >= n) return;
    load_row<V>((const T *)a.logits + t * a.E, col, a.E, vec, ahead);
    if (!a.dw) return;
#pragma unroll
    for (int i = 0; i < kPicks; i++) {
      const int k = i * LP + lane % LP;
      if (k < a.K) {
        pid[i] = __ldg(a.topk + t * a.K + k);
        pw[i] = __ldg(a.w + t * a.K + k);
        pd[i] = __ldg(a.dw + t * a.K + k);
      }
    }
  };
  fetch((blockIdx.x * kWarps + warp) * kTok + sub);
  for (int s0 = (blockIdx.x * kWarps + warp) * kTok; s0 < a.S; s0 += stride) {
    const int s = s0 + sub;
    const int64_t t = (int64_t)r * a.S + s;
    const bool on = s < n;
    float z[V], g[V];
#pragma unroll
    for (int i = 0; i < V; i++) z[i] = ahead[i];
    if (a.dw) {
      float wd = 0.0f;
#pragma unroll
      for (int i = 0; i < kPicks; i++) wd += pw[i] * pd[i];
      wd = group_sum<LP>(wd);
#pragma unroll
      for (int i = 0; i < kPicks; i++)
        if (pid[i] >= 0 && pid[i] < a.E) row[pid[i]] = pw[i] * (pd[i] - wd);
      __syncwarp();
    }
    fetch(s + stride);
#pragma unroll
    for (int i = 0; i < V; i++) g[i] = row[col + i];
    float slope[V];  // d log(score) / d logit
#pragma unroll
    for (int i = 0; i < V; i++) slope[i] = 1.0f;
    if (a.coef || a.sigmoid) {
      float m = 0.0f;
      if (!a.sigmoid) {
        m = z[0];
#pragma unroll
        for (int i = 1; i < V; i++) m = fmaxf(m, z[i]);
#pragma unroll
        for (int o = LP / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      float p[V], Z = 0.0f, pc = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) {
        if (a.sigmoid) {
          // both sigmoid(z) and sigmoid(-z) from one exponential
          const float e = exp_fast(-fabsf(z[i])), q = inverse(1.0f + e);
          p[i] = z[i] < 0.0f ? e * q : q;
          slope[i] = z[i] < 0.0f ? q : e * q;
        } else {
          p[i] = score(z[i], m, false);
        }
        // past the row's end z is -inf and p is 0
        Z += p[i];
        pc += p[i] * cf[i];
      }
      Z = group_sum<LP>(Z);
      pc = group_sum<LP>(pc);
      const float inv = Z == 0.0f ? 0.0f : 1.0f / Z;
      pc *= inv;
      const float f = dl * kCoefUnscale;
#pragma unroll
      for (int i = 0; i < V; i++)
        g[i] = on ? (g[i] + p[i] * inv * (f * (cf[i] - pc))) * slope[i] : 0.0f;
    }
    if (s < a.S) store_row<V>((T *)a.dz + t * a.E, col, a.E, vec, g);
    __syncwarp();
    if (a.dw) {
#pragma unroll
      for (int i = 0; i < V; i++) row[col + i] = 0.0f;
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Any E: one warp per token, several passes over its row.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_backward_long_kernel(RouteBwdArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y;
  const float dl = a.dloss ? *a.dloss : 1.0f;
  for (int s = blockIdx.x * kWarps + warp; s < a.S; s += gridDim.x * kWarps) {
    const int64_t t = (int64_t)r * a.S + s;
    T *out = (T *)a.dz + t * a.E;
    if (s >= a.ntok[r]) {
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
        const float s1 = score(to_f(z[e]), m, a.sigmoid);
        Z += s1;
        pc += s1 * (cf[e] * kCoefScale);
      }
      Z = warp_sum(Z);
      pc = warp_sum(pc);
    }
    const float inv = Z == 0.0f ? 0.0f : 1.0f / Z;
    pc = pc * inv * kCoefUnscale;
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
      if (cf) g = score(x, m, a.sigmoid) * inv * (dl * (cf[e] - pc));
      if (a.sigmoid) g *= one_minus_sigmoid(x);
      put(out + e, g);
    }
    __syncwarp();
    if (id >= 0) {
      const float x = to_f(z[id]);
      float g = wk * (dk - wd);
      if (cf) g += score(x, m, a.sigmoid) * inv * (dl * (cf[id] - pc));
      if (a.sigmoid) g *= one_minus_sigmoid(x);
      put(out + id, g);
    }
  }
}

// How a row of E logits is held: lanes per token and values per lane.  A
// thread to a token of up to 8 experts, four lanes up to 32, then a warp with
// 2 to 16 values per lane; longer rows in shared memory.
enum Form { kThread8, kFour8, kWarp2, kWarp4, kWarp8, kWarp12, kWarp16, kLong };
Form form_of(int E) {
  return E <= 8 ? kThread8 : E <= 32 ? kFour8 : E <= 64 ? kWarp2 : E <= 128 ? kWarp4
         : E <= 256 ? kWarp8 : E <= 384 ? kWarp12 : E <= 512 ? kWarp16 : kLong;
}
int tokens_per_warp(Form f) { return f == kThread8 ? 32 : f == kFour8 ? 8 : 1; }

// Whether rows are whole 16-byte vectors.
bool whole_vectors(int E, int bf16) { return E % (bf16 ? 8 : 4) == 0; }

// Warps of a block of the shared-memory form, two rows of all experts each: at
// four from 1025 experts on, several blocks still fit an SM up to 2048, and one
// up to 4096 (147 KB).
int warps_of(int E) { return E <= 1024 ? kWarps : 4; }
size_t long_smem(int E) { return (size_t)(2 * warps_of(E) + 1) * E * sizeof(float); }

// Blocks per rank of the forward pass: enough for the rank's tokens, at most
// four per SM over all ranks (the selection is a chain of warp-wide steps, so
// it wants warps: two per SM took 48 us for 32768 x 256; rows of 257 logits and
// more need the registers of two and so take two waves) and no more than num_sms
// SMs hold (`held`), but one; a power of two up to the cluster size, then a
// multiple of it.
int blocks_per_rank(int R, int S, int E, int sms, int64_t held) {
  const Form f = form_of(E);
  const int per = (f == kLong ? warps_of(E) : kWarps) * tokens_per_warp(f);
  const int64_t need = ((int64_t)S + per - 1) / per;
  int64_t cap = (4 * sms + R - 1) / R;
  if (held / R < cap) cap = held / R > 0 ? held / R : 1;
  const int64_t b = need < cap ? need : cap;
  if (b >= kCluster) return (int)(b / kCluster * kCluster);
  int p = 1;
  while (p < b && 2 * p <= cap) p <<= 1;
  return p;
}

// The kernel of rows in registers (any form but kLong), and its shared memory.
template <typename T>
auto route_kernel_of(Form f) {
  return f == kThread8 ? route_kernel<T, 1, 8> : f == kFour8 ? route_kernel<T, 4, 8>
         : f == kWarp2 ? route_kernel<T, 32, 2> : f == kWarp4 ? route_kernel<T, 32, 4>
         : f == kWarp8 ? route_kernel<T, 32, 8> : f == kWarp12 ? route_kernel<T, 32, 12>
                                                               : route_kernel<T, 32, 16>;
}
size_t route_smem(Form f, int E, int K) {
  return ((size_t)kWarps * E + ((E + 1) & ~1)) * 4 +
         (size_t)kWarps * tokens_per_warp(f) * K * sizeof(uint2) +
         (tokens_per_warp(f) == 1 ? (size_t)kWarps * 32 * sizeof(uint2) : 0);
}

// Blocks of the forward kernel that num_sms SMs hold.
template <typename T>
int64_t route_held(const moonep_ctx *ctx) {
  const int E = ctx->cfg.E;
  const Form f = form_of(E);
  return f == kLong ? blocks_in_cap(ctx, route_long_kernel<T>, warps_of(E) * 32, long_smem(E))
                    : blocks_in_cap(ctx, route_kernel_of<T>(f), kWarps * 32,
                                    route_smem(f, E, ctx->cfg.K));
}

template <typename T>
cudaError_t launch_forward(const RouteArgs &a, int bpr, cudaStream_t st) {
  const dim3 grid(bpr, a.R);
  const Form f = form_of(a.E);
  if (f == kLong)
    return launch_pdl_ex(route_long_kernel<T>, grid, dim3(warps_of(a.E) * 32), long_smem(a.E), st,
                         false, a.cluster, a);
  return launch_pdl_ex(route_kernel_of<T>(f), grid, dim3(kWarps * 32), route_smem(f, a.E, a.K), st,
                       false, a.cluster, a, whole_vectors(a.E, sizeof(T) == 2));
}

template <typename T>
auto route_backward_kernel_of(Form f) {
  return f == kThread8 ? route_backward_kernel<T, 1, 8> : f == kFour8 ? route_backward_kernel<T, 4, 8>
         : f == kWarp2 ? route_backward_kernel<T, 32, 2>
         : f == kWarp4 ? route_backward_kernel<T, 32, 4>
         : f == kWarp8 ? route_backward_kernel<T, 32, 8>
         : f == kWarp12 ? route_backward_kernel<T, 32, 12>
                        : route_backward_kernel<T, 32, 16>;
}

template <typename T>
cudaError_t launch_backward(const moonep_ctx *ctx, const RouteBwdArgs &a, cudaStream_t st) {
  const Form f = form_of(a.E);
  const int per = kWarps * tokens_per_warp(f), threads = kWarps * 32;
  const int per_sm = f == kWarp16 ? 2 : 3;  // what the registers allow
  const int64_t held = f == kLong
                           ? blocks_in_cap(ctx, route_backward_long_kernel<T>, threads, 0)
                           : blocks_in_cap(ctx, route_backward_kernel_of<T>(f), threads, 0);
  const int64_t need = ((int64_t)a.S + per - 1) / per;
  int64_t cap = ((int64_t)ctx->sms * per_sm + a.R - 1) / a.R;
  if (held / a.R < cap) cap = held / a.R > 0 ? held / a.R : 1;
  const dim3 grid((unsigned)(need < cap ? need : cap), a.R);
  if (f == kLong)
    return launch_pdl(route_backward_long_kernel<T>, grid, dim3(threads), 0, st, false, a);
  return launch_pdl(route_backward_kernel_of<T>(f), grid, dim3(threads), 0, st, false, a,
                    whole_vectors(a.E, sizeof(T) == 2));
}

}  // namespace

cudaError_t route_configure(int E) {
  if (form_of(E) != kLong) return cudaSuccess;
  cudaError_t e = raise_dyn_smem((const void *)route_long_kernel<float>, (int)long_smem(E));
  if (e == cudaSuccess)
    e = raise_dyn_smem((const void *)route_long_kernel<__nv_bfloat16>, (int)long_smem(E));
  return e;
}

int64_t route_scratch_words(int R, int E, int sms) {
  // at most 4 * sms / R + 1 blocks per rank
  return (int64_t)2 * R * ((4 * sms + R - 1) / R / kCluster + 1) * E;
}

int launch_route(moonep_ctx *ctx, const void *logits, int bf16, int scoring, float alpha, int global,
                 const int32_t *num_tokens, int32_t *topk, float *w, int32_t *tpe, float *coef,
                 float *loss, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  RouteArgs a{};
  FinishArgs f{};
  const int bpr = blocks_per_rank(
      c.R, c.S, c.E, ctx->sms, bf16 ? route_held<__nv_bfloat16>(ctx) : route_held<float>(ctx));
  a.R = f.R = c.R;
  a.S = f.S = c.S;
  a.E = f.E = c.E;
  a.K = f.K = c.K;
  a.cluster = bpr < kCluster ? bpr : kCluster;
  f.parts = bpr / a.cluster;
  a.logits = logits;
  a.topk = topk;
  a.w = w;
  a.sigmoid = scoring;
  const int64_t half = (int64_t)c.R * f.parts * c.E;
  a.part_c = ctx->d_route;
  a.part_p = loss ? (float *)(ctx->d_route + half) : nullptr;
  a.tpe = !loss && f.parts == 1 ? tpe : nullptr;
  f.part_c = a.part_c;
  f.part_p = a.part_p;  // the route kernel's sums; global scope reuses their first rows
  f.tpe = tpe;
  f.coef = coef;
  f.loss = loss;
  f.alpha = alpha;
  f.global = global;
  for (int r = 0; r < c.R; r++) a.ntok[r] = f.ntok[r] = num_tokens ? num_tokens[r] : c.S;
  cudaError_t e = bf16 ? launch_forward<__nv_bfloat16>(a, bpr, st) : launch_forward<float>(a, bpr, st);
  if (e == cudaSuccess && !a.tpe)
    e = launch_pdl(route_finish_kernel, dim3(kFinishBlocks), dim3(256), 0, st, false, f);
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
  return cuda_status(bf16 ? launch_backward<__nv_bfloat16>(ctx, a, st)
                          : launch_backward<float>(ctx, a, st));
}

}  // namespace moonep
