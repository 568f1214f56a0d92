// The optimizer's side of a step: the norm of many gradients, AdamW over many
// tensors, and the values of 8-bit moments.
//
//   g' = g min(1, max_norm / norm)
//   m  = b1 m + (1 - b1) g'          v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Everything is computed in fp32.  m and v take each operation's rounding (no
// contraction), so that moments in 8 bits, whose grid has steps, come out the
// same as from any other fp32 evaluation of the formula; the quotient of p uses
// the approximate square root and inverse (a few parts in 2^23 of the update,
// which is itself a small part of p).
//
// Moments in 8 bits: 32 values share a power of two, the smallest that lets
// none saturate (E8M0 byte).  m is E4M3; v, never negative and of a range that
// is the square of the gradient's, has no sign and five exponent bits: code c
// stands for c/8 below 8 and (1 + (c & 7)/8) 2^(c/8 - 1) above, 33 octaves.
// Rounding is to nearest even, or with a seed up with the probability that
// makes it right on average: b2 = 0.999 moves v by a thousandth per step, and
// to nearest on a grid of steps of a tenth it would never move.  A v above zero
// keeps at least the least code, so an update never divides by eps alone for
// want of range.  The stored values' error does not enter the update of its own
// step: p is computed from m and v before they are rounded.
#include <cuda_bf16.h>
#include <math.h>

#include "moonep_internal.cuh"
#include "mx_common.cuh"

namespace moonep {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                     // values of a thread at a time
constexpr int kChunk = kThreads * kPer;     // and of a block
constexpr int kFewTensors = 24, kManyTensors = 384;

__host__ __device__ inline uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x243f6a89u;
  x ^= x >> 15;
  x *= 0xb7e15163u;
  return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9e3779b9u;

// The tensors of one launch, passed by value: a captured launch keeps them.
template <int N>
struct Table {
  void *p[N];
  const void *g[N];
  void *m[N], *v[N];
  uint8_t *ms[N], *vs[N];
  uint16_t *w[N];
  int64_t n[N];
  int32_t first[N + 1];  // chunks before the tensor
  uint8_t vec[N];        // p, g and w start on 16 bytes
  int count;
};

struct Scalars {
  float b1, c1, b2, c2;  // c = 1 - b
  float decay;           // 1 - lr wd
  float rate;            // lr / (1 - b1^t)
  float root;            // 1 / sqrt(1 - b2^t)
  float eps;
  uint32_t key;
};

struct StepArgs {
  Scalars s;
  const float *norm, *lr_dev;
  const int32_t *step_dev;
  float max_norm, lr, wd, log_b1, log_b2;
  int32_t step;
  uint32_t seed;
  int seeded, ordinal;  // number of the table's first tensor
};

__device__ __forceinline__ void load8(const float *p, float f[8]) {
  const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float f[8]) {
  bf16x8(*(const uint4 *)p, f);
}
__device__ __forceinline__ void store8(float *p, const float f[8]) {
  *(float4 *)p = make_float4(f[0], f[1], f[2], f[3]);
  *(float4 *)(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float f[8]) {
  *(uint4 *)p = to_bf16x8(f);
}
__device__ __forceinline__ float get(float v) { return v; }
__device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Eight values from element i on, zeros past the tensor's end.
template <typename T>
__device__ __forceinline__ void load_some(const T *p, int64_t i, int64_t n, bool vec, float f[8]) {
  if (vec && i + 8 <= n) {
    load8(p + i, f);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; k++) f[k] = i + k < n ? get(p[i + k]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_some(T *p, int64_t i, int64_t n, bool vec,
                                           const float f[8]) {
  if (vec && i + 8 <= n) {
    store8(p + i, f);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; k++)
    if (i + k < n) put(p + i + k, f[k]);
}

// Scale byte of a block: OCT octaves from its power to the largest code, whose
// significand's bits are MOST.
template <int OCT, uint32_t MOST>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)(amax >> 23) - OCT + ((amax & 0x7fffffu) > MOST);
  return (uint32_t)(b > 0 ? b : 0);
}

// t >= 0 on the grid of four significant bits and least step 2^(LOW - 3): up
// when the part above the lower neighbour and r/2^16 reach one.
template <int LOW>
__device__ __forceinline__ float grid_up(float t, uint32_t r) {
  const int e = max((int)(__float_as_uint(t) >> 23) - 127, LOW) - 3;
  const float q = __fmul_rn(t, __uint_as_float((uint32_t)(127 - e) << 23));
  return __fmul_rn(floorf(__fadd_rn(q, __fmul_rn((float)r, 0x1p-16f))),
                   __uint_as_float((uint32_t)(127 + e) << 23));
}
template <int LOW>
__device__ __forceinline__ float grid_near(float t) {
  const int e = max((int)(__float_as_uint(t) >> 23) - 127, LOW) - 3;
  return __fmul_rn(rintf(__fmul_rn(t, __uint_as_float((uint32_t)(127 - e) << 23))),
                   __uint_as_float((uint32_t)(127 + e) << 23));
}

// The value of a v code, and the code of a value on the grid.
__device__ __forceinline__ float v_value(uint32_t c) {
  return __uint_as_float(c << 20) * 0x1p126f;
}
__device__ __forceinline__ uint32_t v_code(float q) {
  return __float_as_uint(__fmul_rn(q, 0x1p-126f)) >> 20;
}

// Eight moments from codes and their block's scale.
__device__ __forceinline__ void decode_m(uint2 c, uint32_t s, float f[8]) {
  const float k = mx_value(s);
  const uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 x = mx_e4m3x2(w[i] & 0xffffu);
    f[2 * i] = x.x * k;
    f[2 * i + 1] = x.y * k;
  }
}
__device__ __forceinline__ void decode_v(uint2 c, uint32_t s, float f[8]) {
  const float k = mx_value(s);
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = v_value(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 255u) * k;
}

// Codes of eight moments; word: their random words (seeded).
__device__ __forceinline__ uint2 encode_m(const float f[8], const uint32_t word[8], bool seeded,
                                          uint32_t *scale) {
  const uint32_t s = block_scale<8, 0x600000u>(mx_amax(f));
  const float inv = mx_inverse(s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float t = __fmul_rn(f[i], inv);
    q[i] = seeded ? copysignf(grid_up<-6>(fabsf(t), word[i] & 0xffffu), t) : t;
  }
  *scale = s;
  return make_uint2(mx_pack_e4m3(q[0], q[1], q[2], q[3]), mx_pack_e4m3(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ uint2 encode_v(const float f[8], const uint32_t word[8], bool seeded,
                                          uint32_t *scale) {
  const uint32_t s = block_scale<30, 0x700000u>(mx_amax(f));
  const float inv = mx_inverse(s);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float t = __fmul_rn(f[i], inv);
    uint32_t k = v_code(seeded ? grid_up<0>(t, word[i] >> 16) : grid_near<0>(t));
    if (t > 0.0f) k = max(k, 1u);
    c[i >> 2] |= min(k, 255u) << (8 * (i & 3));
  }
  *scale = s;
  return make_uint2(c[0], c[1]);
}

// The scalars of a step whose rate or number lies in device memory.
__device__ void device_scalars(const StepArgs &a, Scalars *s) {
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const int32_t t = a.step_dev ? *a.step_dev : a.step;
  s->decay = 1.0f - lr * a.wd;
  s->rate = lr / -expm1f((float)t * a.log_b1);
  s->root = 1.0f / sqrtf(-expm1f((float)t * a.log_b2));
  s->key = mix(a.seed + mix((uint32_t)t));
}

template <typename P, typename G, int BITS, int N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<N> tab,
                                                         const __grid_constant__ StepArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ Scalars sh;
  float clip = 1.0f;
  if (a.norm) {
    const float norm = __ldg(a.norm);
    if (!(fabsf(norm) < INFINITY)) return;  // no step on gradients that are not finite
    clip = fminf(1.0f, __fdiv_rn(a.max_norm, norm));
  }
  if (threadIdx.x == 0) {
    sh = a.s;
    if (a.lr_dev || a.step_dev) device_scalars(a, &sh);
  }
  __syncthreads();
  const Scalars s = sh;
  int t = 0;
  for (int c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
    while (c >= tab.first[t + 1]) t++;
    const int64_t n = tab.n[t], i = (int64_t)(c - tab.first[t]) * kChunk + threadIdx.x * kPer;
    // moments come in whole blocks of 32, four lanes to a block
    const bool live = (i & ~(int64_t)31) < n;
    const bool vec = tab.vec[t];
    float p[8], g[8], m[8], v[8];
    load_some((const P *)tab.p[t], i, n, vec, p);
    load_some((const G *)tab.g[t], i, n, vec, g);
#pragma unroll
    for (int k = 0; k < 8; k++) m[k] = v[k] = 0.0f;
    if (BITS == 32 && live) {
      load8((const float *)tab.m[t] + i, m);
      load8((const float *)tab.v[t] + i, v);
    } else if (live) {
      const uint2 cm = *(const uint2 *)((const uint8_t *)tab.m[t] + i);
      const uint2 cv = *(const uint2 *)((const uint8_t *)tab.v[t] + i);
      decode_m(cm, tab.ms[t][i >> 5], m);
      decode_v(cv, tab.vs[t][i >> 5], v);
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float x = __fmul_rn(g[k], clip);
      m[k] = __fadd_rn(__fmul_rn(s.b1, m[k]), __fmul_rn(s.c1, x));
      v[k] = __fadd_rn(__fmul_rn(s.b2, v[k]), __fmul_rn(__fmul_rn(s.c2, x), x));
      float r;
      asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v[k]));
      p[k] = p[k] * s.decay - s.rate * __fdividef(m[k], r * s.root + s.eps);
    }
    uint32_t word[8];
    if (a.seeded) {
      const uint32_t key = mix(s.key + kGolden * (uint32_t)(a.ordinal + t + 1)) ^
                           ((uint32_t)(i >> 32) * kGolden);
#pragma unroll
      for (int k = 0; k < 8; k++) word[k] = mix(key ^ (uint32_t)(i + k));
    }
    uint32_t sm, sv;
    uint2 cm, cv;
    if (BITS == 8) {
      cm = encode_m(m, word, a.seeded, &sm);
      cv = encode_v(v, word, a.seeded, &sv);
    }
    if (!live) continue;
    if (BITS == 32) {
      store8((float *)tab.m[t] + i, m);
      store8((float *)tab.v[t] + i, v);
    } else {
      *(uint2 *)((uint8_t *)tab.m[t] + i) = cm;
      *(uint2 *)((uint8_t *)tab.v[t] + i) = cv;
      if ((i & 31) == 0) {
        tab.ms[t][i >> 5] = (uint8_t)sm;
        tab.vs[t][i >> 5] = (uint8_t)sv;
      }
    }
    if (sizeof(P) == 2 && a.seeded) {
#pragma unroll
      for (int k = 0; k < 8; k++)
        if (fabsf(p[k]) < INFINITY)
          p[k] = __uint_as_float((__float_as_uint(p[k]) + (mix(word[k] + kGolden) & 0xffffu)) &
                                 0xffff0000u);
    }
    store_some((P *)tab.p[t], i, n, vec, p);
    if (tab.w[t]) store_some((__nv_bfloat16 *)tab.w[t], i, n, vec, p);
  }
}

// Sums of squares: fp32 over a thread's eight values, double beyond.
template <typename G, int N>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ Table<N> tab,
                                                          double *part, int add) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  int t = 0;
  for (int c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
    while (c >= tab.first[t + 1]) t++;
    const int64_t i = (int64_t)(c - tab.first[t]) * kChunk + threadIdx.x * kPer;
    float g[8];
    load_some((const G *)tab.g[t], i, tab.n[t], tab.vec[t], g);
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) q = fmaf(g[k], g[k], q);
    sum += (double)q;
  }
  __shared__ double red[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kThreads / 32; k++) sum += red[k];
    part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
  }
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *part, int n, float *norm) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
  __shared__ double red[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kThreads / 32; k++) sum += red[k];
    *norm = (float)sqrt(sum);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    moments_kernel(int64_t n, const uint8_t *m8, const uint8_t *ms, const uint8_t *v8,
                   const uint8_t *vs, T *m, T *v) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPer; i < n;
       i += (int64_t)gridDim.x * kChunk) {
    float f[8];
    decode_m(*(const uint2 *)(m8 + i), ms[i >> 5], f);
    store8(m + i, f);
    decode_v(*(const uint2 *)(v8 + i), vs[i >> 5], f);
    store8(v + i, f);
  }
}

template <typename P, typename G, int N>
auto adamw_kernel_of(int bits) {
  return bits == 32 ? adamw_kernel<P, G, 32, N> : adamw_kernel<P, G, 8, N>;
}

// Blocks: as many as are resident at once on the SMs that the context may use.
template <typename K>
int resident(const moonep_ctx *ctx, K kernel, int64_t chunks) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  const int64_t most = (int64_t)ctx->sms * (n > 0 ? n : 1);
  return (int)(chunks < most ? (chunks > 0 ? chunks : 1) : most);
}

// Fills a table with tensors from `from` on; returns how many it took.
template <int N>
int fill(Table<N> *tab, const AdamwCall &c, int from, bool whole) {
  int k = 0;
  int64_t chunks = 0;
  for (; from + k < c.count && k < N; k++) {
    const int j = from + k;
    const int64_t more = (c.sizes[j] + kChunk - 1) / kChunk;
    if (chunks + more > INT32_MAX - (1 << 20)) break;
    tab->g[k] = c.g[j];
    tab->n[k] = c.sizes[j];
    uintptr_t low = (uintptr_t)c.g[j];
    if (whole) {
      tab->p[k] = c.p[j];
      tab->m[k] = c.m[j];
      tab->v[k] = c.v[j];
      tab->ms[k] = c.ms ? c.ms[j] : nullptr;
      tab->vs[k] = c.vs ? c.vs[j] : nullptr;
      tab->w[k] = c.w ? c.w[j] : nullptr;
      low |= (uintptr_t)c.p[j] | (uintptr_t)tab->w[k];
    }
    tab->vec[k] = (low & 15) == 0;
    tab->first[k] = (int32_t)chunks;
    chunks += more;
  }
  tab->first[k] = (int32_t)chunks;
  tab->count = k;
  return k;
}

template <typename P, typename G, int N>
int adamw_run(moonep_ctx *ctx, const AdamwCall &c, StepArgs a, cudaStream_t st) {
  Table<N> tab;
  for (int from = 0; from < c.count;) {
    a.ordinal = from;
    from += fill(&tab, c, from, true);
    const int chunks = tab.first[tab.count];
    if (chunks == 0) continue;
    auto kern = adamw_kernel_of<P, G, N>(c.bits);
    const cudaError_t e = launch_pdl(kern, dim3(resident(ctx, kern, chunks)), dim3(kThreads), 0,
                                     st, false, tab, a);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return MOONEP_OK;
}

template <typename P, typename G>
int adamw_types(moonep_ctx *ctx, const AdamwCall &c, const StepArgs &a, cudaStream_t st) {
  return c.count <= kFewTensors ? adamw_run<P, G, kFewTensors>(ctx, c, a, st)
                                : adamw_run<P, G, kManyTensors>(ctx, c, a, st);
}

template <typename G, int N>
int norm_run(moonep_ctx *ctx, const AdamwCall &c, double *part, float *norm, cudaStream_t st) {
  Table<N> tab;
  int64_t all = 0;
  for (int k = 0; k < c.count; k++) all += (c.sizes[k] + kChunk - 1) / kChunk;
  const int blocks = (int)(all < norm_blocks(ctx) ? all : norm_blocks(ctx));
  int add = 0;  // every launch after the first adds to the same blocks' sums
  for (int from = 0; from < c.count;) {
    from += fill(&tab, c, from, false);
    if (tab.first[tab.count] == 0) continue;
    const cudaError_t e = launch_pdl(square_kernel<G, N>, dim3(blocks), dim3(kThreads), 0, st,
                                     false, tab, part, add);
    if (e != cudaSuccess) return cuda_status(e);
    add = 1;
  }
  return cuda_status(launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, st, false,
                                (const double *)part, blocks, norm));
}

}  // namespace

int norm_blocks(const moonep_ctx *ctx) { return ctx->sms * 8; }

int launch_grad_norm(moonep_ctx *ctx, const AdamwCall &c, double *part, float *norm,
                     cudaStream_t st) {
  const bool few = c.count <= kFewTensors;
  if (c.g_bf16)
    return few ? norm_run<__nv_bfloat16, kFewTensors>(ctx, c, part, norm, st)
               : norm_run<__nv_bfloat16, kManyTensors>(ctx, c, part, norm, st);
  return few ? norm_run<float, kFewTensors>(ctx, c, part, norm, st)
             : norm_run<float, kManyTensors>(ctx, c, part, norm, st);
}

int launch_adamw(moonep_ctx *ctx, const AdamwCall &c, const moonep_adamw_config &h,
                 cudaStream_t st) {
  StepArgs a{};
  a.norm = h.norm;
  a.max_norm = h.max_norm;
  a.lr_dev = h.lr_dev;
  a.step_dev = h.step_dev;
  a.lr = (float)h.lr;
  a.wd = (float)h.weight_decay;
  a.step = h.step;
  a.seed = h.seed;
  a.seeded = h.seeded != 0;
  a.log_b1 = (float)log(h.beta1);
  a.log_b2 = (float)log(h.beta2);
  const double t = h.step;
  a.s.b1 = (float)h.beta1;
  a.s.c1 = (float)(1.0 - h.beta1);
  a.s.b2 = (float)h.beta2;
  a.s.c2 = (float)(1.0 - h.beta2);
  a.s.decay = (float)(1.0 - h.lr * h.weight_decay);
  a.s.rate = (float)(h.lr / (1.0 - pow(h.beta1, t)));
  a.s.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, t)));
  a.s.eps = (float)h.eps;
  a.s.key = mix(h.seed + mix((uint32_t)h.step));
  if (c.p_bf16)
    return c.g_bf16 ? adamw_types<__nv_bfloat16, __nv_bfloat16>(ctx, c, a, st)
                    : adamw_types<__nv_bfloat16, float>(ctx, c, a, st);
  return c.g_bf16 ? adamw_types<float, __nv_bfloat16>(ctx, c, a, st)
                  : adamw_types<float, float>(ctx, c, a, st);
}

int launch_adamw_moments(moonep_ctx *ctx, int64_t n, const uint8_t *m8, const uint8_t *ms,
                         const uint8_t *v8, const uint8_t *vs, int fp32, void *m, void *v,
                         cudaStream_t st) {
  const int64_t chunks = (n + kChunk - 1) / kChunk;
  if (fp32)
    return cuda_status(launch_pdl(moments_kernel<float>,
                                  dim3(resident(ctx, moments_kernel<float>, chunks)),
                                  dim3(kThreads), 0, st, false, n, m8, ms, v8, vs, (float *)m,
                                  (float *)v));
  return cuda_status(launch_pdl(moments_kernel<__nv_bfloat16>,
                                dim3(resident(ctx, moments_kernel<__nv_bfloat16>, chunks)),
                                dim3(kThreads), 0, st, false, n, m8, ms, v8, vs,
                                (__nv_bfloat16 *)m, (__nv_bfloat16 *)v));
}

}  // namespace moonep
