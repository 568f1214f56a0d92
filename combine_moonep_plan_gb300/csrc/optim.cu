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
// keeps at least the least code, so an update never divides by eps alone because
// of the codes' range.  The stored values' error does not enter the update of its own
// step: p is computed from m and v before they are rounded.
//
// Measured (the kernels alone, 704 million parameters in three tensors): fp32
// moments, parameters and gradients with bf16 copies 2.98 ms, 7.09 TB/s, above
// the plain copy's 6.79, bound by memory; 8-bit moments, rounded at random, 1.81
// ms, 7.0 TB/s; bf16 parameters and gradients with fp32 moments 2.24 ms, 6.9
// TB/s, with 8-bit ones 1.87 ms, 3.8 TB/s, bound by 86 instructions per value (60
// to nearest: a fifth of them are the words for p's rounding).  Pairs of products
// in one instruction, rounding in whole numbers and a hash whose first shift the
// eight values of a thread share took 8-bit moments from 2.44 to 1.86 ms; five
// blocks per SM in place of four (a few registers spilled) to 1.81, bf16
// parameters with six from 2.10 to 1.87.  The norm reads at 7.3 TB/s (fp32) and
// 6.3 (bf16).  Tensors that do not start on 16 bytes go element by element: without
// copies 2.97 for 2.80 ms (fp32, 32 bits), 2.20 for 1.64 (fp32, 8 bits at random),
// 2.37 for 1.89 (bf16, 8 bits at random).
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

__host__ __device__ inline uint32_t mix_rest(uint32_t x) {
  x *= 0x243f6a89u;
  x ^= x >> 15;
  x *= 0xb7e15163u;
  return x ^ (x >> 16);
}
__host__ __device__ inline uint32_t mix(uint32_t x) { return mix_rest(x ^ (x >> 16)); }
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

// The upper halves of eight fp32 numbers, as bf16.
__device__ __forceinline__ void cut_some(float *, int64_t, int64_t, bool, const float *) {}
__device__ __forceinline__ void cut_some(__nv_bfloat16 *p, int64_t i, int64_t n, bool vec,
                                         const float f[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; k++)
    w[k] = __byte_perm(__float_as_uint(f[2 * k]), __float_as_uint(f[2 * k + 1]), 0x7632);
  if (vec && i + 8 <= n) {
    *(uint4 *)(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; k++)
    if (i + k < n) ((uint16_t *)p)[i + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

// Pairs: one instruction for two products or sums, each rounded as usual.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// A sum of two products that were rounded, one by one: an addition of pairs, and a
// product with one as well, is contracted with the product before it in spite of
// its rounding, and one value in four then differs in its last bit.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// Square root; a subnormal's is 0 unless it is asked for (TINY).
template <bool TINY>
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  if (TINY)
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / x for x from 2^-126 to 2^126, which eps and the root's size keep it within.
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scale byte of a block: OCT octaves from its power to the largest code, whose
// significand's bits are MOST.
template <int OCT, uint32_t MOST>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)(amax >> 23) - OCT + ((amax & 0x7fffffu) > MOST);
  return (uint32_t)(b > 0 ? b : 0);
}

// Largest of the four lanes that hold a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// The low bytes of four words as one.
__device__ __forceinline__ uint32_t bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight moments from codes and their block's scale.  A v code's bits from 20 on
// are an fp32 number 2^126 too small, subnormal where the code is.
__device__ __forceinline__ void decode_m(uint2 c, uint32_t s, float2 f[4]) {
  const float2 k = both(mx_value(s));
  const uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; i++) f[i] = mul2(mx_e4m3x2(w[i] & 0xffffu), k);
}
__device__ __forceinline__ void decode_v(uint2 c, uint32_t s, float2 f[4]) {
  const uint32_t w[2] = {c.x, c.y};
  const float2 k = both(mx_value(s)), up = both(0x1p126f);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t lo = w[i >> 1] >> (16 * (i & 1)), hi = lo >> 8;
    f[i] = make_float2(__uint_as_float((lo & 255u) << 20), __uint_as_float((hi & 255u) << 20));
    f[i] = mul2(mul2(f[i], up), k);
  }
}

// Rounding a value to a code: the value times a power that makes 2^-126 of the
// least normal one is an fp32 number whose bits from 20 on are the code, below
// the normals too.  Adding 20 bits' worth of chance to the bits that are cut (r,
// 16 bits) goes up with a probability that is what was cut; adding half and the
// lowest kept bit rounds to nearest even.  In whole numbers: with conversions and
// floors the kernel needed 102 instructions for each value and was bound by them.
__device__ __forceinline__ uint32_t code_bits(float u, uint32_t r, bool seeded) {
  const uint32_t b = __float_as_uint(u);
  return seeded ? b + (r << 4) : b + 0x7ffffu + ((b >> 20) & 1u);
}

// Codes of eight moments; word: their random words (seeded), the low half m's,
// the high half v's.
__device__ __forceinline__ uint2 encode_m(const float2 f[4], const uint32_t word[8], bool seeded,
                                          uint32_t *scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; i++)
    top = max(top, max(__float_as_uint(fabsf(f[i].x)), __float_as_uint(fabsf(f[i].y))));
  const uint32_t s = block_scale<8, 0x600000u>(block_max(top));
  const float2 inv = both(mx_inverse(s)), down = both(0x1p-120f);
  *scale = s;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 t = mul2(mul2(f[i], inv), down);
    const uint32_t x = code_bits(t.x, word[2 * i] & 0xffffu, seeded);
    const uint32_t y = code_bits(t.y, word[2 * i + 1] & 0xffffu, seeded);
    c[2 * i] = ((x >> 20) & 0x7fu) | ((x >> 24) & ~0x7fu);
    c[2 * i + 1] = ((y >> 20) & 0x7fu) | ((y >> 24) & ~0x7fu);
  }
  return make_uint2(bytes(c[0], c[1], c[2], c[3]), bytes(c[4], c[5], c[6], c[7]));
}
__device__ __forceinline__ uint2 encode_v(const float2 f[4], const uint32_t word[8], bool seeded,
                                          uint32_t *scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; i++)
    top = max(top, max(__float_as_uint(f[i].x), __float_as_uint(f[i].y)));
  const uint32_t s = block_scale<30, 0x700000u>(block_max(top));
  const float2 inv = both(mx_inverse(s)), down = both(0x1p-126f);
  *scale = s;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 t = mul2(mul2(f[i], inv), down);
    // a value above zero keeps at least the least code
    c[2 * i] = max(code_bits(t.x, word[2 * i] >> 16, seeded) >> 20,
                   min(__float_as_uint(f[i].x), 1u));
    c[2 * i + 1] = max(code_bits(t.y, word[2 * i + 1] >> 16, seeded) >> 20,
                       min(__float_as_uint(f[i].y), 1u));
  }
  return make_uint2(bytes(c[0], c[1], c[2], c[3]), bytes(c[4], c[5], c[6], c[7]));
}

// The scalars of a step whose rate or number lies in device memory.
__device__ void device_scalars(const StepArgs &a, Scalars *s) {
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const int32_t t = a.step_dev ? max(*a.step_dev, 1) : a.step;
  s->decay = 1.0f - lr * a.wd;
  s->rate = lr / -expm1f((float)t * a.log_b1);
  s->root = 1.0f / sqrtf(-expm1f((float)t * a.log_b2));
  s->key = mix(a.seed + mix((uint32_t)t));
}

// TINY: eps is small enough for the root of a v below 2^-126 to count beside it.
// With 8-bit moments, where instructions count, that root costs 2 to 3 % (704 million
// values rounded at random, fp32 parameters 1.68 ms for 1.64, bf16 1.95 for 1.89; a
// branch on eps in one kernel as much), so they take it only then; with 32-bit ones,
// bound by memory, always.
template <typename P, typename G, int BITS, bool TINY, int N>
__global__ void __launch_bounds__(kThreads, BITS == 8 && sizeof(P) == 4 ? 5 : 6)
    adamw_kernel(const __grid_constant__ Table<N> tab, const __grid_constant__ StepArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ Scalars sh;
  float clip = 1.0f;
  if (a.norm) {
    const float norm = *a.norm;
    if (!(fabsf(norm) < INFINITY)) return;  // no step on gradients that are not finite
    clip = fminf(1.0f, __fdiv_rn(a.max_norm, norm));
  }
  if (threadIdx.x == 0) {
    sh = a.s;
    if (a.lr_dev || a.step_dev) device_scalars(a, &sh);
  }
  __syncthreads();
  const Scalars s = sh;
  // the tensor of the block's first chunk
  int t = 0;
  for (int hi = tab.count - 1; t < hi;) {
    const int mid = (t + hi) >> 1;
    if ((int)blockIdx.x < tab.first[mid + 1]) hi = mid; else t = mid + 1;
  }
  for (int c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
    while (c >= tab.first[t + 1]) t++;
    const int64_t n = tab.n[t], i = (int64_t)(c - tab.first[t]) * kChunk + threadIdx.x * kPer;
    // moments come in whole blocks of 32, four lanes to a block
    const bool live = (i & ~(int64_t)31) < n;
    const bool vec = tab.vec[t];
    float p[8], g[8];
    load_some((const P *)tab.p[t], i, n, vec, p);
    load_some((const G *)tab.g[t], i, n, vec, g);
    float2 m[4], v[4];
    if (BITS == 32) {
      float f[8], h[8];
#pragma unroll
      for (int k = 0; k < 8; k++) f[k] = h[k] = 0.0f;
      if (live) {
        load8((const float *)tab.m[t] + i, f);
        load8((const float *)tab.v[t] + i, h);
      }
#pragma unroll
      for (int k = 0; k < 8; k++) {
        // one by one: pairs of registers would take a block of warps off the SM
        const float x = __fmul_rn(g[k], clip);
        f[k] = __fadd_rn(__fmul_rn(s.b1, f[k]), __fmul_rn(s.c1, x));
        h[k] = __fadd_rn(__fmul_rn(s.b2, h[k]), __fmul_rn(__fmul_rn(s.c2, x), x));
        p[k] = p[k] * s.decay - s.rate * (f[k] * inverse(sqrt_fast<TINY>(h[k]) * s.root + s.eps));
      }
      if (live) {
        store8((float *)tab.m[t] + i, f);
        store8((float *)tab.v[t] + i, h);
      }
    } else {
      uint2 cm = make_uint2(0u, 0u), cv = cm;
      uint32_t sm = 0, sv = 0;
      if (live) {
        cm = *(const uint2 *)((const uint8_t *)tab.m[t] + i);
        cv = *(const uint2 *)((const uint8_t *)tab.v[t] + i);
        sm = tab.ms[t][i >> 5];
        sv = tab.vs[t][i >> 5];
      }
      decode_m(cm, sm, m);
      decode_v(cv, sv, v);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float2 x = mul2(make_float2(g[2 * k], g[2 * k + 1]), both(clip));
        m[k] = add2(mul2(both(s.b1), m[k]), mul2(both(s.c1), x));
        v[k] = add2(mul2(both(s.b2), v[k]), mul2(mul2(both(s.c2), x), x));
        const float2 den = fma2(make_float2(sqrt_fast<TINY>(v[k].x), sqrt_fast<TINY>(v[k].y)),
                                both(s.root), both(s.eps));
        const float2 q = mul2(m[k], make_float2(inverse(den.x), inverse(den.y)));
        const float2 y = fma2(both(-s.rate), q, mul2(make_float2(p[2 * k], p[2 * k + 1]),
                                                     both(s.decay)));
        p[2 * k] = y.x;
        p[2 * k + 1] = y.y;
      }
    }
    uint32_t word[8];
    if (a.seeded) {
      const uint32_t key = mix(s.key + kGolden * (uint32_t)(a.ordinal + t + 1)) ^
                           ((uint32_t)(i >> 32) * kGolden);
      // i is a multiple of eight: the first shift of key ^ (i + k) knows no k
      const uint32_t base = key ^ (uint32_t)i, start = base ^ (base >> 16);
#pragma unroll
      for (int k = 0; k < 8; k++) word[k] = mix_rest(start ^ (uint32_t)k);
    }
    uint32_t sm, sv;
    uint2 cm, cv;
    if (BITS == 8) {
      if (a.seeded) {
        cm = encode_m(m, word, true, &sm);
        cv = encode_v(v, word, true, &sv);
      } else {
        cm = encode_m(m, word, false, &sm);
        cv = encode_v(v, word, false, &sv);
      }
    }
    if (!live) continue;
    if (BITS == 8) {
      *(uint2 *)((uint8_t *)tab.m[t] + i) = cm;
      *(uint2 *)((uint8_t *)tab.v[t] + i) = cv;
      if ((i & 31) == 0) {
        tab.ms[t][i >> 5] = (uint8_t)sm;
        tab.vs[t][i >> 5] = (uint8_t)sv;
      }
    }
    if (sizeof(P) == 2 && a.seeded) {
      // the cut half's chance; a NaN's bits would run over
#pragma unroll
      for (int k = 0; k < 8; k++)
        p[k] = __uint_as_float(__float_as_uint(p[k]) +
                               (p[k] == p[k] ? mix(word[k] + kGolden) & 0xffffu : 0u));
      cut_some((P *)tab.p[t], i, n, vec, p);
      continue;
    }
    store_some((P *)tab.p[t], i, n, vec, p);
    if (tab.w[t]) store_some((__nv_bfloat16 *)tab.w[t], i, n, vec, p);
  }
}

// Sums of squares: fp32 over a thread's eight values, then a pair of fp32 numbers
// whose second one collects the first one's rounding errors (each error exactly,
// by the six operations of the two-sum), and 64 bits beyond the thread.  An
// addition in 64 bits for every eight values took the time of reading them twice.
template <typename G, int N>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ Table<N> tab,
                                                          double *part, int add) {
  pdl_wait();
  pdl_launch_dependents();
  float hi = 0.0f, lo = 0.0f;
  int t = 0;
  const int all = tab.first[tab.count];
  for (int c = blockIdx.x; c < all; c += gridDim.x) {
    while (c >= tab.first[t + 1]) t++;
    const int64_t i = (int64_t)(c - tab.first[t]) * kChunk + threadIdx.x * kPer;
    float g[8];
    load_some((const G *)tab.g[t], i, tab.n[t], tab.vec[t], g);
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) q = fmaf(g[k], g[k], q);
    const float s = __fadd_rn(hi, q), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(q, b)));
    hi = s;
  }
  // an infinite sum has no error to speak of
  double sum = hi < INFINITY ? (double)hi + (double)lo : (double)hi;
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
    float2 f[4];
    decode_m(*(const uint2 *)(m8 + i), ms[i >> 5], f);
    store8(m + i, (const float *)f);
    decode_v(*(const uint2 *)(v8 + i), vs[i >> 5], f);
    store8(v + i, (const float *)f);
  }
}

template <typename P, typename G, int N>
auto adamw_kernel_of(int bits, bool tiny) {
  return bits == 32 ? adamw_kernel<P, G, 32, true, N>
         : tiny     ? adamw_kernel<P, G, 8, true, N> : adamw_kernel<P, G, 8, false, N>;
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

// Blocks of a step.  One chunk to a block where the step is bound by memory, the
// hardware handing blocks out as others end: 704 million fp32 parameters with
// fp32 moments took 2.98 ms, with as many blocks as are resident and many chunks
// to each 3.56.  Moments in 8 bits have more to work out before a block's first
// load: four chunks 1.81 ms, two 1.84, eight 1.86 (at four blocks per SM one chunk
// took 8 % more than four, all resident 13 %); bf16 parameters, bound by
// instructions, sixteen or more 1.94 ms, eight 1.96 (and 9 % more with four).
// Where blocks take several chunks their count is a multiple of the resident
// ones, so that no wave of them is all but empty.
template <typename K>
int64_t step_blocks(const moonep_ctx *ctx, const AdamwCall &c, K kernel, int64_t chunks) {
  const int span = c.bits == 32 ? 1 : c.p_bf16 ? 16 : 4;
  int64_t blocks = chunks;
  if (span > 1) {
    const int64_t wave = resident(ctx, kernel, INT32_MAX);
    blocks = (chunks + span * wave - 1) / (span * wave) * wave;
    if (blocks > chunks) blocks = chunks;
  }
  const int64_t held = blocks_in_cap(ctx, kernel, kThreads, 0);
  return blocks < held ? blocks : held;
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
    auto kern = adamw_kernel_of<P, G, N>(c.bits, c.tiny);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)step_blocks(ctx, c, kern, chunks)),
                                     dim3(kThreads), 0, st, false, tab, a);
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

int launch_adamw(moonep_ctx *ctx, AdamwCall c, const moonep_adamw_config &h, cudaStream_t st) {
  StepArgs a{};
  // v below 2^-126: sqrt(v) / sqrt(1 - b2^t) is below 2^-63 / sqrt(1 - b2), which is
  // half an ulp of any other eps or less
  c.tiny = !(h.eps * sqrt(1.0 - h.beta2) >= 0x1p-39);
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
