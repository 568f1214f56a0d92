// The router with a selection bias and expert groups, and the bias's step.
//
// Row of logits z[E] of a valid token, scores s_e and shares p_e as in the plain
// router; a_e = p_e (softmax) or s_e (sigmoid):
//   c_e = a_e + b_e                                   selects
//   v_g = the largest c in group g, or the sum of its two largest
//   picks = the K largest c among the top groups (equal: lowest index)
//   w_k = scale a_k / sum_picks a, or scale a_k       weighs, without the bias
// Without a bias the order of c is that of the logits, and these are compared.
//
// The order of c is that of its value in 64 bits.  In fp32 two neighbours may
// come out the wrong way round, so the picks are made in fp32 with a bound on
// each value's error, and a row in which a comparison that mattered (neighbours
// among the picks, the last pick and the rest, the last group and the rest) is
// closer than the bounds is done again in 64 bits by its warp: one row in a
// thousand of 256 experts.  Two experts with the same logit and bias have the
// same c and need no second look.
#include "route_common.cuh"

namespace moonep {
namespace {

constexpr int kWarps = kRouteWarps;

struct SelectArgs {
  RouteArgs r;
  const float *bias;  // [E] or null
  int groups, top_groups, sum_two, renormalize;
  float scale;
};

__device__ __forceinline__ uint64_t order_key64(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  if (v != v) return ~0ull;
  return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value64(uint64_t k) {
  if (k == ~0ull) return __longlong_as_double(0x7fffffffffffffffll);
  return __longlong_as_double((int64_t)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

// A row's picks in 64 bits, by one warp: indices into stage[k].y, and the
// logits' keys into stage[k].x.  row: E words of shared memory, of the warp's
// own; best: one word per group.
template <typename T>
__device__ __noinline__ void select_exact(const SelectArgs &a, const T *z, uint64_t *row,
                                          uint64_t *best, uint2 *stage) {
  const int lane = threadIdx.x & 31, E = a.r.E, gs = E / a.groups;
  const bool grouped = a.top_groups < a.groups;
  if (a.bias || grouped) {
    float m = -INFINITY;
    double Z = 1.0;
    if (!a.r.sigmoid) {
      for (int e = lane; e < E; e += 32) m = fmaxf(m, to_f(z[e]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      Z = 0.0;
      if (m > -INFINITY)
        for (int e = lane; e < E; e += 32) Z += exp((double)to_f(z[e]) - (double)m);
#pragma unroll
      for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, o);
    }
    for (int e = lane; e < E; e += 32) {
      const double x = to_f(z[e]);
      double c = a.r.sigmoid ? 1.0 / (1.0 + exp(-x))
                             : (m == -INFINITY && x == x ? 0.0 : exp(x - (double)m) / Z);
      if (a.bias) c += (double)__ldg(a.bias + e);
      row[e] = order_key64(c);
    }
    __syncwarp();
  }
  if (grouped) {
    for (int g = lane; g < a.groups; g += 32) {
      uint64_t one = 0, two = 0;
      for (int i = 0; i < gs; i++) {
        const uint64_t k = row[g * gs + i];
        if (k > one) {
          two = one;
          one = k;
        } else if (k > two) {
          two = k;
        }
      }
      best[g] = a.sum_two && gs > 1 ? order_key64(key_value64(one) + key_value64(two)) : one;
    }
    __syncwarp();
  }
  // what the picks are ordered by; 0 leaves out
  for (int e = lane; e < E; e += 32) {
    bool in = true;
    if (grouped) {
      const int g = e / gs;
      int before = 0;
      for (int h = 0; h < a.groups; h++)
        before += best[h] > best[g] || (best[h] == best[g] && h < g);
      in = before < a.top_groups;
    }
    if (!a.bias) row[e] = (uint64_t)order_key(to_f(z[e]));
    if (!in) row[e] = 0;
  }
  __syncwarp();
  for (int k = 0; k < a.r.K; k++) {
    uint64_t top = 0;
    int at = 0x7fffffff;
    for (int e = lane; e < E; e += 32)
      if (row[e] > top) {
        top = row[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t q = __shfl_xor_sync(0xffffffffu, top, o);
      const int qi = __shfl_xor_sync(0xffffffffu, at, o);
      if (q > top || (q == top && qi < at)) {
        top = q;
        at = qi;
      }
    }
    if (lane == 0) {
      row[at] = 0;
      stage[k] = make_uint2(order_key(to_f(z[at])), at);
    }
    __syncwarp();
  }
}

// Weights, ids and counts of a row's picks (stage: the logits' keys and
// indices); m and inv: the row's largest logit and 1 / sum of its scores, for
// softmax weights that are not normalised.
__device__ __forceinline__ void write_picks(const SelectArgs &a, const uint2 *stage, int64_t t,
                                            bool on, float m, float inv, int32_t *cnt) {
  const int lane = threadIdx.x & 31, K = a.r.K;
  const bool mine = lane < K;
  const float z = mine && on ? key_value(stage[lane].x) : -INFINITY;
  float by = 1.0f, top = m;
  if (a.renormalize && !a.r.sigmoid) {
    top = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  const float v = mine ? score(z, top, a.r.sigmoid) : 0.0f;
  if (a.renormalize) {
    const float sum = warp_sum(v);
    by = sum == 0.0f ? 0.0f : a.scale / sum;
  } else {
    by = a.r.sigmoid ? a.scale : a.scale * inv;
  }
  if (mine) {
    a.r.topk[t * K + lane] = on ? (int)stage[lane].y : 0;
    // no weight beside the smallest scores
    a.r.w[t * K + lane] = on && by != 0.0f ? v * by : 0.0f;
    if (on) atomicAdd(&cnt[stage[lane].y], 1);
  }
}

// Bound on the error of a in fp32 where it is s and the logit x (sigmoid: two
// parts in 2^23 of the exponential and |x| of 2^24 of its argument, halved, and
// the inverse's; softmax: relative to the row's largest logit, and n roundings
// of the sum), twice over, and of adding the bias.
__device__ __forceinline__ float bound(float s, float x, float c, int n) {
  return s * (fminf(fabsf(x), 104.0f) * 0x1p-23f + (float)n * 0x1p-24f) + fabsf(c) * 0x1p-23f;
}

// Rows of up to 32 V logits, a warp to a token, lane l holding columns l V to
// l V + V - 1.
template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32) select_kernel(SelectArgs a, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint64_t words[];
  const int E = a.r.E, K = a.r.K, G = a.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane * V;
  uint64_t *row = words + (size_t)warp * E;                         // [kWarps, E]
  uint64_t *best = words + (size_t)kWarps * E + (size_t)warp * G;   // [kWarps, G]
  uint2 *stage = (uint2 *)(words + (size_t)kWarps * (E + G)) + warp * 64;
  uint2 *few = stage + 32;
  int32_t *cnt = (int32_t *)(words + (size_t)kWarps * (E + G + 64));  // [E]
  const int r = blockIdx.y, n = a.r.ntok[r];
  const bool grouped = a.top_groups < G, sigmoid = a.r.sigmoid;
  const int gs = E / G;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  float sum[V], b[V];
  float most = 0.0f;  // largest finite bias
#pragma unroll
  for (int i = 0; i < V; i++) {
    sum[i] = 0.0f;
    b[i] = a.bias && col + i < E ? __ldg(a.bias + col + i) : 0.0f;
    if (fabsf(b[i]) < INFINITY) most = fmaxf(most, fabsf(b[i]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  // lanes of a group in the search for its best, a power of two
  int per = 1;
  while (2 * per * G <= 32) per *= 2;
  int first[V];  // the first lane of a column's group
#pragma unroll
  for (int i = 0; i < V; i++) first[i] = ((col + i) / gs * per) & 31;
  const int gl = lane / per, sub = lane & (per - 1), turns = (gs + per - 1) / per;
  // whether the whole row's scores are wanted, or logits are enough
  const bool scores = a.r.part_p || a.bias || (grouped && a.sum_two) ||
                      (!sigmoid && !a.renormalize);
  const int need = a.bias ? K + 1 : K;  // the first that is not picked, too
  const int roundings = sigmoid ? 8 : V + 30;
  for (int s = blockIdx.x * kWarps + warp; s < a.r.S; s += gridDim.x * kWarps) {
    const int64_t t = (int64_t)r * a.r.S + s;
    if (s >= n) {
      write_picks(a, stage, t, false, 0.0f, 0.0f, cnt);
      continue;
    }
    const T *zt = (const T *)a.r.logits + t * E;
    float z[V], p[V];
    load_row<V>(zt, col, E, vec, z);
    float m = z[0];
#pragma unroll
    for (int i = 1; i < V; i++) m = fmaxf(m, z[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv = 0.0f;
    if (scores) {
      float Z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) {
        p[i] = score(z[i], m, sigmoid);  // -inf past the row's end: 0
        Z += p[i];
      }
      Z = warp_sum(Z);
      inv = Z == 0.0f ? 0.0f : 1.0f / Z;
    }
    const float unit = sigmoid ? 1.0f : inv;  // from scores to what selects
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; i++)
      key[i] = col + i >= E ? 0u : order_key(a.bias ? __fadd_rn(p[i] * unit, b[i]) : z[i]);
    // a bound for every value of the row
    const float any = bound(unit, sigmoid ? fmaxf(m, 0.3f) : 0.4f, 1.0f + most, roundings);
    bool again = need > 32 || G > 32;
    if (grouped && !again) {
      // groups are compared by logits where these are what selects
      const bool exact = !a.bias && !a.sum_two;
      float *line = (float *)row;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < V; i++)
        if (col + i < E) {
          const float c = a.bias ? key_value(key[i]) : exact ? z[i] : p[i] * unit;
          nan |= c != c;
          line[col + i] = c;
        }
      __syncwarp();
      float one = -INFINITY, two = -INFINITY;
      if (gl < G)
        for (int i = 0; i < turns; i++) {
          // every group starts elsewhere, on banks of its own
          int q = i + gl % turns;
          if (q >= turns) q -= turns;
          const int e = q * per + sub;
          if (e < gs) {
            const float c = line[gl * gs + e];
            two = fmaxf(two, fminf(one, c));
            one = fmaxf(one, c);
          }
        }
      for (int o = 1; o < per; o <<= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, one, o);
        const float y = __shfl_xor_sync(0xffffffffu, two, o);
        two = fmaxf(fmaxf(two, y), fminf(one, x));
        one = fmaxf(one, x);
      }
      const float v = a.sum_two && gs > 1 ? one + two : one;
      uint32_t left = gl < G && sub == 0 ? order_key(v) : 0u, last = 0u;
      unsigned in = 0;  // the chosen groups' lanes
      for (int k = 0; k < a.top_groups; k++) {
        last = __reduce_max_sync(0xffffffffu, left);
        const int src = __ffs(__ballot_sync(0xffffffffu, left == last)) - 1;
        in |= 1u << src;
        if (lane == src) left = 0u;
      }
      const float lowest = key_value(last);
      const float rest = key_value(__reduce_max_sync(0xffffffffu, left));
      again = __any_sync(0xffffffffu, nan) ||
              (!exact && !(lowest - rest > 4.0f * any + fabsf(lowest) * 0x1p-22f));
#pragma unroll
      for (int i = 0; i < V; i++)
        if (!(in >> first[i] & 1u)) key[i] = 0u;
      __syncwarp();
    }
    if (!again) {
      bool done = V >= 4 && pick_few<V>(key, col, need, lane, few, stage);
      for (int k = 0; k < need && !done; k++) {
        uint32_t top = key[0];
#pragma unroll
        for (int i = 1; i < V; i++) top = max(top, key[i]);
        const uint32_t all = __reduce_max_sync(0xffffffffu, top);
        const int src = __ffs(__ballot_sync(0xffffffffu, top == all)) - 1;
        bool look = lane == src;
#pragma unroll
        for (int i = 0; i < V; i++)
          if (look && key[i] == all) {
            key[i] = 0u;
            stage[k] = make_uint2(all, col + i);
            look = false;
          }
        // fewer candidates than picks and one: nothing is left out
        if (all == 0u && lane == 0) stage[k] = make_uint2(0u, 0u);
      }
      __syncwarp();
      if (a.bias) {
        // from the keys of c to those of the logits; neighbours further apart
        // than their errors
        const uint2 q = lane < need ? stage[lane] : make_uint2(0u, 0u);
        const bool there = q.x != 0u;
        const int id = there && q.y < (uint32_t)E ? (int)q.y : 0;
        const float c = key_value(q.x), x = to_f(zt[id]), bx = __ldg(a.bias + id);
        const float as = score(x, m, sigmoid) * unit;
        const float d = bound(as, sigmoid ? x : x - m, c, roundings);
        const float cn = __shfl_down_sync(0xffffffffu, c, 1), dn = __shfl_down_sync(0xffffffffu, d, 1);
        const float xn = __shfl_down_sync(0xffffffffu, x, 1), bn = __shfl_down_sync(0xffffffffu, bx, 1);
        const bool next = __shfl_down_sync(0xffffffffu, there, 1);
        bool close = false;
        if (lane < K - 1)
          close = !(c - cn > d + dn) && !(x == xn && bx == bn);
        else if (lane == K - 1)
          close = next && !(c - cn > d + any);
        again = __any_sync(0xffffffffu, close);
        __syncwarp();
        if (lane < K) stage[lane] = make_uint2(order_key(x), q.y);
        __syncwarp();
      }
    }
    if (again) select_exact(a, zt, row, best, stage);
    write_picks(a, stage, t, true, m, inv, cnt);
    if (a.r.part_p) {
#pragma unroll
      for (int i = 0; i < V; i++) sum[i] += p[i] * inv;
    }
    __syncwarp();
  }
  __syncthreads();
  float *acc = (float *)words;  // [kWarps, E], over the rows
  if (a.r.part_p) {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (col + i < E) acc[(size_t)warp * E + col + i] = sum[i];
  }
  finish_block(a.r, cnt, acc, kWarps);
}

// Any E: every row in 64 bits.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) select_long_kernel(SelectArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint64_t words[];
  const int E = a.r.E, G = a.groups, warps = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t *row = words + (size_t)warp * E;
  uint64_t *best = words + (size_t)warps * E + (size_t)warp * G;
  uint2 *stage = (uint2 *)(words + (size_t)warps * (E + G)) + warp * 32;
  float *acc = (float *)(words + (size_t)warps * (E + G + 32));  // [warps, E]
  int32_t *cnt = (int32_t *)(acc + (size_t)warps * E);           // [E]
  float *mine = acc + (size_t)warp * E;
  const int r = blockIdx.y, n = a.r.ntok[r];
  for (int e = lane; e < E; e += 32) mine[e] = 0.0f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  for (int s = blockIdx.x * warps + warp; s < a.r.S; s += gridDim.x * warps) {
    const int64_t t = (int64_t)r * a.r.S + s;
    if (s >= n) {
      write_picks(a, stage, t, false, 0.0f, 0.0f, cnt);
      continue;
    }
    const T *z = (const T *)a.r.logits + t * E;
    select_exact(a, z, row, best, stage);
    float m = -INFINITY, Z = 0.0f;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, to_f(z[e]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int e = lane; e < E; e += 32) Z += score(to_f(z[e]), m, a.r.sigmoid);
    Z = warp_sum(Z);
    const float inv = Z == 0.0f ? 0.0f : 1.0f / Z;
    write_picks(a, stage, t, true, m, inv, cnt);
    if (a.r.part_p)
      for (int e = lane; e < E; e += 32) mine[e] += score(to_f(z[e]), m, a.r.sigmoid) * inv;
    __syncwarp();
  }
  finish_block(a.r, cnt, acc, warps);
}

struct BiasArgs {
  const int32_t *tpe;  // [R, E]
  float *bias;
  float rate;
  int R, S, E, K;
  int32_t ntok[kMaxRanks];
};

__global__ void __launch_bounds__(1024) bias_kernel(BiasArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  int64_t tokens = 0, padded = 0;
  for (int r = 0; r < a.R; r++) {
    tokens += a.ntok[r];
    padded += a.S - a.ntok[r];
  }
  for (int e = blockIdx.x * blockDim.x + threadIdx.x; e < a.E; e += gridDim.x * blockDim.x) {
    int64_t load = e == 0 ? -padded * a.K : 0;
    for (int r = 0; r < a.R; r++) load += a.tpe[(int64_t)r * a.E + e];
    const int64_t more = tokens * a.K - load * a.E;
    if (more) a.bias[e] += more > 0 ? a.rate : -a.rate;
  }
}

constexpr int kInRegisters = 512;  // longest row in registers
int long_warps(int E) { return E <= 1024 ? 8 : E <= 2048 ? 4 : 2; }

size_t select_smem(int E, int G) {
  if (E <= kInRegisters) return ((size_t)kWarps * (E + G + 64)) * 8 + (size_t)E * 4;
  const size_t w = long_warps(E);
  return w * (E + G + 32) * 8 + (w + 1) * E * 4;
}

template <typename T>
auto select_kernel_of(int E) {
  return E <= 32 ? select_kernel<T, 1> : E <= 64 ? select_kernel<T, 2>
         : E <= 128 ? select_kernel<T, 4> : E <= 256 ? select_kernel<T, 8>
         : E <= 384 ? select_kernel<T, 12> : select_kernel<T, 16>;
}

template <typename T>
int run_select(moonep_ctx *ctx, SelectArgs &a, FinishArgs &f, int32_t *tpe, bool loss,
               cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  const bool reg = c.E <= kInRegisters;
  const int warps = reg ? kWarps : long_warps(c.E);
  const size_t smem = select_smem(c.E, a.groups);
  const void *fn = reg ? (const void *)select_kernel_of<T>(c.E) : (const void *)select_long_kernel<T>;
  cudaError_t e = smem > 48 * 1024 ? raise_dyn_smem(fn, (int)smem) : cudaSuccess;
  if (e != cudaSuccess) return cuda_status(e);
  // as the plain router: at most four blocks per SM, no more than num_sms SMs
  // hold, but one per rank; a power of two up to the cluster, then a multiple
  const int64_t held = reg ? blocks_in_cap(ctx, select_kernel_of<T>(c.E), warps * 32, smem)
                           : blocks_in_cap(ctx, select_long_kernel<T>, warps * 32, smem);
  const int64_t need = ((int64_t)c.S + warps - 1) / warps;
  int64_t cap = (4 * ctx->sms + c.R - 1) / c.R;
  if (held / c.R < cap) cap = held / c.R > 0 ? held / c.R : 1;
  const int64_t b = need < cap ? need : cap;
  int bpr = 1;
  if (b >= kCluster)
    bpr = (int)(b / kCluster * kCluster);
  else
    while (bpr < b && 2 * bpr <= cap) bpr <<= 1;
  a.r.cluster = bpr < kCluster ? bpr : kCluster;
  f.parts = bpr / a.r.cluster;
  const int64_t half = (int64_t)c.R * f.parts * c.E;
  a.r.part_c = ctx->d_route;
  a.r.part_p = loss ? (float *)(ctx->d_route + half) : nullptr;
  a.r.tpe = !loss && f.parts == 1 ? tpe : nullptr;
  f.part_c = a.r.part_c;
  f.part_p = a.r.part_p;
  const dim3 grid(bpr, c.R), block(warps * 32);
  if (reg)
    e = launch_pdl_ex(select_kernel_of<T>(c.E), grid, block, smem, st, false, a.r.cluster, a,
                      c.E % (sizeof(T) == 2 ? 8 : 4) == 0);
  else
    e = launch_pdl_ex(select_long_kernel<T>, grid, block, smem, st, false, a.r.cluster, a);
  if (e == cudaSuccess && !a.r.tpe) e = launch_route_finish(f, st);
  return cuda_status(e);
}

}  // namespace

int launch_select(moonep_ctx *ctx, const void *logits, int bf16, int scoring,
                  const moonep_route_selection &sel, float alpha, int global,
                  const int32_t *num_tokens, int32_t *topk, float *w, int32_t *tpe, float *coef,
                  float *loss, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  SelectArgs a{};
  FinishArgs f{};
  a.r.R = f.R = c.R;
  a.r.S = f.S = c.S;
  a.r.E = f.E = c.E;
  a.r.K = f.K = c.K;
  a.r.logits = logits;
  a.r.topk = topk;
  a.r.w = w;
  a.r.sigmoid = scoring;
  a.bias = sel.bias;
  a.groups = sel.groups;
  a.top_groups = sel.top_groups;
  a.sum_two = sel.group_score == MOONEP_GROUP_TOP2;
  a.renormalize = sel.renormalize;
  a.scale = sel.scale;
  f.tpe = tpe;
  f.coef = coef;
  f.loss = loss;
  f.alpha = alpha;
  f.global = global;
  for (int r = 0; r < c.R; r++) a.r.ntok[r] = f.ntok[r] = num_tokens ? num_tokens[r] : c.S;
  return bf16 ? run_select<__nv_bfloat16>(ctx, a, f, tpe, loss != nullptr, st)
              : run_select<float>(ctx, a, f, tpe, loss != nullptr, st);
}

int launch_route_bias(moonep_ctx *ctx, const int32_t *tpe, const int32_t *num_tokens, float rate,
                      float *bias, cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  BiasArgs a{};
  a.tpe = tpe;
  a.bias = bias;
  a.rate = rate;
  a.R = c.R;
  a.S = c.S;
  a.E = c.E;
  a.K = c.K;
  for (int r = 0; r < c.R; r++) a.ntok[r] = num_tokens ? num_tokens[r] : c.S;
  const int threads = c.E < 1024 ? (c.E + 31) / 32 * 32 : 1024;
  return cuda_status(launch_pdl(bias_kernel, dim3((c.E + threads - 1) / threads), dim3(threads), 0,
                                st, false, a));
}

}  // namespace moonep
