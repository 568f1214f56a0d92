// The router with a selection bias and expert groups, and the bias's step.
//
// Row of logits z[E] of a valid token, scores s_e and shares p_e as in the plain
// router; a_e = p_e (softmax) or s_e (sigmoid):
//   c_e = a_e + b_e                                   selects
//   v_g = the largest c in group g, or the sum of its two largest
//   picks = the K largest c among the top groups (equal: lowest index)
//   w_k = scale a_k / sum_picks a, or scale a_k       weighs, without the bias
// Without a bias the order of c is that of the logits, and these are compared: expert
// with expert, and groups by their largest.
//
// The order of c is that of its value in 64 bits.  In fp32 two neighbours may
// come out the wrong way round, so the picks are made in fp32 with a bound on
// each value's error, and where a comparison that mattered (neighbours among the
// picks, the last pick and the rest, the last group and the rest) is closer than
// the bounds, 64 bits decide, of the few candidates alone (one row in a thousand
// of 256 experts).  Rows with values that are not finite, or with too many
// candidates, are done again as a whole.  Two experts with the same logit and
// bias have the same c and need no second look.
//
// The bound for the values that are not picked is one for the row, with the largest
// finite |b| in it, and at least the rounding of 1.  So a bias of -inf costs nothing,
// but one expert at -10^4 sends many rows to 64 bits and at -10^6 all of them as a
// whole (32768 x 256: 31 us with -inf, 38 with -10^4, 527 with -10^6; in 8 groups 37,
// 91 and 2380), as do softmax rows so peaked that their last pick's share is near
// 10^-6 (logits of deviation 3 42 us, 8 184).
#include "route_common.cuh"

namespace moonep {
namespace {

constexpr int kWarps = kRouteWarps;
constexpr int kCandidates = 36;  // one per lane, and what is read behind them
constexpr int kScratch = 2 * (kCandidates + 32);  // words of a warp: candidates and picks

struct SelectArgs {
  RouteArgs r;
  const float *bias;  // [E] or null
  int groups, top_groups, sum_two, renormalize;
  float scale;
  // Of the search for a group's best: its size; whether it is lanes' whole columns
  // (a power of two of lanes), which then hold it in registers, or read from shared
  // memory by as many lanes as there are for each; the logarithm of the lanes, and
  // the turns they take.
  int size, held, lanes_log, turns;
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

// A row's picks in 64 bits, by one warp, into index.  row: E words of shared
// memory, of the warp's own; best: one word per group.
template <typename T>
__device__ __forceinline__ void select_exact(const SelectArgs &a, const T *z, uint64_t *row,
                                          uint64_t *best, int32_t *index) {
  const int lane = threadIdx.x & 31, E = a.r.E, gs = E / a.groups;
  const bool grouped = a.top_groups < a.groups;
  // as in select_kernel: without a bias the logits themselves order the experts, and
  // groups by their largest (two logits may have one score in 64 bits)
  if (!a.bias && !(grouped && a.sum_two)) {
    for (int e = lane; e < E; e += 32) row[e] = order_key(to_f(z[e]));
    __syncwarp();
  } else {
    float m = -INFINITY;
    double Z = 1.0;
    if (!a.r.sigmoid) {
      for (int e = lane; e < E; e += 32) m = fmaxf(m, to_f(z[e]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      Z = 0.0;
      for (int e = lane; e < E; e += 32) {
        const double x = to_f(z[e]);
        Z += m > -INFINITY ? exp(x - (double)m) : x == x ? 0.0 : x;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, o);
    }
    for (int e = lane; e < E; e += 32) {
      const double x = to_f(z[e]);
      // no share where every logit is -inf, none that is a number beside a NaN
      double c = a.r.sigmoid ? 1.0 / (1.0 + exp(-x))
                             : (m > -INFINITY || Z != Z ? exp(x - (double)m) / Z : 0.0);
      if (a.bias) c += (double)a.bias[e];
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
    if (!a.bias) row[e] = order_key(to_f(z[e]));
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
      index[k] = at;
    }
    __syncwarp();
  }
}

// Weights, ids and counts of a row's picks, one per lane (id, and logit z); m and
// inv: the row's largest logit and 1 / sum of its scores, for softmax weights
// that are not normalised.
__device__ __forceinline__ void write_picks(const SelectArgs &a, bool sigmoid, int id, float z,
                                            int64_t t, bool on, float m, float inv,
                                            int32_t *cnt) {
  const int lane = threadIdx.x & 31, K = a.r.K;
  const bool mine = lane < K;
  if (!on || !mine) z = -INFINITY;
  float by = 1.0f, top = m;
  if (a.renormalize && !sigmoid) {
    top = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  float v = mine ? score(z, top, sigmoid) : 0.0f;
  if (a.renormalize) {
    const float sum = warp_sum(v);
    by = sum == 0.0f ? 0.0f : a.scale * inverse(sum);
    // scale over a sum below 1 may pass the largest number: the shares first, none
    // of which is above 1 (softmax scores add up to 1 or more)
    if (sigmoid && fabsf(by) == INFINITY) {
      v *= inverse(sum);
      by = a.scale;
    }
  } else {
    by = sigmoid ? a.scale : a.scale * inv;
  }
  if (mine) {
    a.r.topk[t * K + lane] = on ? id : 0;
    // no weight beside the smallest scores
    a.r.w[t * K + lane] = on && by != 0.0f ? v * by : 0.0f;
    if (on) atomicAdd(&cnt[id], 1);
  }
}

// Bounds on the error of c = a + b in fp32, some one and a half times what they
// have to be.
//   sigmoid  of e = exp(-x): four parts in 2^24, and |x| parts of its argument's
//            rounding, of which s (1 - s) reaches s; the sum 1 + e, the inverse,
//            and the addition of b.  s (1 - s) |x| is at most 0.28
//   softmax  of exp(x - m): the same, and |x - m| parts of the difference's
//            rounding; the sum of the row's in n + 5 roundings, its terms' errors,
//            which weighted by p are those of |x - m| = 7 (the entropy of 512
//            experts), and its inverse.  p |x - m| is at most 0.4 times the largest p
__device__ __forceinline__ float sigmoid_bound(float s, float x, float c) {
  return s * ((1.0f - s) * (fminf(fabsf(x), 104.0f) * 0x1p-23f + 0x1p-21f) + 3 * 0x1p-23f) +
         fabsf(c) * 0x1p-23f;
}
__device__ __forceinline__ float softmax_bound(float p, float d, float c, int n) {
  return p * (fminf(fabsf(d), 104.0f) * 0x1p-22f + (float)(n + 60) * 0x1p-24f) +
         fabsf(c) * 0x1p-23f;
}

// The values at or above `least` (V per lane, index col + i; NaN: none) side by
// side with their indices, in the order of these; their count, of which more than
// 32 are not written.  By predicates: as branches they were twice the
// instructions.
template <int V>
__device__ __forceinline__ int gather(const float c[V], int col, float least, int lane,
                                      uint2 *list) {
  int mine = 0;
#pragma unroll
  for (int i = 0; i < V; i++)
    asm("{\n .reg .pred p;\n setp.ge.f32 p, %1, %2;\n @p add.s32 %0, %0, 1;\n}"
        : "+r"(mine)
        : "f"(c[i]), "f"(least));
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += u;
  }
  const int n = __shfl_sync(0xffffffffu, at, 31);
  if (n > 32) return n;
  uint32_t to = (uint32_t)__cvta_generic_to_shared(list + at - mine);
#pragma unroll
  for (int i = 0; i < V; i++)
    asm volatile(
        "{\n .reg .pred p;\n setp.ge.f32 p, %1, %2;\n @p st.shared.v2.b32 [%0], {%3, %4};\n"
        " @p add.u32 %0, %0, 8;\n}"
        : "+r"(to)
        : "f"(c[i]), "f"(least), "r"(__float_as_uint(c[i])), "r"(col + i)
        : "memory");
  // what the comparisons by fours read behind them
  if (lane < 4) list[n + lane].x = 0x7fffffffu;
  __syncwarp();
  return n;
}

// Places of a warp's n side-by-side values, largest first, equal ones in order:
// each counts the larger ones, and where that does not tell all apart the equal
// ones before it.
__device__ __forceinline__ int place(const uint2 *list, int n, int lane, float mine) {
  int rank = 0;
  for (int j = 0; j < n; j += 4) {
    const uint4 a = *(const uint4 *)(list + j), b = *(const uint4 *)(list + j + 2);
    rank += __uint_as_float(a.x) > mine;
    rank += __uint_as_float(a.z) > mine;
    rank += __uint_as_float(b.x) > mine;
    rank += __uint_as_float(b.z) > mine;
  }
  if ((int)__reduce_add_sync(0xffffffffu, lane < n ? rank : 0) != n * (n - 1) / 2)
    for (int j = 0; j < n; j++) rank += j < lane && __uint_as_float(list[j].x) == mine;
  return rank;
}

// What selects, in 64 bits: a score, or a share of a row whose largest logit is m
// and whose scores' sum Z is.
__device__ __forceinline__ double exact_value(double x, double m, double Z, bool sigmoid) {
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / Z;
}
template <bool kSigmoid, typename T>
__device__ __forceinline__ double exact_sum(const SelectArgs &a, const T *z, float m) {
  double Z = 0.0;
  if (!kSigmoid) {
    for (int e = threadIdx.x & 31; e < a.r.E; e += 32) Z += exp((double)to_f(z[e]) - (double)m);
#pragma unroll
    for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, o);
  }
  return Z;
}

// The picks among n candidates by their values in 64 bits, into picks[..].y.
template <bool kSigmoid, typename T>
__device__ __noinline__ void refine_picks(const SelectArgs &a, const T *z, const float *bias,
                                          float m, int n, const uint2 *list, uint64_t *keys,
                                          uint2 *picks) {
  const int lane = threadIdx.x & 31, K = a.r.K;
  const double Z = exact_sum<kSigmoid>(a, z, m);
  uint64_t mine = 0;
  int id = 0;
  if (lane < n) {
    id = (int)list[lane].y;
    mine = order_key64(exact_value(to_f(z[id]), m, Z, kSigmoid) + (double)bias[id]);
    keys[lane] = mine;
  }
  __syncwarp();
  int rank = 0;
  for (int j = 0; j < n; j++) {
    const uint64_t o = keys[j];
    rank += o > mine || (o == mine && j < lane);
  }
  if (lane < n && rank < K) picks[rank].y = (uint32_t)id;
  __syncwarp();
}

// The top groups where some values lie within `margin` of the last one's: those
// groups by their values in 64 bits, from the elements that can be among a
// group's two largest.  Lane g has group g's value and its second largest
// element; line: the elements.  Returns the groups as bits.
template <bool kSigmoid, typename T>
__device__ __noinline__ unsigned refine_groups(const SelectArgs &a, const T *z, const float *bias,
                                               float m, const float *line, uint64_t *best,
                                               float value, float second, float last,
                                               float margin, float any) {
  const double Z = exact_sum<kSigmoid>(a, z, m);
  const int lane = threadIdx.x & 31, gs = a.r.E / a.groups;
  const bool group = lane < a.groups, flagged = group && fabsf(value - last) <= margin;
  const unsigned sure = __ballot_sync(0xffffffffu, group && value - last > margin);
  uint64_t mine = 0;
  if (flagged) {
    uint64_t one = 0, two = 0;
    const float least = second - 2.0f * any;
    for (int i = 0; i < gs; i++) {
      const int e = lane * gs + i;
      if (!(line[e] >= least)) continue;
      const uint64_t k =
          order_key64(exact_value(to_f(z[e]), m, Z, kSigmoid) + (double)bias[e]);
      if (k > one) {
        two = one;
        one = k;
      } else if (k > two) {
        two = k;
      }
    }
    mine = a.sum_two && gs > 1 ? order_key64(key_value64(one) + key_value64(two)) : one;
  }
  if (group) best[lane] = mine;
  __syncwarp();
  int rank = __popc(sure);
  for (int h = 0; h < a.groups; h++) {
    const uint64_t o = best[h];
    rank += o > mine || (o == mine && h < lane);
  }
  const unsigned in = __ballot_sync(0xffffffffu, flagged && rank < a.top_groups) | sure;
  __syncwarp();
  return in;
}

// A row's largest logit, and 1 / sum of its scores (0 where that is 0).
template <typename T>
__device__ __forceinline__ float row_max(const T *z, int E) {
  float m = -INFINITY;
  for (int e = threadIdx.x & 31; e < E; e += 32) m = fmaxf(m, to_f(z[e]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
template <typename T>
__device__ __forceinline__ float row_inverse(const T *z, int E, float m, bool sigmoid) {
  float Z = 0.0f;
  for (int e = threadIdx.x & 31; e < E; e += 32) Z += score(to_f(z[e]), m, sigmoid);
  Z = warp_sum(Z);
  return Z == 0.0f ? 0.0f : 1.0f / Z;
}

// A row's picks and weights, by 64-bit values.
template <typename T>
__device__ __noinline__ void again_exact(const SelectArgs &a, const T *z, uint64_t *row,
                                         uint64_t *best, int32_t *index, int64_t t, int32_t *cnt) {
  select_exact(a, z, row, best, index);
  const float m = row_max(z, a.r.E);
  const float inv = a.r.sigmoid || a.renormalize ? 0.0f : row_inverse(z, a.r.E, m, false);
  const int id = (threadIdx.x & 31) < a.r.K ? index[threadIdx.x & 31] : 0;
  write_picks(a, a.r.sigmoid, id, to_f(z[id]), t, true, m, inv, cnt);
  __syncwarp();
}

// Rows of up to 32 V logits, a warp to a token, lane l holding columns l V to
// l V + V - 1.  A row to be done again gets the id -1 as its first pick and its
// turn after the warp's last row.
//
// Bound by instructions, some 800 a row, and the chains between them: with four
// blocks per SM (64 registers, a few of them spilled) 32768 rows of 256 in 8
// groups take 41 us, without groups 32, 65536 bf16 rows of 384 61 us.  Two or three
// blocks without spills took a quarter more; loading the next row ahead took 5 us
// more, sorting the candidates by warp-wide maxima 7.
template <typename T, int V, bool kSigmoid>
__global__ void __launch_bounds__(kWarps * 32, V <= 12 ? 4 : 2)
    select_kernel(SelectArgs a, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint64_t words[];
  const int E = a.r.E, K = a.r.K, G = a.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane * V;
  uint64_t *row = words + (size_t)warp * (E + 32);                        // [kWarps, E + 32]
  uint64_t *best = words + (size_t)kWarps * (E + 32) + (size_t)warp * G;  // [kWarps, G]
  float *bias = (float *)(words + (size_t)kWarps * (E + 32 + G));         // [32 V], 0 past E
  uint2 *list = (uint2 *)(bias + 32 * V + warp * kScratch);               // candidates: value,
  uint2 *picks = list + kCandidates;                                      // index; the picks
  int32_t *cnt = (int32_t *)(bias + 32 * V + kWarps * kScratch);          // [E]
  const int r = blockIdx.y, n = min(a.r.ntok[r], a.r.S);
  const bool grouped = a.top_groups < G;
  constexpr bool sigmoid = kSigmoid;
  const int gs = a.size;
  const float none = __uint_as_float(0x7fffffffu);  // left out: no comparison holds
  for (int e = threadIdx.x; e < 32 * V; e += blockDim.x)
    bias[e] = a.bias && e < E ? a.bias[e] : 0.0f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  float sum[V];
  float most = 0.0f;  // largest finite bias
  bool odd = false;   // one is a NaN
#pragma unroll
  for (int i = 0; i < V; i++) {
    sum[i] = 0.0f;
    const float b = fabsf(bias[col + i]);
    if (b < INFINITY) most = fmaxf(most, b);
    odd |= b != b;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  const bool held = a.held;
  const int per = a.lanes_log, gl = lane >> per, sub = lane & ((1 << per) - 1), turns = a.turns;
  // whether the whole row's scores are wanted, or logits are enough
  const bool scores = a.r.part_p || a.bias || (grouped && a.sum_two) ||
                      (!sigmoid && !a.renormalize);
  const int need = a.bias ? K + 1 : K;  // the first that is not picked, too
  const bool full = E == 32 * V;
  const int step = gridDim.x * kWarps, begin = blockIdx.x * kWarps + warp;
  for (int s = begin; s < a.r.S; s += step) {
    const int64_t t = (int64_t)r * a.r.S + s;
    if (s >= n) {
      write_picks(a, true, 0, 0.0f, t, false, 0.0f, 0.0f, cnt);
      continue;
    }
    const T *zt = (const T *)a.r.logits + t * E;
    float c[V], p[V];
    load_row<V>(zt, col, E, vec, c);
    float m = 0.0f, inv = 0.0f, Z = 0.0f;
    if (!sigmoid) {
      m = c[0];
#pragma unroll
      for (int i = 1; i < V; i++) m = fmaxf(m, c[i]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    bool nan = false;
    if (scores) {
#pragma unroll
      for (int i = 0; i < V; i++) {
        p[i] = score(c[i], m, sigmoid);  // -inf past the row's end: 0
        Z += p[i];
      }
      nan = Z != Z || odd;  // a NaN among the lane's scores, or its biases
      if (!sigmoid && m == -INFINITY)  // scores of 0, whatever the logits
#pragma unroll
        for (int i = 0; i < V; i++) nan |= c[i] != c[i];
      if (a.r.part_p || !sigmoid) {
        Z = warp_sum(Z);
        inv = Z == 0.0f ? 0.0f : 1.0f / Z;
      }
    }
    if (a.r.part_p) {
#pragma unroll
      for (int i = 0; i < V; i++) sum[i] += p[i] * inv;
    }
    const float unit = sigmoid ? 1.0f : inv;  // from scores to what selects
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < V; i++) c[i] = __fmaf_rn(p[i], unit, bias[col + i]);
    } else if (!scores) {
#pragma unroll
      for (int i = 0; i < V; i++) nan |= c[i] != c[i];
    }
    if (!full) {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (col + i >= E) c[i] = none;
    }
    bool again = need > 32 || (grouped && G > 32) || __any_sync(0xffffffffu, nan);
    // a bound for every value of the row
    const float any = sigmoid ? 5.0f * 0x1p-23f + most * 0x1p-23f + 0x1p-23f
                              : softmax_bound(unit, 0.4f, 1.0f + most, V);
    if (grouped && !again) {
      // groups are compared by logits where these are what selects
      const bool logits = !a.bias && !a.sum_two, shares = !a.bias && a.sum_two;
      float one = -INFINITY, two = -INFINITY;
      auto take = [&](float x) {
        two = fmaxf(two, fminf(one, x));
        one = fmaxf(one, x);
      };
      float *line = (float *)row;
      auto spread = [&] {
#pragma unroll
        for (int i = 0; i < V; i++)
          if (col + i < E) line[col + i] = shares ? p[i] * unit : c[i];
        __syncwarp();
      };
      if (held && !shares) {
#pragma unroll
        for (int i = 0; i < V; i++) take(c[i]);
      } else if (held) {
#pragma unroll
        for (int i = 0; i < V; i++) take(p[i] * unit);
      } else {
        spread();
        if (gl < G)
          for (int i = 0; i < turns; i++) {
            // every group starts elsewhere, on banks of its own
            int q = i + gl % turns;
            if (q >= turns) q -= turns;
            q = (q << per) + sub;
            if (q < gs) take(line[gl * gs + q]);
          }
        __syncwarp();
      }
      for (int o = 1; o < 1 << per; o <<= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, one, o);
        const float y = __shfl_xor_sync(0xffffffffu, two, o);
        two = fmaxf(fmaxf(two, y), fminf(one, x));
        one = fmaxf(one, x);
      }
      const float v = a.sum_two && gs > 1 ? one + two : one;
      const uint32_t mine = gl < G && sub == 0 ? order_key(v) : 0u;
      uint32_t left = mine, last = 0u;
      for (int k = 0; k < a.top_groups; k++) {
        last = __reduce_max_sync(0xffffffffu, left);
        if (left == last) left = 0u;  // equal ones together
      }
      // the chosen groups, by their lanes, the first of equal ones
      unsigned in = __ballot_sync(0xffffffffu, mine && mine >= last);
      const bool ties = __popc(in) != a.top_groups;
      if (ties) {
        left = mine;
        in = 0;
        for (int k = 0; k < a.top_groups; k++) {
          last = __reduce_max_sync(0xffffffffu, left);
          const int src = __ffs(__ballot_sync(0xffffffffu, left == last)) - 1;
          in |= 1u << src;
          if (lane == src) left = 0u;
        }
      }
      const float lowest = key_value(last);
      const float rest = key_value(__reduce_max_sync(0xffffffffu, left));
      const float margin = 4.0f * any + fabsf(lowest) * 0x1p-21f;
      if (!logits && !(lowest - rest > margin)) {
        again = true;
        if (fabsf(lowest) < INFINITY && m > -INFINITY && !__any_sync(0xffffffffu, v != v)) {
          if (held) spread();
          const int src = lane << per & 31;
          const float gv = __shfl_sync(0xffffffffu, v, src);
          const float g2 = __shfl_sync(0xffffffffu, gs > 1 ? two : one, src);
          const unsigned groups =
              refine_groups<kSigmoid>(a, zt, bias, m, line, best, gv, g2, lowest, margin, any);
          in = __ballot_sync(0xffffffffu, sub == 0 && gl < G && (groups >> gl & 1u));
          again = false;
        }
      }
      if (held) {
        const bool kept = in >> (lane - sub) & 1u;
#pragma unroll
        for (int i = 0; i < V; i++) c[i] = kept ? c[i] : none;
      } else {
        int g = col / gs, at = col - g * gs;  // the column's group and place in it
#pragma unroll
        for (int i = 0; i < V; i++) {
          if (!(in >> (g << per & 31) & 1u)) c[i] = none;
          if (++at == gs) {
            at = 0;
            g++;
          }
        }
      }
    }
    if (!again) {
      // The need-th largest of the lanes' largest is at most the need-th largest
      // value, so the few at or above it hold the picks.
      float top = c[0];
#pragma unroll
      for (int i = 1; i < V; i++) top = fmaxf(top, c[i]);
      uint32_t lead = top == top ? order_key(top) : 0u, least = 0u;
      for (int k = 0; k < need; k++) {
        least = __reduce_max_sync(0xffffffffu, lead);
        if (lead == least) lead = 0u;  // equal ones together: only more qualify
      }
      const int count = gather<V>(c, col, least ? key_value(least) : -INFINITY, lane, list);
      int id = 0;
      float own = none;  // this lane's pick's value
      if (count <= 32) {
        const uint2 mine = lane < count ? list[lane] : make_uint2(0x7fffffffu, 0u);
        const int rank = place(list, count, lane, __uint_as_float(mine.x));
        if (lane >= count) {
          picks[lane].x = 0x7fffffffu;  // fewer candidates than picks and one
          picks[lane].y = 0u;
        } else if (rank < need) {
          picks[rank] = mine;
        }
        __syncwarp();
        if (lane < need) {
          const uint2 q = picks[lane];
          own = __uint_as_float(q.x);
          id = (int)q.y;
        }
      } else {
        for (int k = 0; k < need; k++) {
          float x = none;
          int at = 0;
#pragma unroll
          for (int i = V - 1; i >= 0; i--)
            if (c[i] == c[i] && !(c[i] < x)) {
              x = c[i];
              at = col + i;
            }
          const uint32_t key = x == x ? order_key(x) : 0u;
          const uint32_t all = __reduce_max_sync(0xffffffffu, key);
          const int src = __ffs(__ballot_sync(0xffffffffu, key == all)) - 1;
          const float xs = __shfl_sync(0xffffffffu, x, src);
          const int is = __shfl_sync(0xffffffffu, at, src);
          if (lane == k && all) {
            own = xs;
            id = is;
          }
#pragma unroll
          for (int i = 0; i < V; i++)
            if (all && col + i == is) c[i] = none;
        }
      }
      float x = to_f(zt[id]);
      if (a.bias) {
        // neighbours have to lie further apart than their errors
        const float bx = bias[id], as = score(x, m, sigmoid) * unit;
        const float d = sigmoid ? sigmoid_bound(as, x, own) : softmax_bound(as, x - m, own, V);
        const float cn = __shfl_down_sync(0xffffffffu, own, 1);
        const float dn = __shfl_down_sync(0xffffffffu, d, 1);
        const float xn = __shfl_down_sync(0xffffffffu, x, 1);
        const float bn = __shfl_down_sync(0xffffffffu, bx, 1);
        bool close = false;
        if (lane < K - 1)
          close = !(own - cn > d + dn) && !(x == xn && bx == bn);
        else if (lane == K - 1)
          close = cn == cn && !(own - cn > d + any);
        again = __any_sync(0xffffffffu, close);
        if (again && count <= 32 && m > -INFINITY) {
          // what may be a pick lies at most twice the bound below the last one
          const float last = __shfl_sync(0xffffffffu, own, K - 1);
          const float low = last - 2.0f * any - fabsf(last) * 0x1p-22f;
          if (fabsf(low) < INFINITY) {
            const int more = gather<V>(c, col, low, lane, list);
            if (more <= 32) {
              refine_picks<kSigmoid>(a, zt, bias, m, more, list, row, picks);
              id = lane < K ? (int)picks[lane].y : 0;
              x = to_f(zt[id]);
              again = false;
            }
          }
        }
      }
      if (!again) write_picks(a, kSigmoid, id, x, t, true, m, inv, cnt);
    }
    if (again && lane == 0) a.r.topk[t * K] = -1;
    __syncwarp();
  }
  // the rows to be done again, found 32 at a time
  for (int s0 = begin; s0 < n; s0 += 32 * step) {
    const int64_t mine = (int64_t)s0 + (int64_t)lane * step;
    const bool again = mine < n && __ldcg(a.r.topk + ((int64_t)r * a.r.S + mine) * K) < 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, again); todo; todo &= todo - 1) {
      const int64_t t = (int64_t)r * a.r.S + s0 + (int64_t)(__ffs(todo) - 1) * step;
      again_exact<T>(a, (const T *)a.r.logits + t * E, row, best, (int32_t *)list, t, cnt);
    }
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

// Any E: every row in 64 bits, K passes over its values, and for every expert one over
// the groups (32768 x 640 in 8 groups 1.52 ms, 32768 x 768 1.46 without groups, 8192 x
// 4096 3.6: some twenty times what a row of 512 takes, of which 16384 take 40 us).
// Shorter rows in more than 32 groups are done so too (32768 x 256 in 64 groups 582 us).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) select_long_kernel(SelectArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint64_t words[];
  const int E = a.r.E, G = a.groups, warps = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t *row = words + (size_t)warp * E;
  uint64_t *best = words + (size_t)warps * E + (size_t)warp * G;
  int32_t *index = (int32_t *)(words + (size_t)warps * (E + G)) + warp * 32;
  float *acc = (float *)(words + (size_t)warps * (E + G + 16));  // [warps, E]
  int32_t *cnt = (int32_t *)(acc + (size_t)warps * E);           // [E]
  float *mine = acc + (size_t)warp * E;
  const int r = blockIdx.y, n = a.r.ntok[r];
  for (int e = lane; e < E; e += 32) mine[e] = 0.0f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  for (int s = blockIdx.x * warps + warp; s < a.r.S; s += gridDim.x * warps) {
    const int64_t t = (int64_t)r * a.r.S + s;
    if (s >= n) {
      write_picks(a, true, 0, 0.0f, t, false, 0.0f, 0.0f, cnt);
      continue;
    }
    const T *z = (const T *)a.r.logits + t * E;
    select_exact(a, z, row, best, index);
    const int id = lane < a.r.K ? index[lane] : 0;
    const float m = row_max(z, E), inv = row_inverse(z, E, m, a.r.sigmoid);
    write_picks(a, a.r.sigmoid, id, to_f(z[id]), t, true, m, inv, cnt);
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
  if (E <= kInRegisters)  // the bias in whole lanes' columns, at most 512
    return ((size_t)kWarps * (E + 32 + G)) * 8 +
           (size_t)(E + kInRegisters + kWarps * kScratch) * 4;
  const size_t w = long_warps(E);
  return w * (E + G + 16) * 8 + (w + 1) * E * 4;
}

// Logits of a lane in the kernel of rows in registers: no more than need be (160
// experts in 8 groups of 20 take 27 us with five, whose lanes hold whole groups, and
// 33 with eight; 32768 x 192 in 8 groups of 24 40 us with six and 51 with eight, without
// groups 33 and 35; sizes whose groups are no lanes' whole columns about the same).
int per_lane(int E) {
  return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : E <= 160 ? 5 : E <= 192 ? 6
         : E <= 256 ? 8 : E <= 384 ? 12 : 16;
}

template <typename T, bool kSigmoid>
auto select_kernel_for(int V) {
  return V == 1 ? select_kernel<T, 1, kSigmoid> : V == 2 ? select_kernel<T, 2, kSigmoid>
         : V == 4 ? select_kernel<T, 4, kSigmoid> : V == 5 ? select_kernel<T, 5, kSigmoid>
         : V == 6 ? select_kernel<T, 6, kSigmoid> : V == 8 ? select_kernel<T, 8, kSigmoid>
         : V == 12 ? select_kernel<T, 12, kSigmoid> : select_kernel<T, 16, kSigmoid>;
}
template <typename T>
auto select_kernel_of(int E, bool sigmoid) {
  const int V = per_lane(E);
  return sigmoid ? select_kernel_for<T, true>(V) : select_kernel_for<T, false>(V);
}

template <typename T>
int run_select(moonep_ctx *ctx, SelectArgs &a, FinishArgs &f, int32_t *tpe, bool loss,
               cudaStream_t st) {
  const moonep_config &c = ctx->cfg;
  const bool reg = c.E <= kInRegisters;
  const int warps = reg ? kWarps : long_warps(c.E);
  const size_t smem = select_smem(c.E, a.groups);
  const auto kernel = select_kernel_of<T>(c.E, a.r.sigmoid);
  const void *fn = reg ? (const void *)kernel : (const void *)select_long_kernel<T>;
  cudaError_t e = smem > 48 * 1024 ? raise_dyn_smem(fn, (int)smem) : cudaSuccess;
  if (e != cudaSuccess) return cuda_status(e);
  // as the plain router: at most four blocks per SM, no more than num_sms SMs
  // hold, but one per rank; a power of two up to the cluster, then a multiple
  const int64_t held = reg ? blocks_in_cap(ctx, kernel, warps * 32, smem)
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
    e = launch_pdl_ex(kernel, grid, block, smem, st, false, a.r.cluster, a,
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
  a.size = c.E / sel.groups;
  const int V = per_lane(c.E), whole = a.size % V == 0 ? a.size / V : 0;
  a.held = whole > 0 && whole <= 32 && (whole & (whole - 1)) == 0;
  while (a.held ? 1 << a.lanes_log < whole : 2 * sel.groups << a.lanes_log <= 32) a.lanes_log++;
  a.turns = (a.size + (1 << a.lanes_log) - 1) >> a.lanes_log;
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
  const int blocks = (c.E + threads - 1) / threads;
  return cuda_status(launch_pdl(bias_kernel, dim3(blocks < ctx->sms ? blocks : ctx->sms),
                                dim3(threads), 0, st, false, a));
}

}  // namespace moonep
