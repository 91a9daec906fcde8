// The k experts of each row of logits, and the gradient of their weights.
//
//   score  = sigmoid(x), or exp(x - max) / sum of them        choice = score + bias
//   weight = scale score / (1, or the sum of the chosen scores)
//
// Without a bias the order of the choices is that of the logits.  With one it
// is that of 64-bit arithmetic: 42 bits of the choices are compared, and where
// these cannot tell the order of two and it matters, the chosen ones and the
// two behind them (or the groups' sums) are formed once more and compared whole.
//
// Renormalised weights are formed from exp(min(x, 0) - most) / (1 + exp(-|x|)),
// the scores times a common factor under which the largest does not underflow.
#include "mhc_experts.h"
#include "mhc_finish.h"

namespace mhc {

namespace {

constexpr int kWaves = 4;
constexpr float kLargest = 3.4028234663852886e38f;
constexpr float kLog2e = 1.4426950408889634f;

// A logit as it counts: NaN is minus infinity (no expert), plus infinity the
// largest number.
__device__ __forceinline__ float clean(float x) { return x != x ? -__builtin_inff() : fminf(x, kLargest); }
__device__ __forceinline__ float logit_at(const void *p, size_t i, bool bf16) {
  return clean(bf16 ? bf16_lo(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i]);
}
template <bool BF16>
__device__ __forceinline__ float logit_at(const void *p, size_t i) {
  return logit_at(p, i, BF16);
}

template <class T>
__device__ __forceinline__ T wave_total(T x) {
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}
template <class T>
__device__ __forceinline__ T wave_max(T x) {
  for (int d = 32; d > 0; d >>= 1) {
    const T y = __shfl_xor(x, d);
    x = y > x ? y : x;
  }
  return x;
}

// What a wave's lanes wrote to LDS is there for its other lanes (its LDS
// accesses keep their order; the compiler has to keep it too).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// -- lane moves -------------------------------------------------------------
//
// Partners of five and six doublings that need no LDS: lane ^ 1, lane ^ 2, the
// mirrored lane in eight and in sixteen (whose sets of lanes are those of
// lane ^ 4 and lane ^ 8 then), the other row of sixteen and the other half.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_mov_dpp((int)w[0], CTRL, 0xF, 0xF, false),
                                          (uint32_t)__builtin_amdgcn_mov_dpp((int)w[1], CTRL, 0xF, 0xF, false)});
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

template <class T>
struct Two {
  T a, b;
};
__device__ __forceinline__ Two<float> swap16(float x) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return {__uint_as_float(s[0]), __uint_as_float(s[1])};
}
__device__ __forceinline__ Two<float> swap32(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return {__uint_as_float(s[0]), __uint_as_float(s[1])};
}
__device__ __forceinline__ Two<double> swap16(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  const auto lo = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
  return {__builtin_bit_cast(double, u32x2{lo[0], hi[0]}), __builtin_bit_cast(double, u32x2{lo[1], hi[1]})};
}
__device__ __forceinline__ Two<double> swap32(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  const auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
  return {__builtin_bit_cast(double, u32x2{lo[0], hi[0]}), __builtin_bit_cast(double, u32x2{lo[1], hi[1]})};
}

// f over a row's L lanes; every one of them has it.
template <int L, class T, class F>
__device__ __forceinline__ T row_join(T x, F f) {
  x = f(x, dpp<kXor1>(x));
  x = f(x, dpp<kXor2>(x));
  x = f(x, dpp<kMirror8>(x));
  x = f(x, dpp<kMirror16>(x));
  if constexpr (L == 64) {
    const Two<T> s = swap16(x);
    x = f(s.a, s.b);
    const Two<T> t = swap32(x);
    x = f(t.a, t.b);
  }
  return x;
}
template <int L>
__device__ __forceinline__ double row_max(double x) {
  return row_join<L>(x, [](double a, double b) { return __builtin_fmax(a, b); });
}
template <int L>
__device__ __forceinline__ float row_max(float x) {
  return row_join<L>(x, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  return row_join<L>(x, [](float a, float b) { return a + b; });
}

// -- keys -------------------------------------------------------------------
//
// A key is the choice as a double whose ten lowest bits hold the index, so that
// one maximum compares the choices and, of equal ones, takes the lowest index.
constexpr int kIndexMask = kMaxExperts - 1;
constexpr double kNoKey = -1e300;  // below every choice

__device__ __forceinline__ double key_of(double choice, int index) {
  const u32x2 w = __builtin_bit_cast(u32x2, choice);
  const uint32_t low = (int)w[1] < 0 ? index : kIndexMask - index;
  return __builtin_bit_cast(double, u32x2{(w[0] & ~(uint32_t)kIndexMask) | low, w[1]});
}
__device__ __forceinline__ int index_of(double key) {
  const u32x2 w = __builtin_bit_cast(u32x2, key);
  const int low = w[0] & kIndexMask;
  return key == kNoKey ? -1 : (int)w[1] < 0 ? low : kIndexMask - low;
}
__device__ __forceinline__ double choice_of(double key) {
  const u32x2 w = __builtin_bit_cast(u32x2, key);
  return __builtin_bit_cast(double, u32x2{w[0] & ~(uint32_t)kIndexMask, w[1]});
}

// exp(x) to 2^-50 of its value, from 2^n exp(r), |r| <= ln 2 / 2, by the power
// series up to r^12 (the next term is below 2^-52); |x| beyond 700 counts as 700.
__device__ __forceinline__ double exp_64(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -700.0), 700.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  // ln 2 in two parts, the upper one with few enough bits for n times it to be exact
  const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, x));
  double p = 1.0 / 479001600.0;
  constexpr double kInverse[] = {1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720,
                                 1.0 / 120,      1.0 / 24,      1.0 / 6,      0.5,         1.0,        1.0};
#pragma unroll
  for (double c : kInverse) p = fma(p, r, c);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / x for x >= 1: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal_64(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(y, fma(-x, y, 1.0), y);
  return fma(y, fma(-x, y, 1.0), y);
}

// The choice of a score and its bias, within what keys hold; kNoKey for a bias
// that takes the expert out.
__device__ __forceinline__ double choice_of_score(double score, float b) {
  const double c = __builtin_fmin(score + (double)b, 1e299) + 0.0;  // (a zero without a sign)
  return c > -1e299 && b == b ? c : kNoKey;
}
__device__ __forceinline__ double key_of_choice(double score, float b, int index) {
  const double c = choice_of_score(score, b);
  return c == kNoKey ? kNoKey : key_of(c, index);
}

// Batcher's odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_keys(double (&x)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = x[i + j], b = x[i + j + q];
            x[i + j] = __builtin_fmax(a, b);
            x[i + j + q] = __builtin_fmin(a, b);
          }
}

// How near two choices may be before their keys cannot tell their order,
// relative to 1 + |choice|: a key's upper bits are off by 2^-42 of the choice,
// the scores by less than 2^-47; twice that for two, and twice for safety.
constexpr double kNear = 0x1p-40;

// The weight (without the scale) of a chosen logit, one a lane of a row's L;
// minus infinity where there is none.  top, all: the row's softmax.
template <int L>
__device__ __forceinline__ float weight_of(const RouteArgs &a, float x, float top, float all) {
  const bool is = x > -__builtin_inff();
  if (a.renorm) {
    const float most = row_max<L>(a.softmax ? x : fminf(x, 0.f));
    float e = 0.f;
    if (is) e = a.softmax ? expf(x - most) : expf(fminf(x, 0.f) - most) / (1.0f + expf(-fabsf(x)));
    const float sum = row_sum<L>(e);
    return is ? e / sum : 0.f;
  }
  return !is ? 0.f : a.softmax ? expf(x - top) / all : 1.0f / (1.0f + expf(-x));
}

constexpr int kAtOnce = 4;  // exponentials a lane works on at a time (all 16 take 216 registers)

struct RouteShape {
  int groups, size;  // groups that are chosen among (1: all experts), experts of one
  int lanes_log;     // lanes of a group: 1 << lanes_log
};

// L lanes take a row, V experts each: those of a group are neighbours, a
// group's lanes are too.  Each lane sorts its keys; then the largest of the
// lanes' first keys is taken k times, and twice more to see what is left out:
// KL >= min(V, k + 2) of a lane's keys can be among them.
template <int V, int KL, int L>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a, RouteShape g,
                                                            const void *__restrict__ logits,
                                                            const float *__restrict__ bias, int32_t *__restrict__ ids,
                                                            float *__restrict__ weights, uint32_t B) {
  extern __shared__ float shared[];  // each wave's rows of logits, then the bias
  constexpr int kRows = 64 / L;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), l = lane & (L - 1), r = lane / L;
  float *x_lds = shared + wave * kRows * a.E, *bias_lds = shared + kWaves * kRows * a.E;
  if (bias) {
    for (int i = threadIdx.x; i < a.E; i += 64 * kWaves) bias_lds[i] = bias[i];
    __syncthreads();
  }
  const float none = -__builtin_inff();
  const int group = l >> g.lanes_log;
  // Lanes start at different ones of their experts, so that their reads fall
  // on different LDS banks.
  const int turn = (L == 64 ? lane / (64 / V) : r + 4 * (l / (64 / V))) & (V - 1);
  const bool sums = a.softmax && (bias || !a.renorm);
  for (uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * kRows; first < B;
       first += (uint64_t)gridDim.x * kWaves * kRows) {
    const uint64_t row = first + r;
    const bool real = row < B;
    const int total = (int)(B - first < kRows ? B - first : kRows) * a.E;
    const float *x_row = x_lds + r * a.E;
    float x[V];
    if (a.bf16) {
      const uint16_t *from = static_cast<const uint16_t *>(logits) + first * a.E;
#pragma unroll
      for (int t = 0; t < V; ++t) x[t] = lane + 64 * t < total ? bf16_lo(from[lane + 64 * t]) : 0.f;
    } else {
      const float *from = static_cast<const float *>(logits) + first * a.E;
#pragma unroll
      for (int t = 0; t < V; ++t) x[t] = lane + 64 * t < total ? from[lane + 64 * t] : 0.f;
    }
#pragma unroll
    for (int t = 0; t < V; ++t)
      if (lane + 64 * t < total) x_lds[lane + 64 * t] = clean(x[t]);
    wave_lds_fence();
    int part = l & ((1 << g.lanes_log) - 1);
    asm volatile("" : "+v"(part));  // or the compiler keeps 64 registers of indexes and addresses over the rows
    const auto index_at = [&](int t) { return group * g.size + part * V + ((t + turn) & (V - 1)); };
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const bool there = real && group < g.groups && part * V + ((t + turn) & (V - 1)) < g.size;
      x[t] = there ? x_row[index_at(t)] : none;
    }
    float top = none;
    double all = 0.0, key[V];
    if (sums) {
#pragma unroll
      for (int t = 0; t < V; ++t) top = fmaxf(top, x[t]);
      top = row_max<L>(top);
#pragma unroll
      for (int t = 0; t < V; ++t) {
        key[t] = x[t] > none ? exp_64((double)x[t] - (double)top) : 0.0;
        all += key[t];
        if (t % kAtOnce == kAtOnce - 1) __builtin_amdgcn_sched_barrier(0);
      }
      all = row_join<L>(all, [](double p, double q) { return p + q; });
    }
    const double share = all > 0.0 ? reciprocal_64(all) : 0.0;
    if (bias) {
#pragma unroll
      for (int t = 0; t < V; ++t) {
        const double score = a.softmax ? key[t] * share : reciprocal_64(1.0 + exp_64(-(double)x[t]));
        key[t] = kNoKey;
        if (x[t] > none) key[t] = key_of_choice(score, bias_lds[index_at(t)], index_at(t));
        if (t % kAtOnce == kAtOnce - 1) __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int t = 0; t < V; ++t)
        key[t] = x[t] > none ? key_of((double)(x[t] + 0.0f), index_at(t)) : kNoKey;  // (a zero without a sign)
    }
    // A candidate's choice once more, with all of its bits.
    const auto whole = [&](double k) {
      const int e = index_of(k);
      if (e < 0) return kNoKey;
      const double z = x_row[e];
      return choice_of_score(a.softmax ? exp_64(z - (double)top) * share : reciprocal_64(1.0 + exp_64(-z)), bias_lds[e]);
    };
    sort_keys<V>(key);
    if (g.groups > 1) {
      // The group's two largest, joined over its lanes.
      double a0 = key[0], a1 = V > 1 ? key[V > 1 ? 1 : 0] : kNoKey;
      const auto join = [&](double b0, double b1) {
        a1 = __builtin_fmax(__builtin_fmin(a0, b0), __builtin_fmax(a1, b1));
        a0 = __builtin_fmax(a0, b0);
      };
      if (g.lanes_log > 0) join(dpp<kXor1>(a0), dpp<kXor1>(a1));
      if (g.lanes_log > 1) join(dpp<kXor2>(a0), dpp<kXor2>(a1));
      if (g.lanes_log > 2) join(dpp<kMirror8>(a0), dpp<kMirror8>(a1));
      if (g.lanes_log > 3) join(dpp<kMirror16>(a0), dpp<kMirror16>(a1));
      if constexpr (L == 64) {
        if (g.lanes_log > 4) {
          const Two<double> p = swap16(a0), q = swap16(a1);
          a0 = p.a, a1 = q.a;
          join(p.b, q.b);
        }
      }
      if (group >= g.groups) a0 = a1 = kNoKey;
      double rank = a0, size = 0.0;  // size: of the choices that a rank is the sum of
      if (bias && a0 != kNoKey) {
        const double c0 = choice_of(a0), c1 = a1 != kNoKey ? choice_of(a1) : 0.0;
        size = __builtin_fmax(__builtin_fabs(c0), __builtin_fabs(c1));
        rank = key_of(c0 + c1 + 0.0, group);
      }
      const double own = rank;
      bool kept = false;
      double last = kNoKey;
      for (int t = 0; t < a.top_groups; ++t) {
        last = row_max<L>(rank);
        if (rank == last) {
          kept = true;
          rank = kNoKey;
        }
      }
      if (bias) {
        const double next = row_max<L>(rank);
        if (__ballot(next != kNoKey && !(last - next > 4 * kNear * (1.0 + row_max<L>(size))))) {
          const double sum = own == kNoKey ? kNoKey : whole(a0) + (a1 != kNoKey ? whole(a1) : 0.0);
          int better = 0;  // groups before the own one
          for (int q = 0; q < g.groups; ++q) {
            const double other = __shfl(sum, (lane & ~(L - 1)) + (q << g.lanes_log));
            better += other > sum || (other == sum && q < group) ? 1 : 0;
          }
          kept = better < a.top_groups;
        }
      }
      if (!kept) {
#pragma unroll
        for (int t = 0; t < KL; ++t) key[t] = kNoKey;
      }
    }
    double chosen = kNoKey, best = kNoKey;  // of lane j: the j-th key
    const auto take = [&](int j) {
      best = row_max<L>(key[0]);
      const bool win = key[0] == best;
#pragma unroll
      for (int t = 0; t + 1 < KL; ++t) key[t] = win ? key[t + 1] : key[t];
      if (win) key[KL - 1] = kNoKey;
      if (l == j) chosen = best;
    };
    for (int j = 0; j < a.k; ++j) take(j);
    int id = index_of(chosen);
    if (bias) {
      // Keys next to each other that are too near, unless they come from the
      // same numbers.  Behind a pair that is too near at the border there may
      // be one more.
      const double edge = best;
      const auto close = [](double p, double q) {
        const double c = choice_of(p);
        return q != kNoKey && !(c - choice_of(q) > kNear * (1.0 + __builtin_fabs(c)));
      };
      take(a.k);
      if (__ballot(close(edge, best))) take(a.k + 1);
      id = index_of(chosen);
      const float z = id >= 0 ? x_row[id] : none, b = id >= 0 ? bias_lds[id] : 0.f;
      const double next = __shfl_down(chosen, 1);
      const bool same = z == __shfl_down(z, 1) && b == __shfl_down(b, 1);
      if (__ballot(l <= a.k && id >= 0 && close(chosen, next) && !same)) {
        const double c = whole(chosen);
        int better = 0;
        for (int q = 0; q < a.k + 2; ++q) {
          const double other = __shfl(c, (lane & ~(L - 1)) + q);
          const int e = __shfl(id, (lane & ~(L - 1)) + q);
          better += other > c || (other == c && (id < 0 ? q < l : e >= 0 && e < id)) ? 1 : 0;
        }
        const int to = (lane & ~(L - 1)) + (l < a.k + 2 ? better : l);
        id = __builtin_amdgcn_ds_permute(4 * to, id);
      }
    }
    const float w = weight_of<L>(a, l < a.k && id >= 0 ? x_row[id] : none, top, (float)all);
    if (real && l < a.k) {
      ids[row * a.k + l] = id;
      weights[row * a.k + l] = w * a.scale;
    }
    wave_lds_fence();  // the next rows' logits go where these were
  }
}

template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void route_bwd_kernel(RouteArgs a, const void *__restrict__ logits,
                                                                const int32_t *__restrict__ ids,
                                                                const float *__restrict__ dweights,
                                                                void *__restrict__ dlogits, uint32_t B) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float none = -__builtin_inff();
  for (uint64_t row = (uint64_t)blockIdx.x * kWaves + wave; row < B; row += (uint64_t)gridDim.x * kWaves) {
    int id = lane < a.k ? ids[row * a.k + lane] : -1;
    if (id >= a.E) id = -1;
    const float x = id >= 0 ? logit_at<BF16>(logits, row * a.E + id) : none;
    const float dw = id >= 0 ? a.scale * dweights[row * a.k + lane] : 0.f;
    float top = none, inv_total = 0.f, along = 0.f;
    float d = 0.f;  // the chosen logit's gradient (without -p along of the plain softmax)
    const bool every = a.softmax && !a.renorm;
    if (every) {
      for (int i = lane; i < a.E; i += 64) top = fmaxf(top, logit_at<BF16>(logits, row * a.E + i));
      top = wave_max(top);
      float total = 0.f;
      for (int i = lane; i < a.E; i += 64) {
        const float y = logit_at<BF16>(logits, row * a.E + i);
        total += y > none ? expf(y - top) : 0.f;
      }
      total = wave_total(total);
      inv_total = total > 0.f ? 1.0f / total : 0.f;
      const float p = x > none ? expf(x - top) * inv_total : 0.f;
      d = p * dw;
      along = wave_total(d);
    } else if (a.renorm) {
      const float z = !(x > none) ? none : a.softmax ? x : fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
      const float most = wave_max(z);
      const float e = z > none ? expf(z - most) : 0.f;
      const float total = wave_total(e);
      const float w = total > 0.f ? e / total : 0.f;
      d = w * (dw - wave_total(w * dw));
    } else {
      d = dw / (1.0f + expf(-x));
    }
    if (!a.softmax) d = x > none ? d / (1.0f + expf(x)) : 0.f;
    for (int i = lane; i - lane < a.E; i += 64) {
      float o = 0.f;
      if (every && i < a.E) {
        const float y = logit_at<BF16>(logits, row * a.E + i);
        o = y > none ? -expf(y - top) * inv_total * along : 0.f;
      }
      for (int j = 0; j < a.k; ++j) {
        const int e = __shfl(id, j);
        const float g = __shfl(d, j);
        if (e == i) o += g;
      }
      if (i >= a.E) continue;
      if constexpr (BF16)
        static_cast<uint16_t *>(dlogits)[row * a.E + i] = (uint16_t)pack_bf16x2(o, 0.f);
      else
        static_cast<float *>(dlogits)[row * a.E + i] = o;
    }
  }
}

uint32_t grid_of(int64_t rows_a_wg, int64_t B) {
  const int64_t wgs = (B + rows_a_wg - 1) / rows_a_wg;
  return (uint32_t)(wgs < (1 << 22) ? wgs : (1 << 22));
}

// Experts a lane, for L lanes a row: 0 where they are not enough.
int experts_a_lane(int L, const RouteArgs &a, RouteShape *g) {
  g->groups = a.top_groups < a.groups ? a.groups : 1;
  g->size = a.E / g->groups;
  if (g->groups > L) return 0;
  g->lanes_log = 0;
  while ((g->groups << (g->lanes_log + 1)) <= L) ++g->lanes_log;
  const int each = (g->size + (1 << g->lanes_log) - 1) >> g->lanes_log;
  int v = 1;
  while (v < each) v *= 2;
  return v;
}

constexpr int64_t kManyRows = 2048;

template <int V, int KL, int L>
hipError_t launch_route_t(int64_t B, const RouteArgs &a, const RouteShape &g, const void *logits, const float *bias,
                          int32_t *ids, float *weights, hipStream_t st) {
  constexpr int kRows = 64 / L;
  const size_t lds = (size_t)(kWaves * kRows + (bias ? 1 : 0)) * a.E * sizeof(float);
  route_kernel<V, KL, L><<<grid_of(kWaves * kRows, B), 64 * kWaves, lds, st>>>(a, g, logits, bias, ids, weights,
                                                                              (uint32_t)B);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(int64_t B, const RouteArgs &a, const void *logits, const float *bias, int32_t *ids,
                        float *weights, hipStream_t st) {
  RouteShape g;
  const int v = experts_a_lane(16, a, &g);
  const auto go = [&](auto kernel) { return kernel(B, a, g, logits, bias, ids, weights, st); };
  if (v > 0 && v <= 16 && a.k <= 14 && B >= kManyRows) {
    switch (v) {
      case 1: return go(launch_route_t<1, 1, 16>);
      case 2: return go(launch_route_t<2, 2, 16>);
      case 4: return go(launch_route_t<4, 4, 16>);
      case 8: return go(launch_route_t<8, 8, 16>);
      default: return a.k <= 8 ? go(launch_route_t<16, 10, 16>) : go(launch_route_t<16, 16, 16>);
    }
  }
  switch (experts_a_lane(64, a, &g)) {
    case 1: return go(launch_route_t<1, 1, 64>);
    case 2: return go(launch_route_t<2, 2, 64>);
    case 4: return go(launch_route_t<4, 4, 64>);
    case 8: return go(launch_route_t<8, 8, 64>);
    case 16: return a.k <= 8 ? go(launch_route_t<16, 10, 64>) : go(launch_route_t<16, 16, 64>);
    case 32: return a.k <= 8 ? go(launch_route_t<32, 10, 64>) : go(launch_route_t<32, 32, 64>);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_route_bwd(int64_t B, const RouteArgs &a, const void *logits, const int32_t *ids,
                            const float *dweights, void *dlogits, hipStream_t st) {
  const uint32_t grid = grid_of(kWaves, B);
  if (a.bf16)
    route_bwd_kernel<true><<<grid, 64 * kWaves, 0, st>>>(a, logits, ids, dweights, dlogits, (uint32_t)B);
  else
    route_bwd_kernel<false><<<grid, 64 * kWaves, 0, st>>>(a, logits, ids, dweights, dlogits, (uint32_t)B);
  return hipGetLastError();
}

}  // namespace mhc
