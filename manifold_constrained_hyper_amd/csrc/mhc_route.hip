// The k experts of each row of logits, and the gradient of their weights.
//
//   score  = sigmoid(x), or exp(x - max) / sum of them        choice = score + bias
//   weight = scale score / (1, or the sum of the chosen scores)
//
// Without a bias the order of the choices is that of the logits.  With one it
// is that of 64-bit arithmetic: 42 bits of the choices are compared, and where
// these cannot tell the order of two and it matters, the chosen ones and the one
// behind them (all of them where two behind are as near, and the groups' sums)
// are formed once more and compared whole.
//
// Bound by vector instructions, mostly: 1437 a wave of four rows of 256 experts
// in eight groups, of which the scores in 64 bits are a quarter, keys, sort and the
// k maxima half.  Four waves a SIMD keep it at them for 71 % of the time that a CU
// is busy (89 % of a wave's life); the rest is start, first loads and tail.  13.9
// us a call at B=16384 (17.8 MB).  By inputs, in a replayed graph: fp32 logits
// 14.8 (9.2 without a bias), bf16 16.5 (10.7), bf16 and a bias of zeros 24 (groups
// as good as each other in some rows), all logits equal 28.  One row takes 5.2.
//
// Renormalised weights are formed from exp(min(x, 0) - most) / (1 + exp(-|x|)),
// the scores times a common factor under which the largest does not underflow.
// Weights are formed in 64 bits and rounded once.
#include "mhc_experts.h"
#include "mhc_finish.h"

namespace mhc {

namespace {

constexpr int kWaves = 4;
constexpr float kLargest = 3.4028234663852886e38f;
constexpr float kLog2e = 1.4426950408889634f;

// A logit as it counts: NaN is minus infinity (no expert), plus infinity the
// largest number.
__device__ __forceinline__ float clean(float x) {
  return fminf(fmaxf(x, -__builtin_inff()), kLargest);  // (the maximum of a NaN and a number is the number)
}
__device__ __forceinline__ float logit_at(const void *p, size_t i, bool bf16) {
  return clean(bf16 ? bf16_lo(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i]);
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
  if constexpr (L >= 32) {
    const Two<T> s = swap16(x);
    x = f(s.a, s.b);
  }
  if constexpr (L == 64) {
    const Two<T> s = swap32(x);
    x = f(s.a, s.b);
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
constexpr double kNoKey = -1e300;  // below every choice; with an index in it, it is one still
__device__ __forceinline__ bool is_key(double key) { return key > -1e299; }

__device__ __forceinline__ double key_of(double choice, int index) {
  const u32x2 w = __builtin_bit_cast(u32x2, __builtin_fmax(choice, kNoKey));
  const uint32_t low = (int)w[1] < 0 ? index : index ^ kIndexMask;
  return __builtin_bit_cast(double, u32x2{(w[0] & ~(uint32_t)kIndexMask) | low, w[1]});
}
__device__ __forceinline__ int index_of(double key) {
  const u32x2 w = __builtin_bit_cast(u32x2, key);
  const int low = w[0] & kIndexMask;
  return !is_key(key) ? -1 : (int)w[1] < 0 ? low : low ^ kIndexMask;
}
__device__ __forceinline__ double choice_of(double key) {
  const u32x2 w = __builtin_bit_cast(u32x2, key);
  return __builtin_bit_cast(double, u32x2{w[0] & ~(uint32_t)kIndexMask, w[1]});
}

// exp of each x, |x| <= 1000, from 2^n exp(r), |r| <= ln 2 / 2, by the power
// series up to r^TERMS: to 2^-50 of its value with 12 terms (the next one is
// below 2^-52), to 2^-36 with 9.  N of them go step by step, as each is a chain
// of dependent products.
__constant__ const double kInverse[] = {1.0,           1.0,            0.5,        1.0 / 6,     1.0 / 24,
                                        1.0 / 120,     1.0 / 720,      1.0 / 5040, 1.0 / 40320, 1.0 / 362880,
                                        1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
// HERE: the constants are formed where they are used; or the compiler keeps them
// in vector registers over the rows (133 of them, and three waves a SIMD, for the
// weights of sixteen experts a lane).
template <bool HERE>
__device__ __forceinline__ double constant(double c) {
  if constexpr (HERE) asm volatile("" : "+s"(c));
  return c;
}
template <int TERMS, bool HERE = false, int N>
__device__ __forceinline__ void exp_64(double (&x)[N]) {
  constexpr double kShift = 0x1.8p52;  // a number added to it is rounded to an integer in the low bits
  double n[N], p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] = fma(x[i], constant<HERE>(1.4426950408889634), kShift);
  int e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    e[i] = (int)__builtin_bit_cast(u32x2, n[i])[0];
    n[i] -= kShift;
  }
  // The reduction of Cody and Waite: ln 2 = kHigh + kLow, kHigh its first 42 bits, so
  // that n times it is exact for n of 11.
  constexpr double kHigh = 0x1.62e42fefa38p-1, kLow = 0x1.ef35793c7673p-45;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fma(n[i], constant<HERE>(-kHigh), x[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fma(n[i], constant<HERE>(-kLow), x[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = constant<HERE>(kInverse[TERMS]);
  constexpr int kStep = TERMS > 9 ? 1 : TERMS;  // (few rows come to the long series: its constants stay in memory)
#pragma unroll kStep
  for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], x[i], constant<HERE>(kInverse[t]));
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __builtin_amdgcn_ldexp(p[i], e[i]);
}
// 1 / x for x >= 1 to 2^-47: the hardware's estimate, to 2^-24, and a Newton
// step, which squares its error.
template <int N>
__device__ __forceinline__ void reciprocal_64(double (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double y = __builtin_amdgcn_rcp(x[i]);
    x[i] = fma(y, fma(-x[i], y, 1.0), y);
  }
}
// WHOLE: to all 64 bits, down to 0; else to 2^-35, and none below exp(-700).
template <bool WHOLE, bool HERE = false, int N>
__device__ __forceinline__ void sigmoid_64(const float (&x)[N], double (&s)[N]) {
  constexpr float kFar = WHOLE ? 1000.0f : 700.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = -(double)__builtin_amdgcn_fmed3f(x[i], -kFar, kFar);
  exp_64<WHOLE ? 12 : 9, HERE>(s);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] += 1.0;
  if constexpr (WHOLE) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 1.0 / s[i];
  } else {
    reciprocal_64(s);
  }
}
// exp(x - top) for x <= top, 0 for minus infinity.
template <bool WHOLE, bool HERE = false, int N>
__device__ __forceinline__ void exp_from(const float (&x)[N], float top, double (&e)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = __builtin_fmax((double)x[i] - (double)top, WHOLE ? -1000.0 : -700.0);
  exp_64<WHOLE ? 12 : 9, HERE>(e);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = x[i] > -__builtin_inff() ? e[i] : 0.0;
}
constexpr int kAtOnce = 2;

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
// relative to 1 + |choice|: the scores are off by less than 2^-35 (of the
// softmax's share of its sum too), a key's upper bits by 2^-42 of the choice;
// twice that for two, and twice for safety.
constexpr double kNear = 0x1p-33;

// The weight (without the scale) of a chosen logit, one a lane of a row's L;
// minus infinity where there is none.  top, all: the row's softmax.  In 64 bits
// to 2^-33, as weights are rounded once, with the scale: in 32 they were off by
// up to three roundings, and sigmoids and shares below 2^-126 were lost before
// the scale came to them.  (An IEEE division: a single weight is 1.)
template <int L>
__device__ __forceinline__ double weight_of(const RouteArgs &a, float x, float top, double all) {
  const bool is = x > -__builtin_inff();
  double w;
  if (a.renorm) {
    const float z[1] = {a.softmax ? x : fminf(x, 0.f)};
    const float most = row_max<L>(z[0]);
    double e[1];
    exp_from<false, true>(z, most, e);
    if (!a.softmax) {
      const float y[1] = {fabsf(x)};
      double s[1];
      sigmoid_64<false, true>(y, s);
      e[0] *= s[0];
    }
    w = e[0] / row_join<L>(is ? e[0] : 0.0, [](double p, double q) { return p + q; });
  } else if (a.softmax) {
    const float z[1] = {x};
    double e[1];
    exp_from<false, true>(z, top, e);
    w = e[0] / all;
  } else {
    const float z[1] = {x};
    double s[1];
    sigmoid_64<false, true>(z, s);
    w = s[0];
  }
  return is ? w : 0.0;
}

struct RouteShape {
  int groups, size;  // groups that are chosen among (1: all experts), experts of one
  int lanes_log;     // lanes of a group: 1 << lanes_log
  uint32_t inverse;  // 2^20 / size, rounded up: (i * inverse) >> 20 is i / size for i < 1024; 0 where group q's
                     // lanes follow on those of q - 1 without a gap, and the groups need not be told apart
};

// A lane's V values in LDS are neighbours, and lanes are apart by as much as
// lets sixteen of them read 16 bytes each without sharing a bank.
template <int V>
struct Slots {
  static constexpr int kPad = V > 4 ? 4 : 0, kApart = V + kPad;
};

// The sorted keys of a lane: two in registers and, where there are 8 to 10, the
// others in LDS (a list that is moved up in registers takes two instructions a
// key and choice: 17.2 us, not 15.3, at B=16384, E=256), else all in registers.  A list
// that can be used up ends with no key; one of k + 2 keys cannot.
template <int V, int KL>
struct List {
  static constexpr bool kInLds = KL >= 8 && KL <= 10;
  static constexpr int kRows = !kInLds ? 0 : KL == V ? KL - 1 : KL - 2;  // of 64 lanes
};
template <int V>
__device__ __forceinline__ void read_slots(const float *from, float (&x)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int t = 0; t < V; t += 4) {
      const f32x4 w = *reinterpret_cast<const f32x4 *>(from + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[t + i] = w[i];
    }
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) x[t] = from[t];
  }
}

// L lanes take a row, V experts each: those of a group are neighbours, a
// group's lanes are too.  Each lane sorts its keys; then the largest of the
// lanes' first keys is taken k times, and twice more to see what is left out:
// KL >= min(V, k + 2) of a lane's keys can be among them.
template <int V, int KL, int L>
__global__ __launch_bounds__(64 * kWaves, V <= 16 ? 3 : 2) void route_kernel(
    RouteArgs a, RouteShape g, const void *__restrict__ logits, const float *__restrict__ bias,
    int32_t *__restrict__ ids, float *__restrict__ weights, uint32_t B) {
  // Each wave's rows of logits and the bias, where the lanes find them.  A
  // lane's places without an expert hold minus infinity.
  extern __shared__ __attribute__((aligned(16))) float shared[];
  constexpr bool kInLds = List<V, KL>::kInLds;
  constexpr int kRows = 64 / L, kPad = Slots<V>::kPad, kApart = Slots<V>::kApart, kRowSize = L * kApart;
  const int wave = uniform((int)threadIdx.x >> 6);
  constexpr int kList = List<V, KL>::kRows * 64;  // (a read past a wave's list is one of what follows, and not used)
  double *list = reinterpret_cast<double *>(shared) + wave * kList;
  float *rows_lds = shared + 2 * kWaves * kList, *x_lds = rows_lds + wave * kRows * kRowSize;
  float *bias_lds = rows_lds + kWaves * kRows * kRowSize;
  const auto place = [&](uint32_t i) {  // of a row's expert i
    const uint32_t q = __umul24(i, g.inverse) >> 20, e = i - __umul24(q, (uint32_t)g.size);
    return e + kPad * (e / V) + q * (uint32_t)(kApart << g.lanes_log);
  };
  const float none = -__builtin_inff();
  if (bias) {
    for (int i = threadIdx.x; i < a.E; i += 64 * kWaves) bias_lds[place(i)] = clean(bias[i]);
    __syncthreads();
  }
  const bool full = a.E == L * V && g.inverse == 0;
  if (!full) {
#pragma unroll
    for (int t = 0; t < V; ++t) x_lds[(threadIdx.x & 63) * kApart + t] = none;
    wave_lds_fence();
  }
  const bool sums = a.softmax && (bias || !a.renorm);
  for (uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * kRows; first < B;
       first += (uint64_t)gridDim.x * kWaves * kRows) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // or the compiler keeps 64 registers of indexes and addresses over the rows
    const int l = lane & (L - 1), r = lane / L, group = l >> g.lanes_log;
    const int base = group * g.size + (l & ((1 << g.lanes_log) - 1)) * V;  // the lane's first expert
    const uint64_t row = first + r;
    const bool real = row < B;
    float *x_row = x_lds + r * kRowSize;
    const float *x_own = x_lds + lane * kApart, *bias_own = bias_lds + l * kApart;
    float x[V];
    if (L * V >= 64 && full && !a.bf16 && B - first >= kRows) {
      const float *from = static_cast<const float *>(logits) + first * a.E;
      float *to = x_lds + lane + kPad * (lane / V);
#pragma unroll
      for (int t = 0; t < V; ++t) x[t] = from[lane + 64 * t];
#pragma unroll
      for (int t = 0; t < V; ++t) to[64 / V * t * kApart] = clean(x[t]);
    } else {
      // (Lanes behind the last expert take it too, and write it where it is.)
      const size_t begin = (real ? row : first) * a.E;
      const auto at = [&](int t) { return min(l + L * t, a.E - 1); };
      if (a.bf16) {
        const uint16_t *from = static_cast<const uint16_t *>(logits) + begin;
#pragma unroll
        for (int t = 0; t < V; ++t) x[t] = bf16_lo(from[at(t)]);
      } else {
        const float *from = static_cast<const float *>(logits) + begin;
#pragma unroll
        for (int t = 0; t < V; ++t) x[t] = from[at(t)];
      }
#pragma unroll
      for (int t = 0; t < V; ++t) x_row[place(at(t))] = real ? clean(x[t]) : none;
    }
    wave_lds_fence();
    read_slots<V>(x_own, x);
    float top = none;
    double all = 0.0, key[V];
    constexpr int kN = V < kAtOnce ? V : kAtOnce;
    // f(x, key) for kN experts at a time.
    const auto by_parts = [&](auto f) {
#pragma unroll
      for (int t = 0; t < V; t += kN) {
        float z[kN];
        double k[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) z[i] = x[t + i];
        f(z, k);
#pragma unroll
        for (int i = 0; i < kN; ++i) key[t + i] = k[i];
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (sums) {
#pragma unroll
      for (int t = 0; t < V; ++t) top = fmaxf(top, x[t]);
      top = row_max<L>(top);
      by_parts([&](const float(&z)[kN], double(&k)[kN]) {
        exp_from<false>(z, top, k);
#pragma unroll
        for (int i = 0; i < kN; ++i) all += k[i];
      });
      all = row_join<L>(all, [](double p, double q) { return p + q; });
    }
    if (bias) {
      if (a.softmax) {
        double share[1] = {__builtin_fmax(all, 1.0)};  // (the largest term of the sum is 1)
        reciprocal_64(share);
#pragma unroll
        for (int t = 0; t < V; ++t) key[t] *= share[0];
      } else {
        by_parts([&](const float(&z)[kN], double(&k)[kN]) { sigmoid_64<false>(z, k); });
      }
      float b[V];
      read_slots<V>(bias_own, b);
#pragma unroll
      for (int t = 0; t < V; ++t) key[t] = key_of(key[t] + (double)(x[t] > none ? b[t] : none), base + t);
    } else {
#pragma unroll
      for (int t = 0; t < V; ++t) key[t] = key_of((double)(x[t] + 0.0f), base + t);  // (a zero without a sign)
    }
    // An expert's choice once more, with all of its bits, and the softmax's sum
    // that it needs (a loop: few rows come here).
    const auto whole_sum = [&]() {
      if (!a.softmax) return 1.0;
      double sum = 0.0;
#pragma unroll 1
      for (int t = 0; t < V; ++t) {
        const float z[1] = {x_own[t]};
        double c[1];
        exp_from<true>(z, top, c);
        sum += c[0];
      }
      return __builtin_fmax(row_join<L>(sum, [](double p, double q) { return p + q; }), 1.0);
    };
    const auto whole = [&](float x, float b, double sum) {
      const float z[1] = {x};
      double c[1];
      if (!a.softmax) {
        sigmoid_64<true>(z, c);
      } else {
        exp_from<true>(z, top, c);
        c[0] /= sum;
      }
      return x > none && b > none ? c[0] + (double)b : kNoKey;
    };
    sort_keys<V>(key);
    bool kept = true;
    if (g.groups > 1) {
      // The group's two largest, joined over its lanes.
      const auto join_lanes = [&](double &a0, double &a1) {
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
      };
      double a0 = key[0], a1 = V > 1 ? key[V > 1 ? 1 : 0] : kNoKey;
      join_lanes(a0, a1);
      if (group >= g.groups) a0 = a1 = kNoKey;
      double rank = a0, size = 0.0;  // size: of the choices that a rank is the sum of
      if (bias && is_key(a0)) {
        const double c0 = choice_of(a0), c1 = is_key(a1) ? choice_of(a1) : 0.0;
        size = __builtin_fmax(__builtin_fabs(c0), __builtin_fabs(c1));
        rank = key_of(c0 + c1, group);
      }
      kept = false;
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
        if (__ballot(is_key(next) && !(last - next > 4 * kNear * (1.0 + row_max<L>(size))))) {
          const double all_64 = whole_sum();
          a0 = a1 = kNoKey;
#pragma unroll 1
          for (int t = 0; t < V; ++t) {
            const double c = whole(x_own[t], bias_own[t], all_64);
            a1 = __builtin_fmax(a1, __builtin_fmin(a0, c));
            a0 = __builtin_fmax(a0, c);
          }
          join_lanes(a0, a1);
          const double sum = a0 + (is_key(a1) ? a1 : 0.0);
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
        for (int t = 0; t < (kInLds ? 1 : KL); ++t) key[t] = kNoKey;
      }
    }
    const double *next_key = list + lane;
    if constexpr (kInLds) {
#pragma unroll
      for (int t = 2; t < KL; ++t) list[64 * (t - 2) + lane] = key[t];
      if constexpr (KL == V) list[64 * (KL - 2) + lane] = kNoKey;
    }
    double chosen = kNoKey, best = kNoKey;  // of lane j: the j-th key
    const auto take = [&](int j) {
      best = row_max<L>(key[0]);
      const bool win = key[0] == best && is_key(best);
      if constexpr (kInLds) {
        if (win) {
          key[0] = key[1];
          key[1] = *next_key;
          next_key += 64;
        }
      } else {
#pragma unroll
        for (int t = 0; t + 1 < KL; ++t) key[t] = win ? key[t + 1] : key[t];
        if (win) key[KL - 1] = kNoKey;
      }
      if (l == j) chosen = best;
    };
    for (int j = 0; j < a.k; ++j) take(j);
    int id = index_of(chosen);
    if (bias) {
      // Keys next to each other that are too near, unless they come from the
      // same numbers.
      const double edge = best;
      const auto close = [](double p, double q) {
        const double c = choice_of(p);
        return is_key(q) && !(c - choice_of(q) > kNear * (1.0 + __builtin_fabs(c)));
      };
      take(a.k);
      bool many = false;  // that are too near at the border
      if (__ballot(close(edge, best))) {
        take(a.k + 1);
        const bool crowd = close(edge, best);
        if (__ballot(crowd)) {
          // Equal numbers are in the order of their indexes already (zeros at
          // the start of a training, logits in bf16); in 32 bits a score is off
          // by less than 2^-20.
          const uint32_t e0 = crowd ? place(index_of(edge)) : 0;
          const float z0 = x_row[e0], b0 = bias_lds[e0];
          const auto choice = [&](float z, float b) {
            return b + (a.softmax ? __builtin_amdgcn_exp2f((z - top) * kLog2e) * __builtin_amdgcn_rcpf((float)all)
                                  : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e)));
          };
          const float c0 = choice(z0, b0), far = 0x1p-18f * (1.0f + fabsf(c0));
          bool other = false;
#pragma unroll 4
          for (int t = 0; t < V; ++t) {
            const float z = x_own[t], b = bias_own[t];
            other |= z > none && !(z == z0 && b == b0) && fabsf(choice(z, b) - c0) < far;
          }
          many = __ballot(crowd && kept && other);
        }
      }
      id = index_of(chosen);
      const uint32_t at_id = id >= 0 ? place(id) : 0;
      const float z = id >= 0 ? x_row[at_id] : none, b = id >= 0 ? bias_lds[at_id] : 0.f;
      const double next = __shfl_down(chosen, 1);
      const bool same = z == __shfl_down(z, 1) && b == __shfl_down(b, 1);
      if (many) {
        const double all_64 = whole_sum();
#pragma unroll 1
        for (int t = 0; t < V; ++t) {  // (key t comes in at the end and moves up to its place)
          const double c = whole(kept ? x_own[t] : none, bias_own[t], all_64);
#pragma unroll
          for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
          key[V - 1] = c;
        }
        for (int j = 0; j < a.k; ++j) {
          double most = kNoKey;
          int at = kMaxExperts;
#pragma unroll
          for (int t = 0; t < V; ++t) {
            const bool ahead = key[t] > most;
            most = ahead ? key[t] : most;
            at = ahead ? base + t : at;
          }
          const double first_of = row_max<L>(most);
          at = -(int)row_max<L>(most == first_of ? -(float)at : none);
#pragma unroll
          for (int t = 0; t < V; ++t) key[t] = base + t == at ? kNoKey : key[t];
          if (l == j) id = is_key(first_of) ? at : -1;
        }
      } else if (__ballot(l <= a.k && id >= 0 && close(chosen, next) && !same)) {
        const double c = whole(z, b, whole_sum());
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
    const double w = weight_of<L>(a, l < a.k && id >= 0 ? x_row[place(id)] : none, top, all);
    if (real && l < a.k) {
      ids[row * a.k + l] = id;
      weights[row * a.k + l] = (float)(w * (double)a.scale);
    }
    wave_lds_fence();  // the next rows' logits go where these were
  }
}

// exp(x) for x <= 0 to 4 roundings; 0 below 2^-126.  The product h = x log2 e is
// off by up to |x| of them, which the factor 1 + (x - h ln 2) makes good, ln 2 in
// two parts (expf took 6.7 us for 6.1 at B=16383, E=100 in bf16).
__device__ __forceinline__ float exp_32(float x) {
  x = fmaxf(x, -200.0f);
  const float h = x * kLog2e, e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, fmaf(h, 1.9046542e-9f, fmaf(h, -0.69314718f, x)), e);
}

// -- gradient ---------------------------------------------------------------
//
//   softmax          dx_i = p_i (dw_i - sum p dw)           over all experts
//   renormalised     dz_j = w_j (dw_j - sum w dw)           over the chosen ones
//   sigmoid          dx_j = dz_j (1 - sigmoid(x_j)), dz_j = sigmoid(x_j) dw_j if
//                    not renormalised
//
// In fp32.  Sigmoids on either side of 0 are formed from exp(-|x|), and the chosen
// ones' shares by expf, so that they have a gradient below 2^-126 too.
//
// L lanes take a row and form its gradient in LDS (the chosen ones' parts are
// added to zeros or to the softmax's), which leaves in memory order, V values a
// lane.  B=16383, E=100, k=6, softmax in bf16: 6.1 us (6.9 MB, and a launch is
// 3.4).
template <int V, int L>
__global__ __launch_bounds__(64 * kWaves) void route_bwd_kernel(RouteArgs a, const void *__restrict__ logits,
                                                                const int32_t *__restrict__ ids,
                                                                const float *__restrict__ dweights,
                                                                void *__restrict__ dlogits, uint32_t B, bool pairs) {
  extern __shared__ float shared[];
  constexpr int kRows = 64 / L;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), l = lane & (L - 1), r = lane / L;
  float *out = shared + wave * kRows * a.E, *out_row = out + r * a.E;
  const float none = -__builtin_inff();
  const bool every = a.softmax && !a.renorm;
  for (uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * kRows; first < B;
       first += (uint64_t)gridDim.x * kWaves * kRows) {
    const uint64_t row = first + r;
    const bool real = row < B, slot = real && l < a.k;
    const int total = (int)(B - first < kRows ? B - first : kRows) * a.E;
    int id = slot ? ids[row * a.k + l] : -1;
    if (id >= a.E) id = -1;
    const float given = slot ? dweights[row * a.k + l] : 0.f;
    const float x = id >= 0 ? logit_at(logits, row * a.E + id, a.bf16) : none;
    const float dw = x > none ? a.scale * given : 0.f;  // (a masked expert's weight is 0 whatever its gradient)
    float d;  // the chosen logit's part
    if (every) {
      float y[V];
#pragma unroll
      for (int t = 0; t < V; ++t)
        y[t] = lane + 64 * t < total ? logit_at(logits, first * a.E + lane + 64 * t, a.bf16) : none;
#pragma unroll
      for (int t = 0; t < V; ++t)
        if (lane + 64 * t < total) out[lane + 64 * t] = y[t];
      wave_lds_fence();
      float top = none, all = 0.f;
#pragma unroll
      for (int t = 0; t < V; ++t) {
        y[t] = real && l + L * t < a.E ? out_row[l + L * t] : none;
        top = fmaxf(top, y[t]);
      }
      top = row_max<L>(top);
#pragma unroll
      for (int t = 0; t < V; ++t) {
        y[t] = exp_32(y[t] - top);  // (0 where there is no expert)
        all += y[t];
      }
      all = row_sum<L>(all);
      const float share = all > 0.f ? 1.0f / all : 0.f;
      d = x > none ? expf(x - top) * share * dw : 0.f;
      const float along = row_sum<L>(d) * share;
      wave_lds_fence();
#pragma unroll
      for (int t = 0; t < V; ++t)
        if (real && l + L * t < a.E) out_row[l + L * t] = -y[t] * along;
    } else {
#pragma unroll
      for (int t = 0; t < V; ++t)
        if (lane + 64 * t < total) out[lane + 64 * t] = 0.f;
      const float u = expf(-fabsf(x)), near = 1.0f / (1.0f + u);  // the sigmoid of |x|; that of -|x| is u near
      float w;
      if (a.renorm) {
        const float z = a.softmax ? x : fminf(x, 0.f), most = row_max<L>(z);
        float e = 0.f;
        if (x > none) e = a.softmax ? expf(z - most) : expf(z - most) * near;
        const float sum = row_sum<L>(e);
        w = x > none ? e / sum : 0.f;
      } else {
        w = x > none ? (x < 0.f ? u * near : near) : 0.f;
      }
      d = w * dw;
      if (a.renorm) d = w * (dw - row_sum<L>(d));
      if (!a.softmax) d *= x < 0.f ? near : u * near;
      if (!(x > none)) d = 0.f;
    }
    // An expert that was given twice: the first of its lanes adds all parts.
    bool lead = id >= 0;
    float part = 0.f;
    for (int q = 0; q < a.k; ++q) {
      const int e = __shfl(id, (lane & ~(L - 1)) + q);
      const float other = __shfl(d, (lane & ~(L - 1)) + q);
      if (e == id) part += other;
      if (e == id && q < l) lead = false;
    }
    wave_lds_fence();
    if (lead) out_row[id] += part;
    wave_lds_fence();
    if (!a.bf16) {
      float *to = static_cast<float *>(dlogits) + first * a.E;
#pragma unroll
      for (int t = 0; t < V; ++t)
        if (lane + 64 * t < total) to[lane + 64 * t] = out[lane + 64 * t];
    } else {
      uint16_t *to = static_cast<uint16_t *>(dlogits) + first * a.E;
      const int even = pairs ? total & ~1 : 0;
      for (int i = 2 * lane; i < even; i += 128)
        *reinterpret_cast<uint32_t *>(to + i) = pack_bf16x2(out[i], out[i + 1]);
      for (int i = even + lane; i < total; i += 64) to[i] = (uint16_t)pack_bf16x2(out[i], 0.f);
    }
    wave_lds_fence();  // the next rows go where these were
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
  const bool close = g->groups == 1 || g->size == v << g->lanes_log;
  g->inverse = close ? 0 : ((1u << 20) + g->size - 1) / g->size;
  return v;
}

// Waves that have a SIMD each.  Two rows share a wave where there are more of
// them than that, and four where there are more than twice as many: a wave's
// chain of dependent steps is what few rows take (E=256 in eight groups, k=8,
// softmax, us with 1, 2 and 4 rows a wave: 6.7, 7.0, 8.1 at 1024 rows; 7.8, 7.1,
// 8.1 at 2048; -, 8.6, 8.1 at 2560).
constexpr int64_t kSimds = 1024;

template <int V, int KL, int L>
hipError_t launch_route_t(int64_t B, const RouteArgs &a, const RouteShape &g, const void *logits, const float *bias,
                          int32_t *ids, float *weights, hipStream_t st) {
  constexpr int kRows = 64 / L;
  const size_t lds = (size_t)(kWaves * kRows + (bias ? 1 : 0)) * L * Slots<V>::kApart * sizeof(float) +
                     (size_t)kWaves * List<V, KL>::kRows * 64 * sizeof(double);
  route_kernel<V, KL, L><<<grid_of(kWaves * kRows, B), 64 * kWaves, lds, st>>>(a, g, logits, bias, ids, weights,
                                                                              (uint32_t)B);
  return hipGetLastError();
}

// Rows from which several share a wave of the gradient (E=256 in fp32, us with
// four a wave and one: 4.9 against 4.3 at 2048 rows, 5.2 against 5.0 at 4096,
// 6.1 against 7.0 at 8192, 9.1 against 11.3 at 16384).
constexpr int64_t kManyRowsBwd = 4096;

template <int V, int L>
hipError_t launch_route_bwd_t(int64_t B, const RouteArgs &a, const void *logits, const int32_t *ids,
                              const float *dweights, void *dlogits, hipStream_t st) {
  constexpr int kRows = 64 / L;
  // Pairs of bf16 are stored together where every wave's rows begin at four bytes.
  const bool pairs = kRows * a.E % 2 == 0 && reinterpret_cast<uintptr_t>(dlogits) % 4 == 0;
  route_bwd_kernel<V, L><<<grid_of(kWaves * kRows, B), 64 * kWaves, (size_t)kWaves * kRows * a.E * sizeof(float), st>>>(
      a, logits, ids, dweights, dlogits, (uint32_t)B, pairs);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(int64_t B, const RouteArgs &a, const void *logits, const float *bias, int32_t *ids,
                        float *weights, hipStream_t st) {
  RouteShape g;
  const auto go = [&](auto kernel) { return kernel(B, a, g, logits, bias, ids, weights, st); };
  // k + 2 lanes of a row hold what is chosen and the next.  With k above 8 the
  // lists of 16 a lane cost more than the fewer waves give (E=200, k=16, 16384
  // rows: 36 us with sixteen lanes a row, 25 with 32).
  const auto fits = [&](int L) {
    const int v = B * L > 32 * kSimds && a.k <= L - 2 ? experts_a_lane(L, a, &g) : 0;
    return v <= (a.k <= 8 ? 16 : 8) ? v : 0;
  };
  switch (fits(16)) {
    case 1: return go(launch_route_t<1, 1, 16>);
    case 2: return go(launch_route_t<2, 2, 16>);
    case 4: return go(launch_route_t<4, 4, 16>);
    case 8: return go(launch_route_t<8, 8, 16>);
    case 16: return go(launch_route_t<16, 10, 16>);
  }
  switch (fits(32)) {
    case 1: return go(launch_route_t<1, 1, 32>);
    case 2: return go(launch_route_t<2, 2, 32>);
    case 4: return go(launch_route_t<4, 4, 32>);
    case 8: return go(launch_route_t<8, 8, 32>);
    case 16: return go(launch_route_t<16, 10, 32>);
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
  const auto go = [&](auto kernel) { return kernel(B, a, logits, ids, dweights, dlogits, st); };
  if (a.k <= 16 && a.E <= 512 && B >= kManyRowsBwd) {
    if (a.E > 256) return go(launch_route_bwd_t<16, 32>);  // (12.6 against 14.3 at E=512, B=16384)
    return a.E <= 64 ? go(launch_route_bwd_t<4, 16>) : a.E <= 128 ? go(launch_route_bwd_t<8, 16>)
                                                                  : go(launch_route_bwd_t<16, 16>);
  }
  return a.E <= 256 ? go(launch_route_bwd_t<4, 64>) : go(launch_route_bwd_t<16, 64>);
}

}  // namespace mhc
