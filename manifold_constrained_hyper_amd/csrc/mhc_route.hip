// The k experts of each row of logits, and the gradient of their weights.
//
//   score  = sigmoid(x), or exp(x - max) / sum of them        choice = score + bias
//   weight = scale score / (1, or the sum of the chosen scores)
//
// The order of the choices is that of 64-bit arithmetic: in 32 bits two scores
// next to each other may change places with the exponential's last bit.
//
// Renormalised weights are a softmax over the chosen: of x, or of
// log sigmoid(x) = min(x, 0) - log(1 + exp(-|x|)), where nothing underflows.
//
// A wave takes a row.
#include "mhc_experts.h"
#include "mhc_device.h"

namespace mhc {

namespace {

constexpr int kWaves = 4;
constexpr float kLargest = 3.4028234663852886e38f;

// A logit as it counts: NaN is minus infinity (no expert), plus infinity the
// largest number.
__device__ __forceinline__ float clean(float x) { return x != x ? -__builtin_inff() : fminf(x, kLargest); }
template <bool BF16>
__device__ __forceinline__ float logit_at(const void *p, size_t i) {
  if constexpr (BF16)
    return clean(bf16_lo(static_cast<const uint16_t *>(p)[i]));
  else
    return clean(static_cast<const float *>(p)[i]);
}

template <class T>
__device__ __forceinline__ T wave_sum(T x) {
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

// The largest value of a wave and, of equal ones, the lowest index.
__device__ __forceinline__ void wave_best(double &v, int &i) {
  for (int d = 32; d > 0; d >>= 1) {
    const double w = __shfl_xor(v, d);
    const int j = __shfl_xor(i, d);
    if (w > v || (w == v && j < i)) {
      v = w;
      i = j;
    }
  }
}

constexpr int kNone = 1 << 30;

template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a, const void *__restrict__ logits,
                                                            const float *__restrict__ bias, int32_t *__restrict__ ids,
                                                            float *__restrict__ weights, uint32_t B) {
  extern __shared__ double choices[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double *choice = choices + wave * a.E;
  const double none = -__builtin_inf();
  for (uint64_t first = (uint64_t)blockIdx.x * kWaves; first < B; first += (uint64_t)gridDim.x * kWaves) {
  const uint64_t at = first + wave;
  const size_t row = at < B ? at : B - 1;  // spare waves do the last row again and write nothing
  double top = none, total = 1.0;
  if (a.softmax) {
    for (int i = lane; i < a.E; i += 64) {
      const double x = logit_at<BF16>(logits, row * a.E + i);
      top = x > top ? x : top;
    }
    top = wave_max(top);
    total = 0.0;
    for (int i = lane; i < a.E; i += 64) {
      const double x = logit_at<BF16>(logits, row * a.E + i);
      total += x > none ? exp(x - top) : 0.0;
    }
    total = wave_sum(total);
  }
  const auto score = [&](double x) { return a.softmax ? exp(x - top) / total : 1.0 / (1.0 + exp(-x)); };
  for (int i = lane; i < a.E; i += 64) {
    const double x = logit_at<BF16>(logits, row * a.E + i);
    double c = none;
    if (x > none) {
      c = score(x) + (bias ? (double)bias[i] : 0.0);
      c = c > none ? c : none;  // NaN
    }
    choice[i] = c;
  }
  __syncthreads();
  if (a.top_groups < a.groups) {
    const int size = a.E / a.groups;
    double best = none, second = none;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double c = choice[lane * size + i];
        second = c > best ? best : c > second ? c : second;
        best = c > best ? c : best;
      }
    double rank = bias && second > none ? best + second : best;
    uint64_t kept = 0;
    bool left = lane < a.groups;
    for (int t = 0; t < a.top_groups; ++t) {
      double v = left ? rank : none;
      int i = left ? lane : kNone;
      wave_best(v, i);
      kept |= 1ull << i;
      left = left && i != lane;
    }
    for (int i = lane; i < a.E; i += 64)
      if (!(kept >> (i / size) & 1)) choice[i] = none;
  }
  __syncthreads();
  int id = -1;  // lane j: the j-th chosen
  for (int j = 0; j < a.k; ++j) {
    double v = none;
    int i = kNone;
    for (int e = lane; e < a.E; e += 64)
      if (choice[e] > v) {
        v = choice[e];
        i = e;
      }
    wave_best(v, i);
    if (i == kNone) break;
    if (lane == j) id = i;
    if (lane == (i & 63)) choice[i] = none;
  }
  const double x = id >= 0 ? logit_at<BF16>(logits, row * a.E + id) : none;
  double w = 0.0;
  if (a.renorm) {
    const double z = id < 0 ? none : a.softmax ? x : fmin(x, 0.0) - log1p(exp(-fabs(x)));
    const double most = wave_max(z);
    const double e = id < 0 ? 0.0 : exp(z - most);
    const double sum = wave_sum(e);
    w = sum > 0.0 ? e / sum : 0.0;
  } else if (id >= 0) {
    w = score(x);
  }
  if (at < B && lane < a.k) {
    ids[row * a.k + lane] = id;
    weights[row * a.k + lane] = (float)(w * a.scale);
  }
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
    total = wave_sum(total);
    inv_total = total > 0.f ? 1.0f / total : 0.f;
    const float p = x > none ? expf(x - top) * inv_total : 0.f;
    d = p * dw;
    along = wave_sum(d);
  } else if (a.renorm) {
    const float z = !(x > none) ? none : a.softmax ? x : fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
    const float most = wave_max(z);
    const float e = z > none ? expf(z - most) : 0.f;
    const float total = wave_sum(e);
    const float w = total > 0.f ? e / total : 0.f;
    d = w * (dw - wave_sum(w * dw));
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

uint32_t grid_of(int64_t B) {
  const int64_t wgs = (B + kWaves - 1) / kWaves;
  return (uint32_t)(wgs < (1 << 22) ? wgs : (1 << 22));
}

}  // namespace

hipError_t launch_route(int64_t B, const RouteArgs &a, const void *logits, const float *bias, int32_t *ids,
                        float *weights, hipStream_t st) {
  const uint32_t grid = grid_of(B);
  const size_t lds = (size_t)kWaves * a.E * sizeof(double);
  if (a.bf16)
    route_kernel<true><<<grid, 64 * kWaves, lds, st>>>(a, logits, bias, ids, weights, (uint32_t)B);
  else
    route_kernel<false><<<grid, 64 * kWaves, lds, st>>>(a, logits, bias, ids, weights, (uint32_t)B);
  return hipGetLastError();
}

hipError_t launch_route_bwd(int64_t B, const RouteArgs &a, const void *logits, const int32_t *ids,
                            const float *dweights, void *dlogits, hipStream_t st) {
  const uint32_t grid = grid_of(B);
  if (a.bf16)
    route_bwd_kernel<true><<<grid, 64 * kWaves, 0, st>>>(a, logits, ids, dweights, dlogits, (uint32_t)B);
  else
    route_bwd_kernel<false><<<grid, 64 * kWaves, 0, st>>>(a, logits, ids, dweights, dlogits, (uint32_t)B);
  return hipGetLastError();
}

}  // namespace mhc
