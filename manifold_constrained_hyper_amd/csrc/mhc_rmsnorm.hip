// Root-mean-square norm of the layer input, with the shortcut's addition, to
// bf16 or to the checkpoint's 8-bit format; and its gradients.
//
//   s = bf16(x + shortcut)   rstd = 1 / sqrt(mean(s^2) + eps)   y = s rstd w
//   n = s rstd, g = dy w:    dx = rstd (g - n mean(g n)) + dsum,  dw = sum over rows of dy n
//
// A workgroup takes a row, which stays in registers between the sum and its
// use, so every tensor is read or written once.  Squares and sums are fp32
// (products of two bf16 values are exact there).
#include "mhc_experts.h"
#include "mhc_finish.h"
#include "mhc_held.h"
#include "mhc_train.h"

namespace mhc {

namespace {

constexpr int kMostWaves = 16;

// Sum over the workgroup, in the order of its waves.  `part` is used again
// only behind the caller's next barrier.
__device__ __forceinline__ float group_total(float x, float *part) {
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  x = wave_sum(x);
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) part[wave] = x;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < waves; ++w) t += part[w];
  return t;
}

__device__ __forceinline__ void load_weight(const float *w, uint32_t v, float (&o)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 1.f;
    return;
  }
  const f32x4 a = reinterpret_cast<const f32x4 *>(w)[2 * (size_t)v], b = reinterpret_cast<const f32x4 *>(w)[2 * (size_t)v + 1];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = a[e];
    o[4 + e] = b[e];
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&y)[8]) {
  return u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
}

// V vectors of eight channels a thread.
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a, uint32_t B, uint32_t cvec, uint32_t blocks,
                                                       float inv_c) {
  __shared__ float part[2][kMostWaves];
  const uint32_t T = blockDim.x;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x, turn ^= 1) {
    const size_t first = (size_t)row * cvec;
    u32x4 s[V];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      s[i] = u32x4{0u, 0u, 0u, 0u};
      if (v < cvec) {
        s[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.x) + first + v);
        if (a.shortcut) {
          const u32x4 c = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.shortcut) + first + v);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            s[i][w] = pack_bf16x2(bf16_lo(s[i][w]) + bf16_lo(c[w]), bf16_hi(s[i][w]) + bf16_hi(c[w]));
          if (a.sum) store16_nt(static_cast<u32x4 *>(a.sum) + first + v, s[i]);
        }
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) sq = dot2_bf16(s[i][w], s[i][w], sq);
    }
    const float rstd = 1.0f / sqrtf(group_total(sq, part[turn]) * inv_c + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      float y[8], w[8];
      widen8(s[i], y);
      if (v < cvec) load_weight(a.weight, v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v < cvec ? y[e] * rstd * w[e] : 0.f;
      if (a.y && v < cvec) store16_nt(static_cast<u32x4 *>(a.y) + first + v, pack8(y));
      if (a.codes) {
        uint32_t amax = 0;  // of the finite values; their bits order like they do
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t m = __float_as_uint(y[e]) & 0x7fffffffu;
          amax = m < 0x7f800000u && m > amax ? m : amax;
        }
        const int sc = ckpt_scale32(quad_max(amax));
        const u32x2 q = held_codes(y, sc);
        if (v < cvec) {
          __builtin_nontemporal_store(q, static_cast<u32x2 *>(a.codes) + first + v);
          if ((v & 3u) == 0) a.scales[(size_t)row * blocks + (v >> 2)] = (uint8_t)sc;
        }
      }
    }
  }
}

template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(NormBwdArgs a, float *partial, uint32_t B, uint32_t cvec,
                                                           float inv_c) {
  __shared__ float part[2][kMostWaves];
  const uint32_t T = blockDim.x;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x, turn ^= 1) {
    const size_t first = (size_t)row * cvec;
    const float rstd = a.rstd[row];
    u32x4 s[V], d[V];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      s[i] = d[i] = u32x4{0u, 0u, 0u, 0u};
      if (v < cvec) {
        s[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.sum) + first + v);
        d[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.dy) + first + v);
        float x[8], g[8], w[8];
        widen8(s[i], x);
        widen8(d[i], g);
        load_weight(a.weight, v, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = x[e] * rstd;
          dw[i][e] = fmaf(g[e], n, dw[i][e]);
          dot = fmaf(g[e] * w[e], n, dot);
        }
      }
    }
    const float mean = group_total(dot, part[turn]) * inv_c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      if (v >= cvec) continue;
      float x[8], g[8], w[8], o[8];
      widen8(s[i], x);
      widen8(d[i], g);
      load_weight(a.weight, v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (g[e] * w[e] - x[e] * rstd * mean);
      if (a.dsum) {
        float p[8];
        widen8(__builtin_nontemporal_load(static_cast<const u32x4 *>(a.dsum) + first + v), p);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += p[e];
      }
      store16_nt(static_cast<u32x4 *>(a.dx) + first + v, pack8(o));
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t v = threadIdx.x + i * T;
    if (v >= cvec) continue;
    f32x4 *p = reinterpret_cast<f32x4 *>(partial) + ((size_t)blockIdx.x * cvec + v) * 2;
    p[0] = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    p[1] = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

// dweight: the partial sums, a sixteenth of them a wave, then the waves'.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void join_dweight_kernel(const f32x4 *partial, uint32_t parts,
                                                                       uint32_t quads, f32x4 *dweight) {
  __shared__ f32x4 sum[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t q = blockIdx.x * 64 + lane;
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
  if (q < quads)
    for (uint32_t p = wave; p < parts; p += kJoinWaves) t += partial[(size_t)p * quads + q];
  sum[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && q < quads) {
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) t += sum[w][lane];
    dweight[q] = t;
  }
}

struct Shape {
  uint32_t threads;
  int v;
};
Shape shape_of(int64_t C) {
  const uint32_t cvec = (uint32_t)(C / 8);
  const uint32_t threads = cvec > 2048 ? 1024 : cvec > 64 ? 256 : 64;
  const uint32_t v = (cvec + threads - 1) / threads;
  return Shape{threads, v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8};
}

}  // namespace

hipError_t launch_rmsnorm(int64_t B, int64_t C, const NormArgs &a, hipStream_t st) {
  const Shape s = shape_of(C);
  const uint32_t grid = (uint32_t)(B < (1 << 21) ? B : (1 << 21)), cvec = (uint32_t)(C / 8);
  const uint32_t blocks = (uint32_t)ckpt_blocks(C);
  const float inv_c = 1.0f / (float)C;
  switch (s.v) {
    case 1: rmsnorm_kernel<1><<<grid, s.threads, 0, st>>>(a, (uint32_t)B, cvec, blocks, inv_c); break;
    case 2: rmsnorm_kernel<2><<<grid, s.threads, 0, st>>>(a, (uint32_t)B, cvec, blocks, inv_c); break;
    case 4: rmsnorm_kernel<4><<<grid, s.threads, 0, st>>>(a, (uint32_t)B, cvec, blocks, inv_c); break;
    default: rmsnorm_kernel<8><<<grid, s.threads, 0, st>>>(a, (uint32_t)B, cvec, blocks, inv_c); break;
  }
  return hipGetLastError();
}

NormBwdPlan plan_rmsnorm_bwd(int64_t B, int64_t C) {
  NormBwdPlan p;
  p.parts = B < 1024 ? B : 1024;
  p.total_bytes = (size_t)p.parts * C * 4;
  return p;
}

hipError_t launch_rmsnorm_bwd(const NormBwdPlan &p, int64_t B, int64_t C, const NormBwdArgs &a, void *ws,
                              hipStream_t st) {
  const Shape s = shape_of(C);
  const uint32_t grid = (uint32_t)p.parts, cvec = (uint32_t)(C / 8);
  const float inv_c = 1.0f / (float)C;
  float *partial = a.dweight ? static_cast<float *>(ws) : nullptr;
  switch (s.v) {
    case 1: rmsnorm_bwd_kernel<1><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    case 2: rmsnorm_bwd_kernel<2><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    case 4: rmsnorm_bwd_kernel<4><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    default: rmsnorm_bwd_kernel<8><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  const uint32_t quads = (uint32_t)(C / 4);
  join_dweight_kernel<<<(quads + 63) / 64, 64 * kJoinWaves, 0, st>>>(reinterpret_cast<const f32x4 *>(partial), grid,
                                                                     quads, reinterpret_cast<f32x4 *>(a.dweight));
  return hipGetLastError();
}

}  // namespace mhc
