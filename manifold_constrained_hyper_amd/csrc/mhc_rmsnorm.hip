// Root-mean-square norm of the layer input, with the shortcut's addition, to
// bf16 or to the checkpoint's 8-bit format; and its gradients.
//
//   s = bf16(x + shortcut)   rstd = 1 / sqrt(mean(s^2) + eps)   y = s rstd w
//   n = s rstd, g = dy w:    dx = rstd (g - n mean(g n)) + dsum,  dw = sum over rows of dy n
//
// A workgroup takes a row at a time (of short rows several), which stays in
// registers between the sum and its use, so that every tensor is read or written
// once.  Two gradient kernels read a row twice, the second time from the cache
// where it holds it: that of rows above C=16384, and that of few rows, by rows
// and by columns.  Squares and sums are fp32 (products of two bf16 values are
// exact there).
//
// Bound by HBM: 139 us for B=16384, C=7168 with the shortcut in 8 bits (826 MB,
// 6.0 TB/s), 160 for its gradients with the shortcut's (940 MB, 5.9 TB/s, of
// which 5 us join dweight).  One row takes 3.1, and its gradients 4.0.
// Long rows, 4096 of them without the shortcut, and their gradients: C=16384 52
// us (5.1 TB/s) and 98 (4.1), C=32768 102 (5.3) and 243 (3.3, read twice).
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
  const f32x4 *from = reinterpret_cast<const f32x4 *>(w) + 2 * (size_t)v;
  const f32x4 a = from[0], b = from[1];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = a[e];
    o[4 + e] = b[e];
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&y)[8]) {
  return u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
}

// Vector v of a row in 8 bits; four neighbouring lanes have a block.
__device__ __forceinline__ void store_codes(const NormArgs &a, float (&y)[8], size_t row, uint32_t v,
                                            size_t first, uint32_t blocks, bool real) {
  uint32_t amax = 0;  // of the finite values; their bits order like they do
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t m = __float_as_uint(y[e]) & 0x7fffffffu;
    amax = m < 0x7f800000u && m > amax ? m : amax;
  }
  const int sc = ckpt_scale32(quad_max(amax));
  const u32x2 q = held_codes(y, sc);
  if (real) {
    __builtin_nontemporal_store(q, static_cast<u32x2 *>(a.codes) + first + v);
    if ((v & 3u) == 0) a.scales[row * blocks + (v >> 2)] = (uint8_t)sc;
  }
}

// V vectors of eight channels a thread, all of a row.
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a, uint32_t B, uint32_t cvec, uint32_t blocks,
                                                       float inv_c) {
  __shared__ float part[2][kMostWaves];
  const uint32_t T = blockDim.x;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x, turn ^= 1) {
    const size_t first = (size_t)row * cvec;
    u32x4 s[V], c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      s[i] = c[i] = u32x4{0u, 0u, 0u, 0u};
      if (v >= cvec) continue;
      s[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.x) + first + v);
      if (a.shortcut) c[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.shortcut) + first + v);
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      if (a.shortcut) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          s[i][q] = pack_bf16x2(bf16_lo(s[i][q]) + bf16_lo(c[i][q]), bf16_hi(s[i][q]) + bf16_hi(c[i][q]));
        if (a.sum && v < cvec) store16_nt(static_cast<u32x4 *>(a.sum) + first + v, s[i]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) sq = dot2_bf16(s[i][q], s[i][q], sq);
    }
    const float rstd = 1.0f / sqrtf(group_total(sq, part[turn]) * inv_c + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      float y[8], w[8];
      widen8(s[i], y);
      load_weight(v < cvec ? a.weight : nullptr, v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v < cvec ? y[e] * rstd * w[e] : 0.f;
      if (a.y && v < cvec) store16_nt(static_cast<u32x4 *>(a.y) + first + v, pack8(y));
      if (a.codes) store_codes(a, y, row, v, first, blocks, v < cvec);
    }
  }
}

// Rows of up to 32 vectors: `lanes` of a wave (a power of two, four at least)
// take one.  us for 65536 rows with the shortcut in 8 bits, and with a
// workgroup a row: C=64 7.8 and 27, C=256 25 and 32, C=512 46 and 44.
constexpr int kShortWaves = 4, kShortVecs = 32;
__device__ __forceinline__ float lanes_sum(float x, uint32_t lanes) {
  for (uint32_t m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
  return x;
}
__global__ __launch_bounds__(64 * kShortWaves) void rmsnorm_short_kernel(NormArgs a, uint32_t B, uint32_t cvec,
                                                                         uint32_t lanes, uint32_t blocks, float inv_c) {
  const uint32_t lane = threadIdx.x & 63, rows = 64 / lanes, v = lane & (lanes - 1);
  const uint64_t step = (uint64_t)gridDim.x * kShortWaves * rows;
  for (uint64_t base = ((uint64_t)blockIdx.x * kShortWaves + (threadIdx.x >> 6)) * rows; base < B; base += step) {
    const uint64_t row = base + lane / lanes;
    const size_t first = row * cvec;
    const bool real = row < B && v < cvec;
    u32x4 s = {0u, 0u, 0u, 0u};
    if (real) {
      s = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.x) + first + v);
      if (a.shortcut) {
        const u32x4 c = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.shortcut) + first + v);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          s[q] = pack_bf16x2(bf16_lo(s[q]) + bf16_lo(c[q]), bf16_hi(s[q]) + bf16_hi(c[q]));
        if (a.sum) store16_nt(static_cast<u32x4 *>(a.sum) + first + v, s);
      }
    }
    float sq = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) sq = dot2_bf16(s[q], s[q], sq);
    const float rstd = 1.0f / sqrtf(lanes_sum(sq, lanes) * inv_c + a.eps);
    if (a.rstd && real && v == 0) a.rstd[row] = rstd;
    float y[8], w[8];
    widen8(s, y);
    load_weight(real ? a.weight : nullptr, v, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = real ? y[e] * rstd * w[e] : 0.f;
    if (a.y && real) store16_nt(static_cast<u32x4 *>(a.y) + first + v, pack8(y));
    if (a.codes) store_codes(a, y, row, v, first, blocks, real);
  }
}

// The partial sums of dweight stay in registers; with one vector a thread the
// weight does too, and the next row is loaded while this one is worked on.
// From four on a row does not fit beside them and is read twice.
template <int V>
struct BwdRow {
  u32x4 s[V], d[V], p[V];
  float rstd;
};
template <int V>
__device__ __forceinline__ void load_row(const NormBwdArgs &a, uint32_t row, uint32_t cvec, uint32_t thread,
                                         uint32_t threads, BwdRow<V> &x) {
  const size_t first = (size_t)row * cvec;
  x.rstd = a.rstd[row];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t v = thread + i * threads;
    x.s[i] = x.d[i] = x.p[i] = u32x4{0u, 0u, 0u, 0u};
    if (v >= cvec) continue;
    x.s[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.sum) + first + v);
    x.d[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.dy) + first + v);
    if (a.dsum) x.p[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.dsum) + first + v);
  }
}

template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(NormBwdArgs a, float *partial, uint32_t B, uint32_t cvec,
                                                           float inv_c) {
  __shared__ float part[2][kMostWaves];
  const uint32_t T = blockDim.x;
  constexpr bool kStay = V == 1, kKeep = V <= 2;
  constexpr int kHeld = kStay ? V : 1;
  float dw[V][8], held[kHeld][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  BwdRow<kHeld> next;
  if constexpr (kStay) {
    load_weight(threadIdx.x < cvec ? a.weight : nullptr, threadIdx.x, held[0]);
    load_row<kHeld>(a, blockIdx.x, cvec, threadIdx.x, T, next);
  }
  const auto weight_at = [&](uint32_t v, float(&w)[8]) {
    if constexpr (kStay) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = held[0][e];
    } else {
      load_weight(v < cvec ? a.weight : nullptr, v, w);
    }
  };
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x, turn ^= 1) {
    const size_t first = (size_t)row * cvec;
    const u32x4 *s = static_cast<const u32x4 *>(a.sum) + first, *d = static_cast<const u32x4 *>(a.dy) + first;
    constexpr int kRow = kKeep ? V : 1;
    BwdRow<kRow> x;
    if constexpr (kStay) {
      x = next;
      if (row + gridDim.x < B) load_row<kHeld>(a, row + gridDim.x, cvec, threadIdx.x, T, next);
    } else if constexpr (kKeep) {
      load_row<kRow>(a, row, cvec, threadIdx.x, T, x);
    } else {
      x.rstd = a.rstd[row];
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      if (!kKeep && v >= cvec) continue;
      float n[8], g[8], w[8];
      widen8(kKeep ? x.s[kKeep ? i : 0] : s[v], n);
      widen8(kKeep ? x.d[kKeep ? i : 0] : d[v], g);
      weight_at(v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= x.rstd;
        dw[i][e] = fmaf(g[e], n[e], dw[i][e]);
        dot = fmaf(g[e] * w[e], n[e], dot);
      }
    }
    const float mean = group_total(dot, part[turn]) * inv_c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t v = threadIdx.x + i * T;
      if (v >= cvec) continue;
      float n[8], g[8], o[8], w[8];
      widen8(kKeep ? x.s[kKeep ? i : 0] : s[v], n);
      widen8(kKeep ? x.d[kKeep ? i : 0] : d[v], g);
      weight_at(v, w);
      if constexpr (kKeep) {
        widen8(x.p[i], o);
      } else {
        widen8(a.dsum ? static_cast<const u32x4 *>(a.dsum)[first + v] : u32x4{0u, 0u, 0u, 0u}, o);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += x.rstd * (g[e] * w[e] - n[e] * x.rstd * mean);
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

// The gradients, of rows of up to 64 vectors (C=64 12 us, 36 with a workgroup a
// row; C=256 30, 43; C=512 55, 55, but 19, 23 for 16384 rows).
constexpr int kShortVecsBwd = 64;
__global__ __launch_bounds__(64 * kShortWaves) void rmsnorm_bwd_short_kernel(NormBwdArgs a, float *partial, uint32_t B,
                                                                             uint32_t cvec, uint32_t lanes,
                                                                             float inv_c) {
  __shared__ float part[kShortWaves][kShortVecsBwd * 8];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rows = 64 / lanes, v = lane & (lanes - 1);
  const uint64_t step = (uint64_t)gridDim.x * kShortWaves * rows;
  float w[8], dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  load_weight(v < cvec ? a.weight : nullptr, v, w);
  for (uint64_t base = ((uint64_t)blockIdx.x * kShortWaves + wave) * rows; base < B; base += step) {
    const uint64_t row = base + lane / lanes;
    const size_t at = row * cvec + v;
    const bool real = row < B && v < cvec;
    u32x4 s = {0u, 0u, 0u, 0u}, d = s, p = s;
    float rstd = 0.f;
    if (real) {
      s = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.sum) + at);
      d = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.dy) + at);
      if (a.dsum) p = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.dsum) + at);
      rstd = a.rstd[row];
    }
    float n[8], g[8], o[8], dot = 0.f;
    widen8(s, n);
    widen8(d, g);
    widen8(p, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      n[e] *= rstd;
      dw[e] = fmaf(g[e], n[e], dw[e]);
      g[e] *= w[e];
      dot = fmaf(g[e], n[e], dot);
    }
    const float mean = lanes_sum(dot, lanes) * inv_c;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += rstd * (g[e] - n[e] * mean);
    if (real) store16_nt(static_cast<u32x4 *>(a.dx) + at, pack8(o));
  }
  if (!partial) return;
  for (uint32_t m = lanes; m < 64; m <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] += __shfl_xor(dw[e], m);
  if (lane < cvec) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[wave][lane * 8 + e] = dw[e];
  }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < cvec * 8; c += 64 * kShortWaves) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kShortWaves; ++i) t += part[i][c];
    partial[(size_t)blockIdx.x * cvec * 8 + c] = t;
  }
}

// Few rows: one launch.  The first workgroups take 32 columns of dweight each,
// which needs no sum over a row (rstd is given), and read dy and the rows a
// second time, from the cache; the others take a row for each `threads` of
// theirs.
constexpr int kColumnVecs = 4;
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_few_kernel(NormBwdArgs a, uint32_t B, uint32_t cvec,
                                                               uint32_t column_wgs, uint32_t threads, float inv_c) {
  __shared__ float part[kMostWaves][kColumnVecs * 8];
  const uint32_t T = blockDim.x;
  if (blockIdx.x < column_wgs) {
    const uint32_t lane = threadIdx.x % kColumnVecs, v = blockIdx.x * kColumnVecs + lane, teams = T / kColumnVecs;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (v < cvec) {
#pragma unroll 4
      for (uint32_t row = threadIdx.x / kColumnVecs; row < B; row += teams) {
        const size_t at = (size_t)row * cvec + v;
        float n[8], g[8];
        widen8(static_cast<const u32x4 *>(a.sum)[at], n);
        widen8(static_cast<const u32x4 *>(a.dy)[at], g);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(g[e], n[e] * rstd, dw[e]);
      }
    }
#pragma unroll
    for (int m = kColumnVecs; m < 64; m *= 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[e] += __shfl_xor(dw[e], m);
    if ((threadIdx.x & 63) < kColumnVecs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[threadIdx.x >> 6][lane * 8 + e] = dw[e];
    }
    __syncthreads();
    const uint32_t c = blockIdx.x * kColumnVecs * 8 + threadIdx.x;
    if (threadIdx.x < kColumnVecs * 8 && c < cvec * 8) {
      float t = 0.f;
      for (uint32_t w = 0; w < T / 64; ++w) t += part[w][threadIdx.x];
      a.dweight[c] = t;
    }
    return;
  }
  const uint32_t wave = uniform((int)threadIdx.x >> 6), waves = threads >> 6, which = wave / waves;
  const uint32_t row = (blockIdx.x - column_wgs) * (T / threads) + which, thread = threadIdx.x - which * threads;
  BwdRow<V> x{};
  if (row < B) load_row<V>(a, row, cvec, thread, threads, x);
  float dot = 0.f, g[V][8], n[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t v = thread + i * threads;
    float w[8];
    widen8(x.s[i], n[i]);
    widen8(x.d[i], g[i]);
    load_weight(v < cvec ? a.weight : nullptr, v, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[i][e] *= w[e];
      n[i][e] *= x.rstd;
      dot = fmaf(g[i][e], n[i][e], dot);
    }
  }
  dot = wave_sum(dot);
  if ((threadIdx.x & 63) == 0) part[wave][0] = dot;
  __syncthreads();
  float mean = 0.f;
  for (uint32_t w = 0; w < waves; ++w) mean += part[which * waves + w][0];
  mean *= inv_c;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t v = thread + i * threads;
    if (row >= B || v >= cvec) continue;
    float o[8];
    widen8(x.p[i], o);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += x.rstd * (g[i][e] - n[i][e] * mean);
    store16_nt(static_cast<u32x4 *>(a.dx) + (size_t)row * cvec + v, pack8(o));
  }
}

// dweight: 16 lanes take 64 columns, 64 teams of them a share of the partial
// sums each, whose sums are then joined in the teams' order.
constexpr int kJoinLanes = 16, kTeams = 64;
__global__ __launch_bounds__(kJoinLanes *kTeams) void join_dweight_kernel(const f32x4 *__restrict__ partial,
                                                                          uint32_t parts, uint32_t quads,
                                                                          f32x4 *__restrict__ dweight) {
  __shared__ f32x4 sum[kTeams][kJoinLanes];
  const int lane = threadIdx.x % kJoinLanes, team = threadIdx.x / kJoinLanes;
  const uint32_t q = blockIdx.x * kJoinLanes + lane;
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
  if (q < quads) {
#pragma unroll 8
    for (uint32_t p = team; p < parts; p += kTeams) t += partial[(size_t)p * quads + q];
  }
  sum[team][lane] = t;
#pragma unroll
  for (int half = kTeams / 2; half > 0; half /= 2) {
    __syncthreads();
    if (team < half) {
      t += sum[team + half][lane];
      sum[team][lane] = t;
    }
  }
  if (team == 0 && q < quads) dweight[q] = t;
}

struct Shape {
  uint32_t threads;
  int v;
};
// Threads for rows of cvec vectors, `wide` of them at most: full waves, with 1,
// 2, 4 or 8 vectors each.
Shape shape_of(int64_t C, uint32_t wide) {
  const uint32_t cvec = (uint32_t)(C / 8), v = (cvec + wide - 1) / wide;
  Shape s{0, v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8};
  s.threads = ((cvec + s.v - 1) / s.v + 63) / 64 * 64;
  return s;
}

// Lanes that take a short row, 0 for one of more than `most` vectors.
uint32_t short_lanes(int64_t C, int most) {
  if (C > 8 * most) return 0;
  uint32_t lanes = 4;
  while (lanes * 8 < C) lanes *= 2;
  return lanes;
}

}  // namespace

hipError_t launch_rmsnorm(int64_t B, int64_t C, const NormArgs &a, hipStream_t st) {
  // Vectors a thread: one where there is little work, as a row's chain is what
  // takes the time, else enough to have four loads in flight, two with the
  // shortcut (its own come on top), in at least a wave.  us with 1, 2 and 4:
  //   C=7168, shortcut, 8 bits  8.2 8.0 9.4 (512 rows)   14.7 13.0 14.8 (1024)  162 147 143 (16384)
  //   C=7168, shortcut, bf16    7.4 7.2 8.6 (512 rows)   14.4 13.3 13.3 (1024)  163 157 161 (16384)
  //   C=7168, bf16              5.2 5.4 6.0 (512 rows)   9.7 8.7 7.8 (1024)     116 107 88 (16384)
  //   C=2048, bf16              4.4 4.7 5.3 (1024 rows)  9.3 8.6 7.5 (4096)     27 27 28 (16384)
  // (Which outputs are asked for has no part in it, so that it changes no bits.)
  const int64_t all = B * C;
  const int v = all < (7 << 20) ? 1 : a.shortcut && (C <= 4096 || all < (56 << 20)) ? 2 : 4;
  const int64_t wide = (C / 8 + v - 1) / v;
  const Shape s = shape_of(C, (uint32_t)(wide < 64 ? 64 : wide < 1024 ? wide : 1024));
  const uint32_t cvec = (uint32_t)(C / 8), blocks = (uint32_t)ckpt_blocks(C), rows = (uint32_t)B;
  const float inv_c = 1.0f / (float)C;
  if (const uint32_t lanes = short_lanes(C, kShortVecs)) {
    const int64_t per = kShortWaves * 64 / lanes, wgs = (B + per - 1) / per;
    rmsnorm_short_kernel<<<(uint32_t)(wgs < (1 << 21) ? wgs : (1 << 21)), 64 * kShortWaves, 0, st>>>(
        a, rows, cvec, lanes, blocks, inv_c);
    return hipGetLastError();
  }
  const uint32_t grid = (uint32_t)(B < (1 << 21) ? B : (1 << 21));
  switch (s.v) {
    case 1: rmsnorm_kernel<1><<<grid, s.threads, 0, st>>>(a, rows, cvec, blocks, inv_c); break;
    case 2: rmsnorm_kernel<2><<<grid, s.threads, 0, st>>>(a, rows, cvec, blocks, inv_c); break;
    case 4: rmsnorm_kernel<4><<<grid, s.threads, 0, st>>>(a, rows, cvec, blocks, inv_c); break;
    default: rmsnorm_kernel<8><<<grid, s.threads, 0, st>>>(a, rows, cvec, blocks, inv_c); break;
  }
  return hipGetLastError();
}

// One launch for the gradients instead of two (us, one against two: C=7168 4.4
// and 6.1 for one row, 4.6 and 7.2 for 64, 7.5 and 11.8 for 256, 12.3 and 12.9
// for 512, 22 and 18 for 1024; C=256 6.7 and 9.6 for 2048 rows, 13 and 10.8 for
// 4096; B=1001, C=1000, more than the L2 caches keep, 10.3 and 8.8).  The
// workspace is as large as without it.
bool few_rows(int64_t B, int64_t C) {
  return C <= 16384 && ((B <= 512 && B * C < (4 << 20)) || (B <= 2048 && B * C <= (3 << 18)));
}

NormBwdPlan plan_rmsnorm_bwd(int64_t B, int64_t C) {
  NormBwdPlan p;
  // Workgroups, each with its own partial sums of dweight: 512, or two waves a
  // SIMD where rows are short, but not fewer than eight rows each (C=1000, us:
  // 9.1 with 256 for 1001 rows, 12.9 with 1024; 34.5 with 1024 for 16384 rows,
  // 37 with 512; C=7168: 164 with 512 for 16384 rows, 169 with 1024).
  // Of short rows a workgroup takes two turns at least.
  constexpr int64_t kPer = 8, kLeast = 256;
  if (const uint32_t lanes = short_lanes(C, kShortVecsBwd)) {
    const int64_t turns = 2 * kShortWaves * 64 / lanes, wgs = (B + turns - 1) / turns;
    p.parts = wgs < 512 ? wgs : 512;
    p.total_bytes = (size_t)p.parts * C * 4;
    return p;
  }
  const int64_t waves = shape_of(C, 1024).threads / 64;
  int64_t parts = 2048 / waves;
  parts = parts < 512 ? 512 : parts;
  parts = parts > B / kPer ? B / kPer : parts;
  parts = parts < kLeast ? kLeast : parts;
  p.parts = B < parts ? B : parts;
  p.total_bytes = (size_t)p.parts * C * 4;
  return p;
}

hipError_t launch_rmsnorm_bwd(const NormBwdPlan &p, int64_t B, int64_t C, const NormBwdArgs &a, void *ws,
                              hipStream_t st) {
  const Shape s = shape_of(C, 1024);
  const uint32_t grid = (uint32_t)p.parts, cvec = (uint32_t)(C / 8);
  const float inv_c = 1.0f / (float)C;
  float *partial = a.dweight ? static_cast<float *>(ws) : nullptr;
  if (few_rows(B, C)) {
    const uint32_t rows = s.threads >= 512 ? 1 : 512 / s.threads;  // a workgroup
    const uint32_t column_wgs = partial ? (cvec + kColumnVecs - 1) / kColumnVecs : 0;
    const uint32_t wgs = column_wgs + ((uint32_t)B + rows - 1) / rows, threads = s.threads * rows;
    const auto kernel = s.v == 1 ? rmsnorm_bwd_few_kernel<1> : rmsnorm_bwd_few_kernel<2>;
    kernel<<<wgs, threads, 0, st>>>(a, (uint32_t)B, cvec, column_wgs, s.threads, inv_c);
    return hipGetLastError();
  }
  const uint32_t lanes = short_lanes(C, kShortVecsBwd);
  switch (lanes ? 0 : s.v) {
    case 0:
      rmsnorm_bwd_short_kernel<<<grid, 64 * kShortWaves, 0, st>>>(a, partial, (uint32_t)B, cvec, lanes, inv_c);
      break;
    case 1: rmsnorm_bwd_kernel<1><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    case 2: rmsnorm_bwd_kernel<2><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    case 4: rmsnorm_bwd_kernel<4><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
    default: rmsnorm_bwd_kernel<8><<<grid, s.threads, 0, st>>>(a, partial, (uint32_t)B, cvec, inv_c); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  const uint32_t quads = (uint32_t)(C / 4);
  join_dweight_kernel<<<(quads + kJoinLanes - 1) / kJoinLanes, kJoinLanes * kTeams, 0, st>>>(
      reinterpret_cast<const f32x4 *>(partial), grid, quads, reinterpret_cast<f32x4 *>(a.dweight));
  return hipGetLastError();
}

}  // namespace mhc
