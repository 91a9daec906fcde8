// Rows into the order of their experts and back.
//
//   order    slot(b, j) = first[e] + earlier pairs of e,  e = ids[b, j]
//   gather   rows[slot(b, j)] = X[b]
//   combine  out[b] = shared[b] + sum_j w(b, j) Y[slot(b, j)]
//   and its gradients dY[slot(b, j)] = w(b, j) dout[b], dw(b, j) = dout[b] . Y[slot(b, j)]
#include "mhc_experts.h"
#include "mhc_finish.h"
#include "mhc_held.h"
#include "mhc_train.h"

namespace mhc {

namespace {

// -- order ------------------------------------------------------------------
//
// A counting sort.  A wave takes a tile of consecutive pairs, 64 at a time:
// ten ballots on the bits of the expert tell a lane which lanes have the same
// one, so its rank is the tile's count so far (LDS) and its earlier peers.
// The second kernel adds what the smaller experts and the earlier tiles count.
constexpr int kOrderWaves = 4;
constexpr int kIdBits = 10;
static_assert(kMaxExperts == 1 << kIdBits, "experts' bits");

__global__ __launch_bounds__(64 * kOrderWaves) void rank_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                                uint32_t tile, uint32_t tiles, int E,
                                                                int32_t *__restrict__ slots, uint32_t *counts) {
  extern __shared__ uint32_t seen_all[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t t = blockIdx.x * kOrderWaves + wave;
  if (t >= tiles) return;
  volatile uint32_t *seen = seen_all + wave * E;
  for (int e = lane; e < E; e += 64) seen[e] = 0;
  const uint64_t first = (uint64_t)t * tile, last = first + tile < pairs ? first + tile : pairs;
  for (uint64_t p0 = first; p0 < last; p0 += 64) {
    const uint64_t p = p0 + lane;
    const int32_t id = p < last ? ids[p] : -1;
    const bool real = id >= 0 && id < E;
    uint64_t peers = __ballot(real);
#pragma unroll
    for (int b = 0; b < kIdBits; ++b) {
      const bool bit = id >> b & 1;
      const uint64_t m = __ballot(bit);
      peers &= bit ? m : ~m;
    }
    const uint32_t before = (uint32_t)__popcll(peers & ((1ull << lane) - 1));
    uint32_t rank = 0;
    if (real) rank = seen[id];
    if (p < last) slots[p] = real ? (int32_t)(rank + before) : -1;
    if (real && before == 0) seen[id] = rank + (uint32_t)__popcll(peers);
  }
  for (int e = lane; e < E; e += 64) counts[(size_t)t * E + e] = seen[e];
}

// Each workgroup takes `per` tiles and adds up the counts that come before.
constexpr int kPlaceThreads = 256;
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                              uint32_t tile, uint32_t tiles, uint32_t per, int E,
                                                              const uint32_t *__restrict__ counts,
                                                              int32_t *__restrict__ slots,
                                                              int32_t *__restrict__ offsets) {
  __shared__ uint32_t base[kMaxExperts], total[kMaxExperts];
  const uint32_t mine = blockIdx.x * per;
  for (int e = threadIdx.x; e < E; e += kPlaceThreads) {
    uint32_t before = 0, all = 0;
    for (uint32_t t = 0; t < tiles; ++t) {
      const uint32_t c = counts[(size_t)t * E + e];
      before += t < mine ? c : 0;
      all += c;
    }
    base[e] = before;
    total[e] = all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t at = 0;
    for (int e = 0; e < E; ++e) {
      const uint32_t all = total[e];
      total[e] = at;
      at += all;
    }
    if (blockIdx.x == 0) offsets[E] = (int32_t)at;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlaceThreads) {
    if (blockIdx.x == 0) offsets[e] = (int32_t)total[e];
    base[e] += total[e];
  }
  for (uint32_t t = mine; t < mine + per && t < tiles; ++t) {
    __syncthreads();
    const uint64_t first = (uint64_t)t * tile, last = first + tile < pairs ? first + tile : pairs;
    for (uint64_t p = first + threadIdx.x; p < last; p += kPlaceThreads) {
      const int32_t id = ids[p];
      if (id >= 0 && id < E) slots[p] += (int32_t)base[id];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) base[e] += counts[(size_t)t * E + e];
  }
}

// -- gather -----------------------------------------------------------------

constexpr int kThreads = 256;

// A thread moves one vector of a row (T: 16 bytes, or 8 or 1) to its places.
template <class T>
__global__ __launch_bounds__(kThreads) void gather_kernel(const T *__restrict__ x, const int32_t *__restrict__ slots,
                                                          T *__restrict__ rows, uint64_t total, uint32_t vecs, int k,
                                                          uint32_t pairs) {
  for (uint64_t t = (uint64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = t / vecs;
    const uint32_t v = (uint32_t)(t - row * vecs);
    const T d = x[t];
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = (uint32_t)slots[row * k + j];
      if (slot < pairs) rows[(size_t)slot * vecs + v] = d;
    }
  }
}

// -- combine ----------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void combine_kernel(const u32x4 *__restrict__ Y,
                                                           const int32_t *__restrict__ slots,
                                                           const float *__restrict__ weights,
                                                           const u32x4 *__restrict__ shared, u32x4 *__restrict__ out,
                                                           uint64_t total, uint32_t cvec, int k, uint32_t pairs) {
  for (uint64_t t = (uint64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = t / cvec;
    const uint32_t v = (uint32_t)(t - row * cvec);
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (shared) widen8(__builtin_nontemporal_load(shared + t), o);
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = (uint32_t)slots[row * k + j];
      if (slot >= pairs) continue;
      const float w = weights ? weights[row * k + j] : 1.0f;
      float y[8];
      widen8(__builtin_nontemporal_load(Y + (size_t)slot * cvec + v), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(w, y[e], o[e]);
    }
    store16_nt(out + t, u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                              pack_bf16x2(o[6], o[7])});
  }
}

// A workgroup takes a row, one slot after the other.
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const u32x4 *__restrict__ Y,
                                                               const int32_t *__restrict__ slots,
                                                               const float *__restrict__ weights,
                                                               const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY,
                                                               float *__restrict__ dweights, uint32_t B,
                                                               uint32_t cvec, int k, uint32_t pairs) {
  __shared__ float part[kMaxChosen][kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x) {
    const u32x4 *d = dout + (size_t)row * cvec;
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = (uint32_t)slots[(size_t)row * k + j];
      float dot = 0.f;
      if (slot < pairs) {
        const float w = weights[(size_t)row * k + j];
        for (uint32_t v = threadIdx.x; v < cvec; v += kThreads) {
          const u32x4 g = d[v], y = __builtin_nontemporal_load(Y + (size_t)slot * cvec + v);
          u32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            dot = dot2_bf16(g[q], y[q], dot);
            o[q] = pack_bf16x2(w * bf16_lo(g[q]), w * bf16_hi(g[q]));
          }
          store16_nt(dY + (size_t)slot * cvec + v, o);
        }
      }
      dot = tree16_sum(dot);
      dot += __shfl_xor(dot, 16);
      dot += __shfl_xor(dot, 32);
      if (lane == 0) part[j][wave] = dot;
    }
    __syncthreads();
    if (threadIdx.x < (uint32_t)k) {
      float t = 0.f;
      for (int w = 0; w < kThreads / 64; ++w) t += part[threadIdx.x][w];
      dweights[(size_t)row * k + threadIdx.x] = t;
    }
    __syncthreads();
  }
}

uint32_t grid_of(uint64_t total, int per) {
  const uint64_t wgs = (total + per - 1) / per;
  return (uint32_t)(wgs < (1u << 22) ? wgs : (1u << 22));
}

template <class T>
hipError_t gather_t(int64_t B, int k, int64_t vecs, const void *x, const int32_t *slots, void *rows, hipStream_t st) {
  const uint64_t total = (uint64_t)B * vecs;
  gather_kernel<T><<<grid_of(total, kThreads), kThreads, 0, st>>>(static_cast<const T *>(x), slots,
                                                                  static_cast<T *>(rows), total, (uint32_t)vecs, k,
                                                                  (uint32_t)(B * k));
  return hipGetLastError();
}

}  // namespace

// Tiles of at least 512 pairs, at most 256 of them: their counts are added up
// by every workgroup of the second kernel.
OrderPlan plan_experts_order(int64_t pairs, int E) {
  OrderPlan p;
  constexpr int64_t kLeast = 512, kMost = 256;
  p.tile = kLeast;
  if (pairs > kLeast * kMost) p.tile = ((pairs + kMost - 1) / kMost + 63) / 64 * 64;
  p.tiles = (pairs + p.tile - 1) / p.tile;
  p.total_bytes = (size_t)p.tiles * E * 4;
  return p;
}

hipError_t launch_experts_order(const OrderPlan &p, int64_t pairs, int E, const int32_t *ids, int32_t *slots,
                                int32_t *offsets, void *ws, hipStream_t st) {
  uint32_t *counts = static_cast<uint32_t *>(ws);
  const uint32_t tiles = (uint32_t)p.tiles, wgs = (tiles + kOrderWaves - 1) / kOrderWaves;
  rank_kernel<<<wgs, 64 * kOrderWaves, (size_t)kOrderWaves * E * 4, st>>>(ids, (uint32_t)pairs, (uint32_t)p.tile,
                                                                          tiles, E, slots, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_kernel<<<tiles, kPlaceThreads, 0, st>>>(ids, (uint32_t)pairs, (uint32_t)p.tile, tiles, 1, E, counts, slots,
                                                offsets);
  return hipGetLastError();
}

hipError_t launch_experts_gather(int64_t B, int k, int64_t C, const void *x, const uint8_t *scales,
                                 const int32_t *slots, void *rows, uint8_t *row_scales, hipStream_t st) {
  if (!scales) return gather_t<u32x4>(B, k, C / 8, x, slots, rows, st);
  const hipError_t e = C % 16 == 0 ? gather_t<u32x4>(B, k, C / 16, x, slots, rows, st)
                                   : gather_t<u32x2>(B, k, C / 8, x, slots, rows, st);
  if (e != hipSuccess) return e;
  return gather_t<uint8_t>(B, k, ckpt_blocks(C), scales, slots, row_scales, st);
}

hipError_t launch_experts_combine(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                  const float *weights, const void *shared, void *out, hipStream_t st) {
  const uint32_t cvec = (uint32_t)(C / 8);
  const uint64_t total = (uint64_t)B * cvec;
  combine_kernel<<<grid_of(total, kThreads), kThreads, 0, st>>>(
      static_cast<const u32x4 *>(Y), slots, weights, static_cast<const u32x4 *>(shared), static_cast<u32x4 *>(out),
      total, cvec, k, (uint32_t)(B * k));
  return hipGetLastError();
}

hipError_t launch_experts_combine_bwd(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                      const float *weights, const void *dout, void *dY, float *dweights,
                                      hipStream_t st) {
  combine_bwd_kernel<<<grid_of((uint64_t)B, 1), kThreads, 0, st>>>(
      static_cast<const u32x4 *>(Y), slots, weights, static_cast<const u32x4 *>(dout), static_cast<u32x4 *>(dY),
      dweights, (uint32_t)B, (uint32_t)(C / 8), k, (uint32_t)(B * k));
  return hipGetLastError();
}

}  // namespace mhc
