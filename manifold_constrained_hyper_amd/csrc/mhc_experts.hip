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
// A counting sort in chunks of consecutive pairs.  A wave takes its part of a
// chunk 64 pairs at a time: ten ballots on the bits of the expert tell a lane
// which lanes have the same one, so its rank is the wave's count so far (LDS)
// and its earlier peers.  The waves' counts are then added up in their order.
// Up to 4096 pairs one workgroup does it all.  Above, each workgroup ranks a
// tile, and a second launch adds the counts of the earlier tiles and of the
// smaller experts, which each of its workgroups sums up for itself.
constexpr int kIdBits = 10;
static_assert(kMaxExperts == 1 << kIdBits, "experts' bits");
constexpr int kRounds = 4;  // of 64 pairs a wave and chunk

// Ranks of the pairs p0 + 64 r + lane among the wave's pairs of the same
// expert; -1 where there is no expert.  `seen` (E counts of this wave, zero
// before) ends as its totals.
__device__ __forceinline__ void wave_ranks(const int32_t (&id)[kRounds], int E, volatile uint16_t *seen,
                                           int32_t (&rank)[kRounds]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool real = id[r] >= 0 && id[r] < E;
    uint64_t peers = __ballot(real);
    if (peers == 0) {
      rank[r] = -1;
      continue;
    }
#pragma unroll
    for (int b = 0; b < kIdBits; ++b) {
      const bool bit = id[r] >> b & 1;
      const uint64_t m = __ballot(bit);
      peers &= bit ? m : ~m;
    }
    const int before = (int)__popcll(peers & ((1ull << lane) - 1));
    const int so_far = real ? seen[id[r]] : 0;
    rank[r] = real ? so_far + before : -1;
    if (real && before == 0) seen[id[r]] = (uint16_t)(so_far + __popcll(peers));
  }
}

// Exclusive sums of x over the threads of the workgroup; *all is the total.
template <int WAVES>
__device__ __forceinline__ uint32_t group_scan(uint32_t x, uint32_t *sums, uint32_t *all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t y = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t z = __shfl_up(y, d);
    y += lane >= d ? z : 0;
  }
  if (lane == 63) sums[wave] = y;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  *all = total;
  return before + y - x;
}

constexpr int kOneWaves = 16, kOnePairs = kOneWaves * 64 * kRounds;
__global__ __launch_bounds__(64 * kOneWaves) void order_kernel(const int32_t *__restrict__ ids, uint32_t pairs, int E,
                                                               int32_t *__restrict__ slots,
                                                               int32_t *__restrict__ offsets) {
  extern __shared__ uint16_t seen[];  // [waves][E]
  __shared__ uint32_t first[kMaxExperts], sums[kOneWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t *mine = seen + wave * E;
  // Each wave takes whole rounds, so that the pairs stay in their order.
  const uint32_t rounds = (pairs + 63) / 64, per = (rounds + kOneWaves - 1) / kOneWaves;
  const uint32_t p0 = wave * per * 64 + lane;
  int32_t id[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) id[r] = (uint32_t)r < per && p0 + 64 * r < pairs ? ids[p0 + 64 * r] : -1;
  for (int e = lane; e < E; e += 64) mine[e] = 0;
  wave_ranks(id, E, mine, rank);
  __syncthreads();
  uint32_t count = 0;  // of the expert that is this thread's index
  if ((int)threadIdx.x < E) {
    for (int w = 0; w < kOneWaves; ++w) {
      const uint32_t c = seen[w * E + threadIdx.x];
      seen[w * E + threadIdx.x] = (uint16_t)count;
      count += c;
    }
  }
  uint32_t all;
  const uint32_t at = group_scan<kOneWaves>(count, sums, &all);
  if ((int)threadIdx.x < E) {
    first[threadIdx.x] = at;
    offsets[threadIdx.x] = (int32_t)at;
  }
  if (threadIdx.x == 0) offsets[E] = (int32_t)all;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if ((uint32_t)r < per && p0 + 64 * r < pairs)
      slots[p0 + 64 * r] = rank[r] < 0 ? -1 : (int32_t)(first[id[r]] + mine[id[r]]) + rank[r];
}

constexpr int kRankWaves = 4, kChunk = kRankWaves * 64 * kRounds;
__global__ __launch_bounds__(64 * kRankWaves) void rank_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                               uint32_t tile, int E, int32_t *__restrict__ slots,
                                                               uint32_t *__restrict__ counts) {
  extern __shared__ uint16_t seen[];  // [waves][E]
  __shared__ uint32_t so_far[kMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t *mine = seen + wave * E;
  const uint64_t first = (uint64_t)blockIdx.x * tile, last = first + tile < pairs ? first + tile : pairs;
  for (int e = threadIdx.x; e < E; e += 64 * kRankWaves) so_far[e] = 0;
  for (uint64_t c = first; c < last; c += kChunk) {
    const uint64_t p0 = c + wave * 64 * kRounds + lane;
    int32_t id[kRounds], rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) id[r] = p0 + 64 * r < last ? ids[p0 + 64 * r] : -1;
    for (int e = lane; e < E; e += 64) mine[e] = 0;
    wave_ranks(id, E, mine, rank);
    __syncthreads();
    uint32_t base[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      base[r] = 0;
      if (rank[r] >= 0) {
        base[r] = so_far[id[r]];
        for (int w = 0; w < wave; ++w) base[r] += seen[w * E + id[r]];
      }
      if (p0 + 64 * r < last) slots[p0 + 64 * r] = rank[r] < 0 ? -1 : (int32_t)base[r] + rank[r];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 64 * kRankWaves) {
      uint32_t t = so_far[e];
#pragma unroll
      for (int w = 0; w < kRankWaves; ++w) t += seen[w * E + e];
      so_far[e] = t;
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < E; e += 64 * kRankWaves) counts[(size_t)blockIdx.x * E + e] = so_far[e];
}

// A workgroup takes a tile.  `stride`: E rounded up to a power of two; the
// threads are kPlaceThreads / stride teams that share the tiles.
constexpr int kPlaceThreads = 1024;
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                              uint32_t tile, uint32_t tiles, int E, uint32_t stride,
                                                              const uint32_t *__restrict__ counts,
                                                              int32_t *__restrict__ slots,
                                                              int32_t *__restrict__ offsets) {
  __shared__ uint32_t before[kPlaceThreads], total[kPlaceThreads], sums[kPlaceThreads / 64];
  const uint32_t tid = threadIdx.x, e = tid & (stride - 1), teams = kPlaceThreads / stride;
  uint32_t b = 0, all = 0;
  if (e < (uint32_t)E) {
#pragma unroll 8
    for (uint32_t t = tid / stride; t < tiles; t += teams) {
      const uint32_t c = counts[(size_t)t * E + e];
      b += t < blockIdx.x ? c : 0;
      all += c;
    }
  }
  before[tid] = b;
  total[tid] = all;
  __syncthreads();
  b = all = 0;
  if (tid < stride)
    for (uint32_t q = 0; q < teams; ++q) {
      b += before[q * stride + e];
      all += total[q * stride + e];
    }
  uint32_t every;
  const uint32_t at = group_scan<kPlaceThreads / 64>(all, sums, &every);  // its barrier is behind the reads above
  if (tid < (uint32_t)E) {
    before[tid] = at + b;
    if (blockIdx.x == 0) offsets[tid] = (int32_t)at;
  }
  if (blockIdx.x == 0 && tid == 0) offsets[E] = (int32_t)every;
  __syncthreads();
  const uint64_t first = (uint64_t)blockIdx.x * tile, last = first + tile < pairs ? first + tile : pairs;
  for (uint64_t p = first + tid; p < last; p += kPlaceThreads) {
    const int32_t id = ids[p];
    if (id >= 0 && id < E) slots[p] += (int32_t)before[id];
  }
}

// -- rows -------------------------------------------------------------------
//
// A row of up to 32 vectors shares a wave with others: `lanes` (a power of
// two) of them a row.  Of a longer one a wave takes 64 vectors at a time; all
// of its lanes have the same row then, and slots and weights come by scalar
// loads.
constexpr int kThreads = 256, kWaves = kThreads / 64;

struct Rows {
  uint64_t units;    // of work, one a wave: 64 vectors of a row, or 64 / lanes rows
  uint32_t segs;     // units a row (LONG)
  uint32_t lanes;    // lanes a row (not LONG)
  uint32_t vecs;     // vectors a row
};

// The row and the vector of a lane in unit u; false where there is none.
template <bool LONG>
__device__ __forceinline__ bool place_of(const Rows &r, uint64_t u, uint64_t B, uint32_t per, uint64_t *row,
                                         uint32_t *v) {
  const uint32_t lane = threadIdx.x & 63;
  if constexpr (LONG) {
    // (units are below 2^32 but for rows beyond a few TB)
    *row = u >> 32 ? u / per : (uint32_t)u / per;
    *v = (uint32_t)(u - *row * per) * 64 + lane;
    return true;
  } else {
    *row = u * (64 / r.lanes) + lane / r.lanes;
    *v = lane & (r.lanes - 1);
    return *row < B;
  }
}

__device__ __forceinline__ uint64_t wave_index() {
  return (uint64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// -- gather -----------------------------------------------------------------
//
// A lane moves a vector (T: 16 or 8 bytes) of a row to the row's places.  A
// row's scale bytes are a further unit of it (LONG), or a lane each.
template <class T, bool LONG>
__global__ __launch_bounds__(kThreads) void gather_kernel(const T *__restrict__ x, const uint8_t *__restrict__ scales,
                                                          const int32_t *__restrict__ slots, T *__restrict__ rows,
                                                          uint8_t *__restrict__ row_scales, Rows r, uint64_t B,
                                                          uint32_t blocks, int k, uint32_t pairs) {
  const uint32_t per = r.segs + (scales ? 1 : 0);
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    if (!place_of<LONG>(r, u, B, per, &row, &v)) continue;
    const int32_t *to = slots + row * k;
    if (LONG ? v >= r.segs * 64 : scales && v < blocks) {
      for (uint32_t i = LONG ? v - r.segs * 64 : v; i < blocks; i += 64) {
        const uint8_t d = scales[row * blocks + i];
        for (int j = 0; j < k; ++j) {
          const uint32_t slot = (uint32_t)to[j];
          if (slot < pairs) row_scales[(size_t)slot * blocks + i] = d;
        }
      }
    }
    if (v >= r.vecs) continue;
    const T d = __builtin_nontemporal_load(x + row * r.vecs + v);
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = (uint32_t)to[j];
      if (slot < pairs) __builtin_nontemporal_store(d, rows + (size_t)slot * r.vecs + v);
    }
  }
}

// -- combine ----------------------------------------------------------------

constexpr int kBatch = 8;  // slots whose rows are in flight at a time

template <bool LONG>
__global__ __launch_bounds__(kThreads) void combine_kernel(const u32x4 *__restrict__ Y,
                                                           const int32_t *__restrict__ slots,
                                                           const float *__restrict__ weights,
                                                           const u32x4 *__restrict__ shared, u32x4 *__restrict__ out,
                                                           Rows r, uint64_t B, int k, uint32_t pairs) {
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    if (!place_of<LONG>(r, u, B, r.segs, &row, &v) || v >= r.vecs) continue;
    const size_t at = row * r.vecs + v;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (shared) widen8(__builtin_nontemporal_load(shared + at), o);
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      u32x4 y[kBatch];
      float w[kBatch];
      bool there[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        there[j] = false;
        if (j0 + j >= k) continue;
        const uint32_t slot = (uint32_t)slots[row * k + j0 + j];
        there[j] = slot < pairs;
        w[j] = weights ? weights[row * k + j0 + j] : 1.0f;
        if (there[j]) y[j] = __builtin_nontemporal_load(Y + (size_t)slot * r.vecs + v);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!there[j]) continue;
        float f[8];
        widen8(y[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w[j], f[e], o[e]);
      }
    }
    store16_nt(out + at, u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                               pack_bf16x2(o[6], o[7])});
  }
}

// -- its gradients ----------------------------------------------------------

// A vector of dY, and its part of the weight's gradient.
__device__ __forceinline__ u32x4 weighted(u32x4 g, float w) {
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(w * bf16_lo(g[q]), w * bf16_hi(g[q]));
  return o;
}
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float acc) {
#pragma unroll
  for (int q = 0; q < 4; ++q) acc = dot2_bf16(a[q], b[q], acc);
  return acc;
}

// A workgroup takes a row.
constexpr int kRowWaves = 16;
__global__ __launch_bounds__(64 * kRowWaves) void combine_bwd_kernel(
    const u32x4 *__restrict__ Y, const int32_t *__restrict__ slots, const float *__restrict__ weights,
    const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY, float *__restrict__ dweights, uint32_t B, uint32_t cvec,
    int k, uint32_t pairs) {
  __shared__ float part[2][kMaxChosen][kRowWaves];
  const uint32_t T = blockDim.x, waves = T >> 6;
  const int wave = threadIdx.x >> 6, row16 = (threadIdx.x & 63) >> 4;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x, turn ^= 1) {
    const u32x4 *d = dout + (size_t)row * cvec;
    const int32_t *from = slots + (size_t)row * k;
    const float *weight = weights + (size_t)row * k;
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      float dot[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) dot[j] = 0.f;
      for (uint32_t v = threadIdx.x; v < cvec; v += T) {
        const u32x4 g = d[v];
        u32x4 y[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (j0 + j >= k) continue;
          const uint32_t slot = (uint32_t)from[j0 + j];
          if (slot < pairs) y[j] = __builtin_nontemporal_load(Y + (size_t)slot * cvec + v);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (j0 + j >= k) continue;
          const uint32_t slot = (uint32_t)from[j0 + j];
          if (slot >= pairs) continue;
          dot[j] = dot8(g, y[j], dot[j]);
          store16_nt(dY + (size_t)slot * cvec + v, weighted(g, weight[j0 + j]));
        }
      }
      wave_sums(dot);  // v[i] of lane row q: the sum of slot i + 2 (q & 1) + 4 (q / 2)
      if ((threadIdx.x & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kBatch / 4; ++i) {
          const int j = j0 + i + kBatch / 4 * (row16 & 1) + kBatch / 2 * (row16 >> 1);
          if (j < k) part[turn][j][wave] = dot[i];
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < (uint32_t)k) {
      float t = 0.f;
      for (uint32_t w = 0; w < waves; ++w) t += part[turn][threadIdx.x][w];
      dweights[(size_t)row * k + threadIdx.x] = t;
    }
  }
}

// Rows of up to 32 vectors, several a wave.
__global__ __launch_bounds__(kThreads) void combine_bwd_short_kernel(
    const u32x4 *__restrict__ Y, const int32_t *__restrict__ slots, const float *__restrict__ weights,
    const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY, float *__restrict__ dweights, Rows r, uint64_t B, int k,
    uint32_t pairs) {
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    const bool real = place_of<false>(r, u, B, 1, &row, &v);
    const bool mine = real && v < r.vecs;
    const u32x4 g = mine ? dout[row * r.vecs + v] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = real ? (uint32_t)slots[row * k + j] : ~0u;
      float dot = 0.f;
      if (mine && slot < pairs) {
        const size_t at = (size_t)slot * r.vecs + v;
        dot = dot8(g, __builtin_nontemporal_load(Y + at), 0.f);
        store16_nt(dY + at, weighted(g, weights[row * k + j]));
      }
      for (uint32_t m = 1; m < r.lanes; m <<= 1) dot += __shfl_xor(dot, m);
      if (real && v == 0) dweights[row * k + j] = dot;
    }
  }
}

uint32_t grid_of(uint64_t total, int per) {
  const uint64_t wgs = (total + per - 1) / per;
  return (uint32_t)(wgs < (1u << 22) ? wgs : (1u << 22));
}

bool is_long(int64_t vecs) { return vecs > 32; }

// more: units a row beside its vectors' (LONG).
Rows rows_of(int64_t B, int64_t vecs, int more) {
  Rows r{};
  r.vecs = (uint32_t)vecs;
  r.segs = (uint32_t)((vecs + 63) / 64);
  r.lanes = 1;
  if (is_long(vecs)) {
    r.units = (uint64_t)B * (r.segs + more);
  } else {
    while (r.lanes < vecs) r.lanes *= 2;
    r.units = ((uint64_t)B * r.lanes + 63) / 64;
  }
  return r;
}

template <class T>
hipError_t gather_t(int64_t B, int k, int64_t vecs, const void *x, const uint8_t *scales, int64_t blocks,
                    const int32_t *slots, void *rows, uint8_t *row_scales, hipStream_t st) {
  const Rows r = rows_of(B, vecs, scales ? 1 : 0);
  const auto kernel = is_long(vecs) ? gather_kernel<T, true> : gather_kernel<T, false>;
  kernel<<<grid_of(r.units, kWaves), kThreads, 0, st>>>(static_cast<const T *>(x), scales, slots,
                                                        static_cast<T *>(rows), row_scales, r, (uint64_t)B,
                                                        (uint32_t)blocks, k, (uint32_t)(B * k));
  return hipGetLastError();
}

}  // namespace

// Tiles of at least 1024 pairs, at most 256 of them: their counts are added up
// by every workgroup of the second kernel.
OrderPlan plan_experts_order(int64_t pairs, int E) {
  OrderPlan p;
  constexpr int64_t kMost = 256;
  const int64_t chunks = (pairs + kChunk - 1) / kChunk;
  p.tile = (chunks + kMost - 1) / kMost * kChunk;
  p.tiles = (pairs + p.tile - 1) / p.tile;
  p.total_bytes = (size_t)p.tiles * E * 4;
  return p;
}

hipError_t launch_experts_order(const OrderPlan &p, int64_t pairs, int E, const int32_t *ids, int32_t *slots,
                                int32_t *offsets, void *ws, hipStream_t st) {
  if (pairs <= kOnePairs) {
    order_kernel<<<1, 64 * kOneWaves, (size_t)kOneWaves * E * 2, st>>>(ids, (uint32_t)pairs, E, slots, offsets);
    return hipGetLastError();
  }
  uint32_t *counts = static_cast<uint32_t *>(ws), stride = 64;
  while (stride < (uint32_t)E) stride *= 2;
  const uint32_t tiles = (uint32_t)p.tiles;
  rank_kernel<<<tiles, 64 * kRankWaves, (size_t)kRankWaves * E * 2, st>>>(ids, (uint32_t)pairs, (uint32_t)p.tile, E,
                                                                          slots, counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_kernel<<<tiles, kPlaceThreads, 0, st>>>(ids, (uint32_t)pairs, (uint32_t)p.tile, tiles, E, stride, counts,
                                                slots, offsets);
  return hipGetLastError();
}

hipError_t launch_experts_gather(int64_t B, int k, int64_t C, const void *x, const uint8_t *scales,
                                 const int32_t *slots, void *rows, uint8_t *row_scales, hipStream_t st) {
  if (!scales) return gather_t<u32x4>(B, k, C / 8, x, nullptr, 0, slots, rows, nullptr, st);
  const int64_t blocks = ckpt_blocks(C);
  return C % 16 == 0 ? gather_t<u32x4>(B, k, C / 16, x, scales, blocks, slots, rows, row_scales, st)
                     : gather_t<u32x2>(B, k, C / 8, x, scales, blocks, slots, rows, row_scales, st);
}

hipError_t launch_experts_combine(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                  const float *weights, const void *shared, void *out, hipStream_t st) {
  const Rows r = rows_of(B, C / 8, 0);
  const auto kernel = is_long(C / 8) ? combine_kernel<true> : combine_kernel<false>;
  kernel<<<grid_of(r.units, kWaves), kThreads, 0, st>>>(static_cast<const u32x4 *>(Y), slots, weights,
                                                        static_cast<const u32x4 *>(shared), static_cast<u32x4 *>(out),
                                                        r, (uint64_t)B, k, (uint32_t)(B * k));
  return hipGetLastError();
}

hipError_t launch_experts_combine_bwd(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                      const float *weights, const void *dout, void *dY, float *dweights,
                                      hipStream_t st) {
  const auto *y = static_cast<const u32x4 *>(Y), *g = static_cast<const u32x4 *>(dout);
  u32x4 *dy = static_cast<u32x4 *>(dY);
  const uint32_t pairs = (uint32_t)(B * k), cvec = (uint32_t)(C / 8);
  if (!is_long(cvec)) {
    const Rows r = rows_of(B, cvec, 0);
    combine_bwd_short_kernel<<<grid_of(r.units, kWaves), kThreads, 0, st>>>(y, slots, weights, g, dy, dweights, r,
                                                                            (uint64_t)B, k, pairs);
  } else {
    const uint32_t waves = (cvec + 63) / 64 < kRowWaves ? (cvec + 63) / 64 : kRowWaves;
    const uint32_t grid = (uint32_t)(B < (1 << 21) ? B : (1 << 21));
    combine_bwd_kernel<<<grid, 64 * waves, 0, st>>>(y, slots, weights, g, dy, dweights, (uint32_t)B, cvec, k, pairs);
  }
  return hipGetLastError();
}

}  // namespace mhc
