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
// tile of 1024 pairs or more, and a second launch adds the counts of the
// earlier tiles and of the smaller experts, which each of its workgroups sums
// up for itself.
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

// A workgroup ranks the pairs of a tile, a chunk at a time.  ONE: there is no
// other, and the slots are final (3.7 us for 8 pairs, 7.2 for 4096).
constexpr int kRankWaves = 16, kChunk = kRankWaves * 64 * kRounds;
template <bool ONE>
__global__ __launch_bounds__(64 * kRankWaves) void rank_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                               uint32_t tile, int E, int32_t *__restrict__ slots,
                                                               uint32_t *__restrict__ counts,
                                                               int32_t *__restrict__ offsets) {
  extern __shared__ uint16_t seen[];  // [waves][E]
  __shared__ uint32_t so_far[kMaxExperts], sums[kRankWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, own = threadIdx.x;  // own: a thread's expert
  uint16_t *mine = seen + wave * E;
  const uint64_t first = (uint64_t)blockIdx.x * tile, last = first + tile < pairs ? first + tile : pairs;
  uint32_t total = 0;  // of the own expert
  for (uint64_t c = first; c < last; c += kChunk) {
    // Each wave takes whole rounds, so that the pairs stay in their order.
    const uint32_t size = last - c < kChunk ? (uint32_t)(last - c) : kChunk;
    const uint32_t per = (size + 64 * kRankWaves - 1) / (64 * kRankWaves), at = wave * per * 64 + lane;
    int32_t id[kRounds], rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) id[r] = (uint32_t)r < per && at + 64 * r < size ? ids[c + at + 64 * r] : -1;
    for (int e = lane; e < E; e += 64) mine[e] = 0;
    wave_ranks(id, E, mine, rank);
    __syncthreads();
    if (own < E) {  // the earlier waves' counts
      uint32_t n = 0;
#pragma unroll
      for (int w = 0; w < kRankWaves; ++w) {
        const uint32_t m = seen[w * E + own];
        seen[w * E + own] = (uint16_t)n;
        n += m;
      }
      so_far[own] = total;
      total += n;
    }
    if constexpr (ONE) {  // the smaller experts' (its barrier is before the store)
      uint32_t all;
      const uint32_t start = group_scan<kRankWaves>(total, sums, &all);
      if (own < E) {
        so_far[own] = start;
        offsets[own] = (int32_t)start;
      }
      if (own == 0) offsets[E] = (int32_t)all;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if ((uint32_t)r < per && at + 64 * r < size)
        slots[c + at + 64 * r] = rank[r] < 0 ? -1 : (int32_t)(so_far[id[r]] + mine[id[r]]) + rank[r];
    if (last - c > kChunk) __syncthreads();
  }
  if (!ONE && own < E) counts[(size_t)blockIdx.x * E + own] = total;
}

// A workgroup takes `share` pairs of a tile.  `stride`: E rounded up to a power
// of two; the threads are kPlaceThreads / stride teams that share the tiles.
constexpr int kPlaceThreads = 1024;
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(const int32_t *__restrict__ ids, uint32_t pairs,
                                                              uint32_t share, uint32_t tile, uint32_t tiles, int E,
                                                              uint32_t stride, const uint32_t *__restrict__ counts,
                                                              int32_t *__restrict__ slots,
                                                              int32_t *__restrict__ offsets) {
  __shared__ uint32_t before[kPlaceThreads], total[kPlaceThreads], sums[kPlaceThreads / 64];
  const uint32_t tid = threadIdx.x, e = tid & (stride - 1), teams = kPlaceThreads / stride;
  const uint64_t first = (uint64_t)blockIdx.x * share, last = first + share < pairs ? first + share : pairs;
  const uint32_t mine = (uint32_t)(first / tile);
  // The thread's first pair (mostly its only one), asked for ahead of the counts.
  const uint64_t own = first + tid;
  const int32_t own_id = own < last ? ids[own] : -1, own_rank = own < last ? slots[own] : 0;
  uint32_t b = 0, all = 0;
  if (e < (uint32_t)E) {
#pragma unroll 8
    for (uint32_t t = tid / stride; t < tiles; t += teams) {
      const uint32_t c = counts[(size_t)t * E + e];
      b += t < mine ? c : 0;
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
  if (own_id >= 0 && own_id < E) slots[own] = own_rank + (int32_t)before[own_id];
  for (uint64_t p = own + kPlaceThreads; p < last; p += kPlaceThreads) {
    const int32_t id = ids[p];
    if (id >= 0 && id < E) slots[p] += (int32_t)before[id];
  }
}

// -- rows -------------------------------------------------------------------
//
// A row of up to 32 vectors shares a wave with others: `lanes` (a power of
// two) of them a row.  The lanes of a wave that works on a longer one have the
// same row, and slots and weights come by scalar loads.
constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ uint64_t wave_index() {
  return (uint64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}
// (u is below 2^32 but for tensors beyond a few TB)
__device__ __forceinline__ uint64_t quotient(uint64_t u, uint32_t d) { return u >> 32 ? u / d : (uint32_t)u / d; }

// Units of work of short rows, one a wave; a lane's row and vector.
struct Short {
  uint64_t units;
  uint32_t lanes, vecs;
};
__device__ __forceinline__ bool place_of(const Short &r, uint64_t u, uint64_t B, uint64_t *row, uint32_t *v) {
  const uint32_t lane = threadIdx.x & 63;
  *row = u * (64 / r.lanes) + lane / r.lanes;
  *v = lane & (r.lanes - 1);
  return *row < B;
}

// -- gather -----------------------------------------------------------------
//
// A wave copies a row (T: vectors of 16 or 8 bytes), or one of `parts` of it,
// to one place, in one piece; the row's k waves share it in the cache.  Bound
// by the writes: 203 us for B=16384, k=8, C=7168 in 8 bits (1.09 GB, 5.4 TB/s;
// 183 for the codes without any read), 363 in bf16 (2.11 GB, 5.8 TB/s).  Waves
// that write 1 KB each to all of a row's places take 20 us more, and scales in
// a launch of their own as much or more (k=8, C=7168, us with the order: 106
// apart, 100 so at 8192 rows; 218, 215 at 16384; 303, 290 at k=2, 65536 rows).
constexpr int kGatherAhead = 8;  // vectors in flight a lane (227 us with the order; with four 260)
template <class T, class S>
__global__ __launch_bounds__(kThreads) void gather_kernel(const T *__restrict__ x, const S *__restrict__ scales,
                                                          const int32_t *__restrict__ slots, T *__restrict__ rows,
                                                          S *__restrict__ row_scales, uint64_t units, uint32_t parts,
                                                          uint32_t part, uint32_t vecs, uint32_t blocks, uint32_t k,
                                                          uint32_t pairs) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < units; u += step) {
    const uint64_t p = quotient(u, parts);
    const uint32_t first = (uint32_t)(u - p * parts) * part, slot = (uint32_t)slots[p];
    if (slot >= pairs) continue;
    const uint64_t row = (uint32_t)p / k;
    const T *from = x + row * vecs;
    T *to = rows + (size_t)slot * vecs;
    const uint32_t last = first + part < vecs ? first + part : vecs;
    // The scales are asked for first and stored last: a further wait at the
    // end of each wave took the call from 213 us to 272.
    const bool more = scales && first == 0;
    S s = 0;
    if (more && lane < blocks) s = scales[row * blocks + lane];
    for (uint32_t v0 = first + lane; v0 < last; v0 += 64 * kGatherAhead) {
      T d[kGatherAhead];
#pragma unroll
      for (int i = 0; i < kGatherAhead; ++i)
        if (v0 + 64 * i < last) d[i] = from[v0 + 64 * i];
#pragma unroll
      for (int i = 0; i < kGatherAhead; ++i)
        if (v0 + 64 * i < last) __builtin_nontemporal_store(d[i], to + v0 + 64 * i);
    }
    if (more) {
      if (lane < blocks) row_scales[(size_t)slot * blocks + lane] = s;
      for (uint32_t i = lane + 64; i < blocks; i += 64)
        row_scales[(size_t)slot * blocks + i] = scales[row * blocks + i];
    }
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void gather_short_kernel(const T *__restrict__ x,
                                                                const uint8_t *__restrict__ scales,
                                                                const int32_t *__restrict__ slots,
                                                                T *__restrict__ rows, uint8_t *__restrict__ row_scales,
                                                                Short r, uint64_t B, uint32_t blocks, int k,
                                                                uint32_t pairs) {
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    if (!place_of(r, u, B, &row, &v) || v >= r.vecs) continue;
    const T d = __builtin_nontemporal_load(x + row * r.vecs + v);
    const bool scale = scales && v < blocks;  // (there are no more of them than vectors)
    const uint8_t sc = scale ? scales[row * blocks + v] : 0;
    for (int j = 0; j < k; ++j) {
      const uint32_t slot = (uint32_t)slots[row * k + j];
      if (slot >= pairs) continue;
      __builtin_nontemporal_store(d, rows + (size_t)slot * r.vecs + v);
      if (scale) row_scales[(size_t)slot * blocks + v] = sc;
    }
  }
}

// -- combine ----------------------------------------------------------------

constexpr int kBatch = 8;  // slots whose rows are in flight at a time

// A lane takes a vector of a row: of a long one (LONG) 64 of a wave's are
// neighbours, and neighbouring waves have neighbouring pieces.
template <bool LONG>
__global__ __launch_bounds__(kThreads) void combine_kernel(const u32x4 *__restrict__ Y,
                                                           const int32_t *__restrict__ slots,
                                                           const float *__restrict__ weights,
                                                           const u32x4 *__restrict__ shared, u32x4 *__restrict__ out,
                                                           Short r, uint32_t segs, uint64_t B, int k, uint32_t pairs) {
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    if constexpr (LONG) {
      row = quotient(u, segs);
      v = (uint32_t)(u - row * segs) * 64 + (threadIdx.x & 63);
    } else if (!place_of(r, u, B, &row, &v)) {
      continue;
    }
    if (v >= r.vecs) continue;
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

// k <= 2 of many rows: a wave takes a pair, reads its row of Y and writes that of dY in one
// piece, and dout comes from the cache for all but the first of a row's waves.
constexpr int kAhead = 4;  // vectors in flight a lane (with eight 33 us, not 30, for 4096 rows at k=1, C=7168)
__global__ __launch_bounds__(kThreads) void combine_bwd_pair_kernel(
    const u32x4 *__restrict__ Y, const int32_t *__restrict__ slots, const float *__restrict__ weights,
    const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY, float *__restrict__ dweights, uint32_t cvec, uint32_t k,
    uint32_t pairs) {
  const uint32_t lane = threadIdx.x & 63, step = gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < pairs; u += step) {
    const uint32_t p = (uint32_t)u, slot = (uint32_t)slots[p];
    float dot = 0.f;
    if (slot < pairs) {
      const float w = weights[p];
      const u32x4 *d = dout + (size_t)(p / k) * cvec, *y = Y + (size_t)slot * cvec;
      u32x4 *to = dY + (size_t)slot * cvec;
      for (uint32_t v0 = 0; v0 < cvec; v0 += 64 * kAhead) {
        u32x4 a[kAhead], g[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t v = v0 + 64 * i + lane;
          if (v >= cvec) continue;
          a[i] = __builtin_nontemporal_load(y + v);
          g[i] = d[v];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t v = v0 + 64 * i + lane;
          if (v >= cvec) continue;
          dot = dot8(g[i], a[i], dot);
          store16_nt(to + v, weighted(g[i], w));
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) dweights[p] = dot;
  }
}

// A workgroup takes a row.
constexpr int kRowWaves = 16;
__global__ __launch_bounds__(64 * kRowWaves) void combine_bwd_kernel(
    const u32x4 *__restrict__ Y, const int32_t *__restrict__ slots, const float *__restrict__ weights,
    const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY, float *__restrict__ dweights, uint32_t B, uint32_t cvec,
    int k, uint32_t pairs) {
  __shared__ float part[kMaxChosen][kRowWaves];
  const uint32_t T = blockDim.x, waves = T >> 6;
  const int wave = threadIdx.x >> 6, row16 = (threadIdx.x & 63) >> 4;
  for (uint64_t row = blockIdx.x; row < B; row += gridDim.x) {
    const u32x4 *d = dout + row * cvec;
    const int32_t *from = slots + row * k;
    const float *weight = weights + row * k;
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
      wave_sums(dot);  // dot[i] of lane row q: the sum of slot i + 2 (q & 1) + 4 (q / 2)
      if ((threadIdx.x & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kBatch / 4; ++i) {
          const int j = j0 + i + kBatch / 4 * (row16 & 1) + kBatch / 2 * (row16 >> 1);
          if (j < k) part[j][wave] = dot[i];
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < (uint32_t)k) {
      float t = 0.f;
      for (uint32_t w = 0; w < waves; ++w) t += part[threadIdx.x][w];
      dweights[row * k + threadIdx.x] = t;
    }
    __syncthreads();
  }
}

// Short rows, several a wave, BATCH rows of Y in flight.
template <int BATCH>
__global__ __launch_bounds__(kThreads) void combine_bwd_short_kernel(
    const u32x4 *__restrict__ Y, const int32_t *__restrict__ slots, const float *__restrict__ weights,
    const u32x4 *__restrict__ dout, u32x4 *__restrict__ dY, float *__restrict__ dweights, Short r, uint64_t B, int k,
    uint32_t pairs) {
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  for (uint64_t u = wave_index(); u < r.units; u += step) {
    uint64_t row;
    uint32_t v;
    const bool real = place_of(r, u, B, &row, &v);
    const bool mine = real && v < r.vecs;
    const u32x4 g = mine ? dout[row * r.vecs + v] : u32x4{0u, 0u, 0u, 0u};
    for (int j0 = 0; j0 < k; j0 += BATCH) {
      u32x4 y[BATCH];
      float dot[BATCH];
      uint32_t slot[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) slot[j] = mine && j0 + j < k ? (uint32_t)slots[row * k + j0 + j] : ~0u;
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (slot[j] < pairs) y[j] = __builtin_nontemporal_load(Y + (size_t)slot[j] * r.vecs + v);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        dot[j] = 0.f;
        if (slot[j] >= pairs) continue;
        dot[j] = dot8(g, y[j], 0.f);
        store16_nt(dY + (size_t)slot[j] * r.vecs + v, weighted(g, weights[row * k + j0 + j]));
      }
      for (uint32_t m = 1; m < r.lanes; m <<= 1)
#pragma unroll
        for (int j = 0; j < BATCH; ++j) dot[j] += __shfl_xor(dot[j], m);
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (real && v == 0 && j0 + j < k) dweights[row * k + j0 + j] = dot[j];
    }
  }
}

uint32_t grid_of(uint64_t total, int per) {
  const uint64_t wgs = (total + per - 1) / per;
  return (uint32_t)(wgs < (1u << 22) ? wgs : (1u << 22));
}

bool is_long(int64_t vecs) { return vecs > 32; }

Short short_of(int64_t B, int64_t vecs) {
  Short r{0, 1, (uint32_t)vecs};
  while (r.lanes < vecs) r.lanes *= 2;
  r.units = ((uint64_t)B * r.lanes + 63) / 64;
  return r;
}

// Waves that the chip holds about once: with fewer pairs a row is shared by
// several waves (512 rows, k=8, C=7168 in 8 bits: 14.4 us so, 18.0 with four
// times the waves; from 2048 rows on they are the same).
constexpr int64_t kManyWaves = 4096;

template <class T, class S>
hipError_t gather_long(int64_t B, int k, int64_t vecs, const void *x, const void *scales, int64_t blocks,
                       const int32_t *slots, void *rows, void *row_scales, hipStream_t st) {
  const int64_t pairs = B * k, segs = (vecs + 63) / 64;
  int64_t parts = (kManyWaves + pairs - 1) / pairs;
  parts = parts < segs ? parts : segs;
  const int64_t part = (segs + parts - 1) / parts * 64;
  parts = (vecs + part - 1) / part;
  const uint64_t units = (uint64_t)(pairs * parts);
  gather_kernel<T, S><<<grid_of(units, kWaves), kThreads, 0, st>>>(
      static_cast<const T *>(x), static_cast<const S *>(scales), slots, static_cast<T *>(rows),
      static_cast<S *>(row_scales), units, (uint32_t)parts, (uint32_t)part, (uint32_t)vecs, (uint32_t)blocks,
      (uint32_t)k, (uint32_t)pairs);
  return hipGetLastError();
}

template <class T>
hipError_t gather_t(int64_t B, int k, int64_t vecs, const void *x, const uint8_t *scales, int64_t blocks,
                    const int32_t *slots, void *rows, uint8_t *row_scales, hipStream_t st) {
  if (is_long(vecs)) {
    // Scale bytes four at a time where rows and tensors allow it.
    const uintptr_t where = reinterpret_cast<uintptr_t>(scales) | reinterpret_cast<uintptr_t>(row_scales);
    if (blocks % 4 == 0 && where % 4 == 0)
      return gather_long<T, uint32_t>(B, k, vecs, x, scales, blocks / 4, slots, rows, row_scales, st);
    return gather_long<T, uint8_t>(B, k, vecs, x, scales, blocks, slots, rows, row_scales, st);
  }
  const Short r = short_of(B, vecs);
  gather_short_kernel<T><<<grid_of(r.units, kWaves), kThreads, 0, st>>>(
      static_cast<const T *>(x), scales, slots, static_cast<T *>(rows), row_scales, r, (uint64_t)B, (uint32_t)blocks,
      k, (uint32_t)(B * k));
  return hipGetLastError();
}

}  // namespace

// Small tiles are ranked by more workgroups, but their counts are added up by
// every workgroup of the second kernel (all of them read 4 tiles E bytes).  us
// with tiles of 1024, 2048 and 4096 pairs, E=256: 7.6, 8.5, 10.2 for 8192 pairs;
// 9.4, 9.4, 10.7 for 32768; 16.1, 12.9, 12.6 for 131072; E=1024 44, 27, 20 there.
// Above 2^20 pairs, where 4096 pairs a tile make 256 of them, tiles are whole chunks
// and there are 129 to 256 (29.8 us with 256 tiles at 2^20 pairs, 26.3 with 129 at
// eight more).
OrderPlan plan_experts_order(int64_t pairs, int E) {
  OrderPlan p;
  constexpr int64_t kMost = 256;
  const int64_t chunks = (pairs + kChunk - 1) / kChunk;
  const auto fits = [&](int64_t tile, int64_t counts) {
    const int64_t tiles = (pairs + tile - 1) / tile;
    return chunks > 1 && tiles <= kMost && tiles * E <= counts;
  };
  p.tile = fits(1024, 8192) ? 1024 : fits(2048, 12288) ? 2048 : (chunks + kMost - 1) / kMost * kChunk;
  p.tiles = (pairs + p.tile - 1) / p.tile;
  p.total_bytes = (size_t)p.tiles * E * 4;
  return p;
}

hipError_t launch_experts_order(const OrderPlan &p, int64_t pairs, int E, const int32_t *ids, int32_t *slots,
                                int32_t *offsets, void *ws, hipStream_t st) {
  uint32_t *counts = static_cast<uint32_t *>(ws), stride = 64;
  const uint32_t tiles = (uint32_t)p.tiles, tile = (uint32_t)p.tile;
  const size_t lds = (size_t)kRankWaves * E * 2;
  if (tiles == 1) {
    rank_kernel<true><<<1, 64 * kRankWaves, lds, st>>>(ids, (uint32_t)pairs, tile, E, slots, counts, offsets);
    return hipGetLastError();
  }
  rank_kernel<false><<<tiles, 64 * kRankWaves, lds, st>>>(ids, (uint32_t)pairs, tile, E, slots, counts, offsets);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  while (stride < (uint32_t)E) stride *= 2;
  // Shares divide a tile; 128 workgroups at least where there are pairs enough.
  uint32_t share = tile;
  while (share > kPlaceThreads && pairs / share < 128) share /= 2;
  place_kernel<<<(uint32_t)((pairs + share - 1) / share), kPlaceThreads, 0, st>>>(ids, (uint32_t)pairs, share, tile,
                                                                                  tiles, E, stride, counts, slots,
                                                                                  offsets);
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
  const auto *y = static_cast<const u32x4 *>(Y), *add = static_cast<const u32x4 *>(shared);
  u32x4 *o = static_cast<u32x4 *>(out);
  const uint32_t pairs = (uint32_t)(B * k), segs = (uint32_t)((C / 8 + 63) / 64);
  if (is_long(C / 8)) {
    const Short r{(uint64_t)B * segs, 64, (uint32_t)(C / 8)};
    combine_kernel<true><<<grid_of(r.units, kWaves), kThreads, 0, st>>>(y, slots, weights, add, o, r, segs,
                                                                        (uint64_t)B, k, pairs);
  } else {
    const Short r = short_of(B, C / 8);
    combine_kernel<false><<<grid_of(r.units, kWaves), kThreads, 0, st>>>(y, slots, weights, add, o, r, segs,
                                                                         (uint64_t)B, k, pairs);
  }
  return hipGetLastError();
}

hipError_t launch_experts_combine_bwd(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                      const float *weights, const void *dout, void *dY, float *dweights,
                                      hipStream_t st) {
  const auto *y = static_cast<const u32x4 *>(Y), *g = static_cast<const u32x4 *>(dout);
  u32x4 *dy = static_cast<u32x4 *>(dY);
  const uint32_t pairs = (uint32_t)(B * k), cvec = (uint32_t)(C / 8);
  if (!is_long(cvec)) {
    const Short r = short_of(B, cvec);
    // Rows of Y in flight, us with 1, 4 and 8: 16384 rows at k=8 C=64 15.2, 10.8, 9.0,
    // C=128 19.3, 17.0, 15.1; C=256 30.5, 31.0, 32.1 there, but 8.1, 5.6, 5.5 for 64
    // rows, and with 4 and 8 11.1, 9.1 for 4096, 17.0, 15.1 for 8192, 68.3, 70.9 for
    // 40000.  At k=4 with 1 and 4: C=64 8.6, 6.3, C=256 16.9, 15.6.
    const auto kernel = k == 1   ? combine_bwd_short_kernel<1>
                        : k <= 4 ? combine_bwd_short_kernel<4>
                                 : combine_bwd_short_kernel<8>;
    kernel<<<grid_of(r.units, kWaves), kThreads, 0, st>>>(y, slots, weights, g, dy, dweights, r, (uint64_t)B, k, pairs);
  } else if (k <= 2 && B >= 768) {
    // A workgroup a row has few loads in flight at k = 1 and 2 (C=7168, us: 30
    // against 40 for 4096 rows at k=1, 51 against 59 at k=2, 10.4 against 11.0
    // for 768 at k=1, 14.1 against 14.4 at k=2); from k = 3 on it is faster (183
    // against 188 at k=8), and with fewer rows (7.2 against 8.7 for 512 at k=1).
    combine_bwd_pair_kernel<<<grid_of(pairs, kWaves), kThreads, 0, st>>>(y, slots, weights, g, dy, dweights, cvec,
                                                                         (uint32_t)k, pairs);
  } else {
    const uint32_t waves = (cvec + 63) / 64 < kRowWaves ? (cvec + 63) / 64 : kRowWaves;
    combine_bwd_kernel<<<(uint32_t)(B < (1 << 21) ? B : (1 << 21)), 64 * waves, 0, st>>>(
        y, slots, weights, g, dy, dweights, (uint32_t)B, cvec, k, pairs);
  }
  return hipGetLastError();
}

}  // namespace mhc
