// The first layer's residual stream from token embeddings, and the embedding
// table's gradient.
//
//   X_0[b, i, :] = bf16(scale * table[token[b], :])      for every stream i
//   dtable[v, :] = scale * sum over {b : token[b] = v} and i of dX_0[b, i, :]
//
// The gradient goes over the rows in the order of their tokens (and of their
// index where tokens are equal): equal tokens are neighbours then, each table
// row is summed in a fixed order without atomics, and dX_0 is read once.
#include "mhc_device.h"
#include "mhc_train.h"

#include <type_traits>
#include <utility>

namespace mhc {

namespace {

constexpr int kThreads = 256;

// A lane reads eight channels of the table's row and writes them to every
// stream.  Bound by the writes: 184 us at n=4, C=7168, B=16384 (1.01 GB, of
// which 0.94 are X_0; 5.5 TB/s); one token takes a launch (6.3 us).
template <int NS>
__global__ __launch_bounds__(kThreads) void embed_kernel(const int64_t *__restrict__ tokens,
                                                         const u32x4 *__restrict__ table, float scale,
                                                         u32x4 *__restrict__ X, uint64_t total, uint32_t cvec,
                                                         int64_t V) {
  for (uint64_t t = (uint64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = t / cvec;
    const uint32_t v = (uint32_t)(t - row * cvec);
    const int64_t id = tokens[row];
    u32x4 o = {0u, 0u, 0u, 0u};
    if (id >= 0 && id < V) {
      const u32x4 w = table[(size_t)id * cvec + v];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(scale * bf16_lo(w[q]), scale * bf16_hi(w[q]));
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) store16_nt(X + (row * NS + i) * cvec + v, o);
  }
}

// -- the rows in the order of their tokens ----------------------------------
//
// A key is (token << 32) | row; tokens outside the table get kNoToken, which
// sorts last.  Keys are all different, so any correct sort gives the same
// order.  Tiles of 1024 keys are sorted in one workgroup each; then runs are
// joined 16 at a time: a key's place in the joined run is its place in its
// own run plus, for each other run, the number of smaller keys there (a
// binary search).  One launch for up to 1024 rows (5.5 us), two for up to
// 16384 (19 us: the tiles' bitonic sort and the join are chains of lane moves
// and LDS reads).
typedef unsigned long long u64;
constexpr uint32_t kNoToken = 0xffffffffu;
constexpr uint32_t kTile = 1024, kJoin = 16;

__device__ __forceinline__ uint32_t token_of(u64 key) { return (uint32_t)(key >> 32); }

// The value of lane ^ D, without LDS: DPP inside rows of 16 lanes, row and
// half swaps beyond.
template <int D>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
  const auto dpp = [](uint32_t v, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xF, 0xF, false);
  };
  if constexpr (D == 1) return dpp(x, std::integral_constant<int, 0xB1>{});
  if constexpr (D == 2) return dpp(x, std::integral_constant<int, 0x4E>{});
  // 7 - lane in its eight, then 3 - lane in its four
  if constexpr (D == 4) return dpp(dpp(x, std::integral_constant<int, 0x141>{}), std::integral_constant<int, 0x1B>{});
  if constexpr (D == 8) return dpp(x, std::integral_constant<int, 0x128>{});  // lane + 8 in its row
  if constexpr (D == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return threadIdx.x & 16 ? s[0] : s[1];
  }
  if constexpr (D == 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return threadIdx.x & 32 ? s[0] : s[1];
  }
}
template <int D>
__device__ __forceinline__ u64 lane_xor64(u64 x) {
  return ((u64)lane_xor<D>((uint32_t)(x >> 32)) << 32) | lane_xor<D>((uint32_t)x);
}

// Bitonic sort, one key a thread: a step's partners are D apart.
template <int SIZE, int D>
__device__ __forceinline__ void sort_steps(u64 &key, u64 *swap, uint32_t t) {
  u64 other;
  if constexpr (D >= 64) {
    __syncthreads();
    swap[t] = key;
    __syncthreads();
    other = swap[t ^ D];
  } else {
    other = lane_xor64<D>(key);
  }
  const bool up = (t & SIZE) == 0, low = (t & D) == 0;
  key = (up == low) == (key < other) ? key : other;
  if constexpr (D > 1) sort_steps<SIZE, D / 2>(key, swap, t);
}
template <int SIZE>
__device__ __forceinline__ void sort_tile(u64 &key, u64 *swap, uint32_t t) {
  sort_steps<SIZE, SIZE / 2>(key, swap, t);
  if constexpr (SIZE < (int)kTile) sort_tile<2 * SIZE>(key, swap, t);
}

__global__ __launch_bounds__(kTile) void sort_tiles_kernel(const int64_t *__restrict__ tokens, uint32_t B, int64_t V,
                                                           u64 *__restrict__ keys) {
  __shared__ u64 swap[kTile];
  const uint32_t t = threadIdx.x;
  const uint64_t row = (uint64_t)blockIdx.x * kTile + t;
  u64 key = ~0ull;
  if (row < B) {
    const int64_t id = tokens[row];
    key = ((u64)(id >= 0 && id < V ? (uint32_t)id : kNoToken) << 32) | row;
  }
  sort_tile<2>(key, swap, t);
  if (row < B) keys[row] = key;
}

// Runs of `run` sorted keys (a power of two) -> runs of kJoin times that.  The
// searches of a key in the other runs go side by side, as each is a chain of
// dependent loads.
__global__ __launch_bounds__(kThreads) void join_runs_kernel(const u64 *__restrict__ in, u64 *__restrict__ out,
                                                             uint32_t B, uint64_t run, int log_run) {
  const uint64_t p = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (p >= B) return;
  const u64 key = in[p];
  const uint64_t mine = p >> log_run, first = mine / kJoin * kJoin;
  uint64_t less[kJoin];  // keys of each run found to be smaller
#pragma unroll
  for (uint32_t u = 0; u < kJoin; ++u) less[u] = 0;
  for (uint64_t step = run; step > 0; step >>= 1) {
#pragma unroll
    for (uint32_t u = 0; u < kJoin; ++u) {
      // the first less[u] keys are smaller; are the next `step` ones too?
      const uint64_t upto = less[u] + step, at = ((first + u) << log_run) + upto - 1;
      const bool there = upto <= run && at < B;
      const u64 other = in[there ? at : p];
      less[u] = there && other < key ? upto : less[u];
    }
  }
  uint64_t place = first << log_run;
#pragma unroll
  for (uint32_t u = 0; u < kJoin; ++u) place += less[u];  // its own run counts the keys before it
  out[place] = key;
}

// The same for the first level, whose runs are the tiles: their tokens fit
// LDS (64 KiB), where a step of the searches costs a tenth of what it does in
// the cache.  Of equal tokens the rows of an earlier tile come first.  TILES:
// kJoin, or fewer where there are no more.
constexpr uint32_t kJoinThreads = 512;  // a workgroup's keys are of one tile
template <uint32_t TILES>
__global__ __launch_bounds__(kJoinThreads) void join_tiles_kernel(const u64 *__restrict__ in, u64 *__restrict__ out,
                                                                  uint32_t B) {
  constexpr uint32_t kAll = TILES * kTile, kLoads = kAll / 2 / kJoinThreads;
  __shared__ uint32_t tok[kAll];
  const uint32_t p = blockIdx.x * kJoinThreads + threadIdx.x;
  const uint32_t first = p / kAll * kAll, count = B - first < kAll ? B - first : kAll;
  // Two keys a load, all of a thread's loads in flight at once.
  ulonglong2 two[kLoads];
#pragma unroll
  for (uint32_t k = 0; k < kLoads; ++k) {
    const uint32_t at = 2 * (threadIdx.x + k * kJoinThreads);
    two[k] = at + 1 < count ? *reinterpret_cast<const ulonglong2 *>(in + first + at)
                            : ulonglong2{at < count ? in[first + at] : ~0ull, ~0ull};
  }
#pragma unroll
  for (uint32_t k = 0; k < kLoads; ++k)
    *reinterpret_cast<uint2 *>(tok + 2 * (threadIdx.x + k * kJoinThreads)) = uint2{token_of(two[k].x), token_of(two[k].y)};
  __syncthreads();
  if (p >= B) return;
  const u64 key = in[p];
  const uint32_t mine = (p - first) / kTile, token = token_of(key);
  uint32_t less[TILES];
#pragma unroll
  for (uint32_t u = 0; u < TILES; ++u) less[u] = 0;
  for (uint32_t step = kTile; step > 0; step >>= 1) {
#pragma unroll
    for (uint32_t u = 0; u < TILES; ++u) {
      // (places past the last key hold ~0, which no token exceeds)
      const uint32_t upto = less[u] + step, there = tok[u * kTile + (upto <= kTile ? upto : kTile) - 1];
      const bool before = there < token || (there == token && u < mine);
      less[u] = before && upto <= kTile ? upto : less[u];
    }
  }
  uint32_t place = first;
#pragma unroll
  for (uint32_t u = 0; u < TILES; ++u) place += u == mine ? p - first - mine * kTile : less[u];
  out[place] = key;
}

// First place whose token is not below `token`.
__device__ __forceinline__ uint32_t first_place(const u64 *keys, uint32_t B, u64 token) {
  uint32_t lo = 0, len = B;
  while (len > 0) {
    const uint32_t half = len >> 1;
    if ((keys[lo + half] >> 32) < token) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo;
}

// -- the table's gradient ---------------------------------------------------

__device__ __forceinline__ void write_row(f32x4 *o, const float (&acc)[8], float scale, bool accumulate) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 x = f32x4{acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]} * scale;
    if (accumulate) x += o[h];
    o[h] = x;  // half of every 32 bytes: the cache joins the two (streaming stores cost 45 us more)
  }
}

// A wave takes `rb` places of the sorted order (a block) and 512 channels and
// adds up each token's rows in their order.  A token whose rows all lie in
// the block is written to the table; a block's first token that began before
// it, and its last that goes on after it, are left in `part` ([blocks][2][C]:
// from the left, to the right) for the join below.  Workgroups from sum_wgs
// on write zeros to the table rows that have no token: kZeroBytes or a row each,
// kZeroRows at most (with 8 rows each the table of n=4, C=7168, B=16384,
// V=32768 took 405 us, not 396, and V=65536, C=64 with 300 rows 30, not 18).
//
// Bound by HBM where there are many rows: 336 us of the call's 398 at n=4,
// C=7168, B=16384, V=32768, for 0.94 GB of dX_0 and 0.94 of the table (5.6
// TB/s), 250 where it adds to the table (1.24 GB); by latency where there are
// few (8 us at n=2, C=1000, B=1001).
constexpr int kAhead = 16;  // 16-byte loads a lane has in flight
constexpr uint32_t kZeroRows = 32, kZeroBytes = 1 << 14;

// Eight lanes search for a row's token together, nine parts a step; a wave
// searches for eight rows.  All threads then write the absent ones, whatever
// their width.
__device__ __forceinline__ void zero_rows(const u64 *keys, uint32_t B, uint64_t v0, uint32_t rows, uint32_t V, uint32_t cvec,
                                          f32x4 *dtable) {
  static_assert(kZeroRows == kThreads / 8, "eight lanes for each row");
  __shared__ uint8_t absent[kZeroRows];
  const uint32_t lane = threadIdx.x & 63, s = lane & 7, shift = lane & 56;
  const u64 token = v0 + (threadIdx.x >> 3);
  uint32_t lo = 0, len = (threadIdx.x >> 3) < rows ? B : 0;  // [lo, lo + len] holds the first place not below the token
  while (__any(len > 0)) {
    const uint32_t part = (len + 8) / 9, at = lo + s * part + part - 1;
    const bool probe = len > 0 && s * part + part <= len;
    const uint32_t probes = (uint32_t)__builtin_popcountll((__ballot(probe) >> shift) & 0xff);
    const bool below = probe && (keys[at] >> 32) < token;
    const uint32_t found = (uint32_t)__builtin_popcountll((__ballot(below) >> shift) & 0xff);
    lo += found * part;
    len = len == 0 ? 0 : found == probes ? len - found * part : part - 1;
  }
  if (s == 0 && (threadIdx.x >> 3) < rows) absent[threadIdx.x >> 3] = token < V && (lo >= B || token_of(keys[lo]) != token);
  __syncthreads();
  const uint32_t width = 2 * cvec, down = kThreads / width, along = kThreads % width;
  uint32_t row = threadIdx.x / width, c = threadIdx.x % width;
  while (row < rows) {
    if (absent[row]) __builtin_nontemporal_store(f32x4{0.f, 0.f, 0.f, 0.f}, dtable + (v0 + row) * width + c);
    row += down;
    c += along;
    if (c >= width) c -= width, ++row;
  }
  __syncthreads();
}

template <int NS>
__device__ __forceinline__ void sum_block(const u64 *__restrict__ keys, const u32x4 *__restrict__ G, float scale,
                                          bool accumulate, f32x4 *__restrict__ dtable, float *__restrict__ part,
                                          uint32_t B, uint32_t cvec, uint32_t rb, uint32_t block, uint32_t slice) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t v = slice * 64 + lane;
  const uint32_t p0 = block * rb, m = B - p0 < rb ? B - p0 : rb;
  const u64 key = lane < m ? keys[p0 + lane] : ~0ull;
  const uint32_t tok = token_of(key), row = (uint32_t)key;
  const uint32_t before = p0 > 0 ? token_of(keys[p0 - 1]) : kNoToken;
  const uint32_t after = p0 + m < B ? token_of(keys[p0 + m]) : kNoToken;
  constexpr int U = kAhead / NS;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool began = __builtin_amdgcn_readlane((int)tok, 0) != (int)before;
  for (uint32_t base = 0; base < m; base += U) {
    u32x4 g[U][NS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t q = base + u;
      if (q >= m || v >= cvec || (uint32_t)__builtin_amdgcn_readlane((int)tok, (int)q) == kNoToken) continue;
      const uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)row, (int)q);
#pragma unroll
      for (int i = 0; i < NS; ++i) g[u][i] = __builtin_nontemporal_load(G + ((size_t)r * NS + i) * cvec + v);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t q = base + u;
      if (q >= m) break;
      const uint32_t here = (uint32_t)__builtin_amdgcn_readlane((int)tok, (int)q);
      if (here == kNoToken) return;  // and so are all after it
      const uint32_t next = q + 1 < m ? (uint32_t)__builtin_amdgcn_readlane((int)tok, (int)(q + 1)) : after;
      if (v < cvec) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            acc[2 * w] += bf16_lo(g[u][i][w]);
            acc[2 * w + 1] += bf16_hi(g[u][i][w]);
          }
        const bool ends = next != here;
        if (ends && began) {
          write_row(dtable + ((size_t)here * cvec + v) * 2, acc, scale, accumulate);
        } else if (ends || q + 1 == m) {
          f32x4 *o = reinterpret_cast<f32x4 *>(part) + (((size_t)block * 2 + (began ? 1 : 0)) * cvec + v) * 2;
          o[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
          o[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
        }
      }
      if (next != here) {
        began = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
    }
  }
}

template <int NS>
__global__ __launch_bounds__(kThreads) void table_kernel(const u64 *__restrict__ keys, const u32x4 *__restrict__ G,
                                                         float scale, bool accumulate, f32x4 *__restrict__ dtable,
                                                         float *__restrict__ part, uint32_t B, uint32_t cvec,
                                                         uint32_t slices, uint32_t rb, uint64_t items,
                                                         uint64_t sum_wgs, uint64_t all_wgs, uint32_t zero, uint32_t V) {
  for (uint64_t wg = blockIdx.x; wg < all_wgs; wg += gridDim.x) {
    if (wg >= sum_wgs) {
      zero_rows(keys, B, (wg - sum_wgs) * zero, zero, V, cvec, dtable);
      continue;
    }
    const uint64_t item = (uint64_t)uniform((int64_t)(wg * (kThreads / 64) + (threadIdx.x >> 6)));
    if (item >= items) continue;
    const uint64_t block = item / slices;
    sum_block<NS>(keys, G, scale, accumulate, dtable, part, B, cvec, rb, (uint32_t)block,
                  (uint32_t)(item - block * slices));
  }
}

// The tokens whose rows span blocks: the piece that begins one, then the
// pieces of the blocks that follow, in their order.  A workgroup a block and
// slice; its four waves take a quarter of the following blocks each, and the
// quarters are added in their order.
__device__ __forceinline__ void join_part(const u64 *__restrict__ keys, const float *__restrict__ part, float scale,
                                          bool accumulate, f32x4 *__restrict__ dtable, uint32_t B, uint32_t cvec,
                                          uint32_t rb, uint32_t block, uint32_t slice) {
  constexpr int W = kThreads / 64;
  __shared__ float quarter[W - 1][8][64];
  const uint32_t p0 = block * rb, p1 = p0 + rb;
  if (p1 >= B) return;
  const uint32_t tok = token_of(keys[p1]);
  if (tok == kNoToken || token_of(keys[p1 - 1]) != tok) return;               // nothing goes on to the right
  if (p0 > 0 && token_of(keys[p0]) == tok && token_of(keys[p0 - 1]) == tok) return;  // it did not begin here
  const uint32_t last = (first_place(keys, B, (u64)tok + 1) - 1) / rb;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, v = slice * 64 + lane;
  const uint32_t follow = last - block, each = (follow + W - 1) / W;
  const uint32_t lo = block + 1 + wave * each;
  const uint32_t hi = lo + each < last + 1 ? lo + each : last + 1;
  const f32x4 *src = reinterpret_cast<const f32x4 *>(part);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  if (v < cvec) {
    if (wave == 0) {
      const f32x4 *s = src + (((size_t)block * 2 + 1) * cvec + v) * 2;
      const f32x4 a = s[0], b = s[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = a[e], acc[4 + e] = b[e];
    }
    for (uint32_t k = lo; k < hi; k += 8) {
      f32x4 a[8], b[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u)
        if (k + u < hi) {
          const f32x4 *s = src + ((size_t)(k + u) * 2 * cvec + v) * 2;
          a[u] = s[0], b[u] = s[1];
        }
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u)
        if (k + u < hi) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += a[u][e], acc[4 + e] += b[u][e];
        }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) quarter[wave - 1][e][lane] = acc[e];
  }
  __syncthreads();
  if (wave > 0 || v >= cvec) return;
#pragma unroll
  for (int w = 0; w < W - 1; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += quarter[w][e][lane];
  write_row(dtable + ((size_t)tok * cvec + v) * 2, acc, scale, accumulate);
}

__global__ __launch_bounds__(kThreads) void join_parts_kernel(const u64 *__restrict__ keys,
                                                              const float *__restrict__ part, float scale,
                                                              bool accumulate, f32x4 *__restrict__ dtable, uint32_t B,
                                                              uint32_t cvec, uint32_t slices, uint32_t rb,
                                                              uint64_t items) {
  for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint64_t block = item / slices;
    join_part(keys, part, scale, accumulate, dtable, B, cvec, rb, (uint32_t)block, (uint32_t)(item - block * slices));
    __syncthreads();
  }
}

uint32_t wgs(uint64_t work, uint64_t per, uint64_t most) {
  const uint64_t g = (work + per - 1) / per;
  return (uint32_t)(g < most ? g : most);
}

template <int NS>
hipError_t embed_n(int64_t B, int64_t C, int64_t V, const int64_t *tokens, const void *table, float scale, void *X,
                   hipStream_t st) {
  const uint32_t cvec = (uint32_t)(C / 8);
  const uint64_t total = (uint64_t)B * cvec;
  embed_kernel<NS><<<wgs(total, kThreads, 1u << 22), kThreads, 0, st>>>(
      tokens, static_cast<const u32x4 *>(table), scale, static_cast<u32x4 *>(X), total, cvec, V);
  return hipGetLastError();
}

template <int NS>
hipError_t table_n(const EmbedBwdPlan &p, int64_t B, int64_t C, int64_t V, const int64_t *tokens, const void *G,
                   float scale, bool accumulate, float *dtable, char *ws, hipStream_t st) {
  const uint32_t cvec = (uint32_t)(C / 8), slices = (cvec + 63) / 64, rows = (uint32_t)B, rb = (uint32_t)p.rb;
  u64 *keys = reinterpret_cast<u64 *>(ws + p.keys), *other = reinterpret_cast<u64 *>(ws + p.other);
  float *part = reinterpret_cast<float *>(ws + p.part);
  f32x4 *out = reinterpret_cast<f32x4 *>(dtable);
  hipError_t e;
  sort_tiles_kernel<<<(uint32_t)((B + kTile - 1) / kTile), kTile, 0, st>>>(tokens, rows, V, keys);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  int log_run = 10;
  for (uint64_t run = kTile; run < (uint64_t)B; run *= kJoin, log_run += 4) {
    if (run == kTile) {  // (a call of 1100 rows: 21 us with two tiles, 28 with kJoin)
      const uint32_t grid = (uint32_t)((B + kJoinThreads - 1) / kJoinThreads);
      if (B <= 2 * kTile)
        join_tiles_kernel<2><<<grid, kJoinThreads, 0, st>>>(keys, other, rows);
      else if (B <= 4 * kTile)
        join_tiles_kernel<4><<<grid, kJoinThreads, 0, st>>>(keys, other, rows);
      else if (B <= 8 * kTile)
        join_tiles_kernel<8><<<grid, kJoinThreads, 0, st>>>(keys, other, rows);
      else
        join_tiles_kernel<kJoin><<<grid, kJoinThreads, 0, st>>>(keys, other, rows);
    } else {
      join_runs_kernel<<<(uint32_t)((B + kThreads - 1) / kThreads), kThreads, 0, st>>>(keys, other, rows, run, log_run);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    std::swap(keys, other);
  }
  const uint64_t blocks = (B + rb - 1) / rb, items = blocks * slices;
  const uint64_t sum_wgs = (items + kThreads / 64 - 1) / (kThreads / 64);
  uint32_t zero = kZeroRows;
  while (zero > 1 && (uint64_t)zero * C * 4 > kZeroBytes) zero /= 2;
  const uint64_t all_wgs = sum_wgs + (accumulate ? 0 : (uint64_t)(V + zero - 1) / zero);
  table_kernel<NS><<<wgs(all_wgs, 1, 1u << 22), kThreads, 0, st>>>(keys, static_cast<const u32x4 *>(G), scale,
                                                                   accumulate, out, part, rows, cvec, slices, rb,
                                                                   items, sum_wgs, all_wgs, zero, (uint32_t)V);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (blocks > 1)
    join_parts_kernel<<<wgs(items, 1, 1u << 22), kThreads, 0, st>>>(keys, part, scale, accumulate, out, rows, cvec,
                                                                    slices, rb, items);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(int n, int64_t B, int64_t C, int64_t V, const int64_t *tokens, const void *table, float scale,
                        void *X_0, hipStream_t st) {
  switch (n) {
    case 1: return embed_n<1>(B, C, V, tokens, table, scale, X_0, st);
    case 2: return embed_n<2>(B, C, V, tokens, table, scale, X_0, st);
    case 4: return embed_n<4>(B, C, V, tokens, table, scale, X_0, st);
    case 8: return embed_n<8>(B, C, V, tokens, table, scale, X_0, st);
    default: return hipErrorInvalidValue;
  }
}

EmbedBwdPlan plan_embed_bwd(int64_t B, int64_t C) {
  EmbedBwdPlan p;
  const int64_t slices = (C + 511) / 512;
  // Long blocks where there are rows enough for one round of waves (4 on each
  // SIMD of the 256 compute units), short ones for latency otherwise.  In us,
  // one call at a time (V = 32768, the last one 5003; * what is taken):
  //     rows a block                   4     8    16    32    64
  //     n=4, C=7168, B=16384         440   405   391   381   367*
  //     n=4, C=1024, B=16384        92.8  82.4* 79.0  83.4   110
  //     n=4, C=256, B=3000          27.0* 29.2  36.4  51.5  80.0
  //     n=2, C=1000, B=1001         19.5* 21.2  25.9  36.4  59.0
  p.rb = 4;
  while (p.rb < 64 && B * slices / p.rb > (p.rb == 4 ? 1024 : 4096)) p.rb *= 2;
  const size_t list = ((size_t)B * 8 + 15) / 16 * 16;
  p.keys = 0;
  p.other = list;
  p.part = 2 * list;
  p.total_bytes = p.part + (size_t)((B + p.rb - 1) / p.rb) * 2 * (size_t)C * 4;
  return p;
}

hipError_t launch_embed_bwd(const EmbedBwdPlan &p, int n, int64_t B, int64_t C, int64_t V, const int64_t *tokens,
                            const void *dX_0, float scale, bool accumulate, float *dtable, void *ws, hipStream_t st) {
  char *w = static_cast<char *>(ws);
  switch (n) {
    case 1: return table_n<1>(p, B, C, V, tokens, dX_0, scale, accumulate, dtable, w, st);
    case 2: return table_n<2>(p, B, C, V, tokens, dX_0, scale, accumulate, dtable, w, st);
    case 4: return table_n<4>(p, B, C, V, tokens, dX_0, scale, accumulate, dtable, w, st);
    case 8: return table_n<8>(p, B, C, V, tokens, dX_0, scale, accumulate, dtable, w, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mhc
