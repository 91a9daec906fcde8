// The first layer's residual stream from token embeddings, and the embedding
// table's gradient.
//
//   X_0[b, i, :] = bf16(scale * table[token[b], :])      for every stream i
//   dtable[v, :] = scale * sum over {b : token[b] = v} and i of dX_0[b, i, :]
//
// The gradient goes over the rows in the order of their tokens (and of their
// index where tokens are equal), so that a table row is summed by one
// workgroup in a fixed order, without atomics.
#include "mhc_device.h"
#include "mhc_train.h"

namespace mhc {

namespace {

constexpr int kThreads = 256;

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

// Position of each row in the order of (token, row), by counting the rows
// before it.
__global__ __launch_bounds__(kThreads) void order_kernel(const int64_t *__restrict__ tokens, uint32_t B,
                                                         int64_t *__restrict__ keys, int32_t *__restrict__ rows) {
  __shared__ int64_t tile[kThreads];
  const uint64_t b = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t mine = b < B ? tokens[b] : 0;
  uint32_t before = 0;
  for (uint64_t t0 = 0; t0 < B; t0 += kThreads) {
    const uint64_t t = t0 + threadIdx.x;
    __syncthreads();
    if (t < B) tile[threadIdx.x] = tokens[t];
    __syncthreads();
    const uint32_t m = (uint32_t)(B - t0 < kThreads ? B - t0 : kThreads);
    for (uint32_t k = 0; k < m; ++k) before += tile[k] < mine || (tile[k] == mine && t0 + k < b);
  }
  if (b < B) {
    keys[before] = mine;
    rows[before] = (int32_t)b;
  }
}

__global__ __launch_bounds__(kThreads) void zero_table_kernel(f32x4 *__restrict__ p, uint64_t count) {
  for (uint64_t t = (uint64_t)blockIdx.x * kThreads + threadIdx.x; t < count; t += (uint64_t)gridDim.x * kThreads)
    p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// A workgroup for each place in the sorted order that begins a token.
template <int NS>
__global__ __launch_bounds__(kThreads) void table_kernel(const int64_t *__restrict__ keys,
                                                         const int32_t *__restrict__ rows,
                                                         const u32x4 *__restrict__ G, float scale, bool accumulate,
                                                         f32x4 *__restrict__ dtable, uint32_t B, uint32_t cvec,
                                                         int64_t V) {
  for (uint32_t p = blockIdx.x; p < B; p += gridDim.x) {
    const int64_t id = keys[p];
    if (id < 0 || id >= V || (p > 0 && keys[p - 1] == id)) continue;
    for (uint32_t v = threadIdx.x; v < cvec; v += kThreads) {
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      for (uint32_t q = p; q < B && keys[q] == id; ++q) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const u32x4 g = G[((size_t)rows[q] * NS + i) * cvec + v];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            acc[2 * w] += bf16_lo(g[w]);
            acc[2 * w + 1] += bf16_hi(g[w]);
          }
        }
      }
      f32x4 *o = dtable + ((size_t)id * cvec + v) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 x = f32x4{acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]} * scale;
        if (accumulate) x += o[h];
        o[h] = x;
      }
    }
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
  const uint32_t cvec = (uint32_t)(C / 8);
  int64_t *keys = reinterpret_cast<int64_t *>(ws + p.keys);
  int32_t *rows = reinterpret_cast<int32_t *>(ws + p.rows);
  f32x4 *out = reinterpret_cast<f32x4 *>(dtable);
  hipError_t e;
  if (!accumulate) {
    const uint64_t count = (uint64_t)V * cvec * 2;
    zero_table_kernel<<<wgs(count, kThreads, 1u << 22), kThreads, 0, st>>>(out, count);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  order_kernel<<<(uint32_t)((B + kThreads - 1) / kThreads), kThreads, 0, st>>>(tokens, (uint32_t)B, keys, rows);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  table_kernel<NS><<<wgs(B, 1, 1u << 22), kThreads, 0, st>>>(keys, rows, static_cast<const u32x4 *>(G), scale,
                                                             accumulate, out, (uint32_t)B, cvec, V);
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

EmbedBwdPlan plan_embed_bwd(int64_t B, int n, int64_t C, int64_t V) {
  (void)n, (void)C, (void)V;
  EmbedBwdPlan p;
  p.keys = 0;
  p.rows = (size_t)B * 8;
  p.total_bytes = (p.rows + (size_t)B * 4 + 15) / 16 * 16;
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
