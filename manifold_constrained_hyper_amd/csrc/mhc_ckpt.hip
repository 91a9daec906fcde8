// The residual stream's 8-bit checkpoint: packing before the stream is
// dropped, unpacking where a bf16 stream is needed again (mhc_held.h has the
// number format).
//
// A lane takes eight channels (one 16-byte vector) of a stream; the four
// lanes of a block of 32 channels find its scale from the largest magnitude
// among them with two lane moves.  Bound by HBM: 2 bytes in and 1 + 1/32 out
// a channel.  A pack and an unpack of n=4, C=7168, B=16384 take 473 us for
// 2.85 GB (6.0 TB/s); of n=2, C=1000, B=1001 11.5, their two launches.
#include "mhc_held.h"
#include "mhc_finish.h"
#include "mhc_train.h"

namespace mhc {

namespace {

constexpr int kThreads = 256;

// slots: four lanes for every block of every stream of every row; cvec
// vectors a stream (the last block's lanes past it carry zeros).
__global__ __launch_bounds__(kThreads) void pack_kernel(const u32x4 *__restrict__ X, u32x2 *__restrict__ codes,
                                                        uint8_t *__restrict__ scales, uint64_t slots, uint32_t cvec,
                                                        uint32_t slots_per_stream) {
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < slots; g += (uint64_t)gridDim.x * kThreads) {
    const uint64_t stream = g / slots_per_stream;
    const uint32_t v = (uint32_t)(g - stream * slots_per_stream);
    const uint64_t at = stream * cvec + v;
    u32x4 x = {0u, 0u, 0u, 0u};
    if (v < cvec) x = __builtin_nontemporal_load(X + at);
    uint32_t amax = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t m = finite_magnitude(x[w]);
      amax = amax > m ? amax : m;
    }
    const int s = ckpt_scale(quad_max(amax));
    float y[8];
    widen8(x, y);
    const u32x2 q = held_codes(y, s);
    if (v < cvec) codes[at] = q;
    if ((v & 3u) == 0) scales[g >> 2] = (uint8_t)s;
  }
}

__global__ __launch_bounds__(kThreads) void unpack_kernel(const u32x2 *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, u32x4 *__restrict__ X,
                                                          uint64_t slots, uint32_t cvec, uint32_t slots_per_stream) {
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < slots; g += (uint64_t)gridDim.x * kThreads) {
    const uint64_t stream = g / slots_per_stream;
    const uint32_t v = (uint32_t)(g - stream * slots_per_stream);
    if (v >= cvec) continue;
    const uint64_t at = stream * cvec + v;
    X[at] = held_bf16(__builtin_nontemporal_load(codes + at), scales[g >> 2]);
  }
}

struct Slots {
  uint64_t total;
  uint32_t cvec, per_stream, grid;
};
Slots slots_of(int n, int64_t B, int64_t C) {
  Slots s;
  s.cvec = (uint32_t)(C / 8);
  s.per_stream = (uint32_t)(4 * ckpt_blocks(C));
  s.total = (uint64_t)B * n * s.per_stream;
  const uint64_t wgs = (s.total + kThreads - 1) / kThreads;
  s.grid = (uint32_t)(wgs < (1u << 22) ? wgs : (1u << 22));
  return s;
}

}  // namespace

hipError_t launch_ckpt_pack(int n, int64_t B, int64_t C, const void *X, void *codes, uint8_t *scales,
                            hipStream_t st) {
  const Slots s = slots_of(n, B, C);
  pack_kernel<<<s.grid, kThreads, 0, st>>>(static_cast<const u32x4 *>(X), static_cast<u32x2 *>(codes), scales, s.total,
                                           s.cvec, s.per_stream);
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack(int n, int64_t B, int64_t C, const void *codes, const uint8_t *scales, void *X,
                              hipStream_t st) {
  const Slots s = slots_of(n, B, C);
  unpack_kernel<<<s.grid, kThreads, 0, st>>>(static_cast<const u32x2 *>(codes), scales, static_cast<u32x4 *>(X),
                                             s.total, s.cvec, s.per_stream);
  return hipGetLastError();
}

}  // namespace mhc
