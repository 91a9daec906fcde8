// Gradients of the apply X_next[i] = sum_j H_res[i,j] X_t[j] + H_post[i] F_out
// ([mHC-cutile], page "mHC 算法分析 & cutile 高效实现", sections 2.5 and 3.4)
// with respect to F_out and to the coefficients.  With G = dX_next, a row has
//
//   dF_out[c]    = sum_i H_post[i] G[i][c]
//   dH_post[i]   = sum_c G[i][c] F_out[c]
//   dH_res[i][j] = sum_c G[i][c] X_t[j][c]
//
// Every input is read once; the n + n*n sums over the channels stay in
// registers (fp32) and are joined over a row's lanes and waves in a fixed
// order.  Products of two bf16 values go two at a time through dot2_bf16 (exact
// products, fp32 sums), straight from the packed words.  The gradient
// with respect to X_t is not formed here: it needs the gradient of the layer's
// input, which comes later, and is then one pass over G with everything else
// that flows into X_t (mhc_coeffs_pre_bwd.hip).
//
// Bound by HBM: 320 us at n=4, C=7168, B=16384 from the checkpoint (1.90 GB,
// 5.9 TB/s), 428 from the stream (2.35 GB, 5.5 TB/s), 205 at n=8, C=4096,
// B=8192 (1.21 GB, 5.9 TB/s).  64 rows of n=4, C=7168 take 7.1, which is the
// launch (6.2 of the kernel).
#include "mhc_finish.h"
#include "mhc_held.h"
#include "mhc_train.h"

namespace mhc {

namespace {

// Sums of K values (a multiple of 4) over a wave's lanes.  Two halvings trade
// half of the values between half-waves, then between rows of 16 lanes, so
// that each lane goes on with a quarter of them; the rest are lane moves
// inside a row.  Afterwards v[k], k < K / 4, of any lane holds the sum of
// value k + K/4 (row & 1) + K/2 (row / 2), row = lane / 16.
template <int K>
__device__ __forceinline__ void wave_sums(float (&v)[K]) {
  static_assert(K % 4 == 0, "quarters");
#pragma unroll
  for (int k = 0; k < K / 2; ++k) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + K / 2]), false, false);
    v[k] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int k = 0; k < K / 4; ++k) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + K / 4]), false, false);
    v[k] = tree16_sum(__uint_as_float(s[0]) + __uint_as_float(s[1]));
  }
}

template <int NS, bool CK>
__device__ __forceinline__ u32x4 x_words(const Held8<CK> &x) {
  if constexpr (CK)
    return held_bf16(x.v, x.s);
  else
    return x.v;
}

template <int NS>
constexpr int max_waves() { return NS == 8 ? 8 : 16; }  // n = 8 needs more than 128 registers

template <int NS, bool CK>
__global__ __launch_bounds__(64 * max_waves<NS>()) void post_res_bwd_kernel(
    const void *__restrict__ X, const uint8_t *__restrict__ scales, const u32x4 *__restrict__ F,
    const float *__restrict__ H, const u32x4 *__restrict__ G, u32x4 *__restrict__ dF, float *__restrict__ dH,
    uint32_t B, uint32_t cvec, uint32_t blocks) {
  constexpr int N = NS * NS + 2 * NS;
  constexpr int K = NS * NS + NS, KP = (K + 3) / 4 * 4;
  __shared__ float part[max_waves<NS>()][KP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, threads = blockDim.x;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x) {
    const float *h = H + (size_t)row * N;
    float hpost[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) hpost[i] = h[NS + i];
    float acc[KP];  // [dH_post | dH_res row-major]
#pragma unroll
    for (int k = 0; k < KP; ++k) acc[k] = 0.f;
    const size_t first = (size_t)row * NS * cvec;
    for (uint32_t v = threadIdx.x; v < cvec; v += threads) {
      u32x4 g[NS];
      Held8<CK> x[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) g[i] = __builtin_nontemporal_load(G + first + (size_t)i * cvec + v);
      const u32x4 f = __builtin_nontemporal_load(F + (size_t)row * cvec + v);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        x[j].load(X, scales, first + (size_t)j * cvec + v, ((size_t)row * NS + j) * blocks + (v >> 2));
      float out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        float gw[8];
        widen8(g[i], gw);
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = fmaf(hpost[i], gw[e], out[e]);
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[i] = dot2_bf16(g[i][w], f[w], acc[i]);
      }
      const u32x4 o = {pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]), pack_bf16x2(out[4], out[5]),
                       pack_bf16x2(out[6], out[7])};
      store16_nt(dF + (size_t)row * cvec + v, o);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const u32x4 xw = x_words<NS>(x[j]);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < NS; ++i) acc[NS + i * NS + j] = dot2_bf16(g[i][w], xw[w], acc[NS + i * NS + j]);
      }
    }
    wave_sums(acc);
    if ((lane & 15) == 0) {
      float *p = part[wave] + KP / 4 * ((lane >> 4) & 1) + KP / 2 * (lane >> 5);
#pragma unroll
      for (int k = 0; k < KP / 4; ++k) p[k] = acc[k];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < N; k += threads) {
      float a = 0.f;
      if (k >= NS) {
        for (int w = 0; w < threads / 64; ++w) a += part[w][k - NS];
      }
      dH[(size_t)row * N + k] = a;  // no gradient of H_pre from the apply
    }
    __syncthreads();
  }
}

// Waves a row: two steps of 512 channels each, at most eight, where there are
// rows enough to fill the chip so; a wave a step where there are not.  In us
// (n=4, C=7168 from the checkpoint, from the stream; n=8, C=4096):
//     rows                 256           512            768           1024           4096
//     a wave a step     8.0  8.8 11.5  12.6 13.8 16.0  19.2 19.3 24.0  25.0 26.7 29.6  91.7  96.5 110.5
//     two steps a wave  8.3  9.0 14.4  11.1 14.3 18.8  15.8 19.8 23.8  20.9 25.8 28.3  79.4 103.4 104.1
constexpr int64_t kManyRows = 768;
int waves_of(int most, int64_t B, int64_t C) {
  const int64_t steps = (C + 511) / 512, want = B >= kManyRows ? (steps + 1) / 2 : steps;
  const int64_t cap = B >= kManyRows ? 8 : most;
  return (int)(want < cap ? want : cap);
}

template <int NS, bool CK>
hipError_t launch_t(int64_t B, int64_t C, HeldX X, const void *F, const float *H, const void *G, void *dF, float *dH,
                    hipStream_t st) {
  const int W = waves_of(max_waves<NS>(), B, C);
  const uint32_t grid = (uint32_t)(B < (1 << 22) ? B : (1 << 22));
  post_res_bwd_kernel<NS, CK><<<grid, 64 * W, 0, st>>>(
      X.x, X.scales, static_cast<const u32x4 *>(F), H, static_cast<const u32x4 *>(G), static_cast<u32x4 *>(dF), dH,
      (uint32_t)B, (uint32_t)(C / 8), (uint32_t)ckpt_blocks(C));
  return hipGetLastError();
}

template <int NS>
hipError_t launch_n(int64_t B, int64_t C, HeldX X, const void *F, const float *H, const void *G, void *dF, float *dH,
                    hipStream_t st) {
  return X.scales ? launch_t<NS, true>(B, C, X, F, H, G, dF, dH, st)
                  : launch_t<NS, false>(B, C, X, F, H, G, dF, dH, st);
}

}  // namespace

hipError_t launch_post_res_bwd(int n, int64_t B, int64_t C, HeldX X, const void *F_out, const float *H,
                               const void *dX_next, void *dF_out, float *dH, hipStream_t st) {
  switch (n) {
    case 1: return launch_n<1>(B, C, X, F_out, H, dX_next, dF_out, dH, st);
    case 2: return launch_n<2>(B, C, X, F_out, H, dX_next, dF_out, dH, st);
    case 4: return launch_n<4>(B, C, X, F_out, H, dX_next, dF_out, dH, st);
    case 8: return launch_n<8>(B, C, X, F_out, H, dX_next, dF_out, dH, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mhc
