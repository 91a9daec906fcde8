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
// order.  The gradient with respect to X_t is not formed here: it needs the
// gradient of the layer's input, which comes later, and is then one pass over
// G with everything else that flows into X_t (mhc_coeffs_pre_bwd.hip).
#include "mhc_held.h"
#include "mhc_train.h"

namespace mhc {

namespace {

template <int NS, bool CK, int W>
__global__ __launch_bounds__(64 * W) void post_res_bwd_kernel(
    const void *__restrict__ X, const uint8_t *__restrict__ scales, const u32x4 *__restrict__ F,
    const float *__restrict__ H, const u32x4 *__restrict__ G, u32x4 *__restrict__ dF, float *__restrict__ dH,
    uint32_t B, uint32_t cvec, uint32_t blocks) {
  constexpr int N = NS * NS + 2 * NS;
  constexpr int K = NS * NS + NS;
  __shared__ float part[W][K];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x) {
    const float *h = H + (size_t)row * N;
    float hpost[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) hpost[i] = h[NS + i];
    float acc[K];  // [dH_post | dH_res row-major]
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] = 0.f;
    const size_t first = (size_t)row * NS * cvec;
    for (uint32_t v = threadIdx.x; v < cvec; v += 64 * W) {
      u32x4 g[NS];
      Held8<CK> x[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) g[i] = __builtin_nontemporal_load(G + first + (size_t)i * cvec + v);
      const u32x4 f = __builtin_nontemporal_load(F + (size_t)row * cvec + v);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        x[j].load(X, scales, first + (size_t)j * cvec + v, ((size_t)row * NS + j) * blocks + (v >> 2));
      float fw[8], gw[NS][8], out[8];
      widen8(f, fw);
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        widen8(g[i], gw[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          out[e] = fmaf(hpost[i], gw[i][e], out[e]);
          acc[i] = fmaf(gw[i][e], fw[e], acc[i]);
        }
      }
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float xw[8];
        x[j].widen(xw);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[NS + i * NS + j] = fmaf(gw[i][e], xw[e], acc[NS + i * NS + j]);
      }
      const u32x4 o = {pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]), pack_bf16x2(out[4], out[5]),
                       pack_bf16x2(out[6], out[7])};
      store16_nt(dF + (size_t)row * cvec + v, o);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) acc[k] += __shfl_xor(acc[k], d);
      if (lane == 0) part[wave][k] = acc[k];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < N; k += 64 * W) {
      float a = 0.f;
      if (k >= NS) {
#pragma unroll
        for (int w = 0; w < W; ++w) a += part[w][k - NS];
      }
      dH[(size_t)row * N + k] = a;  // no gradient of H_pre from the apply
    }
    __syncthreads();
  }
}

template <int NS, bool CK>
hipError_t launch_t(int64_t B, int64_t C, HeldX X, const void *F, const float *H, const void *G, void *dF, float *dH,
                    hipStream_t st) {
  constexpr int W = 4;
  const uint32_t grid = (uint32_t)(B < (1 << 22) ? B : (1 << 22));
  post_res_bwd_kernel<NS, CK, W><<<grid, 64 * W, 0, st>>>(
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
