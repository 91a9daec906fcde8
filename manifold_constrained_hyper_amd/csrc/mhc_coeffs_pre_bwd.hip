// Gradients of the coefficients, of the pre-mix and of the residual path of
// one layer ([mHC-cutile], page "mHC 算法分析 & cutile 高效实现", sections
// 2.1-2.5), given G = dX_next, the gradients of H_post and H_res, and dF_pre.
// Per row (b's index left out):
//
//   dH_pre[i] = sum_c dF_pre[c] X_t[i][c]
//   z = alpha logit / r + b
//   dz_pre  = dH_pre s(z) s(-z),  dz_post = dH_post 2 s(z) s(-z)  (s: sigmoid)
//   dz_res: the 20 row and column normalisations backwards.  One of them,
//     y = x / total, gives dx = (dy - sum(dy y)) / total over the same row or
//     column; then dz = dm exp(z).
//   dlogit = alpha dz / r,  turn = -sum_k dlogit_k logit_k / (n C r^2)
//     (r = sqrt(sum x^2 / (n C)), so dr/dx = x / (n C r))
//   dX[j] = sum_i H_res[i][j] G[i] + H_pre[j] dF_pre + dlogit . phi_j^T + turn X_t[j]
//
// and over the rows dphi = X_t^T dlogit, dalpha = sum dz logit / r, db = sum dz.
//
// dH_pre needs the whole row before dlogit is known, so X_t and dF_pre are
// read twice: once by the row dot products, once where dX and dphi are formed.
#include "mhc_held.h"
#include "mhc_finish.h"
#include "mhc_train.h"

namespace mhc {

namespace {

constexpr int kSumThreads = 256;
constexpr int64_t kMaxSumBlocks = 512;

// dH_pre [B, n]: a workgroup a row.
template <int NS, bool CK, int W>
__global__ __launch_bounds__(64 * W) void pre_dots_kernel(const void *__restrict__ X,
                                                          const uint8_t *__restrict__ scales,
                                                          const u32x4 *__restrict__ dF, float *__restrict__ dpre,
                                                          uint32_t B, uint32_t cvec, uint32_t blocks) {
  __shared__ float part[W][NS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t row = blockIdx.x; row < B; row += gridDim.x) {
    float acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = 0.f;
    const size_t first = (size_t)row * NS * cvec;
    for (uint32_t v = threadIdx.x; v < cvec; v += 64 * W) {
      Held8<CK> x[NS];
      const u32x4 f = __builtin_nontemporal_load(dF + (size_t)row * cvec + v);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        x[j].load(X, scales, first + (size_t)j * cvec + v, ((size_t)row * NS + j) * blocks + (v >> 2));
      float fw[8];
      widen8(f, fw);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float xw[8];
        x[j].widen(xw);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j] = fmaf(fw[e], xw[e], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) acc[j] += __shfl_xor(acc[j], d);
      if (lane == 0) part[wave][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < NS) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) a += part[w][threadIdx.x];
      dpre[(size_t)row * NS + threadIdx.x] = a;
    }
    __syncthreads();
  }
}

// Sum over the n lanes that hold a row (AXIS 2: lanes differ in j) or a
// column (AXIS 1: lanes differ in i) of an n x n matrix, one element a lane
// at lane i*n + j of an aligned group of n*n lanes.
template <int NS, int AXIS>
__device__ __forceinline__ float axis_sum(float x) {
#pragma unroll
  for (int d = 1; d < NS; d <<= 1) x += __shfl_xor(x, AXIS == 2 ? d : d * NS);
  return x;
}

// The coefficients' gradient of each row: n*n lanes a row, one element of the
// n x n matrix each.  Every division is an IEEE one and the exponentials are
// the accurate ones: a 1 x 1 matrix normalises to exactly 1 and its gradient
// to exactly 0, as in the definition.  The partial sums of db and dalpha are
// kept in fp64 (few adds, and gates' gradients cancel over a batch).
template <int NS>
__global__ __launch_bounds__(kSumThreads) void coeffs_bwd_kernel(
    const float *__restrict__ logits, const float *__restrict__ r_in, float alpha_pre, float alpha_post,
    float alpha_res, const float *__restrict__ b_pre, const float *__restrict__ b_post,
    const float *__restrict__ b_res, const float *__restrict__ dH, const float *__restrict__ dpre,
    float *__restrict__ dl, float *__restrict__ turn, double *__restrict__ sums, uint32_t B, double inv_k) {
  constexpr int NN = NS * NS, N = NN + 2 * NS, R = kSumThreads / NN;
  constexpr int GATES = (2 * NS + NN - 1) / NN;  // gates a lane: 2 at n = 1, else 1
  constexpr int IT = kSinkhornIters;
  __shared__ double part[R][N + 3];
  const int e = threadIdx.x % NN, slot = threadIdx.x / NN;
  double sum_res = 0.0, sum_gate[GATES] = {}, sum_a[3] = {};
  const uint32_t stride = gridDim.x * R;
  for (uint32_t row0 = blockIdx.x * R; row0 < B; row0 += stride) {
    const uint32_t at = row0 + slot;
    const bool in = at < B;
    const uint32_t row = in ? at : B - 1;  // lanes past the end redo the last row and write nothing
    const float *lg = logits + (size_t)row * N;
    const float *up = dH + (size_t)row * N;
    const float r = r_in[row];
    float scaled = 0.f;  // sum of dlogit * logit over the lane's coefficients

    float dz_gate[GATES], dl_gate[GATES];
#pragma unroll
    for (int q = 0; q < GATES; ++q) {
      const int k = e + q * NN;
      dz_gate[q] = dl_gate[q] = 0.f;
      if (k < 2 * NS) {
        const bool post = k >= NS;
        const float a = post ? alpha_post : alpha_pre;
        const float z = a * lg[k] / r + (post ? b_post[k - NS] : b_pre[k]);
        const float s0 = 1.0f / (1.0f + expf(-z)), s1 = 1.0f / (1.0f + expf(z));
        const float g = post ? 2.0f * up[k] : dpre[(size_t)row * NS + k];
        dz_gate[q] = g * s0 * s1;
        dl_gate[q] = a * dz_gate[q] / r;
        scaled = fmaf(dl_gate[q], lg[k], scaled);
      }
    }

    const float lr = lg[2 * NS + e];
    const float m0 = expf(alpha_res * lr / r + b_res[e]);
    float y[2 * IT], total[2 * IT], m = m0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      total[2 * it] = axis_sum<NS, 2>(m);
      y[2 * it] = m = m / total[2 * it];
      total[2 * it + 1] = axis_sum<NS, 1>(m);
      y[2 * it + 1] = m = m / total[2 * it + 1];
    }
    float d = up[2 * NS + e];
#pragma unroll
    for (int it = IT - 1; it >= 0; --it) {
      d = (d - axis_sum<NS, 1>(d * y[2 * it + 1])) / total[2 * it + 1];
      d = (d - axis_sum<NS, 2>(d * y[2 * it])) / total[2 * it];
    }
    const float dz = d * m0;
    const float dlr = alpha_res * dz / r;
    scaled = fmaf(dlr, lr, scaled);
#pragma unroll
    for (int o = 1; o < NN; o <<= 1) scaled += __shfl_xor(scaled, o);

    if (in) {
      float *out = dl + (size_t)row * N;
      out[2 * NS + e] = dlr;
      if (e == 0) turn[row] = (float)(-(double)scaled * inv_k / ((double)r * r));
      sum_res += dz;
      sum_a[2] += (double)dz * lr / r;
#pragma unroll
      for (int q = 0; q < GATES; ++q) {
        const int k = e + q * NN;
        if (k < 2 * NS) {
          out[k] = dl_gate[q];
          sum_gate[q] += dz_gate[q];
          sum_a[k >= NS ? 1 : 0] += (double)dz_gate[q] * lg[k] / r;
        }
      }
    }
  }
  // [db_pre | db_post | db_res | dalpha_pre, _post, _res] of this workgroup
  part[slot][2 * NS + e] = sum_res;
#pragma unroll
  for (int q = 0; q < GATES; ++q)
    if (e + q * NN < 2 * NS) part[slot][e + q * NN] = sum_gate[q];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 1; o < NN; o <<= 1) sum_a[k] += __shfl_xor(sum_a[k], o);
    if (e == 0) part[slot][N + k] = sum_a[k];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < N + 3; k += kSumThreads) {
    double a = 0.0;
    for (int s = 0; s < R; ++s) a += part[s][k];
    sums[(size_t)blockIdx.x * (N + 3) + k] = a;
  }
}

// The workgroups' partial sums of db and dalpha, in their order.
__global__ __launch_bounds__(128) void sums_kernel(const double *__restrict__ sums, int blocks, int n,
                                                   float *__restrict__ dalpha, float *__restrict__ db_pre,
                                                   float *__restrict__ db_post, float *__restrict__ db_res) {
  const int N = n * n + 2 * n;
  for (int k = threadIdx.x; k < N + 3; k += 128) {
    double a = 0.0;
    for (int b = 0; b < blocks; ++b) a += sums[(size_t)b * (N + 3) + k];
    float *out = k < n ? db_pre + k : k < 2 * n ? db_post + (k - n) : k < N ? db_res + (k - 2 * n) : dalpha + (k - N);
    *out = (float)a;
  }
}

// dX: a lane takes eight channels of all streams of a row.
template <int NS, bool CK>
__global__ __launch_bounds__(256) void dx_kernel(const void *__restrict__ X, const uint8_t *__restrict__ scales,
                                                 const uint16_t *__restrict__ phi, const float *__restrict__ H,
                                                 const u32x4 *__restrict__ G, const u32x4 *__restrict__ dF,
                                                 const float *__restrict__ dl, const float *__restrict__ turn,
                                                 u32x4 *__restrict__ dX, uint64_t total, uint32_t cvec,
                                                 uint32_t blocks) {
  constexpr int N = NS * NS + 2 * NS;
  for (uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (uint64_t)gridDim.x * 256) {
    const uint64_t row = t / cvec;
    const uint32_t v = (uint32_t)(t - row * cvec);
    const float *h = H + row * N, *d = dl + row * N;
    const float c = turn[row];
    float gw[NS][8], fw[8];
#pragma unroll
    for (int i = 0; i < NS; ++i) widen8(G[(row * NS + i) * cvec + v], gw[i]);
    widen8(dF[row * cvec + v], fw);
    for (int j = 0; j < NS; ++j) {
      Held8<CK> x;
      x.load(X, scales, (row * NS + j) * cvec + v, (row * NS + j) * blocks + (v >> 2));
      float o[8], xw[8];
      x.widen(xw);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        o[q] = fmaf(c, xw[q], h[j] * fw[q]);
        const uint16_t *p = phi + ((size_t)j * cvec * 8 + (size_t)v * 8 + q) * N;
        for (int k = 0; k < N; ++k) o[q] = fmaf(d[k], __uint_as_float((uint32_t)p[k] << 16), o[q]);
#pragma unroll
        for (int i = 0; i < NS; ++i) o[q] = fmaf(h[2 * NS + i * NS + j], gw[i][q], o[q]);
      }
      dX[(row * NS + j) * cvec + v] = u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                            pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
    }
  }
}

// Partial dphi over a range of rows: a lane takes eight rows of phi (eight
// channels of a stream) and eight of its columns.
template <int NS, bool CK>
__global__ __launch_bounds__(256) void dphi_kernel(const void *__restrict__ X, const uint8_t *__restrict__ scales,
                                                   const float *__restrict__ dl, float *__restrict__ out, uint32_t B,
                                                   uint32_t rows, uint32_t cvec, uint32_t blocks) {
  constexpr int N = NS * NS + 2 * NS;
  const uint32_t kv = blockIdx.x * 256 + threadIdx.x;
  if (kv >= NS * cvec) return;
  const uint32_t j = kv / cvec, v = kv - j * cvec, col = blockIdx.y * 8;
  const uint32_t lo = blockIdx.z * rows, hi = min(B, lo + rows);
  float acc[8][8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int m = 0; m < 8; ++m) acc[q][m] = 0.f;
  for (uint32_t row = lo; row < hi; ++row) {
    Held8<CK> x;
    x.load(X, scales, ((size_t)row * NS + j) * cvec + v, ((size_t)row * NS + j) * blocks + (v >> 2));
    float xw[8];
    x.widen(xw);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float d = col + m < N ? dl[(size_t)row * N + col + m] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q][m] = fmaf(xw[q], d, acc[q][m]);
    }
  }
  float *o = out + ((size_t)blockIdx.z * NS * cvec * 8 + (size_t)kv * 8) * N;
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int m = 0; m < 8; ++m)
      if (col + m < N) o[(size_t)q * N + col + m] = acc[q][m];
}

// dphi: the partial sums in the order of their row ranges.
__global__ __launch_bounds__(256) void dphi_sum_kernel(const float *__restrict__ part, float *__restrict__ dphi,
                                                       uint64_t count, uint32_t split) {
  for (uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x; t < count; t += (uint64_t)gridDim.x * 256) {
    float a = 0.f;
    for (uint32_t s = 0; s < split; ++s) a += part[s * count + t];
    dphi[t] = a;
  }
}

__global__ __launch_bounds__(256) void zero_kernel(float *p, uint64_t count) {
  for (uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x; t < count; t += (uint64_t)gridDim.x * 256) p[t] = 0.f;
}

uint32_t wgs(uint64_t work, uint64_t per, uint64_t most) {
  const uint64_t g = (work + per - 1) / per;
  return (uint32_t)(g < most ? g : most);
}

template <int NS, bool CK>
hipError_t launch_t(const CoeffsBwdPlan &p, int64_t B, int64_t C, const CoeffsBwdArgs &a, char *ws, hipStream_t st) {
  constexpr int N = NS * NS + 2 * NS;
  float *dl = reinterpret_cast<float *>(ws + p.dl), *turn = reinterpret_cast<float *>(ws + p.turn);
  float *dpre = reinterpret_cast<float *>(ws + p.dpre), *part = reinterpret_cast<float *>(ws + p.dphi);
  double *sums = reinterpret_cast<double *>(ws + p.sums);
  const uint32_t cvec = (uint32_t)(C / 8), blocks = (uint32_t)ckpt_blocks(C), rows = (uint32_t)B;
  const u32x4 *dF = static_cast<const u32x4 *>(a.dF_pre);
  hipError_t e;
  pre_dots_kernel<NS, CK, 4><<<wgs(B, 1, 1u << 22), 256, 0, st>>>(a.X.x, a.X.scales, dF, dpre, rows, cvec, blocks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  coeffs_bwd_kernel<NS><<<(uint32_t)p.sum_blocks, kSumThreads, 0, st>>>(
      a.logits, a.r, a.alpha[0], a.alpha[1], a.alpha[2], a.b_pre, a.b_post, a.b_res, a.dH, dpre, dl, turn, sums, rows,
      1.0 / ((double)NS * (double)C));
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sums_kernel<<<1, 128, 0, st>>>(sums, (int)p.sum_blocks, NS, a.dalpha, a.db_pre, a.db_post, a.db_res);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const uint64_t total = (uint64_t)B * cvec;
  dx_kernel<NS, CK><<<wgs(total, 256, 1u << 22), 256, 0, st>>>(
      a.X.x, a.X.scales, static_cast<const uint16_t *>(a.phi), a.H, static_cast<const u32x4 *>(a.dX_next), dF, dl,
      turn, static_cast<u32x4 *>(a.dX), total, cvec, blocks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 grid(wgs((uint64_t)NS * cvec, 256, UINT32_MAX), (N + 7) / 8, (uint32_t)p.split);
  dphi_kernel<NS, CK><<<grid, 256, 0, st>>>(a.X.x, a.X.scales, dl, part, rows, (uint32_t)p.rows, cvec, blocks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const uint64_t count = (uint64_t)NS * C * N;
  dphi_sum_kernel<<<wgs(count, 256, 1u << 22), 256, 0, st>>>(part, a.dphi, count, (uint32_t)p.split);
  return hipGetLastError();
}

template <int NS>
hipError_t launch_n(const CoeffsBwdPlan &p, int64_t B, int64_t C, const CoeffsBwdArgs &a, char *ws, hipStream_t st) {
  return a.X.scales ? launch_t<NS, true>(p, B, C, a, ws, st) : launch_t<NS, false>(p, B, C, a, ws, st);
}

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

}  // namespace

CoeffsBwdPlan plan_coeffs_pre_bwd(int64_t B, int n, int64_t C) {
  CoeffsBwdPlan p;
  const int64_t N = (int64_t)n * n + 2 * n, K = (int64_t)n * C;
  p.split = B < 1024 ? 1 : B < 8192 ? 4 : 16;
  p.rows = (B + p.split - 1) / p.split;
  const int64_t per = kSumThreads / (n * n), groups = (B + per - 1) / per;
  p.sum_blocks = groups < kMaxSumBlocks ? groups : kMaxSumBlocks;
  p.dl = 0;
  p.turn = up16(p.dl + (size_t)B * N * 4);
  p.dpre = up16(p.turn + (size_t)B * 4);
  p.sums = up16(p.dpre + (size_t)B * n * 4);
  p.dphi = up16(p.sums + (size_t)p.sum_blocks * (N + 3) * 8);
  p.total_bytes = up16(p.dphi + (size_t)p.split * K * N * 4);
  return p;
}

hipError_t launch_coeffs_pre_bwd(const CoeffsBwdPlan &p, int n, int64_t B, int64_t C, const CoeffsBwdArgs &a,
                                 void *ws, hipStream_t st) {
  char *w = static_cast<char *>(ws);
  switch (n) {
    case 1: return launch_n<1>(p, B, C, a, w, st);
    case 2: return launch_n<2>(p, B, C, a, w, st);
    case 4: return launch_n<4>(p, B, C, a, w, st);
    case 8: return launch_n<8>(p, B, C, a, w, st);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_zero_f32(float *p, int64_t count, hipStream_t st) {
  if (count <= 0) return hipSuccess;
  zero_kernel<<<wgs((uint64_t)count, 256, 1u << 22), 256, 0, st>>>(p, (uint64_t)count);
  return hipGetLastError();
}

}  // namespace mhc
