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

#include <type_traits>

namespace mhc {

namespace {

constexpr int64_t kMaxSumBlocks = 1024;

typedef short s16x8 __attribute__((ext_vector_type(8)));

// How dx_dphi_kernel splits the work for n streams.
template <int NS>
struct Tiles {
  static constexpr int N = NS * NS + 2 * NS;
  static constexpr int KS = (N + 31) / 32;      // 32-wide steps over the coefficients (dlogit . phi^T)
  static constexpr int MT = (N + 15) / 16;      // 16-row tiles of dphi^T
  static constexpr int JW = NS == 8 ? 2 : NS;   // streams a wave forms dX and dphi of
  static constexpr int GROUPS = NS / JW;        // waves that share a tile of rows and channels
  static constexpr int CW = 32;                 // channels a wave
  // What dx_dphi_kernel needs of a tile of 16 rows, a record written by
  // coeffs_bwd_kernel: dlogit, then the factors of dX
  //   mix   [KH][16 rows] fp32  H_pre and H_res
  //   turn  [16 rows] fp32      the factor of X_t that r contributes
  static constexpr int KH = NS + NS * NS;
  // dlogit as the matrix core's operands (byte offsets; every part is a
  // multiple of 16), bf16 parts whose sum is dlogit to 2^-17 (hi + mid: for
  // dX, which is rounded to bf16) or 2^-25 (hi + mid + low: for dphi, fp32) of
  // it:
  //   rows_b  [hi, mid][KS][lane][8]  B operand of dlogit . phi^T: lane
  //           16 q + i has coefficients 32 ks + 8 q .. + 7 of row i
  //   cols_a  [MT][lane][8]  A operand of dphi^T += dlogit^T X: lane 16 q + m
  //           has hi, then mid, of rows 4 q .. + 3 of coefficient 16 mt + m
  //   cols_c  [MT][lane][4]  the same with the low parts
  static constexpr int kColsA = 2 * KS * 1024, kColsC = kColsA + MT * 1024, kOperands = kColsC + MT * 512;
  // At n = 4 a tile's dlogit goes out as it is, [16][N] fp32, and
  // dx_dphi_kernel forms the operands in LDS: they have 3.3 times the bytes,
  // read by every workgroup along the channels (625 us against 638 at C=7168,
  // B=16384 from the checkpoint; few rows take 0.3 us longer).  At n = 8, with
  // 80 coefficients, forming them there costs more than the bytes (570 us
  // against 552 at C=4096, B=8192), and at n = 1 and 2 the tiles are short
  // (n=1, B=120: 23 us against 20).
  static constexpr bool kLate = NS == 4;
  static constexpr int kDlogit = kLate ? 16 * N * 4 : kOperands;
  static constexpr int kTurn = kDlogit + KH * 64, kEnd = kTurn + 64, kMix = kEnd - kDlogit;
  static constexpr int kStride = kLate ? kEnd : (kEnd + 1023) / 1024 * 1024;
};

__device__ __forceinline__ float bf16_round(float x) { return bf16_lo(pack_bf16x2(x, 0.f)); }

// One wave's part `item` (below KS: a step of rows_b, then a tile of cols) of
// a tile's operands, from its dlogit dl[row * STRIDE + coefficient].
// Coefficients past N are zeros.
template <int NS, int STRIDE>
__device__ __forceinline__ void form_operands(const float *dl, int item, int lane, char *to) {
  using T = Tiles<NS>;
  constexpr int N = T::N, KS = T::KS;
  const int lo16 = lane & 15, q = lane >> 4;
  if (item < KS) {
    const int k0 = 32 * item + 8 * q;
    float v[8];
    if constexpr (STRIDE % 4 == 0) {
      f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
      if (k0 < N) {
        const f32x4 *row = reinterpret_cast<const f32x4 *>(dl + lo16 * STRIDE + k0);
        a = row[0], b = row[1];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = k0 + j < N ? dl[lo16 * STRIDE + k0 + j] : 0.f;
    }
    u32x4 hi, mid;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      mid[j] = pack_bf16x2(v[2 * j] - bf16_lo(hi[j]), v[2 * j + 1] - bf16_hi(hi[j]));
    }
    reinterpret_cast<u32x4 *>(to)[item * 64 + lane] = hi;
    reinterpret_cast<u32x4 *>(to)[(KS + item) * 64 + lane] = mid;
  } else {
    const int mt = item - KS, k = 16 * mt + lo16;
    float v[4], h[4], m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = k < N ? dl[(4 * q + j) * STRIDE + k] : 0.f;
      h[j] = bf16_round(v[j]);
      m[j] = bf16_round(v[j] - h[j]);
      v[j] = v[j] - h[j] - m[j];
    }
    reinterpret_cast<u32x4 *>(to + T::kColsA)[mt * 64 + lane] =
        u32x4{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(m[0], m[1]), pack_bf16x2(m[2], m[3])};
    reinterpret_cast<u32x2 *>(to + T::kColsC)[mt * 64 + lane] = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// dH_pre [B, n]: a workgroup a row (106 us at n=4, C=7168, B=16384 from the
// checkpoint, 0.72 GB at 6.8 TB/s; 174 from the stream, 1.17 GB at 6.7).
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
// at lane i*n + j of an aligned group of n*n lanes; every lane of the row or
// column gets the same bits (each step adds two values that its partner adds
// too).  Lane moves inside rows of 16 lanes are DPP; n = 8 swaps rows and
// halves of the wave beside.
__device__ __forceinline__ float dpp_add_ror8(float x) {  // lane ^ 8 in its row of 16
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x128, 0xF, 0xF, false));
}
template <int NS, int AXIS>
__device__ __forceinline__ float axis_sum(float x) {
  static_assert(NS == 8, "");
  if constexpr (AXIS == 2) return group_sum<NS>(x);
  x = dpp_add_ror8(x);
  const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
  const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}
template <int CTRL>
__device__ __forceinline__ double dpp_add(double x) {
  const int lo = __builtin_amdgcn_mov_dpp(__double2loint(x), CTRL, 0xF, 0xF, false);
  const int hi = __builtin_amdgcn_mov_dpp(__double2hiint(x), CTRL, 0xF, 0xF, false);
  return x + __hiloint2double(hi, lo);
}
template <int NS, int AXIS>
__device__ __forceinline__ double axis_sum(double x) {
  static_assert(NS == 2 || NS == 4, "");
  if constexpr (NS == 2) return dpp_add<AXIS == 2 ? 0xB1 : 0x4E>(x);  // lane ^ 1, lane ^ 2
  if constexpr (AXIS == 2) return dpp_add<0x4E>(dpp_add<0xB1>(x));
  return dpp_add<0x124>(dpp_add<0x128>(x));  // lane ^ 8, then lane ^ 4 (lane + 4, as lanes 8 apart are equal)
}
// 1 / x to about an ulp: the hardware's reciprocal and a Newton step.
__device__ __forceinline__ float recip(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return fmaf(r, fmaf(-x, r, 1.0f), r);
}
__device__ __forceinline__ double recip(double x) {  // two steps: 2^-23, 2^-46, 2^-52
  double r = __builtin_amdgcn_rcp(x);
  r = fma(r, fma(-x, r, 1.0), r);
  return fma(r, fma(-x, r, 1.0), r);
}

// The coefficients' gradient of each row: n*n lanes a row, one element of the
// n x n matrix each, with the accurate exponentials.  A 1 x 1 matrix is 1
// whatever its logit and has no gradient.  The first division is an IEEE one
// (its totals are sums of exponentials of any size); the later ones, whose
// totals are near 1, multiply by a reciprocal.  The 80 sums and divisions of a
// row depend on each other, so the kernel is bound by their latency (and at
// n = 8, 64 lanes a row, by their number).
//
// What is summed over a batch cancels, so the partial sums of db and dalpha
// and the gates' derivatives are fp64 (a few operations a row), and up to
// n = 4 so are the normalisations: most of dH_res cancels in them (at n = 2
// all but one degree of freedom), and fp32 left errors of 1e-6 of small
// batches' sums.  That costs 5 us at n=4, B=16384 (19 against 14).  At n = 8,
// with 49 degrees of freedom, fp32 leaves dz within 1.1 * 2^-24 of a row's
// largest dH_res, and sums over 333 rows within 6e-8 of the sums of their
// terms' magnitudes, from balanced matrices to ones that 20 iterations do not
// balance; 64 bits would not fit the registers of 1024 threads.
//
// dlogit leaves in tiles of 16 rows; rows past the last are zeros.
template <int NS>
constexpr int sum_threads() { return NS == 8 ? 1024 : 256; }  // a multiple of 16 rows a workgroup

// With Dots (where X_t is), the row dot products are formed here too, by eight
// waves, rather than in a launch of their own.
struct NoDots {};
template <bool CK>
struct Dots {
  const void *X;
  const uint8_t *scales;
  const u32x4 *dF;
  uint32_t cvec, blocks;
};
template <class D>
constexpr bool kFused = !std::is_same<D, NoDots>::value;
template <int NS, bool FUSED>
constexpr int coeff_threads() { return FUSED ? 512 : sum_threads<NS>(); }
template <int NS>
constexpr int kDotRows = NS == 4 ? 2 : 8 / NS;  // rows a wave has under way

template <int NS, bool CK>
__device__ __forceinline__ void row_dots(const Dots<CK> &d, uint32_t row0, uint32_t rows, uint32_t B, float (*out)[NS]) {
  constexpr int U = kDotRows<NS>;
  const uint32_t lane = threadIdx.x & 63, wave = (uint32_t)uniform((int)(threadIdx.x >> 6)), W = blockDim.x >> 6;
  for (uint32_t base = wave * U; base < rows && row0 + base < B; base += W * U) {
    float acc[U][NS];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NS; ++j) acc[u][j] = 0.f;
    for (uint32_t v = lane; v < d.cvec; v += 64) {
      Held8<CK> x[U][NS];
      u32x4 f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t row = row0 + base + u < B ? row0 + base + u : B - 1;
        f[u] = __builtin_nontemporal_load(d.dF + (size_t)row * d.cvec + v);
#pragma unroll
        for (int j = 0; j < NS; ++j)
          x[u][j].load(d.X, d.scales, ((size_t)row * NS + j) * d.cvec + v, ((size_t)row * NS + j) * d.blocks + (v >> 2));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float fw[8];
        widen8(f[u], fw);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          float xw[8];
          x[u][j].widen(xw);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[u][j] = fmaf(fw[e], xw[e], acc[u][j]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) acc[u][j] += __shfl_xor(acc[u][j], o);
        if (lane == 0) out[base + u][j] = acc[u][j];
      }
  }
}

template <int NS, class D>
__global__ __launch_bounds__((coeff_threads<NS, kFused<D>>())) void coeffs_bwd_kernel(
    D dots, const float *__restrict__ logits, const float *__restrict__ r_in, float alpha_pre, float alpha_post,
    float alpha_res, const float *__restrict__ b_pre, const float *__restrict__ b_post,
    const float *__restrict__ b_res, const float *__restrict__ dH, const float *__restrict__ dpre,
    const float *__restrict__ H, char *__restrict__ records, double *__restrict__ sums,
    uint32_t B, double inv_k) {
  using T = Tiles<NS>;
  constexpr int TH = coeff_threads<NS, kFused<D>>();
  constexpr int NN = NS * NS, N = NN + 2 * NS, R = sum_threads<NS>() / NN;
  constexpr int IT = kSinkhornIters;
  constexpr int NP = N | 1;  // odd: rows start in different LDS banks
  __shared__ float row_dot[kFused<D> ? R : 1][NS];
  __shared__ float along[R];  // a row's sum of dlogit * logit over the res block
  __shared__ union {
    float dl[R][NP];
    double part[R][N + 3];
  } sh;
  const int e = threadIdx.x % NN, slot = threadIdx.x / NN;  // the thread's element of a row's matrix
  const bool mine = slot < R;  // (whole waves: the other waves have no element)
  const int gk = threadIdx.x % (2 * NS);                    // and its gate, of any row
  const bool post = gk >= NS;
  const float alpha_gate = post ? alpha_post : alpha_pre, b_gate = post ? b_post[gk - NS] : b_pre[gk];
  double sum_res = 0.0, sum_gate = 0.0, sum_a_res = 0.0, sum_a_gate = 0.0;
  const uint32_t stride = gridDim.x * R;
  for (uint32_t row0 = blockIdx.x * R; row0 < B; row0 += stride) {
    if constexpr (kFused<D>) {
      row_dots<NS>(dots, row0, R, B, row_dot);
      __syncthreads();
    }
    for (int w = threadIdx.x; w < R * 2 * NS; w += TH) {
      const int gs = w / (2 * NS);
      const size_t row = row0 + gs;
      float dl = 0.f;
      if (row < B) {
        const float l = logits[row * N + gk], r = r_in[row];
        const double z = (double)alpha_gate * l / r + b_gate;
        const double t = exp(-fabs(z));  // s(z) s(-z) = t / (1 + t)^2
        const double dz = (post ? 2.0f * dH[row * N + gk] : kFused<D> ? row_dot[kFused<D> ? gs : 0][gk] : dpre[row * NS + gk]) * t / ((1.0 + t) * (1.0 + t));
        dl = (float)(alpha_gate * dz / r);
        sum_gate += dz;
        sum_a_gate += dz * l / r;
      }
      sh.dl[gs][gk] = dl;
    }

    if (mine) {
      const uint32_t at = row0 + slot;
      const bool in = at < B;
      const uint32_t row = in ? at : B - 1;  // lanes past the end redo the last row and write nothing
      const float r = r_in[row], lr = logits[(size_t)row * N + 2 * NS + e];
      typedef typename std::conditional<NS <= 4, double, float>::type real;
      real dz = 0;
      if constexpr (NS > 1) {
        const real z = (real)alpha_res * lr / r + b_res[e];
        real m0;
        if constexpr (NS <= 4)
          m0 = exp(z);
        else
          m0 = expf(z);
        real y[IT], inv[2 * IT];  // every second y: the others are a product away (registers)
        const real total = axis_sum<NS, 2>(m0);
        real m = y[0] = m0 / total;
#pragma unroll
        for (int k = 1; k < 2 * IT; ++k) {
          inv[k] = recip(k % 2 ? axis_sum<NS, 1>(m) : axis_sum<NS, 2>(m));
          m *= inv[k];
          if (k % 2 == 0) y[k / 2] = m;
        }
        real d = dH[(size_t)row * N + 2 * NS + e];
#pragma unroll
        for (int k = 2 * IT - 1; k > 0; --k) {
          real yk = y[k / 2];
          if (k % 2) {
            asm("" : "+v"(yk));  // (or the compiler keeps the products)
            yk *= inv[k];
          }
          const real dy = d * yk;
          d = (d - (k % 2 ? axis_sum<NS, 1>(dy) : axis_sum<NS, 2>(dy))) * inv[k];
        }
        // dz = m0 (d - sum) / total, with m0 / total = y[0]
        dz = y[0] * (d - axis_sum<NS, 2>(d * y[0]));
      }
      const float dlr = (float)(alpha_res * dz / r);
      float res = dlr * lr;
#pragma unroll
      for (int o = 1; o < NN; o <<= 1) res += __shfl_xor(res, o);
      sh.dl[slot][2 * NS + e] = in ? dlr : 0.f;
      if (e == 0) along[slot] = res;
      if (in) {
        sum_res += dz;
        sum_a_res += (double)dz * lr / r;
      }
    }
    __syncthreads();
    const uint32_t tiles = (B + 15) / 16;
    if constexpr (T::kLate) {
      for (int w = threadIdx.x; w < R * N; w += TH) {
        const int i = w / N, k = w - i * N;
        if (row0 + i < tiles * 16)
          reinterpret_cast<float *>(records + (size_t)(row0 + i) / 16 * T::kStride)[(i & 15) * N + k] = sh.dl[i][k];
      }
    } else {
      constexpr int kItems = T::KS + T::MT;
      for (int w = threadIdx.x >> 6; w < R / 16 * kItems; w += TH / 64) {
        const size_t tile = row0 / 16 + w / kItems;
        if (tile < tiles)
          form_operands<NS, NP>(sh.dl[w / kItems * 16], w % kItems, threadIdx.x & 63, records + tile * T::kStride);
      }
    }
    for (int w = threadIdx.x; w < R * (T::KH + 1); w += TH) {
      const int i = w & 15, k = (w >> 4) % (T::KH + 1), tl = (w >> 4) / (T::KH + 1);
      const size_t tile = row0 / 16 + tl, row = tile * 16 + i;
      if (tile >= tiles) continue;
      float x = 0.f;
      if (k == T::KH && row < B) {
        const double r = r_in[row];
        double all = along[tl * 16 + i];
#pragma unroll
        for (int g = 0; g < 2 * NS; ++g) all += (double)sh.dl[tl * 16 + i][g] * logits[row * N + g];
        x = (float)(-all * inv_k / (r * r));
      } else if (row < B) {
        x = H[row * N + (k < NS ? k : k + NS)];  // the post block is not needed
      }
      reinterpret_cast<float *>(records + tile * T::kStride + T::kDlogit)[k * 16 + i] = x;
    }
    __syncthreads();
  }
  // [db_pre | db_post | db_res | dalpha_pre, _post, _res] of this workgroup
  for (int w = threadIdx.x; w < R * (N + 3); w += TH) (&sh.part[0][0])[w] = 0.0;
  __syncthreads();
  if (mine) sh.part[slot][2 * NS + e] = sum_res;
#pragma unroll
  for (int o = 1; o < NN; o <<= 1) sum_a_res += __shfl_xor(sum_a_res, o);
  if (mine && e == 0) sh.part[slot][N + 2] = sum_a_res;
#pragma unroll
  for (int o = 1; o < NS; o <<= 1) sum_a_gate += __shfl_xor(sum_a_gate, o);
  if (threadIdx.x < R * 2 * NS) {
    const int gs = threadIdx.x / (2 * NS);
    sh.part[gs][gk] = sum_gate;
    if (gk % NS == 0) sh.part[gs][N + (post ? 1 : 0)] = sum_a_gate;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < N + 3; k += TH) {
    double a = 0.0;
    for (int s = 0; s < R; ++s) a += sh.part[s][k];
    sums[(size_t)blockIdx.x * (N + 3) + k] = a;
  }
}

// The sums over the rows besides dphi: the coefficient kernel's workgroups'
// parts, and where they go.
struct Sums {
  const double *part;
  int blocks;
  float *dalpha, *db_pre, *db_post, *db_res;
  template <int NS>
  __device__ __forceinline__ float *out(int k) const {
    constexpr int N = NS * NS + 2 * NS;
    return k < NS ? db_pre + k : k < 2 * NS ? db_post + (k - NS) : k < N ? db_res + (k - 2 * NS) : dalpha + (k - N);
  }
};

// dX and the partial dphi, in one pass over G, X_t and dF_pre.
//
// A wave takes 16 rows and 32 channels at a time: lane 16 q + i has channels
// 8 q .. 8 q + 7 of row i, of every stream.  That is the matrix core's A
// layout (16 x 32, bf16), and the C layout of a product whose rows are
// channels and whose columns are the tile's rows, so both products happen
// where the data is:
//
//  * dlogit . phi^T: A = phi of 16 channels (in registers for the whole
//    kernel), B = dlogit of the 16 rows.  Two of them, for channels
//    8 q + 0..3 and + 4..7 of each lane, leave each lane its own eight sums;
//    the row's terms (H_res, H_pre and the r term) are added in fp32 and dX is
//    rounded once.
//  * dphi^T += dlogit^T X needs X with its rows along K.  X times a 32 x 16
//    selection (ones and zeros) moves it there: the product is X itself,
//    exactly, with lane 16 q + c holding rows 4 q .. 4 q + 3 of channel c --
//    the B layout.  dlogit^T goes in three bf16 parts (coeffs_bwd_kernel), two
//    of them in one 32-deep product against the same X twice, so dphi has
//    fp32's accuracy (the third's product has zeros in its other half: with a
//    16x16x16 product before a 16x16x32 one on the same sums results changed
//    from run to run, for a cause that was not found).  Sums over a workgroup's rows stay in
//    registers and are joined over the row ranges by join_kernel, in their
//    order.
//
// A NaN in X_t reaches dphi in the 32 channels around it (NaN times the
// selection's zeros); a row with one has no finite r either.
//
// Memory: in that layout the lanes of a quad have four different rows, so
// loads straight into it touch 64 separate 16-byte pieces each (measured 915
// us at n=4, C=7168, B=16384 from the checkpoint).  Direct-to-LDS loads take a
// tile of the workgroup's channels in memory order instead (512 bytes of a row
// at a time at n = 4, 128 at n = 8), one or two tiles ahead, without
// registers; a row's 16-byte pieces are exchanged by an xor with the row, so
// that the reads in the matrix layout meet no bank twice.  dX takes G's or
// X_t's place in LDS and is stored from there, four or eight lanes a row.
//
// A tile's record is staged the same way; where the operands are formed here,
// dlogit one tile further ahead: the waves form a share each, a tile before
// the use.
//
// Measured at n=4, C=7168, B=16384 from the checkpoint: 487 us (460 on the
// fastest card) for 2.77 GB (5.7 TB/s); from the stream 585 for 3.11 (5.3).
// Without the arithmetic the call from the checkpoint takes 618 us, not 628:
// bound by HBM and the order in which it is reached.  At n=8, C=4096, B=8192
// from the stream 407 us for 1.81 GB (4.5 TB/s): the registers of a compute
// unit hold phi and dphi of 64 channels, so rows are read 128 bytes at a time
// (without the arithmetic the call takes 511 us, not 525; with 1 KB of the
// record instead of 19, 493).
//
// Waits: vmcnt counts in order, and between a tile's loads and their use the
// wave issues the loads and dX stores of the tiles in between and no other
// memory access (Stage::kYounger of them at least), so "at most that many
// outstanding" means that the tile has landed.  Where fewer may be issued (the
// first and last tiles, waves past the channels) the wait is for all.
__device__ __attribute__((aligned(256))) uint32_t g_train_zero[64];  // what loads past the edges read

// (M0 is reserved, of which the compiler warns where it is on a clobber list;
// the entry keeps it from relying on M0's old value.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void dma(const void *src, uint32_t lds_addr) {  // lane l's data lands at lds_addr + BYTES l
  lds_addr = (uint32_t)uniform((int)lds_addr);
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds_addr)
                 : "m0", "memory");
  else if constexpr (BYTES == 4)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds_addr)
                 : "m0", "memory");
  else  // one byte, zero-extended to the lane's four
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off" ::"v"(src), "s"(lds_addr)
                 : "m0", "memory");
}
#pragma clang diagnostic pop
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_addr_of(const char *p) { return (uint32_t)(uintptr_t)(lds_char *)p; }

template <int NS, bool CK>
struct Stage {
  using T = Tiles<NS>;
  static constexpr int kWaves = 8, kAlong = kWaves / T::GROUPS;
  static constexpr bool kShared = T::GROUPS > 1;  // G is read by waves of other streams
  // Stages of LDS; loads are issued kStages - 1 tiles ahead.
  static constexpr int kStages = NS == 4 ? 2 : 3;
  static constexpr int kDist = kStages - 1;
  // Bytes of a stage: G, X_t, dF_pre, scale bytes (a dword each).
  static constexpr int kG = kAlong * NS * 1024;
  static constexpr int kX = kWaves * T::JW * (CK ? 512 : 1024);
  static constexpr int kF = kAlong * 1024;
  static constexpr int kS = CK ? kWaves * 256 : 0;
  static constexpr int kBytes = kG + kX + kF + kS;
  // dX takes the place of G in LDS (a wave's own columns of it), or where G is
  // shared that of X_t, or (from codes) a place of its own.
  static constexpr bool kOwnOut = kShared && CK;
  static constexpr int kOutBytes = kOwnOut ? kWaves * T::JW * 1024 : 16;
  // Loads a wave issues for a tile at least (without its share of dlogit and mix),
  // and its stores of a tile: what may be younger than a tile's loads.
  static constexpr int kLoads = (kShared ? T::JW : NS + 1) + (CK ? T::JW / 2 + 1 : T::JW);
  static constexpr int kStores = T::JW;
  static constexpr int kYounger = kDist == 1 ? kStores : 2 * kStores + kLoads;
};

template <int NS, bool CK>
__global__ __launch_bounds__(512, 2) void dx_dphi_kernel(
    const char *__restrict__ X, const uint8_t *__restrict__ scales, const uint16_t *__restrict__ phi,
    const char *__restrict__ G, const char *__restrict__ dF, const char *__restrict__ records, char *__restrict__ dX,
    float *__restrict__ out, uint32_t B, uint32_t cvec, uint32_t blocks, uint32_t slices, uint32_t split, int wc,
    Sums sums) {
  using T = Tiles<NS>;
  using S = Stage<NS, CK>;
  constexpr int N = T::N, KS = T::KS, MT = T::MT, JW = T::JW, GROUPS = T::GROUPS;
  __shared__ __attribute__((aligned(1024))) char stage[S::kStages][S::kBytes];
  __shared__ __attribute__((aligned(16))) char record[S::kStages][T::kStride];
  __shared__ __attribute__((aligned(16))) char formed[T::kLate ? 2 : 1][T::kLate ? T::kOperands : 16];
  __shared__ __attribute__((aligned(16))) char own_out[S::kOutBytes];
  if (blockIdx.x == slices * split) {  // with one row range there is no join_kernel
    for (int k = threadIdx.x; k < N + 3; k += blockDim.x) {
      double a = 0.0;
#pragma unroll 8
      for (int b = 0; b < sums.blocks; ++b) a += sums.part[(size_t)b * (N + 3) + k];
      *sums.out<NS>(k) = (float)a;
    }
    return;
  }
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  // wc waves along the channels, GROUPS along the streams.
  const int cw = wave / GROUPS, group = wave % GROUPS, waves = wc * GROUPS;
  const uint32_t slice = blockIdx.x % slices, range = blockIdx.x / slices;
  const uint32_t v_wg = slice * (uint32_t)wc * 4;  // the workgroup's first vector of eight channels
  const uint32_t v_wave = v_wg + cw * 4;
  const int lo16 = lane & 15, q = lane >> 4, j0 = group * JW;
  // Its tiles: every `split`th, from `range` on, so that all workgroups move
  // through the rows together (with a run of rows each, 14 us slower at n=4,
  // C=7168, B=16384).
  const uint32_t count = ((B + 15) / 16 - range + split - 1) / split;
  const auto tile_at = [&](uint32_t k) { return range + k * split; };
  const size_t row_bytes = (size_t)cvec * 16;  // a stream of a row

  // A stream's tile in LDS: 16 rows of 1 << lg 16-byte pieces, piece p of row
  // r at p ^ turn(r, lg): reads of one piece of every row meet 16 different
  // places of the 256 bytes that the banks span.
  const int lg = __builtin_ctz(wc) + 2;
  const auto turn = [](int row, int l) { return l >= 4 ? row : (row >> (4 - l)) & ((1 << l) - 1); };
  const auto piece_of = [&](int row, int p, int l) { return ((row << l) + (p ^ turn(row, l))) * 16; };

  const auto issue_part = [&](uint32_t tile, int from, auto bytes, int st) {
    constexpr int count = decltype(bytes)::value;
    const char *src = records + (size_t)tile * T::kStride + from;
    for (int k = wave * 1024; k < count; k += waves * 1024)
      if (count % 1024 == 0 || k + lane * 16 < count) dma<16>(src + k + lane * 16, lds_addr_of(record[st]) + from + k);
  };
  // A tile's tensors and mix, and its dlogit or (where the operands are formed
  // here, a tile before their use) the next one's.
  const auto issue = [&](uint32_t k, int st) {
    const uint32_t tile = tile_at(k);
    const char *zero = reinterpret_cast<const char *>(g_train_zero);
    const uint32_t at = lds_addr_of(stage[st]), row0 = tile * 16;
    // bf16 tiles: KiB cw of a stream's.
    const int at_lane = cw * 64 + lane, r = at_lane >> lg, p = (at_lane & ((1 << lg) - 1)) ^ turn(r, lg);
    const uint32_t row = row0 + r, v = v_wg + p, kib = 256u << lg;  // (bytes of a stream's tile)
    const bool in = row < B && v < cvec;
    const size_t o = ((size_t)row * NS * cvec + v) * 16;
#pragma unroll
    for (int k = 0; k < (S::kShared ? JW : NS); ++k) {
      const int i = S::kShared ? j0 + k : k;
      dma<16>(in ? G + o + (size_t)i * row_bytes : zero, at + i * kib + cw * 1024);
    }
    if (!S::kShared || group == 0)
      dma<16>(in ? dF + (size_t)row * row_bytes + (size_t)v * 16 : zero, at + S::kG + S::kX + cw * 1024);
    if constexpr (!CK) {
#pragma unroll
      for (int jj = 0; jj < JW; ++jj)
        dma<16>(in ? X + o + (size_t)(j0 + jj) * row_bytes : zero, at + S::kG + (j0 + jj) * kib + cw * 1024);
    } else {
      // Codes: the same with rows of half as many pieces; 16 bytes a lane
      // where a stream's codes are that aligned, else four.
      const size_t stream = (size_t)cvec * 8;
      const int lc = lg - 1, all = JW * 256 << lc;
      const uint32_t x_at = at + S::kG + (j0 * 256 << lc);
      const auto code = [&](int byte) -> const char * {
        const int jj = byte >> (8 + lc), cr = (byte >> (4 + lc)) & 15;
        const int cp = ((byte >> 4) & ((1 << lc) - 1)) ^ turn(cr, lc);
        const uint32_t code_row = row0 + cr, ch = v_wg * 8 + cp * 16 + (byte & 15);
        return code_row < B && ch < cvec * 8 ? X + ((size_t)code_row * NS + j0 + jj) * stream + ch : zero;
      };
      if (cvec % 2 == 0) {
        for (int b = cw * 1024; b < all; b += wc * 1024)
          if (b + lane * 16 < all) dma<16>(code(b + lane * 16), x_at + b);
      } else {
        for (int b = cw * 256; b < all; b += wc * 256) dma<4>(code(b + lane * 4), x_at + b);
      }
      // One scale byte for each row and stream.
      const uint32_t s_row = row0 + lo16;
      dma<1>(s_row < B && v_wave < cvec && q < JW
                 ? reinterpret_cast<const char *>(scales) + ((size_t)s_row * NS + j0 + q) * blocks + (v_wave >> 2)
                 : zero,
             at + S::kG + S::kX + S::kF + (uint32_t)wave * 256);
    }
    if constexpr (T::kLate) {
      issue_part(tile, T::kDlogit, std::integral_constant<int, T::kMix>{}, st);
      if (k + 1 < count) issue_part(tile_at(k + 1), 0, std::integral_constant<int, T::kDlogit>{}, st + 1 == S::kStages ? 0 : st + 1);
    } else {
      issue_part(tile, 0, std::integral_constant<int, T::kStride>{}, st);
    }
  };
  const auto form = [&](const char *dl, char *to) {
    if constexpr (T::kLate)
      for (int item = wave; item < KS + MT; item += waves)
        form_operands<NS, N>(reinterpret_cast<const float *>(dl), item, lane, to);
  };
  if constexpr (T::kLate) issue_part(tile_at(0), 0, std::integral_constant<int, T::kDlogit>{}, 0);
#pragma unroll
  for (int k = 0; k < S::kDist; ++k)
    if ((uint32_t)k < count) issue(k, k);

  // phi: operand (stream, t, ks), lane 16 q + m: coefficients 32 ks + 8 q .. + 7
  // of the wave's channel 8 (m / 4) + 4 t + m % 4.
  bf16x8 pa[JW][2][KS];
#pragma unroll
  for (int jj = 0; jj < JW; ++jj)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t v = v_wave + (lo16 >> 2);
        const int k0 = 32 * ks + 8 * q;
        u32x4 a = {0u, 0u, 0u, 0u};
        if (v < cvec && k0 < N) {
          const size_t at = ((size_t)(j0 + jj) * cvec * 8 + (size_t)v * 8 + 4 * t + (lo16 & 3)) * N + k0;
          if constexpr (N % 8 == 0) {
            a = load16(phi + at);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k0 + k < N) a[k / 2] |= (uint32_t)phi[at + k] << (16 * (k & 1));
          }
        }
        pa[jj][t][ks] = __builtin_bit_cast(bf16x8, a);
      }
  // Selections: channels 16 s .. 16 s + 15 of the 32.
  s16x8 sel[2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j) sel[s][j] = 8 * q + j == 16 * s + lo16 ? (short)0x3f80 : (short)0;
  f32x4 acc[JW][2][MT];
#pragma unroll
  for (int jj = 0; jj < JW; ++jj)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[jj][s][mt] = f32x4{0.f, 0.f, 0.f, 0.f};

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  // Where all of the wave's pieces have channels, every store is issued each
  // tile.
  const bool full = v_wave + 4 <= cvec;
  if constexpr (T::kLate) {
    // (The builtin, so that the compiler knows phi's loads to have ended and
    // puts no wait of its own into the loop.)
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    form(record[0], formed[0]);
  }
  int st = 0;  // the tile's stage
  for (uint32_t k = 0; k < count; ++k) {
    const uint32_t tile = tile_at(k);
    if (k < S::kDist || k + S::kDist > count || !full)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kYounger) : "memory");
    // The other waves' share of the tile has landed, and everybody has read
    // the last of the stage that the next loads fill.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (k + S::kDist < count) issue(k + S::kDist, st == 0 ? S::kStages - 1 : st - 1);
    char *mine = stage[st];
    const char *now = T::kLate ? formed[T::kLate ? k & 1 : 0] : record[st], *factors = record[st] + T::kDlogit;
    st = st + 1 == S::kStages ? 0 : st + 1;
    if (T::kLate && k + 1 < count) form(record[st], formed[T::kLate ? (k + 1) & 1 : 0]);
    const char *const f_at = mine + S::kG + S::kX;
    const uint32_t *const s_at = reinterpret_cast<const uint32_t *>(f_at + S::kF + wave * 256);
    bf16x8 bh[KS], bm[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      bh[ks] = reinterpret_cast<const bf16x8 *>(now)[ks * 64 + lane];
      bm[ks] = reinterpret_cast<const bf16x8 *>(now)[(KS + ks) * 64 + lane];
    }
    const float *mix = reinterpret_cast<const float *>(factors) + lo16;
    const float c = mix[T::KH * 16];
    const bf16x8 *cols_a = reinterpret_cast<const bf16x8 *>(now + T::kColsA) + lane;
    const u32x2 *cols_c = reinterpret_cast<const u32x2 *>(now + T::kColsC) + lane;
    const int at = piece_of(lo16, cw * 4 + q, lg);
    u32x4 x[JW];
#pragma unroll
    for (int jj = 0; jj < JW; ++jj) {
      if constexpr (CK) {
        const char *codes = mine + S::kG + ((j0 + jj) * 256 << (lg - 1)) + piece_of(lo16, cw * 2 + (q >> 1), lg - 1);
        x[jj] = held_bf16(*reinterpret_cast<const u32x2 *>(codes + (q & 1) * 8), (int)s_at[jj * 16 + lo16]);
      } else {
        x[jj] = *reinterpret_cast<const u32x4 *>(mine + S::kG + ((j0 + jj) * 256 << lg) + at);
      }
    }
    float o[JW][8];
#pragma unroll
    for (int jj = 0; jj < JW; ++jj) {
      f32x4 d[2] = {zero, zero};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 2; ++t) d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pa[jj][t][ks], bm[ks], d[t], 0, 0, 0);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 2; ++t) d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pa[jj][t][ks], bh[ks], d[t], 0, 0, 0);
      float xw[8];
      widen8(x[jj], xw);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[jj][e] = fmaf(c, xw[e], d[e >> 2][e & 3]);
    }
    {
      float fw[8];
      widen8(*reinterpret_cast<const u32x4 *>(f_at + at), fw);
#pragma unroll
      for (int jj = 0; jj < JW; ++jj) {
        const float hpre = mix[(j0 + jj) * 16];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[jj][e] = fmaf(hpre, fw[e], o[jj][e]);
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float gw[8];
      widen8(*reinterpret_cast<const u32x4 *>(mine + (i * 256 << lg) + at), gw);
#pragma unroll
      for (int jj = 0; jj < JW; ++jj) {
        const float hres = mix[(NS + i * NS + j0 + jj) * 16];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[jj][e] = fmaf(hres, gw[e], o[jj][e]);
      }
    }
    // dX out in memory order, the wave's own pieces: 64 bytes of a row a store
    // (whole rows of the workgroup's, after another barrier, measured 15 us
    // slower at n=4, C=7168, B=16384).
    char *const o_at = S::kOwnOut ? own_out + wave * (JW * 1024) : S::kShared ? mine + S::kG + (j0 * 256 << lg) : mine;
    const int ol = S::kOwnOut ? 2 : lg, ow = S::kOwnOut ? 0 : cw * 4;  // pieces of a row there, the wave's first
    const int o_write = S::kOwnOut ? piece_of(lo16, q, 2) : at;
    const int mr = lane >> 2, mp = (lane & 3) ^ (turn(mr, ol) & 3), o_read = piece_of(mr, ow + mp, ol);
#pragma unroll
    for (int jj = 0; jj < JW; ++jj)
      *reinterpret_cast<u32x4 *>(o_at + (jj * 256 << ol) + o_write) =
          u32x4{pack_bf16x2(o[jj][0], o[jj][1]), pack_bf16x2(o[jj][2], o[jj][3]), pack_bf16x2(o[jj][4], o[jj][5]),
                pack_bf16x2(o[jj][6], o[jj][7])};
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    {
      const uint32_t row = tile * 16 + mr, v = v_wave + mp;
      char *const dst = dX + ((size_t)row * NS + j0) * row_bytes + (size_t)v * 16;
      u32x4 y[JW];
#pragma unroll
      for (int jj = 0; jj < JW; ++jj) y[jj] = *reinterpret_cast<const u32x4 *>(o_at + (jj * 256 << ol) + o_read);
      if (row < B && v < cvec) {
#pragma unroll
        for (int jj = 0; jj < JW; ++jj) *reinterpret_cast<u32x4 *>(dst + (size_t)jj * row_bytes) = y[jj];
      }
    }
    bf16x8 twice[JW][2];
#pragma unroll
    for (int jj = 0; jj < JW; ++jj)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const f32x4 m = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, x[jj]), __builtin_bit_cast(bf16x8, sel[s]), zero, 0, 0, 0);
        const uint32_t p0 = pack_bf16x2(m[0], m[1]), p1 = pack_bf16x2(m[2], m[3]);
        twice[jj][s] = __builtin_bit_cast(bf16x8, u32x4{p0, p1, p0, p1});
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const u32x2 low = cols_c[mt * 64];
      const bf16x8 ca = cols_a[mt * 64], cc = __builtin_bit_cast(bf16x8, u32x4{low[0], low[1], 0u, 0u});
#pragma unroll
      for (int jj = 0; jj < JW; ++jj)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc[jj][s][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cc, twice[jj][s], acc[jj][s][mt], 0, 0, 0);
#pragma unroll
      for (int jj = 0; jj < JW; ++jj)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc[jj][s][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ca, twice[jj][s], acc[jj][s][mt], 0, 0, 0);
    }
  }

  // Lane 16 q + c of acc[jj][s][mt]: coefficients 16 mt + 4 q .. + 3 of the
  // wave's channel 16 s + c.
  float *po = out + (size_t)range * NS * cvec * 8 * N;
#pragma unroll
  for (int jj = 0; jj < JW; ++jj)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const f32x4 a = acc[jj][s][mt];
        const uint32_t ch = v_wave * 8 + 16 * s + lo16;
        const int k = 16 * mt + 4 * q;
        if (ch < cvec * 8 && k < N) {
          float *p = po + ((size_t)(j0 + jj) * cvec * 8 + ch) * N + k;
          if constexpr (N % 4 == 0) {
            *reinterpret_cast<f32x4 *>(p) = a;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (k + e < N) p[e] = a[e];
          }
        }
      }
}

// The last joins.  Workgroups below N + 3: a sum of db or dalpha each, from
// the coefficient kernel's workgroups (a thread every 256th, then a tree).
// The others: dphi from its row ranges, 64 vectors of four a workgroup, four
// threads a vector that take a quarter of the ranges each, in order.
template <int NS>
__global__ __launch_bounds__(256) void join_kernel(Sums sums, const f32x4 *__restrict__ part,
                                                   f32x4 *__restrict__ dphi, uint64_t vecs, uint32_t split) {
  constexpr int N = NS * NS + 2 * NS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x < (uint32_t)N + 3) {
    __shared__ double waves[4];
    const int k = blockIdx.x;
    double a = 0.0;
    for (int b = threadIdx.x; b < sums.blocks; b += 256) a += sums.part[(size_t)b * (N + 3) + k];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) a += __shfl_xor(a, o);
    if (lane == 0) waves[wave] = a;
    __syncthreads();
    if (threadIdx.x == 0) *sums.out<NS>(k) = (float)((waves[0] + waves[1]) + (waves[2] + waves[3]));
    return;
  }
  __shared__ f32x4 quarter[3][64];
  const uint32_t each = (split + 3) / 4, lo = wave * each, hi = lo + each < split ? lo + each : split;
  for (uint64_t v0 = (uint64_t)(blockIdx.x - N - 3) * 64; v0 < vecs; v0 += (uint64_t)(gridDim.x - N - 3) * 64) {
    const uint64_t v = v0 + lane;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (v < vecs) {
      for (uint32_t s = lo; s < hi; s += 8) {
        f32x4 x[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
          if (s + u < hi) x[u] = __builtin_nontemporal_load(part + (s + u) * vecs + v);
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
          if (s + u < hi) a += x[u];
      }
    }
    if (wave > 0) quarter[wave - 1][lane] = a;
    __syncthreads();
    if (wave == 0 && v < vecs) dphi[v] = ((a + quarter[0][lane]) + quarter[1][lane]) + quarter[2][lane];
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void zero_kernel(float *p, uint64_t count) {
  for (uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x; t < count; t += (uint64_t)gridDim.x * 256) p[t] = 0.f;
}

uint32_t wgs(uint64_t work, uint64_t per, uint64_t most) {
  const uint64_t g = (work + per - 1) / per;
  return (uint32_t)(g < most ? g : most);
}

// Few steps of the row dot products a wave cost less than a launch (2.7 us):
// with up to two, n=4, B=16, C=512 takes 15.6 us, not 18.1, and with four
// (C=2048) 18.4, not 18.0.  At n = 8 the kernel's 1024 threads have no
// registers for it (1 us slower).
constexpr int64_t kFusedSteps = 2;
template <int NS>
bool fused_dots(int64_t B, int64_t C) {
  if (NS == 8) return false;
  constexpr int R = sum_threads<NS>() / (NS * NS), at_once = coeff_threads<NS, true>() / 64 * kDotRows<NS>;
  const int64_t rows = B < R ? B : R;
  return (rows + at_once - 1) / at_once * ((C + 511) / 512) <= kFusedSteps && (B + R - 1) / R <= 256;
}

template <int NS, bool CK>
hipError_t launch_t(const CoeffsBwdPlan &p, int64_t B, int64_t C, const CoeffsBwdArgs &a, char *ws, hipStream_t st) {
  using T = Tiles<NS>;
  char *records = ws + p.records;
  float *dpre = reinterpret_cast<float *>(ws + p.dpre);
  double *sums = reinterpret_cast<double *>(ws + p.sums);
  float *part = p.split > 1 ? reinterpret_cast<float *>(ws + p.dphi) : a.dphi;
  const uint32_t cvec = (uint32_t)(C / 8), blocks = (uint32_t)ckpt_blocks(C), rows = (uint32_t)B;
  const u32x4 *dF = static_cast<const u32x4 *>(a.dF_pre);
  hipError_t e;
  const double inv_k = 1.0 / ((double)NS * (double)C);
  if (fused_dots<NS>(B, C)) {
    if constexpr (NS < 8)
      coeffs_bwd_kernel<NS><<<(uint32_t)p.sum_blocks, coeff_threads<NS, true>(), 0, st>>>(
          Dots<CK>{a.X.x, a.X.scales, dF, cvec, blocks}, a.logits, a.r, a.alpha[0], a.alpha[1], a.alpha[2], a.b_pre,
          a.b_post, a.b_res, a.dH, dpre, a.H, records, sums, rows, inv_k);
  } else {
    pre_dots_kernel<NS, CK, 4><<<wgs(B, 1, 1u << 22), 256, 0, st>>>(a.X.x, a.X.scales, dF, dpre, rows, cvec, blocks);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    coeffs_bwd_kernel<NS><<<(uint32_t)p.sum_blocks, coeff_threads<NS, false>(), 0, st>>>(
        NoDots{}, a.logits, a.r, a.alpha[0], a.alpha[1], a.alpha[2], a.b_pre, a.b_post, a.b_res, a.dH, dpre, a.H,
        records, sums, rows, inv_k);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const uint32_t slices = (uint32_t)p.slices, split = (uint32_t)p.split;
  const Sums join{sums, (int)p.sum_blocks, a.dalpha, a.db_pre, a.db_post, a.db_res};
  dx_dphi_kernel<NS, CK><<<slices * split + (split == 1 ? 1 : 0), 64 * T::GROUPS * p.wc, 0, st>>>(
      static_cast<const char *>(a.X.x), a.X.scales, static_cast<const uint16_t *>(a.phi),
      static_cast<const char *>(a.dX_next), static_cast<const char *>(a.dF_pre), records, static_cast<char *>(a.dX),
      part, rows, cvec, blocks, slices, split, p.wc, join);
  if ((e = hipGetLastError()) != hipSuccess || split == 1) return e;
  const uint64_t vecs = (uint64_t)NS * C * T::N / 4;
  join_kernel<NS><<<T::N + 3 + wgs(vecs, 64, 1u << 20), 256, 0, st>>>(
      join, reinterpret_cast<const f32x4 *>(part), reinterpret_cast<f32x4 *>(a.dphi), vecs, split);
  return hipGetLastError();
}

template <int NS>
hipError_t launch_n(const CoeffsBwdPlan &p, int64_t B, int64_t C, const CoeffsBwdArgs &a, char *ws, hipStream_t st) {
  return a.X.scales ? launch_t<NS, true>(p, B, C, a, ws, st) : launch_t<NS, false>(p, B, C, a, ws, st);
}

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

constexpr int64_t kRound = 256, kMinTiles = 4;

template <int NS>
CoeffsBwdPlan plan_n(int64_t B, int64_t C) {
  using T = Tiles<NS>;
  CoeffsBwdPlan p;
  const int64_t K = (int64_t)NS * C, tiles = (B + 15) / 16;
  p.wc = 1;  // waves along the channels, as many as there are channels for
  while (p.wc < 8 / T::GROUPS && p.wc * T::CW < C) p.wc *= 2;
  p.slices = (C + p.wc * T::CW - 1) / (p.wc * T::CW);
  // Row ranges: as many workgroups as the compute units hold of full ones
  // (eight waves on each), down to a tile a range; smaller workgroups share a
  // unit, and then a range gets kMinTiles tiles at least, as each costs a copy
  // of dphi.
  const int64_t room = kRound * (8 / (T::GROUPS * p.wc)) / p.slices;
  int64_t split = kRound / p.slices;
  if (split < (room < tiles / kMinTiles ? room : tiles / kMinTiles)) split = room < tiles / kMinTiles ? room : tiles / kMinTiles;
  if (split > tiles) split = tiles;
  if (split < 1) split = 1;
  // One range, which needs no join, where its further tiles cost less than the
  // join's launch and the copies of dphi, written and read (in us, measured:
  // 2 a tile at n = 4 and 8, 0.7 and 0.3 at n = 2 and 1; 2.7 a launch; 6 TB/s.
  // 16 rows of n=4, C=512: 18.1 us with one range or several, 20.7 with the
  // join; 60 rows of n=8, C=7168: 40 with one range, 53 with two; 120 rows of
  // n=4, C=512: 34 with one range, 20 with eight).
  const double tile_us = T::JW * (T::MT + 1) / 6.0, copy_us = (double)K * T::N * 8 / 6e6;
  if ((double)(tiles - (tiles + split - 1) / split) * tile_us <= 2.7 + (double)split * copy_us) split = 1;
  p.split = split;
  const int64_t per = sum_threads<NS>() / (NS * NS), groups = (B + per - 1) / per;
  p.sum_blocks = groups < kMaxSumBlocks ? groups : kMaxSumBlocks;
  p.records = 0;
  p.dpre = p.records + (size_t)tiles * T::kStride;
  p.sums = up16(p.dpre + (size_t)B * NS * 4);
  p.dphi = up16(p.sums + (size_t)p.sum_blocks * (T::N + 3) * 8);
  p.total_bytes = up16(p.dphi + (p.split > 1 ? (size_t)p.split * K * T::N * 4 : 0));
  return p;
}

}  // namespace

CoeffsBwdPlan plan_coeffs_pre_bwd(int64_t B, int n, int64_t C) {
  switch (n) {
    case 1: return plan_n<1>(B, C);
    case 2: return plan_n<2>(B, C);
    case 4: return plan_n<4>(B, C);
    default: return plan_n<8>(B, C);
  }
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
