// Host-side launch interface of the kernels around a layer of experts (norm,
// choice of experts, rows into the experts' order and back).  Arguments are
// validated by the caller; these functions only pick launch shapes and enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mhc {

constexpr int kMaxExperts = 1024;     // E
constexpr int kMaxChosen = 32;        // k
constexpr int kMaxGroups = 64;
constexpr int64_t kMaxNormC = 65536;  // channels of a normalised row

struct NormArgs {
  const void *x, *shortcut;  // shortcut may be null, as weight, sum, y, codes and scales, rstd
  const float *weight;
  float eps;
  void *sum, *y, *codes;
  uint8_t *scales;
  float *rstd;
};
hipError_t launch_rmsnorm(int64_t B, int64_t C, const NormArgs &a, hipStream_t st);

// Workspace of the norm's gradient: fp32 [parts, C] partial sums of dweight.
struct NormBwdPlan {
  int64_t parts;
  size_t total_bytes;
};
NormBwdPlan plan_rmsnorm_bwd(int64_t B, int64_t C);
struct NormBwdArgs {
  const void *sum;
  const float *weight, *rstd;  // weight may be null
  const void *dy, *dsum;       // dsum may be null
  void *dx;
  float *dweight;  // may be null
};
hipError_t launch_rmsnorm_bwd(const NormBwdPlan &p, int64_t B, int64_t C, const NormBwdArgs &a, void *ws,
                              hipStream_t st);

struct RouteArgs {
  int E, k, groups, top_groups;
  bool softmax, renorm, bf16;
  float scale;
};
hipError_t launch_route(int64_t B, const RouteArgs &a, const void *logits, const float *bias, int32_t *ids,
                        float *weights, hipStream_t st);
hipError_t launch_route_bwd(int64_t B, const RouteArgs &a, const void *logits, const int32_t *ids,
                            const float *dweights, void *dlogits, hipStream_t st);

// Workspace of the experts' order: int32 [tiles, E] counts of each tile of
// `tile` consecutive pairs.
struct OrderPlan {
  int64_t tile, tiles;
  size_t total_bytes;
};
OrderPlan plan_experts_order(int64_t pairs, int E);
hipError_t launch_experts_order(const OrderPlan &p, int64_t pairs, int E, const int32_t *ids, int32_t *slots,
                                int32_t *offsets, void *ws, hipStream_t st);

// bf16 rows of C channels, or codes of C and scales of ceil(C / 32) bytes
// (scales non-null).
hipError_t launch_experts_gather(int64_t B, int k, int64_t C, const void *x, const uint8_t *scales,
                                 const int32_t *slots, void *rows, uint8_t *row_scales, hipStream_t st);
// weights may be null (1 for every slot), shared too (nothing is added).
hipError_t launch_experts_combine(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                  const float *weights, const void *shared, void *out, hipStream_t st);
hipError_t launch_experts_combine_bwd(int64_t B, int k, int64_t C, const void *Y, const int32_t *slots,
                                      const float *weights, const void *dout, void *dY, float *dweights,
                                      hipStream_t st);

}  // namespace mhc
