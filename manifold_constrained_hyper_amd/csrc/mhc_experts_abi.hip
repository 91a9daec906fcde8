// C ABI of the calls around a layer of experts (declared in include/mhc.h):
// host-side argument checks, then the kernel launches.  Nothing here
// allocates, synchronises or prints.
#include "mhc_check.h"
#include "mhc_experts.h"
#include "mhc_train.h"

using namespace mhc;

namespace {

constexpr bool kOptional = true;

int check_rows(int64_t B, int64_t C, int64_t most) {
  if (B < 0 || C < 1) return MHC_ERR_INVALID_ARG;
  if (C % 8 != 0 || C > most || B > kMaxB || B > kMaxElems / C) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

// eps is a number that keeps the root real.
bool bad_eps(float eps) { return !(eps >= 0.0f) || eps > 3.4028234e38f; }

constexpr int32_t kRouteFlags = MHC_ROUTE_SOFTMAX | MHC_ROUTE_RENORM | MHC_ROUTE_BF16;

int check_route(int64_t B, int32_t E, int32_t k, int32_t flags) {
  if (B < 0 || E < 1 || k < 1 || k > E || (flags & ~kRouteFlags)) return MHC_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMaxChosen || B > kMaxB) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

int check_pairs(int64_t B, int32_t k) {
  if (B < 0 || k < 1) return MHC_ERR_INVALID_ARG;
  if (k > kMaxChosen || B > kMaxB / k) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

// B * k rows of C channels.
int check_pair_rows(int64_t B, int32_t k, int64_t C) {
  if (C < 1) return MHC_ERR_INVALID_ARG;
  const int st = check_pairs(B, k);
  if (st != MHC_OK) return st;
  if (C % 8 != 0 || C > kMaxK || (B > 0 && B * k > kMaxElems / C)) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

RouteArgs route_args(int32_t E, int32_t k, int32_t groups, int32_t top_groups, int32_t flags, float scale) {
  return RouteArgs{E, k, groups, top_groups, (flags & MHC_ROUTE_SOFTMAX) != 0, (flags & MHC_ROUTE_RENORM) != 0,
                   (flags & MHC_ROUTE_BF16) != 0, scale};
}

}  // namespace

extern "C" {

int mhc_rmsnorm(int64_t B, int64_t C, const void *x, const void *shortcut, const float *weight, float eps, void *sum,
                void *y, void *codes, uint8_t *scales, float *rstd, void *stream) {
  int st = check_rows(B, C, kMaxNormC);
  if (st != MHC_OK) return st;
  if (bad_eps(eps)) return MHC_ERR_INVALID_ARG;
  if (B == 0) return MHC_OK;
  if ((!y && !codes) || !codes != !scales || (sum && !shortcut)) return MHC_ERR_INVALID_ARG;
  const size_t row = (size_t)B * C * 2;
  st = check_buffers({{x, row, 16}, {shortcut, row, 16, kOptional}, {weight, (size_t)C * 4, 16, kOptional}},
                     {{sum, row, 16, kOptional}, {y, row, 16, kOptional}, {codes, (size_t)B * C, 16, kOptional},
                      {scales, (size_t)(B * ckpt_blocks(C)), 1, kOptional}, {rstd, (size_t)B * 4, 4, kOptional}});
  if (st != MHC_OK) return st;
  return from_hip(launch_rmsnorm(B, C, NormArgs{x, shortcut, weight, eps, sum, y, codes, scales, rstd},
                                 static_cast<hipStream_t>(stream)));
}

size_t mhc_rmsnorm_bwd_workspace_size(int64_t B, int64_t C) {
  if (check_rows(B, C, kMaxNormC) != MHC_OK || B == 0) return 0;
  return plan_rmsnorm_bwd(B, C).total_bytes;
}

int mhc_rmsnorm_bwd(int64_t B, int64_t C, const void *sum, const float *weight, const float *rstd, const void *dy,
                    const void *dsum, void *dx, float *dweight, void *workspace, size_t workspace_bytes,
                    void *stream) {
  int st = check_rows(B, C, kMaxNormC);
  if (st != MHC_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Buf gain{dweight, (size_t)C * 4, 16, kOptional};
  if (B == 0) {  // the gain's gradient of no rows: zeros
    st = check_buffers({}, {gain});
    return st != MHC_OK || !dweight ? st : from_hip(launch_zero_f32(dweight, C, s));
  }
  const NormBwdPlan plan = plan_rmsnorm_bwd(B, C);
  const size_t row = (size_t)B * C * 2;
  // Without dweight the workspace is neither looked at nor needed.
  const Buf ws{dweight ? workspace : nullptr, plan.total_bytes, 16, !dweight};
  st = check_buffers({{sum, row, 16}, {weight, (size_t)C * 4, 16, kOptional}, {rstd, (size_t)B * 4, 4}, {dy, row, 16},
                      {dsum, row, 16, kOptional}},
                     {{dx, row, 16}, gain, ws});
  if (st != MHC_OK) return st;
  if (dweight && workspace_bytes < plan.total_bytes) return MHC_ERR_WORKSPACE;
  return from_hip(launch_rmsnorm_bwd(plan, B, C, NormBwdArgs{sum, weight, rstd, dy, dsum, dx, dweight}, workspace, s));
}

int mhc_route(int64_t B, int32_t E, int32_t k, int32_t groups, int32_t top_groups, int32_t flags, float scale,
              const void *logits, const float *bias, int32_t *ids, float *weights, void *stream) {
  int st = check_route(B, E, k, flags);
  if (st == MHC_ERR_INVALID_ARG) return st;
  if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      k > (int64_t)top_groups * (E / groups))
    return MHC_ERR_INVALID_ARG;
  if (st != MHC_OK) return st;
  if (groups > kMaxGroups) return MHC_ERR_UNSUPPORTED;
  if (B == 0) return MHC_OK;
  const RouteArgs a = route_args(E, k, groups, top_groups, flags, scale);
  const size_t one = a.bf16 ? 2 : 4, pairs = (size_t)B * k * 4;
  st = check_buffers({{logits, (size_t)B * E * one, one}, {bias, (size_t)E * 4, 4, kOptional}},
                     {{ids, pairs, 4}, {weights, pairs, 4}});
  if (st != MHC_OK) return st;
  return from_hip(launch_route(B, a, logits, bias, ids, weights, static_cast<hipStream_t>(stream)));
}

int mhc_route_bwd(int64_t B, int32_t E, int32_t k, int32_t flags, float scale, const void *logits, const int32_t *ids,
                  const float *dweights, void *dlogits, void *stream) {
  int st = check_route(B, E, k, flags);
  if (st != MHC_OK || B == 0) return st;
  const RouteArgs a = route_args(E, k, 1, 1, flags, scale);
  const size_t one = a.bf16 ? 2 : 4, pairs = (size_t)B * k * 4, all = (size_t)B * E * one;
  st = check_buffers({{logits, all, one}, {ids, pairs, 4}, {dweights, pairs, 4}}, {{dlogits, all, one}});
  if (st != MHC_OK) return st;
  return from_hip(launch_route_bwd(B, a, logits, ids, dweights, dlogits, static_cast<hipStream_t>(stream)));
}

size_t mhc_experts_order_workspace_size(int64_t B, int32_t k, int32_t E) {
  if (check_pairs(B, k) != MHC_OK || B == 0 || E < 1 || E > kMaxExperts) return 0;
  return plan_experts_order(B * k, E).total_bytes;
}

int mhc_experts_order(int64_t B, int32_t k, int32_t E, const int32_t *ids, int32_t *slots, int32_t *offsets,
                      void *workspace, size_t workspace_bytes, void *stream) {
  if (E < 1) return MHC_ERR_INVALID_ARG;
  int st = check_pairs(B, k);
  if (st != MHC_OK) return st;
  if (E > kMaxExperts) return MHC_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Buf starts{offsets, (size_t)(E + 1) * 4, 4};
  if (B == 0) {  // no pairs: every expert starts and ends at 0
    st = check_buffers({}, {starts});
    return st != MHC_OK ? st : from_hip(launch_zero_f32(reinterpret_cast<float *>(offsets), E + 1, s));
  }
  const OrderPlan plan = plan_experts_order(B * k, E);
  const size_t pairs = (size_t)B * k * 4;
  st = check_buffers({{ids, pairs, 4}}, {{slots, pairs, 4}, starts, {workspace, plan.total_bytes, 16}});
  if (st != MHC_OK) return st;
  if (workspace_bytes < plan.total_bytes) return MHC_ERR_WORKSPACE;
  return from_hip(launch_experts_order(plan, B * k, E, ids, slots, offsets, workspace, s));
}

int mhc_experts_gather(int64_t B, int32_t k, int64_t C, const void *X, const int32_t *slots, void *rows,
                       void *stream) {
  int st = check_pair_rows(B, k, C);
  if (st != MHC_OK || B == 0) return st;
  st = check_buffers({{X, (size_t)B * C * 2, 16}, {slots, (size_t)B * k * 4, 4}}, {{rows, (size_t)B * k * C * 2, 16}});
  if (st != MHC_OK) return st;
  return from_hip(
      launch_experts_gather(B, k, C, X, nullptr, slots, rows, nullptr, static_cast<hipStream_t>(stream)));
}

int mhc_experts_gather_ckpt(int64_t B, int32_t k, int64_t C, const void *codes, const uint8_t *scales,
                            const int32_t *slots, void *row_codes, uint8_t *row_scales, void *stream) {
  int st = check_pair_rows(B, k, C);
  if (st != MHC_OK || B == 0) return st;
  const size_t blocks = (size_t)(B * ckpt_blocks(C));
  st = check_buffers({{codes, (size_t)B * C, 16}, {scales, blocks, 1}, {slots, (size_t)B * k * 4, 4}},
                     {{row_codes, (size_t)B * k * C, 16}, {row_scales, blocks * k, 1}});
  if (st != MHC_OK) return st;
  return from_hip(
      launch_experts_gather(B, k, C, codes, scales, slots, row_codes, row_scales, static_cast<hipStream_t>(stream)));
}

int mhc_experts_combine(int64_t B, int32_t k, int64_t C, const void *Y, const int32_t *slots, const float *weights,
                        const void *shared, void *F_out, void *stream) {
  int st = check_pair_rows(B, k, C);
  if (st != MHC_OK || B == 0) return st;
  const size_t row = (size_t)B * C * 2, pairs = (size_t)B * k * 4;
  st = check_buffers(
      {{Y, row * k, 16}, {slots, pairs, 4}, {weights, pairs, 4, kOptional}, {shared, row, 16, kOptional}},
      {{F_out, row, 16}});
  if (st != MHC_OK) return st;
  return from_hip(
      launch_experts_combine(B, k, C, Y, slots, weights, shared, F_out, static_cast<hipStream_t>(stream)));
}

int mhc_experts_combine_bwd(int64_t B, int32_t k, int64_t C, const void *Y, const int32_t *slots, const float *weights,
                            const void *dF_out, void *dY, float *dweights, void *stream) {
  int st = check_pair_rows(B, k, C);
  if (st != MHC_OK || B == 0) return st;
  const size_t row = (size_t)B * C * 2, pairs = (size_t)B * k * 4;
  st = check_buffers({{Y, row * k, 16}, {slots, pairs, 4}, {weights, pairs, 4}, {dF_out, row, 16}},
                     {{dY, row * k, 16}, {dweights, pairs, 4}});
  if (st != MHC_OK) return st;
  return from_hip(
      launch_experts_combine_bwd(B, k, C, Y, slots, weights, dF_out, dY, dweights, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
