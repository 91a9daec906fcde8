// C ABI of the training calls (declared in include/mhc.h): host-side argument
// checks, then the kernel launches.  Nothing here allocates, synchronises or
// prints.
#include "mhc_check.h"
#include "mhc_train.h"

#include <initializer_list>

using namespace mhc;

namespace {

// Every buffer of a call: where it is, how far it reaches, its alignment.
struct Buf {
  const void *p;
  size_t bytes;
  uintptr_t align;
  Span span() const { return mhc::span(p, bytes); }
};

// NULL, then misalignment, then an output over an input or another output.
int check_buffers(std::initializer_list<Buf> in, std::initializer_list<Buf> out) {
  for (const auto *l : {&in, &out})
    for (const Buf &b : *l)
      if (!b.p) return MHC_ERR_INVALID_ARG;
  for (const auto *l : {&in, &out})
    for (const Buf &b : *l)
      if (!aligned(b.p, b.align)) return MHC_ERR_UNSUPPORTED;
  for (const Buf *o = out.begin(); o != out.end(); ++o) {
    for (const Buf &i : in)
      if (overlaps(o->span(), i.span())) return MHC_ERR_INVALID_ARG;
    for (const Buf *q = out.begin(); q != o; ++q)
      if (overlaps(o->span(), q->span())) return MHC_ERR_INVALID_ARG;
  }
  return MHC_OK;
}

// Bytes of a call's tensors.
struct Sizes {
  size_t stream, vec, codes, scales, phi, coef, row, N, K;
  Sizes(int64_t B, int32_t n, int64_t C)
      : stream((size_t)B * n * C * 2), vec((size_t)B * C * 2), codes((size_t)B * n * C),
        scales((size_t)B * n * ckpt_blocks(C)), phi((size_t)n * C * ncoef(n) * 2), coef((size_t)B * ncoef(n) * 4),
        row((size_t)B * 4), N((size_t)ncoef(n)), K((size_t)n * C) {}
};

// X_t of a gradient call: the bf16 stream, or codes and scales (held twice in
// the buffer list, so that both calls have the same list).
struct XBufs {
  Buf x, s;
};
XBufs x_bufs(const void *X, const uint8_t *scales, bool ckpt, const Sizes &z) {
  if (!ckpt) return {Buf{X, z.stream, 16}, Buf{X, z.stream, 16}};
  return {Buf{X, z.codes, 16}, Buf{scales, z.scales, 1}};
}

int post_res_bwd(bool ckpt, int64_t B, int32_t n, int64_t C, const void *X, const uint8_t *scales, const void *F_out,
                 const float *H, const void *dX_next, void *dF_out, float *dH, void *stream) {
  int st = check_shape(B, n, C);
  if (st != MHC_OK || B == 0) return st;
  const Sizes z(B, n, C);
  const XBufs x = x_bufs(X, scales, ckpt, z);
  st = check_buffers({x.x, x.s, {F_out, z.vec, 16}, {H, z.coef, 4}, {dX_next, z.stream, 16}},
                     {{dF_out, z.vec, 16}, {dH, z.coef, 4}});
  if (st != MHC_OK) return st;
  return from_hip(launch_post_res_bwd(n, B, C, HeldX{X, ckpt ? scales : nullptr}, F_out, H, dX_next, dF_out, dH,
                                      static_cast<hipStream_t>(stream)));
}

// The parameters' gradients of no rows: zeros.
int zero_grads(int32_t n, int64_t C, float *dphi, float *dalpha, float *db_pre, float *db_post, float *db_res,
               hipStream_t s) {
  const Sizes z(0, n, C);
  const int st = check_buffers({}, {{dphi, z.phi * 2, 16}, {dalpha, 12, 4}, {db_pre, (size_t)n * 4, 4},
                                    {db_post, (size_t)n * 4, 4}, {db_res, (size_t)n * n * 4, 4}});
  if (st != MHC_OK) return st;
  hipError_t e = launch_zero_f32(dphi, (int64_t)(z.K * z.N), s);
  if (e == hipSuccess) e = launch_zero_f32(dalpha, 3, s);
  if (e == hipSuccess) e = launch_zero_f32(db_pre, n, s);
  if (e == hipSuccess) e = launch_zero_f32(db_post, n, s);
  if (e == hipSuccess) e = launch_zero_f32(db_res, n * n, s);
  return from_hip(e);
}

int coeffs_pre_bwd(bool ckpt, int64_t B, int32_t n, int64_t C, const CoeffsBwdArgs &a, void *workspace,
                   size_t workspace_bytes, void *stream) {
  int st = check_shape(B, n, C);
  if (st != MHC_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (B == 0) return zero_grads(n, C, a.dphi, a.dalpha, a.db_pre, a.db_post, a.db_res, s);
  const Sizes z(B, n, C);
  const CoeffsBwdPlan plan = plan_coeffs_pre_bwd(B, n, C);
  const XBufs x = x_bufs(a.X.x, a.X.scales, ckpt, z);
  const size_t nb = (size_t)n * 4, nr = (size_t)n * n * 4;
  st = check_buffers({x.x, x.s, {a.phi, z.phi, 16}, {a.b_pre, nb, 4}, {a.b_post, nb, 4}, {a.b_res, nr, 4},
                      {a.logits, z.coef, 4}, {a.r, z.row, 4}, {a.H, z.coef, 4}, {a.dX_next, z.stream, 16},
                      {a.dH, z.coef, 4}, {a.dF_pre, z.vec, 16}},
                     {{a.dX, z.stream, 16}, {a.dphi, z.phi * 2, 16}, {a.dalpha, 12, 4}, {a.db_pre, nb, 4},
                      {a.db_post, nb, 4}, {a.db_res, nr, 4}, {workspace, plan.total_bytes, 16}});
  if (st != MHC_OK) return st;
  if (workspace_bytes < plan.total_bytes) return MHC_ERR_WORKSPACE;
  CoeffsBwdArgs b = a;
  if (!ckpt) b.X.scales = nullptr;
  return from_hip(launch_coeffs_pre_bwd(plan, n, B, C, b, workspace, s));
}

// The embedding calls' shape: V rows of C in the table.
int check_table(int64_t B, int32_t n, int64_t C, int64_t V) {
  if (V < 1) return MHC_ERR_INVALID_ARG;
  const int st = check_shape(B, n, C);
  if (st != MHC_OK) return st;
  return V > kMaxB || V > kMaxElems / C ? MHC_ERR_UNSUPPORTED : MHC_OK;
}

}  // namespace

extern "C" {

int64_t mhc_ckpt_scales_per_row(int32_t n, int64_t C) {
  return check_shape(0, n, C) == MHC_OK ? n * ckpt_blocks(C) : 0;
}

int mhc_ckpt_pack(int64_t B, int32_t n, int64_t C, const void *X_t, void *codes, uint8_t *scales, void *stream) {
  int st = check_shape(B, n, C);
  if (st != MHC_OK || B == 0) return st;
  const Sizes z(B, n, C);
  st = check_buffers({{X_t, z.stream, 16}}, {{codes, z.codes, 16}, {scales, z.scales, 1}});
  if (st != MHC_OK) return st;
  return from_hip(launch_ckpt_pack(n, B, C, X_t, codes, scales, static_cast<hipStream_t>(stream)));
}

int mhc_ckpt_unpack(int64_t B, int32_t n, int64_t C, const void *codes, const uint8_t *scales, void *X_t,
                    void *stream) {
  int st = check_shape(B, n, C);
  if (st != MHC_OK || B == 0) return st;
  const Sizes z(B, n, C);
  st = check_buffers({{codes, z.codes, 16}, {scales, z.scales, 1}}, {{X_t, z.stream, 16}});
  if (st != MHC_OK) return st;
  return from_hip(launch_ckpt_unpack(n, B, C, codes, scales, X_t, static_cast<hipStream_t>(stream)));
}

int mhc_post_res_bwd(int64_t B, int32_t n, int64_t C, const void *X_t, const void *F_out, const float *H,
                     const void *dX_next, void *dF_out, float *dH, void *stream) {
  return post_res_bwd(false, B, n, C, X_t, nullptr, F_out, H, dX_next, dF_out, dH, stream);
}

int mhc_post_res_bwd_ckpt(int64_t B, int32_t n, int64_t C, const void *codes, const uint8_t *scales,
                          const void *F_out, const float *H, const void *dX_next, void *dF_out, float *dH,
                          void *stream) {
  return post_res_bwd(true, B, n, C, codes, scales, F_out, H, dX_next, dF_out, dH, stream);
}

size_t mhc_coeffs_pre_bwd_workspace_size(int64_t B, int32_t n, int64_t C) {
  if (check_shape(B, n, C) != MHC_OK || B == 0) return 0;
  return plan_coeffs_pre_bwd(B, n, C).total_bytes;
}

int mhc_coeffs_pre_bwd(int64_t B, int32_t n, int64_t C, const void *X_t, const void *phi, float alpha_pre,
                       float alpha_post, float alpha_res, const float *b_pre, const float *b_post, const float *b_res,
                       const float *logits, const float *r, const float *H, const void *dX_next, const float *dH,
                       const void *dF_pre, void *dX_t, float *dphi, float *dalpha, float *db_pre, float *db_post,
                       float *db_res, void *workspace, size_t workspace_bytes, void *stream) {
  const CoeffsBwdArgs a{{X_t, nullptr}, phi, {alpha_pre, alpha_post, alpha_res}, b_pre, b_post, b_res, logits, r, H,
                        dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre, db_post, db_res};
  return coeffs_pre_bwd(false, B, n, C, a, workspace, workspace_bytes, stream);
}

int mhc_coeffs_pre_bwd_ckpt(int64_t B, int32_t n, int64_t C, const void *codes, const uint8_t *scales,
                            const void *phi, float alpha_pre, float alpha_post, float alpha_res, const float *b_pre,
                            const float *b_post, const float *b_res, const float *logits, const float *r,
                            const float *H, const void *dX_next, const float *dH, const void *dF_pre, void *dX_t,
                            float *dphi, float *dalpha, float *db_pre, float *db_post, float *db_res, void *workspace,
                            size_t workspace_bytes, void *stream) {
  const CoeffsBwdArgs a{{codes, scales}, phi, {alpha_pre, alpha_post, alpha_res}, b_pre, b_post, b_res, logits, r, H,
                        dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre, db_post, db_res};
  return coeffs_pre_bwd(true, B, n, C, a, workspace, workspace_bytes, stream);
}

int mhc_embed(int64_t B, int32_t n, int64_t C, int64_t V, const int64_t *tokens, const void *table, float scale,
              void *X_0, void *stream) {
  int st = check_table(B, n, C, V);
  if (st != MHC_OK || B == 0) return st;
  st = check_buffers({{tokens, (size_t)B * 8, 8}, {table, (size_t)V * C * 2, 16}}, {{X_0, (size_t)B * n * C * 2, 16}});
  if (st != MHC_OK) return st;
  return from_hip(launch_embed(n, B, C, V, tokens, table, scale, X_0, static_cast<hipStream_t>(stream)));
}

size_t mhc_embed_bwd_workspace_size(int64_t B, int32_t n, int64_t C, int64_t V) {
  if (check_table(B, n, C, V) != MHC_OK || B == 0) return 0;
  return plan_embed_bwd(B, C).total_bytes;
}

int mhc_embed_bwd(int64_t B, int32_t n, int64_t C, int64_t V, const int64_t *tokens, const void *dX_0, float scale,
                  int32_t accumulate, float *dtable, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_table(B, n, C, V);
  if (st != MHC_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Buf table{dtable, (size_t)V * C * 4, 16};
  if (B == 0) {  // the gradient of no tokens: zeros, or nothing to add
    st = check_buffers({}, {table});
    return st != MHC_OK || accumulate ? st : from_hip(launch_zero_f32(dtable, V * C, s));
  }
  const EmbedBwdPlan plan = plan_embed_bwd(B, C);
  st = check_buffers({{tokens, (size_t)B * 8, 8}, {dX_0, (size_t)B * n * C * 2, 16}},
                     {table, {workspace, plan.total_bytes, 16}});
  if (st != MHC_OK) return st;
  if (workspace_bytes < plan.total_bytes) return MHC_ERR_WORKSPACE;
  return from_hip(launch_embed_bwd(plan, n, B, C, V, tokens, dX_0, scale, accumulate != 0, dtable, workspace, s));
}

}  // extern "C"
