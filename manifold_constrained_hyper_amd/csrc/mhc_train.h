// Host-side launch interface of the training kernels (8-bit checkpoints of
// the stream, gradients, embeddings).  Arguments are validated by the caller;
// these functions only pick launch shapes and enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mhc {

// A checkpoint gives one scale byte to every 32 channels of a stream; a
// stream's last block may be shorter.
constexpr int64_t kCkptBlock = 32;
inline int64_t ckpt_blocks(int64_t C) { return (C + kCkptBlock - 1) / kCkptBlock; }

// X_t as the gradient calls get it: the bf16 stream (scales null) or the
// codes and scales of its checkpoint.
struct HeldX {
  const void *x;
  const uint8_t *scales;
};

hipError_t launch_ckpt_pack(int n, int64_t B, int64_t C, const void *X, void *codes, uint8_t *scales, hipStream_t st);
hipError_t launch_ckpt_unpack(int n, int64_t B, int64_t C, const void *codes, const uint8_t *scales, void *X,
                              hipStream_t st);

hipError_t launch_post_res_bwd(int n, int64_t B, int64_t C, HeldX X, const void *F_out, const float *H,
                               const void *dX_next, void *dF_out, float *dH, hipStream_t st);

// Workspace of the coefficient and pre-mix gradient (bytes from its start):
//   records                  a record for each tile of 16 rows: dlogit and what
//                            else its dX needs of H and r
//                            (mhc_coeffs_pre_bwd.hip)
//   dpre   fp32 [B, n]       gradient of H_pre
//   sums   fp64 [sum_blocks, N + 3]  partial sums of the bias and alpha gradients
//   dphi   fp32 [split, K, N]        partial sums of dphi (split > 1)
struct CoeffsBwdPlan {
  int wc;              // waves along the channels in a workgroup
  int64_t slices;      // workgroups along the channels
  int64_t split;       // row ranges (every split-th tile of 16 rows)
  int64_t sum_blocks;  // workgroups of the coefficient kernel
  size_t records, dpre, sums, dphi, total_bytes;
};
CoeffsBwdPlan plan_coeffs_pre_bwd(int64_t B, int n, int64_t C);

struct CoeffsBwdArgs {
  HeldX X;
  const void *phi;
  float alpha[3];
  const float *b_pre, *b_post, *b_res, *logits, *r, *H;
  const void *dX_next;
  const float *dH;
  const void *dF_pre;
  void *dX;
  float *dphi, *dalpha, *db_pre, *db_post, *db_res;
};
hipError_t launch_coeffs_pre_bwd(const CoeffsBwdPlan &p, int n, int64_t B, int64_t C, const CoeffsBwdArgs &a, void *ws,
                                 hipStream_t st);

hipError_t launch_embed(int n, int64_t B, int64_t C, int64_t V, const int64_t *tokens, const void *table, float scale,
                        void *X_0, hipStream_t st);

// Workspace of the embedding gradient (bytes from its start): two lists of
// [B] sort keys (uint64), then fp32 [ceil(B / rb), 2, C] partial sums of the
// tokens whose rows span blocks of rb places of the sorted order.
struct EmbedBwdPlan {
  int64_t rb;
  size_t keys, other, part, total_bytes;
};
EmbedBwdPlan plan_embed_bwd(int64_t B, int64_t C);
hipError_t launch_embed_bwd(const EmbedBwdPlan &p, int n, int64_t B, int64_t C, int64_t V, const int64_t *tokens,
                            const void *dX_0, float scale, bool accumulate, float *dtable, void *ws, hipStream_t st);

// Zero-fills count fp32 values.
hipError_t launch_zero_f32(float *p, int64_t count, hipStream_t st);

}  // namespace mhc
