// Host-only check of libmhc's training calls, built like abi_host_check.cpp
// with AddressSanitizer and UndefinedBehaviorSanitizer on the host code (no
// check here launches a kernel where a device is visible).
//
// Drives the argument checks of the training entry points in include/mhc.h
// with fake device addresses (never dereferenced on the host), their size
// functions and workspace plans over ordinary and extreme shapes, and -- on a
// host with no HIP device -- calls that pass the checks, which must report
// MHC_ERR_HIP.  Exits non-zero on the first failed check; the sanitizers abort
// on any error they find.
#include "mhc.h"
#include "mhc_train.h"

#include <cstdint>
#include <cstdio>
#include <cstdlib>

namespace {

int g_checks = 0;

#define CHECK(cond)                                                                 \
  do {                                                                              \
    ++g_checks;                                                                     \
    if (!(cond)) {                                                                  \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      std::exit(1);                                                                 \
    }                                                                               \
  } while (0)

struct Shape {
  int64_t B;
  int32_t n;
  int64_t C, V;
};
constexpr Shape kGood{16, 4, 40, 100};

// Every tensor of a call, as fake, 16-byte aligned addresses far apart, and
// what `over` replaces of them.
constexpr int kMost = 24;
struct Args {
  char *p[kMost];
  Args() {
    for (int k = 0; k < kMost; ++k) p[k] = reinterpret_cast<char *>(uintptr_t(1) << 44 | (uintptr_t)(k + 1) << 38);
  }
  float *f(int k) const { return reinterpret_cast<float *>(p[k]); }
  uint8_t *b(int k) const { return reinterpret_cast<uint8_t *>(p[k]); }
  int64_t *l(int k) const { return reinterpret_cast<int64_t *>(p[k]); }
};

constexpr size_t kAll = ~size_t(0);  // "the size the call asks for"

// One entry point: how many tensors, which of them are outputs (bit k), their
// alignments, and the call.
struct Call {
  const char *name;
  int tensors;
  uint32_t outputs;
  const uint8_t *align;
  int (*run)(const Shape &, const Args &, size_t ws);
  size_t (*workspace)(const Shape &);  // null where there is none
};

size_t no_workspace(const Shape &) { return 0; }
size_t coeffs_ws(const Shape &s) { return mhc_coeffs_pre_bwd_workspace_size(s.B, s.n, s.C); }
size_t embed_ws(const Shape &s) { return mhc_embed_bwd_workspace_size(s.B, s.n, s.C, s.V); }

int pack(const Shape &s, const Args &a, size_t) { return mhc_ckpt_pack(s.B, s.n, s.C, a.p[0], a.p[1], a.b(2), nullptr); }
int unpack(const Shape &s, const Args &a, size_t) {
  return mhc_ckpt_unpack(s.B, s.n, s.C, a.p[0], a.b(1), a.p[2], nullptr);
}
int post(const Shape &s, const Args &a, size_t) {
  return mhc_post_res_bwd(s.B, s.n, s.C, a.p[0], a.p[1], a.f(2), a.p[3], a.p[4], a.f(5), nullptr);
}
int post_ckpt(const Shape &s, const Args &a, size_t) {
  return mhc_post_res_bwd_ckpt(s.B, s.n, s.C, a.p[0], a.b(1), a.p[2], a.f(3), a.p[4], a.p[5], a.f(6), nullptr);
}
int coeffs(const Shape &s, const Args &a, size_t ws) {
  return mhc_coeffs_pre_bwd(s.B, s.n, s.C, a.p[0], a.p[1], 0.1f, 0.1f, 0.1f, a.f(2), a.f(3), a.f(4), a.f(5), a.f(6),
                            a.f(7), a.p[8], a.f(9), a.p[10], a.p[11], a.f(12), a.f(13), a.f(14), a.f(15), a.f(16),
                            a.p[17], ws == kAll ? coeffs_ws(s) : ws, nullptr);
}
int coeffs_ckpt(const Shape &s, const Args &a, size_t ws) {
  return mhc_coeffs_pre_bwd_ckpt(s.B, s.n, s.C, a.p[0], a.b(1), a.p[2], 0.1f, 0.1f, 0.1f, a.f(3), a.f(4), a.f(5),
                                 a.f(6), a.f(7), a.f(8), a.p[9], a.f(10), a.p[11], a.p[12], a.f(13), a.f(14), a.f(15),
                                 a.f(16), a.f(17), a.p[18], ws == kAll ? coeffs_ws(s) : ws, nullptr);
}
int embed(const Shape &s, const Args &a, size_t) {
  return mhc_embed(s.B, s.n, s.C, s.V, a.l(0), a.p[1], 0.5f, a.p[2], nullptr);
}
int embed_bwd(const Shape &s, const Args &a, size_t ws) {
  return mhc_embed_bwd(s.B, s.n, s.C, s.V, a.l(0), a.p[1], 0.5f, 0, a.f(2), a.p[3], ws == kAll ? embed_ws(s) : ws,
                       nullptr);
}

const uint8_t kPack[] = {16, 16, 1}, kUnpack[] = {16, 1, 16}, kPost[] = {16, 16, 4, 16, 16, 4},
              kPostCkpt[] = {16, 1, 16, 4, 16, 16, 4},
              kCoeffs[] = {16, 16, 4, 4, 4, 4, 4, 4, 16, 4, 16, 16, 16, 4, 4, 4, 4, 16},
              kCoeffsCkpt[] = {16, 1, 16, 4, 4, 4, 4, 4, 4, 16, 4, 16, 16, 16, 4, 4, 4, 4, 16}, kEmbed[] = {8, 16, 16},
              kEmbedBwd[] = {8, 16, 16, 16};
const Call kCalls[] = {
    {"mhc_ckpt_pack", 3, 0b110, kPack, pack, no_workspace},
    {"mhc_ckpt_unpack", 3, 0b100, kUnpack, unpack, no_workspace},
    {"mhc_post_res_bwd", 6, 0b110000, kPost, post, no_workspace},
    {"mhc_post_res_bwd_ckpt", 7, 0b1100000, kPostCkpt, post_ckpt, no_workspace},
    {"mhc_coeffs_pre_bwd", 18, 0x7fu << 11, kCoeffs, coeffs, coeffs_ws},
    {"mhc_coeffs_pre_bwd_ckpt", 19, 0x7fu << 12, kCoeffsCkpt, coeffs_ckpt, coeffs_ws},
    {"mhc_embed", 3, 0b100, kEmbed, embed, no_workspace},
    {"mhc_embed_bwd", 4, 0b1100, kEmbedBwd, embed_bwd, embed_ws},
};

void check_call(const Call &c, bool no_device) {
  std::printf("%s\n", c.name);
  const Args ok;
  const auto shaped = [&](int64_t B, int32_t n, int64_t C) { return c.run(Shape{B, n, C, 100}, ok, 0); };
  CHECK(shaped(-1, 4, 40) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(INT64_MIN, 4, 40) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(16, 0, 40) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(16, INT32_MIN, 40) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(16, 4, 0) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(16, 4, INT64_MIN) == MHC_ERR_INVALID_ARG);
  CHECK(shaped(16, 3, 40) == MHC_ERR_UNSUPPORTED);
  CHECK(shaped(16, INT32_MAX, 40) == MHC_ERR_UNSUPPORTED);
  CHECK(shaped(16, 4, 12) == MHC_ERR_UNSUPPORTED);
  CHECK(shaped(16, 4, INT64_MAX - 7) == MHC_ERR_UNSUPPORTED);
  CHECK(shaped(INT64_MAX, 4, 40) == MHC_ERR_UNSUPPORTED);
  CHECK(shaped(int64_t(1) << 30, 8, int64_t(1) << 26) == MHC_ERR_UNSUPPORTED);
  for (int k = 0; k < c.tensors; ++k) {
    Args a;
    a.p[k] = nullptr;
    CHECK(c.run(kGood, a, kAll) == MHC_ERR_INVALID_ARG);
    if (c.align[k] > 1) {
      a.p[k] = ok.p[k] + c.align[k] / 2;
      CHECK(c.run(kGood, a, kAll) == MHC_ERR_UNSUPPORTED);
    }
    if (!(c.outputs >> k & 1)) continue;
    for (int q = 0; q < c.tensors; ++q) {  // an output over each other tensor, and 16 bytes before it
      if (q == k) continue;
      a.p[k] = ok.p[q];
      CHECK(c.run(kGood, a, kAll) == MHC_ERR_INVALID_ARG);
      if (!no_device) continue;
      a.p[k] = ok.p[q] - 16;  // the shortest outputs end before it
      const int st = c.run(kGood, a, kAll);
      CHECK(st == MHC_ERR_INVALID_ARG || st == MHC_ERR_HIP);
    }
  }
  if (c.workspace(kGood)) {
    CHECK(c.run(kGood, ok, c.workspace(kGood) - 1) == MHC_ERR_WORKSPACE);
    CHECK(c.run(kGood, ok, 0) == MHC_ERR_WORKSPACE);
  }
  if (!no_device) return;
  for (int32_t n : {1, 2, 4, 8})
    for (int64_t B : {int64_t(1), int64_t(17), int64_t(1000), int64_t(20000)})
      for (int64_t C : {int64_t(8), int64_t(1000), int64_t(7168)})
        CHECK(c.run(Shape{B, n, C, 100}, ok, kAll) == MHC_ERR_HIP);
}

// Plans and sizes over the whole accepted range.
void check_sizes() {
  const int64_t Bs[] = {0, 1, 15, 16, 17, 256, 257, 1000, 16384, 1 << 20, (int64_t(1) << 31) - 1, int64_t(1) << 31,
                        INT64_MAX, -1, INT64_MIN};
  const int32_t ns[] = {1, 2, 3, 4, 8, 0, -4, INT32_MAX, INT32_MIN};
  const int64_t Cs[] = {8, 24, 40, 512, 1000, 7168, 1 << 20, int64_t(1) << 27, int64_t(1) << 30, int64_t(1) << 62,
                        INT64_MAX - 7, INT64_MAX, 0, -8, 12};
  const int64_t Vs[] = {1, 100, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX, 0, -1, INT64_MIN};
  for (int32_t n : ns)
    for (int64_t C : Cs) {
      const bool shape = (n == 1 || n == 2 || n == 4 || n == 8) && C > 0 && C % 8 == 0 && C <= (int64_t(1) << 30) / n;
      CHECK(mhc_ckpt_scales_per_row(n, C) == (shape ? n * ((C + 31) / 32) : 0));
      for (int64_t B : Bs) {
        const bool rows = shape && B > 0 && B < (int64_t(1) << 31) && B <= (int64_t(1) << 40) / (n * C);
        const size_t ws = mhc_coeffs_pre_bwd_workspace_size(B, n, C);
        CHECK((ws > 0) == rows);
        if (rows) {
          const mhc::CoeffsBwdPlan p = mhc::plan_coeffs_pre_bwd(B, n, C);
          const int64_t tiles = (B + 15) / 16;
          CHECK(p.total_bytes == ws && p.split >= 1 && p.split <= tiles && p.slices >= 1 && p.sum_blocks >= 1);
          CHECK((p.slices * p.split + 1) * 512 < int64_t(1) << 32);  // the grid's threads
          CHECK(p.dpre % 4 == 0 && p.sums % 16 == 0 && p.dphi % 16 == 0);
          CHECK(p.records < p.dpre && p.dpre < p.sums && p.sums < p.dphi && p.dphi <= p.total_bytes);
          CHECK(p.wc >= 1 && p.wc <= 8 && (p.wc & (p.wc - 1)) == 0);
        }
        for (int64_t V : Vs) {
          const bool table = rows && V > 0 && V < (int64_t(1) << 31) && V <= (int64_t(1) << 40) / C;
          const size_t we = mhc_embed_bwd_workspace_size(B, n, C, V);
          CHECK((we > 0) == table);
          if (!table) continue;
          const mhc::EmbedBwdPlan p = mhc::plan_embed_bwd(B, C);
          CHECK(p.total_bytes == we && p.rb >= 4 && p.rb <= 64 && p.keys + (size_t)B * 8 <= p.other &&
                p.other + (size_t)B * 8 <= p.part && p.part % 16 == 0);
        }
      }
    }
}

}  // namespace

int main(int argc, char **argv) {
  const bool no_device = argc > 1 && argv[1][0] == '1';
  check_sizes();
  for (const Call &c : kCalls) check_call(c, no_device);

  // Tables.
  const Args a;
  for (auto f : {embed, embed_bwd}) {
    CHECK(f(Shape{16, 4, 40, 0}, a, kAll) == MHC_ERR_INVALID_ARG);
    CHECK(f(Shape{16, 4, 40, INT64_MIN}, a, kAll) == MHC_ERR_INVALID_ARG);
    CHECK(f(Shape{16, 4, 40, INT64_MAX}, a, kAll) == MHC_ERR_UNSUPPORTED);
    CHECK(f(Shape{1, 4, 1 << 12, 1 << 30}, a, kAll) == MHC_ERR_UNSUPPORTED);
  }
  // No rows: nothing needed, or the pointers of what is to be zeros.
  const Shape none{0, 4, 40, 100};
  Args null;
  for (auto &p : null.p) p = nullptr;
  for (const Call &c : kCalls) {
    const bool zeros = c.workspace(kGood) != 0;
    CHECK(c.run(none, null, 0) == (zeros ? MHC_ERR_INVALID_ARG : MHC_OK));
    if (zeros && no_device) CHECK(c.run(none, a, 0) == MHC_ERR_HIP);
  }
  CHECK(mhc_embed_bwd(0, 4, 40, 100, nullptr, nullptr, 1.0f, 1, a.f(2), nullptr, 0, nullptr) == MHC_OK);
  std::printf("%d checks passed\n", g_checks);
  return 0;
}
