// Host-only check of libmhc's calls around a layer of experts, built like
// train_host_check.cpp with AddressSanitizer and UndefinedBehaviorSanitizer on
// the host code (no check here launches a kernel where a device is visible).
//
// Drives the argument checks of these entry points in include/mhc.h with fake
// device addresses (never dereferenced on the host), their size functions and
// workspace plans over ordinary and extreme shapes, and -- on a host with no
// HIP device -- calls that pass the checks, which must report MHC_ERR_HIP.
// Exits non-zero on the first failed check; the sanitizers abort on any error
// they find.
#include "mhc.h"
#include "mhc_experts.h"

#include <cmath>
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
  int64_t B, C;
  int32_t k, E;
};
constexpr Shape kGood{16, 40, 4, 12};

// Every tensor of a call, as fake, 16-byte aligned addresses far apart.
constexpr int kMost = 10;
struct Args {
  char *p[kMost];
  Args() {
    for (int k = 0; k < kMost; ++k) p[k] = reinterpret_cast<char *>(uintptr_t(1) << 44 | (uintptr_t)(k + 1) << 40);
  }
  float *f(int k) const { return reinterpret_cast<float *>(p[k]); }
  uint8_t *b(int k) const { return reinterpret_cast<uint8_t *>(p[k]); }
  int32_t *i(int k) const { return reinterpret_cast<int32_t *>(p[k]); }
};

constexpr size_t kAll = ~size_t(0);  // "the size the call asks for"

// One entry point: its tensors, which of them are outputs and which may be
// left out (bit k), their alignments, which sizes it takes, and the call.
struct Call {
  const char *name;
  int tensors;
  uint32_t outputs, optional;
  const uint8_t *align;
  bool C, k, E;
  int (*run)(const Shape &, const Args &, size_t ws);
  size_t (*workspace)(const Shape &);  // null where there is none
};

size_t norm_ws(const Shape &s) { return mhc_rmsnorm_bwd_workspace_size(s.B, s.C); }
size_t order_ws(const Shape &s) { return mhc_experts_order_workspace_size(s.B, s.k, s.E); }

int norm(const Shape &s, const Args &a, size_t) {
  return mhc_rmsnorm(s.B, s.C, a.p[0], a.p[1], a.f(2), 1e-5f, a.p[3], a.p[4], a.p[5], a.b(6), a.f(7), nullptr);
}
int norm_bwd(const Shape &s, const Args &a, size_t ws) {
  return mhc_rmsnorm_bwd(s.B, s.C, a.p[0], a.f(1), a.f(2), a.p[3], a.p[4], a.p[5], a.f(6), a.p[7],
                         ws == kAll ? norm_ws(s) : ws, nullptr);
}
int route(const Shape &s, const Args &a, size_t) {
  return mhc_route(s.B, s.E, s.k, 1, 1, MHC_ROUTE_RENORM, 1.0f, a.p[0], a.f(1), a.i(2), a.f(3), nullptr);
}
int route_bwd(const Shape &s, const Args &a, size_t) {
  return mhc_route_bwd(s.B, s.E, s.k, MHC_ROUTE_SOFTMAX, 1.0f, a.p[0], a.i(1), a.f(2), a.p[3], nullptr);
}
int order(const Shape &s, const Args &a, size_t ws) {
  return mhc_experts_order(s.B, s.k, s.E, a.i(0), a.i(1), a.i(2), a.p[3], ws == kAll ? order_ws(s) : ws, nullptr);
}
int gather(const Shape &s, const Args &a, size_t) {
  return mhc_experts_gather(s.B, s.k, s.C, a.p[0], a.i(1), a.p[2], nullptr);
}
int gather_ckpt(const Shape &s, const Args &a, size_t) {
  return mhc_experts_gather_ckpt(s.B, s.k, s.C, a.p[0], a.b(1), a.i(2), a.p[3], a.b(4), nullptr);
}
int combine(const Shape &s, const Args &a, size_t) {
  return mhc_experts_combine(s.B, s.k, s.C, a.p[0], a.i(1), a.f(2), a.p[3], a.p[4], nullptr);
}
int combine_bwd(const Shape &s, const Args &a, size_t) {
  return mhc_experts_combine_bwd(s.B, s.k, s.C, a.p[0], a.i(1), a.f(2), a.p[3], a.p[4], a.f(5), nullptr);
}

const uint8_t kNorm[] = {16, 16, 16, 16, 16, 16, 1, 4}, kNormBwd[] = {16, 16, 4, 16, 16, 16, 16, 16},
              kRoute[] = {4, 4, 4, 4}, kRouteBwd[] = {4, 4, 4, 4}, kOrder[] = {4, 4, 4, 16}, kGather[] = {16, 4, 16},
              kGatherCkpt[] = {16, 1, 4, 16, 1}, kCombine[] = {16, 4, 4, 16, 16},
              kCombineBwd[] = {16, 4, 4, 16, 16, 4};
const Call kCalls[] = {
    // (of sum, y, codes and scales what is left out decides what the others may be)
    {"mhc_rmsnorm", 8, 0b11111000, 0b11111110, kNorm, true, false, false, norm, nullptr},
    {"mhc_rmsnorm_bwd", 8, 0b11100000, 0b11010010, kNormBwd, true, false, false, norm_bwd, norm_ws},
    {"mhc_route", 4, 0b1100, 0b0010, kRoute, false, true, true, route, nullptr},
    {"mhc_route_bwd", 4, 0b1000, 0, kRouteBwd, false, true, true, route_bwd, nullptr},
    {"mhc_experts_order", 4, 0b1110, 0, kOrder, false, true, true, order, order_ws},
    {"mhc_experts_gather", 3, 0b100, 0, kGather, true, true, false, gather, nullptr},
    {"mhc_experts_gather_ckpt", 5, 0b11000, 0, kGatherCkpt, true, true, false, gather_ckpt, nullptr},
    {"mhc_experts_combine", 5, 0b10000, 0b01100, kCombine, true, true, false, combine, nullptr},
    {"mhc_experts_combine_bwd", 6, 0b110000, 0, kCombineBwd, true, true, false, combine_bwd, nullptr},
};

void check_call(const Call &c, bool no_device) {
  std::printf("%s\n", c.name);
  const Args ok;
  const auto shaped = [&](Shape s) { return c.run(s, ok, kAll); };
  for (int64_t B : {int64_t(-1), INT64_MIN}) CHECK(shaped({B, 40, 4, 12}) == MHC_ERR_INVALID_ARG);
  for (int64_t B : {int64_t(1) << 31, INT64_MAX}) CHECK(shaped({B, 40, 4, 12}) == MHC_ERR_UNSUPPORTED);
  if (c.C) {
    for (int64_t C : {int64_t(0), int64_t(-8), INT64_MIN}) CHECK(shaped({16, C, 4, 12}) == MHC_ERR_INVALID_ARG);
    for (int64_t C : {int64_t(12), int64_t(1) << 40, INT64_MAX - 7}) CHECK(shaped({16, C, 4, 12}) == MHC_ERR_UNSUPPORTED);
    CHECK(shaped({int64_t(1) << 28, int64_t(1) << 16, 4, 12}) == MHC_ERR_UNSUPPORTED);
  }
  if (c.k) {
    for (int32_t k : {0, -1, INT32_MIN}) CHECK(shaped({16, 40, k, 1000}) == MHC_ERR_INVALID_ARG);
    CHECK(shaped({16, 40, 33, 1000}) == MHC_ERR_UNSUPPORTED);
    CHECK(shaped({16, 40, INT32_MAX, INT32_MAX}) == MHC_ERR_UNSUPPORTED);
  }
  if (c.E) {
    for (int32_t E : {0, -1, INT32_MIN}) CHECK(shaped({16, 40, 4, E}) == MHC_ERR_INVALID_ARG);
    for (int32_t E : {1025, INT32_MAX}) CHECK(shaped({16, 40, 4, E}) == MHC_ERR_UNSUPPORTED);
  }
  for (int k = 0; k < c.tensors; ++k) {
    Args a;
    if (!(c.optional >> k & 1)) {
      a.p[k] = nullptr;
      CHECK(c.run(kGood, a, kAll) == MHC_ERR_INVALID_ARG);
    }
    if (c.align[k] > 1) {
      a.p[k] = ok.p[k] + c.align[k] / 2;
      CHECK(c.run(kGood, a, kAll) == MHC_ERR_UNSUPPORTED);
    }
    if (!(c.outputs >> k & 1)) continue;
    for (int q = 0; q < c.tensors; ++q) {  // an output over each other tensor
      if (q == k) continue;
      a.p[k] = ok.p[q];
      CHECK(c.run(kGood, a, kAll) == MHC_ERR_INVALID_ARG);
    }
  }
  if (c.workspace) {
    CHECK(c.run(kGood, ok, c.workspace(kGood) - 1) == MHC_ERR_WORKSPACE);
    CHECK(c.run(kGood, ok, 0) == MHC_ERR_WORKSPACE);
  }
  if (!no_device) return;
  for (int64_t B : {int64_t(1), int64_t(17), int64_t(513), int64_t(4096), int64_t(20000), int64_t(1) << 25})
    for (int64_t C : {int64_t(8), int64_t(264), int64_t(1000), int64_t(7168), int64_t(65536)})
      for (int32_t E : {1, 7, 64, 256, 300, 1000, 1024})
        for (int32_t k : {1, 2, 9, 32})
          if (k <= E && B * k * C <= int64_t(1) << 36) CHECK(c.run(Shape{B, C, k, E}, ok, kAll) == MHC_ERR_HIP);
}

// Plans and sizes over the whole accepted range.
void check_sizes() {
  const int64_t Bs[] = {0,       1,          15,        256,           1000, 4097, 16384, 1 << 20, (int64_t(1) << 31) - 1,
                        int64_t(1) << 31, INT64_MAX, -1,  INT64_MIN};
  const int64_t Cs[] = {8, 24, 1000, 7168, 8200, 16384, 65536, 65544, int64_t(1) << 40, INT64_MAX - 7, 0, -8, 12};
  const int32_t ks[] = {1, 2, 8, 32, 33, 0, -1, INT32_MAX, INT32_MIN}, Es[] = {1, 7, 256, 1024, 1025, 0, -1, INT32_MAX};
  for (int64_t B : Bs) {
    for (int64_t C : Cs) {
      const bool rows = B > 0 && B < (int64_t(1) << 31) && C > 0 && C % 8 == 0 && C <= 65536 &&
                        B <= (int64_t(1) << 40) / C;
      const size_t ws = mhc_rmsnorm_bwd_workspace_size(B, C);
      CHECK((ws > 0) == rows);
      if (!rows) continue;
      const mhc::NormBwdPlan p = mhc::plan_rmsnorm_bwd(B, C);
      CHECK(p.total_bytes == ws && p.parts >= 1 && p.parts <= B && p.parts <= 2048);
      CHECK(ws == (size_t)p.parts * (size_t)C * 4);
    }
    for (int32_t k : ks)
      for (int32_t E : Es) {
        const bool pairs = B > 0 && B < (int64_t(1) << 31) && k > 0 && k <= 32 && B * k < (int64_t(1) << 31) && E > 0 &&
                           E <= 1024;
        const size_t ws = mhc_experts_order_workspace_size(B, k, E);
        CHECK((ws > 0) == pairs);
        if (!pairs) continue;
        const mhc::OrderPlan p = mhc::plan_experts_order(B * k, E);
        CHECK(p.total_bytes == ws && p.tiles >= 1 && p.tiles <= 256 && p.tile % 1024 == 0);
        CHECK(p.tile * p.tiles >= B * k && p.tile * (p.tiles - 1) < B * k);
        CHECK(ws == (size_t)p.tiles * (size_t)E * 4);
      }
  }
}

}  // namespace

int main(int argc, char **argv) {
  const bool no_device = argc > 1 && argv[1][0] == '1';
  check_sizes();
  for (const Call &c : kCalls) check_call(c, no_device);

  const Args a;
  const auto groups = [&](int32_t E, int32_t k, int32_t n, int32_t top, int32_t flags) {
    return mhc_route(16, E, k, n, top, flags, 1.0f, a.p[0], nullptr, a.i(2), a.f(3), nullptr);
  };
  for (int32_t n : {0, -1, INT32_MIN, 5, 24, INT32_MAX}) CHECK(groups(12, 4, n, 1, 0) == MHC_ERR_INVALID_ARG);
  for (int32_t t : {0, -1, INT32_MIN, 4, INT32_MAX}) CHECK(groups(12, 4, 3, t, 0) == MHC_ERR_INVALID_ARG);
  CHECK(groups(12, 5, 3, 1, 0) == MHC_ERR_INVALID_ARG);
  CHECK(groups(12, 13, 1, 1, 0) == MHC_ERR_INVALID_ARG);
  CHECK(groups(1024, 4, 128, 128, 0) == MHC_ERR_UNSUPPORTED);
  for (int32_t f : {8, -1, INT32_MIN, INT32_MAX}) CHECK(groups(12, 4, 3, 2, f) == MHC_ERR_INVALID_ARG);
  for (float eps : {-1.0f, -0x1p-149f, NAN, INFINITY})
    CHECK(mhc_rmsnorm(16, 40, a.p[0], nullptr, nullptr, eps, nullptr, a.p[1], nullptr, nullptr, nullptr, nullptr) ==
          MHC_ERR_INVALID_ARG);

  // No rows: nothing needed, or the pointer of what is to be zeros.
  const Shape none{0, 40, 4, 12};
  Args null;
  for (auto &p : null.p) p = nullptr;
  for (const Call &c : kCalls) {
    CHECK(c.run(none, null, 0) == (c.run == order ? MHC_ERR_INVALID_ARG : MHC_OK));
    if ((c.run == order || c.run == norm_bwd) && no_device) CHECK(c.run(none, a, 0) == MHC_ERR_HIP);
  }
  std::printf("%d checks passed\n", g_checks);
  return 0;
}
