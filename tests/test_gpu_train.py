"""The training calls on the GPU against the fp64 oracle: the 8-bit
checkpoint, the gradients of the apply and of the coefficients and pre-mix,
the embedding lookup and its gradient.

Tolerances (u = 2^-24, the fp32 rounding; bf16 rounds by at most 2^-8 of the
value; A = the sum of the absolute values of an output's terms):

  checkpoint      equal bits (x * 2^-e is exact, the rounding is E4M3's own)
  dF_out          2^-8 |value| + (n + 1) u A
  dH              (C + 8) u A: at most C adds in a row, each rounding once
  dX              2^-8 |value| + 2^-8 T + e, where e = (2N + n + 4) u A plus what an error of
                  dlogit adds (below) and T = e is the part of the value that e itself moves;
                  dlogit may be held in two bf16 parts, 2^-16 of each term
  dz, dlogit      gates: dH_pre's own sum (C + 8) u A, and 16 u of the value and of z (exp and
                  its argument).  The res block: each of the 40 normalisations rounds n + 3
                  times and later ones pass an error on by a bounded factor (their matrices
                  have rows and columns that sum to 1; 8 is allowed for), so
                  e_res = 320 (n + 3) u max|dH_res| of the row, and 16 u (1 + |z|) of it
  dphi            (rows + 8) u A + sum |X| e_dlogit, and 2^-22 A where dlogit is held in parts
  dalpha, db      sums of dz over the rows: rows u A + sum e_dz (times |logit / r|)
  X_0             2^-8 |value|, on the fp32 product
  dtable          (count n + 2) u A
"""

import sys

import numpy as np
import pytest
import torch

import manifold_constrained_hyper_amd as mhc
import oracle
import synth
from oracle import backward
from tests import eight_streams, train_replay

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
TINY = 1e-37


def _say(msg):
    print(f"[gpu-test] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    mhc.load()
    mhc.mhc_tuning_reset()
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A tensor between two bands of a known byte; check() says whether a call
    wrote outside it."""

    BAND = 4096

    def __init__(self, *shape, dtype=torch.float32, fill=0x7F):
        count = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        pad = (-count) % 16
        self.raw = torch.full((2 * self.BAND + count + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.lo, self.hi = self.BAND, self.BAND + count
        self.raw[self.lo:self.hi] = fill
        self.t = self.raw[self.lo:self.hi].view(dtype).view(*shape)

    def check(self):
        return bool((self.raw[:self.lo] == 0xA5).all()) and bool((self.raw[self.hi:] == 0xA5).all())


# -- checkpoint -------------------------------------------------------------------------------------

CKPT_SHAPES = [(1, 1, 8), (3, 2, 24), (5, 4, 32), (7, 4, 40), (2, 8, 264), (33, 1, 1000), (130, 2, 136), (64, 4, 256),
               (9, 8, 64)]


def _pack(x, n, C):
    B = x.shape[0]
    codes = Guarded(B, n * C, dtype=torch.uint8)
    scales = Guarded(B, mhc.mhc_ckpt_scales_per_row(n, C), dtype=torch.uint8)
    mhc.mhc_ckpt_pack(B, n, C, x, codes.t, scales.t)
    torch.cuda.synchronize()
    assert codes.check() and scales.check()
    return codes.t, scales.t


def _same_codes(got, want):
    """Equal codes; where the definition has NaN either NaN code will do."""
    got, want = got.cpu().numpy(), want
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("B,n,C", CKPT_SHAPES)
def test_ckpt_matches_oracle(B, n, C):
    _say(f"ckpt B={B} n={n} C={C}")
    gen = torch.Generator().manual_seed(B * 1000 + C)
    x = synth._draw_rows(gen, B, n * C, "student_t4", "cpu") * torch.exp2(torch.randint(-30, 30, (B, 1)).float())
    x = x.to(torch.bfloat16).cuda()
    codes, scales = _pack(x, n, C)
    want_c, want_s = backward.ckpt_encode(f64(x), n, C)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    _same_codes(codes, want_c)
    back = Guarded(B, n * C, dtype=torch.bfloat16)
    mhc.mhc_ckpt_unpack(B, n, C, codes, scales, back.t)
    torch.cuda.synchronize()
    assert back.check()
    assert np.array_equal(f64(back.t), backward.ckpt_decode(want_c, want_s, n, C))


def test_ckpt_borders():
    """Blocks of zeros, of the smallest and largest numbers, with amax at and
    next to 448 * 2^k, with Inf and NaN among finite values and alone, and
    every bf16 mantissa at several exponents (all E4M3 roundings and ties)."""
    n, C = 1, 32
    rows = [torch.zeros(C), -torch.zeros(C)]
    for top in (448.0, 450.0, 446.0, 1.75, 1.7578125, 2.0 ** -126, 2.0 ** -133, 2.0 ** -120, 3.3895e38, 2.0 ** 127):
        r = torch.linspace(-1, 1, C) * top
        r[5] = top
        rows.append(r)
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 5, C)
        r[7] = bad
        rows.append(r)
        rows.append(torch.full((C,), bad))
    mant = torch.arange(128).float() / 128 + 1
    for e in range(-12, 9):
        for k in range(0, 128, C - 1):
            r = torch.zeros(C)
            part = mant[k:k + C - 1] * 2.0 ** e
            r[1:1 + len(part)] = part
            r[0] = 448.0
            rows.append(r)
            rows.append(-r)
    x = torch.stack(rows).to(torch.bfloat16).cuda()
    codes, scales = _pack(x, n, C)
    want_c, want_s = backward.ckpt_encode(f64(x), n, C)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    _same_codes(codes, want_c)
    assert torch.equal(torch.signbit(x[1]), codes[1].ge(128))      # the sign of zero stays
    back = torch.empty_like(x)
    mhc.mhc_ckpt_unpack(len(rows), n, C, codes, scales, back)
    got, want = f64(back), backward.ckpt_decode(codes.cpu().numpy(), scales.cpu().numpy(), n, C)
    assert np.array_equal(got, want, equal_nan=True)


def test_ckpt_every_code_and_scale():
    """Unpacking all 256 codes under every scale byte a checkpoint can have."""
    n, C = 1, 256
    s = torch.arange(1, 248, dtype=torch.uint8)
    codes = torch.arange(256, dtype=torch.uint8).repeat(len(s), 1).cuda()
    scales = s[:, None].repeat(1, 8).contiguous().cuda()
    back = torch.empty(len(s), C, dtype=torch.bfloat16, device="cuda")
    mhc.mhc_ckpt_unpack(len(s), n, C, codes, scales, back)
    want = torch.from_numpy(backward.ckpt_decode(codes.cpu().numpy(), scales.cpu().numpy(), n, C)).to(torch.bfloat16)
    got = back.cpu()
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


# -- the layer's gradients --------------------------------------------------------------------------

SHAPES = [(1, 1, 8), (1, 4, 8), (2, 2, 40), (5, 4, 72), (17, 8, 64), (16, 4, 256), (65, 4, 520), (33, 8, 136),
          (130, 2, 1000), (300, 1, 264), (70, 4, 1032), (257, 2, 64), (515, 4, 32), (40, 8, 1024), (1100, 4, 64)]


def _inputs(B, n, C, seed, alpha=0.7, scale=1.0):
    inp = synth.make_inputs(n, C, B, "student_t4", seed=seed, device="cuda")
    inp["X"] = (inp["X"].float() * scale).to(torch.bfloat16)
    inp["alphas"] = (alpha, -0.6 * alpha, 1.3 * alpha)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    inp["G"] = (torch.randn(B, n * C, generator=gen, device="cuda") / 64).to(torch.bfloat16)
    inp["dF_pre"] = (torch.randn(B, C, generator=gen, device="cuda") / 64).to(torch.bfloat16)
    N = n * n + 2 * n
    logits, r, H = (torch.empty(B, N, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, N, device="cuda"))
    ws = torch.empty(max(16, mhc.mhc_coeffs_workspace_size(B, n, C)), dtype=torch.uint8, device="cuda")
    mhc.mhc_coeffs(B, n, C, inp["X"], inp["phi"], *inp["alphas"], inp["b_pre"], inp["b_post"], inp["b_res"], logits, r,
                   H, ws)
    inp.update(logits=logits, r=r, H=H)
    return inp


def _held(inp, x, n, C):
    """The tensors a call takes for X_t, and the values they stand for."""
    if x == "bf16":
        return (inp["X"],), f64(inp["X"])
    codes, scales = _pack(inp["X"], n, C)
    return (codes, scales), backward.ckpt_decode(codes.cpu().numpy(), scales.cpu().numpy(), n, C)


def _post_res_bwd(inp, held, B, n, C):
    N = n * n + 2 * n
    dF, dH = Guarded(B, C, dtype=torch.bfloat16), Guarded(B, N)
    call = mhc.mhc_post_res_bwd if len(held) == 1 else mhc.mhc_post_res_bwd_ckpt
    call(B, n, C, *held, inp["F_out"], inp["H"], inp["G"], dF.t, dH.t)
    torch.cuda.synchronize()
    assert dF.check() and dH.check()
    return dF.t, dH.t


def _coeffs_pre_bwd(inp, held, dH, B, n, C, stream=None, keep=None):
    N = n * n + 2 * n
    out = {"dX": Guarded(B, n * C, dtype=torch.bfloat16), "dphi": Guarded(n * C, N), "dalpha": Guarded(3),
           "db_pre": Guarded(n), "db_post": Guarded(n), "db_res": Guarded(n * n)}
    ws = Guarded(mhc.mhc_coeffs_pre_bwd_workspace_size(B, n, C), dtype=torch.uint8, fill=0xFF)  # NaN everywhere
    call = mhc.mhc_coeffs_pre_bwd if len(held) == 1 else mhc.mhc_coeffs_pre_bwd_ckpt
    torch.cuda.synchronize()
    call(B, n, C, *held, inp["phi"], *inp["alphas"], inp["b_pre"], inp["b_post"], inp["b_res"], inp["logits"],
         inp["r"], inp["H"], inp["G"], dH, inp["dF_pre"], *(o.t for o in out.values()), ws.t, stream=stream)
    if keep is not None:      # not waited for: the caller holds the workspace until it is done
        keep.append(ws)
    else:
        torch.cuda.synchronize()
        for k, o in out.items():
            assert o.check(), k
        assert ws.check()
    return {k: o.t for k, o in out.items()}


def _near(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    off = np.abs(got - want) - tol
    assert np.all(off <= 0), f"{what}: {np.sum(~(off <= 0))} of {off.size} beyond the tolerance, worst by {np.nanmax(off)}"


def _check_post_res(inp, held, xv, B, n, C):
    dF, dH = _post_res_bwd(inp, held, B, n, C)
    g, f, H = f64(inp["G"]), f64(inp["F_out"]), f64(inp["H"])
    want_F, want_H = backward.post_res_bwd(xv, f, H, g, n, C)
    abs_F, abs_H = backward.post_res_bwd(np.abs(xv), np.abs(f), np.abs(H), np.abs(g), n, C)
    _near(dF, want_F, HALF_BF16 * np.abs(want_F) + (n + 1) * U * abs_F * (1 + HALF_BF16) + TINY, "dF_out")
    _near(dH, want_H, (C + 8) * U * abs_H + TINY, "dH")
    assert not dH[:, :n].any()
    return dH


def _check_coeffs_pre(inp, held, xv, dH, B, n, C, got=None):
    got = _coeffs_pre_bwd(inp, held, dH, B, n, C) if got is None else got
    N = n * n + 2 * n
    phi, lg, r, H = (f64(inp[k]) for k in ("phi", "logits", "r", "H"))
    g, dF, up = f64(inp["G"]), f64(inp["dF_pre"]), f64(dH)
    bias = [f64(inp[k]) for k in ("b_pre", "b_post", "b_res")]
    want = backward.coeffs_pre_bwd(xv, phi, inp["alphas"], bias, lg, r, H, g, up, dF, n, C)
    # errors of dz and dlogit
    alpha = np.abs(np.concatenate([np.full(n, inp["alphas"][0]), np.full(n, inp["alphas"][1]),
                                   np.full(n * n, inp["alphas"][2])]))
    x3 = xv.reshape(B, n, C)
    a_pre = np.stack([np.sum(np.abs(x3[:, i] * dF), axis=1) for i in range(n)], 1)
    z = alpha * np.abs(lg) / r[:, None] + np.abs(np.concatenate(bias))
    e_dz = 16 * U * (1 + z) * np.abs(want["dz"])
    e_dz[:, :n] += (C + 8) * U * a_pre
    most = np.max(np.abs(up[:, 2 * n:]), axis=1, keepdims=True)
    if n > 1:
        e_dz[:, 2 * n:] += (320 * (n + 3) + 16 * (1 + np.max(z, axis=1, keepdims=True))) * U * most
    e_dl = alpha * e_dz / r[:, None] + 4 * U * np.abs(want["dlogits"])
    # dX
    terms = backward.coeffs_pre_bwd(np.abs(xv), np.abs(phi), np.abs(inp["alphas"]), bias, np.abs(lg), r, np.abs(H),
                                    np.abs(g), np.zeros_like(up), np.abs(dF), n, C)  # apply and pre-mix parts
    a_mix = np.zeros((B, n, C))
    for j in range(n):
        a_mix[:, j] = np.abs(H[:, j:j + 1] * dF)
        for i in range(n):
            a_mix[:, j] += np.abs(H[:, 2 * n + i * n + j, None] * g.reshape(B, n, C)[:, i])
    del terms
    a_phi = (np.abs(want["dlogits"]) @ np.abs(phi).T).reshape(B, n, C)
    e_phi = (e_dl @ np.abs(phi).T).reshape(B, n, C) + 2.0 ** -16 * a_phi
    a_turn = np.sum(np.abs(want["dlogits"] * lg), axis=1) / (n * C * r * r)
    e_turn = np.sum(e_dl * np.abs(lg), axis=1) / (n * C * r * r) + (N + 8) * U * a_turn
    e = ((2 * N + n + 4) * U * (a_mix + a_phi + a_turn[:, None, None] * np.abs(x3)) + e_phi
         + e_turn[:, None, None] * np.abs(x3)).reshape(B, -1)
    _near(got["dX"], want["dX"], HALF_BF16 * np.abs(want["dX"]) + e * (1 + HALF_BF16) + TINY, "dX")
    a = np.abs(xv).T
    _near(got["dphi"], want["dphi"], ((B + 8) * U + 2.0 ** -22) * (a @ np.abs(want["dlogits"])) + a @ e_dl + TINY, "dphi")
    e_db = np.sum(e_dz, axis=0) + (B + 8) * U * np.sum(np.abs(want["dz"]), axis=0) + TINY
    for k, sl in (("db_pre", slice(0, n)), ("db_post", slice(n, 2 * n)), ("db_res", slice(2 * n, N))):
        _near(got[k], want[k], e_db[sl], k)
    ratio = np.abs(lg) / r[:, None]
    e_a = np.sum(e_dz * ratio, axis=0) + (B + 8) * U * np.sum(np.abs(want["dz"]) * ratio, axis=0)
    _near(got["dalpha"], want["dalpha"], np.array([e_a[:n].sum(), e_a[n:2 * n].sum(), e_a[2 * n:].sum()]) + TINY, "dalpha")
    return got


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,C", SHAPES)
def test_layer_gradients_match_oracle(B, n, C, x):
    _say(f"layer gradients B={B} n={n} C={C} x={x}")
    inp = _inputs(B, n, C, seed=B + 7 * C + n)
    held, xv = _held(inp, x, n, C)
    dH = _check_post_res(inp, held, xv, B, n, C)
    _check_coeffs_pre(inp, held, xv, dH, B, n, C)


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,C", [(30, 4, 512), (16, 4, 1024), (34, 4, 1032), (250, 4, 40), (64, 2, 512), (31, 2, 1024),
                                   (200, 2, 264), (61, 1, 1024), (259, 1, 512), (118, 1, 2048), (30, 8, 2056),
                                   (55, 8, 1160)])
def test_layer_gradients_of_few_rows(B, n, C, x):
    """Both sides of the choices by size: row dot products in the coefficient
    kernel or before it, dphi from one range of rows or from several."""
    _say(f"layer gradients of few rows B={B} n={n} C={C} x={x}")
    inp = _inputs(B, n, C, seed=B + 7 * C + n)
    held, xv = _held(inp, x, n, C)
    _check_coeffs_pre(inp, held, xv, _check_post_res(inp, held, xv, B, n, C), B, n, C)


def test_one_stream_has_no_res_gradient():
    """n = 1: H_res is 1 exactly, so its bias gets exactly nothing."""
    inp = _inputs(50, 1, 64, seed=3)
    held, xv = _held(inp, "bf16", 1, 64)
    _, dH = _post_res_bwd(inp, held, 50, 1, 64)
    got = _coeffs_pre_bwd(inp, held, dH, 50, 1, 64)
    assert got["db_res"].item() == 0.0 and got["dalpha"][2].item() == 0.0


@pytest.mark.parametrize("n", [1, 2, 4, 8])
def test_sums_that_cancel(n):
    """db_post, and up to n = 4 db_res, are sums over the rows of 64-bit terms of
    fp32 inputs, whatever they cancel to: off by the one rounding of the
    result, 2^-24 of it, and 2^-40 of their terms (64-bit arithmetic, 2^-53
    each, through a few hundred operations)."""
    B, C = 333, 40
    inp = _inputs(B, n, C, seed=51 + n)
    gen = torch.Generator(device="cuda").manual_seed(n)
    dH = torch.randn(B, n * n + 2 * n, generator=gen, device="cuda")
    got = _coeffs_pre_bwd(inp, (inp["X"],), dH, B, n, C)
    want = backward.coeffs_pre_bwd(f64(inp["X"]), f64(inp["phi"]), [float(np.float32(a)) for a in inp["alphas"]],
                                   [f64(inp[k]) for k in ("b_pre", "b_post", "b_res")], f64(inp["logits"]),
                                   f64(inp["r"]), f64(inp["H"]), f64(inp["G"]), f64(dH), f64(inp["dF_pre"]), n, C)
    for k, sl in (("db_post", slice(n, 2 * n)),) + ((("db_res", slice(2 * n, None)),) if n in (2, 4) else ()):
        terms = np.sum(np.abs(f64(dH)[:, sl]), axis=0)
        _near(got[k], want[k], U * np.abs(want[k]) + 2.0 ** -40 * terms, k)


@pytest.mark.parametrize("alpha,scale", [(0.01, 1.0), (6.0, 1.0), (0.5, 2.0 ** -40), (0.5, 2.0 ** 30)])
def test_ranges(alpha, scale):
    """The training start's alpha, gates far into saturation and a matrix far
    from balanced, and streams of very small and very large values."""
    B, n, C = 70, 4, 104
    inp = _inputs(B, n, C, seed=11, alpha=alpha, scale=scale)
    for x in ("bf16", "e4m3"):
        held, xv = _held(inp, x, n, C)
        dH = _check_post_res(inp, held, xv, B, n, C)
        _check_coeffs_pre(inp, held, xv, dH, B, n, C)


def test_a_row_without_a_scale_stays_alone():
    """X_t = 0 in a row: r = 0, no gradient there (NaN), and dX of the other
    rows as without it."""
    B, n, C = 37, 4, 72
    inp = _inputs(B, n, C, seed=21)
    held, _ = _held(inp, "bf16", n, C)
    _, dH = _post_res_bwd(inp, held, B, n, C)
    want = _coeffs_pre_bwd(inp, held, dH, B, n, C)["dX"].clone()
    inp["X"][17] = 0
    inp["r"][17] = 0
    inp["logits"][17] = 0
    got = _coeffs_pre_bwd(inp, (inp["X"],), dH, B, n, C)["dX"]
    assert torch.isnan(got[17]).all()
    keep = torch.arange(B, device="cuda") != 17
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
def test_nan_in_the_stream_stays_in_its_row(x):
    """Inf and NaN in X_t of one row: NaN comes out there, nothing elsewhere
    (dphi sums over rows, so its row of that channel is NaN)."""
    B, n, C = 21, 2, 72
    inp = _inputs(B, n, C, seed=22)
    inp["X"][5, 3] = float("nan")
    inp["X"][5, 100] = float("inf")
    held, _ = _held(inp, x, n, C)
    _, dH = _post_res_bwd(inp, held, B, n, C)
    assert torch.isnan(dH[5]).any() and torch.isfinite(dH[torch.arange(B) != 5]).all()
    got = _coeffs_pre_bwd(inp, held, dH.nan_to_num(nan=1.0, posinf=1.0, neginf=1.0), B, n, C)
    assert torch.isnan(got["dX"][5]).any() and torch.isfinite(got["dX"][torch.arange(B) != 5]).all()
    assert torch.isnan(got["dphi"][3]).any()


@pytest.mark.parametrize("B,n,C", [(515, 4, 520), (70, 8, 136), (2100, 2, 64)])
def test_same_bits_twice(B, n, C):
    inp = _inputs(B, n, C, seed=31)
    for x in ("bf16", "e4m3"):
        held, _ = _held(inp, x, n, C)
        a, b = (_post_res_bwd(inp, held, B, n, C) for _ in range(2))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        a, b = (_coeffs_pre_bwd(inp, held, a[1], B, n, C) for _ in range(2))
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_no_rows_gives_zero_gradients():
    n, C = 4, 40
    N = n * n + 2 * n
    out = [Guarded(n * C, N), Guarded(3), Guarded(n), Guarded(n), Guarded(n * n)]
    e = torch.empty(0, device="cuda")
    for held in ((e,), (e, e)):
        call = mhc.mhc_coeffs_pre_bwd if len(held) == 1 else mhc.mhc_coeffs_pre_bwd_ckpt
        for o in out:
            o.t.fill_(3.0)
        call(0, n, C, *held, e, 0.1, 0.1, 0.1, e, e, e, e, e, e, e, e, e, e, *(o.t for o in out), None)
        torch.cuda.synchronize()
        assert all(o.check() and not o.t.any() for o in out)
    table = Guarded(10, C)
    mhc.mhc_embed_bwd(0, n, C, 10, e, e, 1.0, table.t, None)
    torch.cuda.synchronize()
    assert table.check() and not table.t.any()
    table.t.fill_(3.0)
    mhc.mhc_embed_bwd(0, n, C, 10, e, e, 1.0, table.t, None, accumulate=True)
    torch.cuda.synchronize()
    assert table.check() and bool((table.t == 3.0).all())


# -- embeddings -------------------------------------------------------------------------------------

EMBED_SHAPES = [(1, 1, 8, 1), (1, 4, 40, 7), (3, 2, 64, 5), (50, 4, 1000, 11), (300, 8, 24, 1000), (700, 2, 264, 3),
                (1030, 1, 72, 50), (2500, 4, 32, 400), (64, 4, 4104, 9)]


def _tokens(B, V, seed, how):
    gen = torch.Generator().manual_seed(seed)
    if how == "one":
        return torch.full((B,), V // 2, dtype=torch.int64, device="cuda")
    if how == "sorted":
        return torch.sort(torch.randint(0, V, (B,), generator=gen)).values.cuda()
    t = torch.randint(-1 if how == "padded" else 0, V + (2 if how == "padded" else 0), (B,), generator=gen)
    if how == "padded":
        t[t == V] = 2 ** 40 + 1      # an id whose low 32 bits are inside the table
    return t.cuda()


@pytest.mark.parametrize("how", ["any", "padded", "one", "sorted"])
@pytest.mark.parametrize("B,n,C,V", EMBED_SHAPES)
def test_embedding_matches_oracle(B, n, C, V, how):
    _say(f"embedding B={B} n={n} C={C} V={V} {how}")
    gen = torch.Generator(device="cuda").manual_seed(B + V)
    tokens = _tokens(B, V, B + C, how)
    table = torch.randn(V, C, generator=gen, device="cuda").to(torch.bfloat16)
    scale = 5.3
    X = Guarded(B, n * C, dtype=torch.bfloat16)
    mhc.mhc_embed(B, n, C, V, tokens, table, scale, X.t)
    torch.cuda.synchronize()
    assert X.check()
    s = float(np.float32(scale))
    want = backward.embed(tokens.tolist(), f64(table), s, n)
    _near(X.t, want, (HALF_BF16 + 2 * U) * np.abs(want), "X_0")

    G = torch.randn(B, n * C, generator=gen, device="cuda").to(torch.bfloat16)
    ws = Guarded(mhc.mhc_embed_bwd_workspace_size(B, n, C, V), dtype=torch.uint8, fill=0xFF)
    d = Guarded(V, C)
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, scale, d.t, ws.t)
    torch.cuda.synchronize()
    assert d.check() and ws.check()
    want = backward.embed_bwd(tokens.tolist(), f64(G), s, n, C, V)
    total = backward.embed_bwd(tokens.tolist(), np.abs(f64(G)), s, n, C, V)
    count = np.bincount([t for t in tokens.tolist() if 0 <= t < V], minlength=V)[:, None]
    _near(d.t, want, (count * n + 2) * U * total, "dtable")
    assert not d.t[torch.from_numpy(count[:, 0] == 0).cuda()].any()

    again = torch.full((V, C), 2.0, device="cuda")
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, scale, again, ws.t, accumulate=True)
    torch.cuda.synchronize()
    _near(again, want + 2, (count * n + 3) * U * (total + 2), "dtable, added to")
    assert bool((again[torch.from_numpy(count[:, 0] == 0).cuda()] == 2.0).all())
    twice = torch.empty_like(d.t)
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, scale, twice, ws.t)
    assert torch.equal(twice, d.t)


@pytest.mark.parametrize("how", ["any", "padded", "one"])
@pytest.mark.parametrize("B,n,C,V", [(17001, 2, 4104, 900), (40000, 1, 8, 70000), (16384, 1, 520, 2), (2048, 2, 16, 300), (6001, 1, 16, 900)])
def test_embedding_gradient_of_many_rows(B, n, C, V, how):
    """More rows than one joining pass sorts, long blocks, and tokens whose
    rows span hundreds of blocks (64-bit sums by torch)."""
    _say(f"embedding gradient B={B} n={n} C={C} V={V} {how}")
    gen = torch.Generator(device="cuda").manual_seed(B)
    tokens = _tokens(B, V, B + C, how)
    G = torch.randn(B, n * C, generator=gen, device="cuda").to(torch.bfloat16)
    ws = Guarded(mhc.mhc_embed_bwd_workspace_size(B, n, C, V), dtype=torch.uint8, fill=0xFF)
    d = Guarded(V, C)
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, 0.25, d.t, ws.t)
    torch.cuda.synchronize()
    assert d.check() and ws.check()
    fine = (tokens >= 0) & (tokens < V)
    g = G[fine].double().view(-1, n, C)
    want = torch.zeros(V, C, dtype=torch.float64, device="cuda").index_add_(0, tokens[fine], 0.25 * g.sum(1))
    total = torch.zeros_like(want).index_add_(0, tokens[fine], 0.25 * g.abs().sum(1))
    count = torch.bincount(tokens[fine], minlength=V)[:, None]
    assert bool(((d.t.double() - want).abs() <= (count * n + 2) * U * total).all())


@pytest.mark.parametrize("B,n,C,V", [(5, 2, 8, 70001), (700, 1, 56, 4999), (9, 1, 2056, 333), (3, 4, 8192, 7)])
def test_embedding_gradient_of_few_rows(B, n, C, V):
    """Most of the table has no token: narrow rows, of which a workgroup writes
    many zeros, and wide ones, the last of them at the table's end.  Every
    element is B n values of either sign, a product and B n + 1 roundings."""
    _say(f"embedding gradient of few rows B={B} n={n} C={C} V={V}")
    gen = torch.Generator(device="cuda").manual_seed(V)
    tokens = torch.randint(0, V, (B,), generator=gen, device="cuda")
    tokens[0], tokens[B // 2] = V - 1, 0
    G = torch.randn(B, n * C, generator=gen, device="cuda").to(torch.bfloat16)
    ws = Guarded(mhc.mhc_embed_bwd_workspace_size(B, n, C, V), dtype=torch.uint8, fill=0xFF)
    d = Guarded(V, C)
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, 0.75, d.t, ws.t)
    torch.cuda.synchronize()
    assert d.check() and ws.check()
    g = G.double().view(B, n, C)
    want = torch.zeros(V, C, dtype=torch.float64, device="cuda").index_add_(0, tokens, 0.75 * g.sum(1))
    total = torch.zeros_like(want).index_add_(0, tokens, 0.75 * g.abs().sum(1))
    assert bool(((d.t.double() - want).abs() <= (B * n + 2) * U * total).all())


def test_offsets_past_32_bits():
    """A stream of more than 2^32 values and a table of more than 2^31: the last
    rows come out as they do in a call of their own."""
    B, n, C, last = 66000, 8, 8192, 2048
    _say(f"offsets past 32 bits B={B} n={n} C={C}")
    N, e = n * n + 2 * n, lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")
    b = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(3)
    X, G = (e(B, n * C, d=b).normal_(generator=gen) for _ in range(2))
    F, dFp = (e(B, C, d=b).normal_(generator=gen) for _ in range(2))
    phi = (torch.randn(n * C, N, generator=gen, device="cuda") / 256).to(b)
    logits, H = torch.randn(B, N, generator=gen, device="cuda"), torch.rand(B, N, generator=gen, device="cuda")
    r = torch.rand(B, generator=gen, device="cuda") + 0.5
    bias = [torch.randn(k, generator=gen, device="cuda") for k in (n, n, n * n)]

    def calls(lo, hi):
        m, s = hi - lo, slice(lo, hi)
        codes, scales = e(m, n * C, d=torch.uint8), e(m, mhc.mhc_ckpt_scales_per_row(n, C), d=torch.uint8)
        mhc.mhc_ckpt_pack(m, n, C, X[s], codes, scales)
        dF, dH, dX = e(m, C, d=b), e(m, N), e(m, n * C, d=b)
        mhc.mhc_post_res_bwd_ckpt(m, n, C, codes, scales, F[s], H[s], G[s], dF, dH)
        ws = e(mhc.mhc_coeffs_pre_bwd_workspace_size(m, n, C), d=torch.uint8)
        grads = [e(n * C, N), e(3), e(n), e(n), e(n * n)]
        mhc.mhc_coeffs_pre_bwd_ckpt(m, n, C, codes, scales, phi, 0.5, 0.5, 0.5, *bias, logits[s], r[s], H[s], G[s], dH,
                                    dFp[s], dX, *grads, ws)
        assert all(bool(torch.isfinite(g).all()) for g in grads)
        back = e(last, n * C, d=b)
        mhc.mhc_ckpt_unpack(last, n, C, codes[m - last:], scales[m - last:], back)
        return [t[m - last:].clone() for t in (codes, scales, dF, dH, dX)] + [back]

    for whole, own in zip(calls(0, B), calls(B - last, B)):
        assert torch.equal(whole, own)

    del X
    V = 2 ** 31 // C + 1000
    table = e(V, C, d=b).normal_(generator=gen)
    tokens = torch.randint(0, V, (B,), generator=gen, device="cuda")
    tokens[-last:] = torch.randperm(last, generator=gen, device="cuda") + V - last
    tokens[:-last] %= V - last
    X_0 = e(B, n * C, d=b)
    mhc.mhc_embed(B, n, C, V, tokens, table, 2.0, X_0)
    assert torch.equal(X_0[-last:].view(last, n, C), (2 * table[tokens[-last:]])[:, None].expand(last, n, C))
    ws = e(mhc.mhc_embed_bwd_workspace_size(B, n, C, V), d=torch.uint8)
    dtable = e(V, C)
    mhc.mhc_embed_bwd(B, n, C, V, tokens, G, 2.0, dtable, ws)
    g = G[-last:].view(last, n, C).double()
    want, total = 2 * g.sum(1), 2 * g.abs().sum(1)
    assert bool(((dtable[tokens[-last:]].double() - want).abs() <= (n + 2) * U * total).all())


# -- a training step --------------------------------------------------------------------------------

class Model:
    """Token embeddings, L mHC layers whose layer F is F_out = F_pre * w (w one
    weight a channel, held by torch), and the sum of the streams at the end:
    a training step's calls in their order."""

    def __init__(self, B, n, C, V, L, ckpt, seed=0):
        self.B, self.n, self.C, self.V, self.L, self.ckpt = B, n, C, V, L, ckpt
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.N = n * n + 2 * n
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.tokens = torch.randint(0, V, (B,), generator=gen, device="cuda")
        self.table = rand(V, C).to(torch.bfloat16)
        self.scale = 1.5
        self.alphas = (0.3, 0.2, 0.4)
        self.layers = [{"phi": (rand(n * C, self.N) / (n * C) ** 0.5).to(torch.bfloat16), "b_pre": 0.1 * rand(n),
                        "b_post": 0.1 * rand(n),
                        "b_res": (2 * torch.eye(n, device="cuda").reshape(-1) + 0.1 * rand(n * n)).contiguous(),
                        "w": rand(C).to(torch.bfloat16)} for _ in range(L)]
        self.out = (rand(B, C) / 64).to(torch.bfloat16)      # gradient of the summed streams
        e = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        b = torch.bfloat16
        self.X = [e(B, n * C, d=b) for _ in range(L + 1)]
        self.co = [{"logits": e(B, self.N), "r": e(B), "H": e(B, self.N), "F_pre": e(B, C, d=b)} for _ in range(L)]
        self.F = [e(B, C, d=b) for _ in range(L)]
        self.kept = [(e(B, n * C, d=torch.uint8), e(B, mhc.mhc_ckpt_scales_per_row(n, C), d=torch.uint8))
                     for _ in range(L)]
        size = max(mhc.mhc_coeffs_pre_workspace_size(B, n, C), mhc.mhc_post_res_coeffs_pre_workspace_size(B, n, C),
                   mhc.mhc_coeffs_pre_bwd_workspace_size(B, n, C), mhc.mhc_embed_bwd_workspace_size(B, n, C, V), 16)
        self.ws = e(size, d=torch.uint8)
        self.G = [e(B, n * C, d=b) for _ in range(L + 1)]
        self.dF, self.dFp, self.dH = e(B, C, d=b), e(B, C, d=b), e(B, self.N)
        self.grads = [{"dphi": e(n * C, self.N), "dalpha": e(3), "db_pre": e(n), "db_post": e(n), "db_res": e(n * n)}
                      for _ in range(L)]
        self.dtable = e(V, C)

    def _next(self, l):
        p, c = self.layers[l], self.co[l]
        return (p["phi"], *self.alphas, p["b_pre"], p["b_post"], p["b_res"], c["logits"], c["r"], c["H"], c["F_pre"],
                self.ws)

    def step(self):
        B, n, C = self.B, self.n, self.C
        mhc.mhc_embed(B, n, C, self.V, self.tokens, self.table, self.scale, self.X[0])
        mhc.mhc_coeffs_pre(B, n, C, self.X[0], *self._next(0))
        for l in range(self.L):
            if self.ckpt:
                mhc.mhc_ckpt_pack(B, n, C, self.X[l], *self.kept[l])
            torch.mul(self.co[l]["F_pre"], self.layers[l]["w"], out=self.F[l])
            if l + 1 < self.L:
                mhc.mhc_post_res_coeffs_pre(B, n, C, self.X[l], self.F[l], self.co[l]["H"], self.X[l + 1],
                                            *self._next(l + 1))
            else:
                mhc.mhc_post_res(B, n, C, self.X[l], self.F[l], self.co[l]["H"], self.X[l + 1])
        self.G[self.L].view(B, n, C).copy_(self.out[:, None])
        for l in reversed(range(self.L)):
            p, c, g = self.layers[l], self.co[l], self.grads[l]
            rest = (p["phi"], *self.alphas, p["b_pre"], p["b_post"], p["b_res"], c["logits"], c["r"], c["H"],
                    self.G[l + 1], self.dH, self.dFp, self.G[l], g["dphi"], g["dalpha"], g["db_pre"], g["db_post"],
                    g["db_res"], self.ws)
            post = (self.F[l], c["H"], self.G[l + 1], self.dF, self.dH)
            if self.ckpt:
                mhc.mhc_post_res_bwd_ckpt(B, n, C, *self.kept[l], *post)
            else:
                mhc.mhc_post_res_bwd(B, n, C, self.X[l], *post)
            torch.mul(self.dF, p["w"], out=self.dFp)
            if self.ckpt:
                mhc.mhc_coeffs_pre_bwd_ckpt(B, n, C, *self.kept[l], *rest)
            else:
                mhc.mhc_coeffs_pre_bwd(B, n, C, self.X[l], *rest)
        mhc.mhc_embed_bwd(B, n, C, self.V, self.tokens, self.G[0], self.scale, self.dtable, self.ws)

    def results(self):
        return {"dtable": self.dtable, **{f"{k}{l}": v for l, g in enumerate(self.grads) for k, v in g.items()}}

    def by_autograd(self):
        """The same gradients by torch.autograd in 64 bits, on the CPU."""
        B, n, C, N = self.B, self.n, self.C, self.N
        d = lambda t: t.detach().double().cpu()  # noqa: E731
        table = d(self.table).requires_grad_()
        params = [{k: d(v).requires_grad_(k != "w") for k, v in p.items()} for p in self.layers]
        alphas = [torch.tensor(self.alphas, dtype=torch.float64).requires_grad_() for _ in range(self.L)]
        x = (self.scale * table[self.tokens.cpu()])[:, None].expand(B, n, C)
        for p, a in zip(params, alphas):
            lg = x.reshape(B, n * C) @ p["phi"]
            r = x.square().mean((1, 2)).sqrt()[:, None]
            pre, post, res = (a[k] * v / r + p[b] for k, (v, b) in enumerate(zip(
                lg.split([n, n, n * n], 1), ("b_pre", "b_post", "b_res"))))
            m = res.reshape(B, n, n).exp()
            for _ in range(20):
                m = m / m.sum(2, keepdim=True)
                m = m / m.sum(1, keepdim=True)
            f = (torch.sigmoid(pre)[:, :, None] * x).sum(1) * p["w"]
            x = m @ x + 2 * torch.sigmoid(post)[:, :, None] * f[:, None]
        (x.sum(1) * d(self.out)).sum().backward()
        got = {"dtable": table.grad}
        for l, (p, a) in enumerate(zip(params, alphas)):
            got.update({f"dphi{l}": p["phi"].grad, f"dalpha{l}": a.grad, f"db_pre{l}": p["b_pre"].grad,
                        f"db_post{l}": p["b_post"].grad, f"db_res{l}": p["b_res"].grad})
        return got


@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,C,V,L", [(300, 4, 256, 50, 2), (37, 2, 96, 20, 3), (64, 8, 64, 30, 2)])
def test_training_step(B, n, C, V, L, ckpt):
    """A whole step against autograd in 64 bits.  Every stored stream and
    gradient is rounded to bf16 (2^-8 of it at most, 2^-9 and less on average,
    independent from value to value) in up to 6 places a layer, and a
    checkpoint moves X_t by up to 2^-4 of a value, 2^-5 on average: by 2-norm
    at most 6 L 2^-8, and with a checkpoint 2^-4 more for what X_t is a factor
    of.  Sums over rows that nearly cancel are measured against the norm of
    the parameter's whole gradient, which these two bounds are shares of; the
    gates' own small vectors (n values) get four times as much.

    db_res can be next to 0 against its terms, and 320 (n + 3) u max|dH_res| a
    row (see the top of this file) is then what its rounding leaves, so that is
    allowed for beside its share.  Last layer: the streams are summed, so
    dH_res[i,j] = <out, X_j> is the same d_j for every i, and the last
    normalisation, over columns that sum to 1, passes on
    d_j - d_j sum_i m[i,j] = 0.  First layer: the streams are equal, so
    dH_res[i,j] = <G_i, X> is the same for every j, and rows sum to 1 as far as
    the iteration has converged.  |dH_res[i,j]| <= (1 + 2^-4) sum |G_i| |X_j|."""
    _say(f"training step B={B} n={n} C={C} V={V} L={L} ckpt={ckpt}")
    m = Model(B, n, C, V, L, ckpt, seed=B)
    m.step()
    torch.cuda.synchronize()
    want = m.by_autograd()
    bound = 6 * L * 2.0 ** -8 + (2.0 ** -4 if ckpt else 0.0)
    for k, v in m.results().items():
        w = want[k].reshape(v.shape)
        if k.startswith("db_res"):
            l = int(k[6:])
            x, g = (s.double().view(B, n, C).abs() for s in (m.X[l], m.G[l + 1]))
            most = (g @ x.transpose(1, 2).contiguous()).amax((1, 2)).sum().item()
            off = float((v.double().cpu() - w).norm())
            assert off <= 4 * bound * float(w.norm()) + n * 320 * (n + 3) * U * (1 + 2.0 ** -4) * most, k
            continue
        rel = float((v.double().cpu() - w).norm() / w.norm())
        _say(f"  {k}: {rel:.2e}")
        assert rel <= (bound if k.startswith(("dtable", "dphi")) else 4 * bound), k


@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "e4m3"])
def test_training_step_from_a_graph(ckpt):
    """A captured step, replayed with eager steps and spoiled outputs in
    between, gives the eager step's bits each time."""
    m = Model(300, 4, 160, 50, 2, ckpt, seed=5)
    m.step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in m.results().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    for k in range(4):
        for v in m.results().values():
            v.fill_(float("nan"))
        m.ws.fill_(0xA5 if k % 2 else 0xFF)
        for t in m.G:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for name, v in m.results().items():
            assert torch.equal(v, want[name]), (k, name)
        m.step()                      # eager work between the replays
        torch.cuda.synchronize()
        for name, v in m.results().items():
            assert torch.equal(v, want[name]), (k, name)


def test_two_streams_at_once():
    """Two calls on two streams with a workspace each: the results of one
    after the other."""
    B, n, C = 520, 4, 512
    a, b = _inputs(B, n, C, seed=41), _inputs(B, n, C, seed=42)
    work = []
    for inp in (a, b):
        held, _ = _held(inp, "e4m3", n, C)
        _, dH = _post_res_bwd(inp, held, B, n, C)
        work.append((inp, held, dH, _coeffs_pre_bwd(inp, held, dH, B, n, C)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        keep = []
        got = [_coeffs_pre_bwd(inp, held, dH, B, n, C, stream=s, keep=keep)
               for (inp, held, dH, _), s in zip(work, streams)]
        torch.cuda.synchronize()
        for (_, _, _, want), g in zip(work, got):
            assert all(torch.equal(want[k], g[k]) for k in want)


# -- eight streams ----------------------------------------------------------------------------------

def _eight_streams_call(logits, r, b, dH, seed):
    """The coefficient gradients of rows with these logits (alpha_res = 1)."""
    B, n, C = len(r), 8, 8
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    inp = {"X": rand(B, n * C).to(torch.bfloat16), "phi": rand(n * C, n * n + 2 * n).to(torch.bfloat16),
           "alphas": (0.3, 0.2, 1.0), "b_pre": rand(n), "b_post": rand(n), "b_res": dev(b), "logits": dev(logits),
           "r": dev(r), "H": torch.rand(B, n * n + 2 * n, generator=gen, device="cuda"),
           "G": rand(B, n * C).to(torch.bfloat16), "dF_pre": rand(B, C).to(torch.bfloat16)}
    return inp, _coeffs_pre_bwd(inp, (inp["X"],), dev(dH), B, n, C)


@pytest.mark.parametrize("diag,spread", eight_streams.SPREADS)
def test_eight_streams_row_by_row(diag, spread):
    """One row's db_res is its dz: within the bound of tests/eight_streams.py,
    which a missing iteration exceeds."""
    logits, r, b, dH, z = eight_streams.inputs(diag, spread, 12, seed=5)
    want, bound = eight_streams.exact(z, dH[:, 16:]), eight_streams.row_bound(z, dH[:, 16:])
    for k in range(len(r)):
        _say(f"eight streams diag={diag} spread={spread} row {k}")
        _, got = _eight_streams_call(logits[k:k + 1], r[k:k + 1], b, dH[k:k + 1], seed=k)
        off = np.abs(f64(got["db_res"]).reshape(8, 8) - want[k]).max()
        _say(f"  {off / (U * np.abs(dH[k, 16:]).max()):.2f} u max|dH_res|")
        assert off <= bound[k]


@pytest.mark.parametrize("diag,spread", eight_streams.SPREADS)
def test_eight_streams_sums_over_rows(diag, spread):
    """Rows' errors are independent and have no side, so what they add up to
    is compared with six times the root of their squared bounds; the sums
    themselves are 64-bit (db_res, dalpha), or as at the top of this file
    (dphi)."""
    B, n, C = 333, 8, 8
    _say(f"eight streams sums diag={diag} spread={spread}")
    logits, r, b, dH, z = eight_streams.inputs(diag, spread, B, seed=6)
    inp, got = _eight_streams_call(logits, r, b, dH, seed=7)
    want = eight_streams.exact(z, dH[:, 16:]).reshape(B, 64)
    bound, lg, r64 = eight_streams.row_bound(z, dH[:, 16:]), logits[:, 16:].astype(np.float64), r.astype(np.float64)
    db = want.sum(0)
    _say(f"  off by {np.max(np.abs(f64(got['db_res']) - db) / np.abs(want).sum(0)):.1e} of the terms")
    _near(got["db_res"], db, 6 * np.sqrt(np.sum(bound ** 2)) + U * np.abs(db), "db_res")
    ratio = lg / r64[:, None]
    da = np.sum(want * ratio)
    _near(got["dalpha"][2:], np.array([da]),
          np.array([6 * np.sqrt(np.sum((bound * np.abs(ratio).sum(1)) ** 2)) + U * abs(da)]), "dalpha")
    x, dl = f64(inp["X"]), want / r64[:, None]
    terms = np.abs(x).T @ np.abs(dl)
    _near(got["dphi"][:, 16:].contiguous(), x.T @ dl,
          6 * np.sqrt((x ** 2).T @ ((bound / r64)[:, None] ** 2)) + ((B + 8) * U + 2.0 ** -22) * terms, "dphi")


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,C", [(767, 4, 2056), (768, 4, 2056), (768, 8, 2056), (3, 4, 7176), (2, 8, 8200), (5, 1, 9000)])
def test_apply_gradients_by_waves_a_row(B, n, C, x):
    """Both sides of the choice of waves a row, and rows of as many as there are."""
    _say(f"apply gradients B={B} n={n} C={C} x={x}")
    gen = torch.Generator(device="cuda").manual_seed(B + C)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    inp = {"X": rand(B, n * C).to(torch.bfloat16), "F_out": rand(B, C).to(torch.bfloat16),
           "H": rand(B, n * n + 2 * n), "G": rand(B, n * C).to(torch.bfloat16)}
    held, xv = _held(inp, x, n, C)
    _check_post_res(inp, held, xv, B, n, C)


# Many tiles a range of rows and several slices of channels, and a launch of
# each other number of streams.
@pytest.mark.parametrize("B,n,C", [(4096, 4, 2048), (3000, 1, 1032), (5000, 2, 520), (2100, 8, 264)])
def test_same_bits_of_many_tiles(B, n, C):
    _say(f"same bits B={B} n={n} C={C}")
    inp = _inputs(B, n, C, seed=32)
    for x in ("bf16", "e4m3"):
        held = (inp["X"],) if x == "bf16" else _pack(inp["X"], n, C)
        dH = _post_res_bwd(inp, held, B, n, C)[1]
        want = _coeffs_pre_bwd(inp, held, dH, B, n, C)
        for _ in range(4):
            assert torch.equal(_post_res_bwd(inp, held, B, n, C)[1], dH)
            got = _coeffs_pre_bwd(inp, held, dH, B, n, C)
            assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("alpha,scale", [(0.01, 1.0), (6.0, 1.0), (0.5, 2.0 ** -40), (0.5, 2.0 ** 30)])
def test_ranges_of_eight_streams(alpha, scale):
    B, n, C = 70, 8, 104
    inp = _inputs(B, n, C, seed=12, alpha=alpha, scale=scale)
    for x in ("bf16", "e4m3"):
        held, xv = _held(inp, x, n, C)
        dH = _check_post_res(inp, held, xv, B, n, C)
        _check_coeffs_pre(inp, held, xv, dH, B, n, C)


# -- a training step, closely -----------------------------------------------------------------------

@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,C,V", [(300, 4, 256, 50), (37, 2, 96, 20), (64, 8, 64, 30)])
def test_training_step_against_its_replay(B, n, C, V, ckpt):
    """Four layers whose streams differ, against the same step in 64 bits with
    the same values rounded (tests/train_replay.py), so that what is left is
    the calls' own arithmetic and the few stored values that it moves across
    a rounding border.

    Bounds, from replays whose values were moved by 2e-6 of themselves before
    each rounding (32-bit sums and the forward's exponentials move them by some
    2^-24 = 6e-8, a thirtieth, and the number of values that cross a border,
    whose root is the distance, goes down with it): the table's gradient moved
    by 1.1e-3 of its norm and dphi by 4.2e-3, 2^-9 and 2^-8 are allowed; the
    small vectors, which are sums over rows that cancel, by 9.3e-4 of `noise`
    (db_res: 1e-5, most of dH_res cancels), 2^-11 and 2^-17 are, and 2^-9 of
    their norm.  A gradient of half its size fails in each of these but db_res
    of the first and the last layer, which are next to 0 (see
    test_training_step)."""
    _say(f"training step and replay B={B} n={n} C={C} V={V} ckpt={ckpt}")
    L = 4
    m = Model(B, n, C, V, L, ckpt, seed=B + 1)
    gen = torch.Generator(device="cuda").manual_seed(B)
    for p in m.layers:
        p["b_pre"].mul_(10)
        p["b_post"].mul_(10)
        p["b_res"].add_(0.5 * torch.randn(n * n, generator=gen, device="cuda"))
    m.step()
    torch.cuda.synchronize()
    want, noise = train_replay.step(
        {"tokens": m.tokens.tolist(), "table": f64(m.table), "scale": m.scale, "out": f64(m.out),
         "alphas": [float(np.float32(a)) for a in m.alphas],
         "layers": [{k: f64(v) for k, v in p.items()} for p in m.layers]}, B, n, C, ckpt)
    for k, v in m.results().items():
        w = want[k]
        norm, off = np.linalg.norm(w), np.linalg.norm(f64(v).reshape(w.shape) - w)
        if k.startswith(("dtable", "dphi")):
            bound = (2.0 ** -9 if k == "dtable" else 2.0 ** -8) * norm
        else:
            size = np.sqrt(w.size) * noise[int(k[-1])]
            bound = 2.0 ** -9 * norm + (2.0 ** -17 if k.startswith("db_res") else 2.0 ** -11) * size
            if not (k.startswith("db_res") and k[-1] in "03"):
                assert norm / 2 > bound, k
        _say(f"  {k}: off by {off / norm:.1e} of the norm, {off / bound:.2f} of the bound")
        assert off <= bound, k
