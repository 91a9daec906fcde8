"""The calls around a layer of experts on the GPU against the fp64 oracle: the
root-mean-square norm and its gradients, the choice of experts and its
gradient, the rows into the experts' order and back.

Tolerances (u = 2^-24, the fp32 rounding; bf16 rounds by at most 2^-8 of the
value, E4M3 by 2^-4 or, below its smallest normal number, by 2^-10 of the
scale; A = the sum of the absolute values of an output's terms):

  sum        2^-8 |value| on the fp32 sum: (2^-8 + u) |value|
  rstd       a lane adds at most 8 * 8 squares (exact products) in a row, then 6 + 16 joins: 86 roundings of
             the sum of positive terms, halved by the root, and 5 of the division, 1 / C, eps, the root:
             50 u of the value
  y          2^-8 |y| + 54 u |y|
  codes      2^-4 |y| + 2^-10 scale + 54 u |y|; the scale is the least one for amax within 54 u of it
  dx         e = rstd (|n| (96 u A / C) + 8 u (|g| + |n mean|)) + u |dx|; 2^-8 (|dx| + e) + e
  dweight    (rows + 40) u A: at most one add a row, and the joins
  weights    (32 + |x - top|) u of the value: the exponent's argument rounds by u |x - top|, the sum of E <= 1024
             terms adds 16 + 6 times, and exp, log1p, division and scale take the rest
  dlogits    (48 + |x - top|) u (|value| + its cancelled part), and the type's rounding
  slots, offsets, ids and rows: equal
  F_out      2^-8 |value| + (k + 2) u A (1 + 2^-8)
  dY         2^-8 |value| + 2 u |value|
  dweights   (C + 8) u A
"""

import sys

import numpy as np
import pytest
import torch

import manifold_constrained_hyper_amd as mhc
from oracle import backward, experts

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
TINY = 1e-37
BF = torch.bfloat16


def _say(msg):
    print(f"[gpu-test] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    mhc.load()
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


def _checked(*guards):
    torch.cuda.synchronize()
    for g in guards:
        assert g is None or g.check()


def _normal(gen, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()


def _near(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want)
    bad = ~(off <= tol + TINY)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(off - tol)} at {np.argwhere(bad)[:3]}"


# -- norm -------------------------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (1, 7168), (3, 24), (5, 40), (64, 512), (33, 520), (130, 1000), (7, 2048), (9, 2056), (2, 4104),
               (17, 8192), (3, 8200), (2, 16384), (2, 32776), (1, 65536), (700, 72), (2100, 264),
               (4100, 200), (4096, 1040), (4097, 2056)]


def _rmsnorm(x, weight, shortcut, eps=1e-5, y=True, codes=True):
    B, C = x.shape
    out = {"sum": Guarded(B, C, dtype=BF) if shortcut is not None else None,
           "y": Guarded(B, C, dtype=BF) if y else None,
           "codes": Guarded(B, C, dtype=torch.uint8) if codes else None,
           "scales": Guarded(B, -(-C // 32), dtype=torch.uint8) if codes else None, "rstd": Guarded(B)}
    mhc.mhc_rmsnorm(B, C, x, weight, shortcut=shortcut, eps=eps, **{k: v and v.t for k, v in out.items()})
    _checked(*out.values())
    return {k: v and v.t for k, v in out.items()}


def _check_codes(codes, scales, y, extra=54 * U):
    """codes and scales hold y (float64 [B, C]): values within E4M3's rounding, scales the least that do."""
    B, C = y.shape
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy().reshape(B, -1)
    got = backward.ckpt_decode(codes, scales, 1, C)
    step = np.repeat(np.exp2(scales - 127.0), 32, axis=1)[:, :C]
    _near(got, y, (2.0 ** -4 + extra) * np.abs(y) + 2.0 ** -10 * step, "codes")
    for k in range(scales.shape[1]):
        amax = np.max(np.abs(y[:, 32 * k:32 * k + 32]), axis=1)
        s = np.exp2(scales[:, k] - 127.0)
        assert np.all(amax <= 448 * s * (1 + extra))
        assert np.all((scales[:, k] == 1) | (amax > 224 * s * (1 - extra)))


@pytest.mark.parametrize("B,C", NORM_SHAPES)
def test_rmsnorm(B, C):
    _say(f"rmsnorm B={B} C={C}")
    gen = torch.Generator().manual_seed(B * 7 + C)
    x = (torch.randn(B, C, generator=gen) * torch.exp2(torch.randint(-12, 12, (B, 1), generator=gen))).to(BF).cuda()
    short, w = _normal(gen, B, C), 1 + _normal(gen, C, scale=0.3, dtype=torch.float32)
    for shortcut in (None, short):
        for weight in (None, w):
            o = _rmsnorm(x, weight, shortcut)
            s = f64(x)
            if shortcut is not None:
                want = s + f64(short)
                _near(o["sum"], want, (HALF_BF16 + U) * np.abs(want), "sum")
                s = f64(o["sum"])
            y, rstd = experts.rmsnorm(s, None if weight is None else f64(w))
            _near(o["rstd"], rstd, 50 * U * rstd, "rstd")
            _near(o["y"], y, (HALF_BF16 + 54 * U) * np.abs(y), "y")
            _check_codes(o["codes"], o["scales"], y)
            # What is asked for does not change what comes out.
            part = _rmsnorm(x, weight, shortcut, codes=False)
            assert torch.equal(part["y"], o["y"]) and torch.equal(part["rstd"], o["rstd"])
            part = _rmsnorm(x, weight, shortcut, y=False)
            assert torch.equal(part["codes"], o["codes"]) and torch.equal(part["scales"], o["scales"])


@pytest.mark.parametrize("B,C", [(8195, 7168), (1100, 7168), (4000, 2048), (3600, 2056), (8200, 1024), (900, 16392)])
def test_rmsnorm_many_values(B, C):
    """Sizes from which a thread takes several vectors of a row, and rows that end inside them."""
    _say(f"rmsnorm many values B={B} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(B + C)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, short, w = (normal(B, C) * torch.exp2(normal(B, 1))).to(BF), normal(B, C).to(BF), 1 + 0.3 * normal(C)
    for shortcut in (None, short):
        o = _rmsnorm(x, w, shortcut)
        s = x.double()
        if shortcut is not None:
            s = s + short.double()
            assert torch.all((o["sum"] - s).abs() <= (HALF_BF16 + U) * s.abs())
            s = o["sum"].double()
        rstd = 1 / (s.square().mean(1) + 1e-5).sqrt()
        assert torch.all((o["rstd"] - rstd).abs() <= 50 * U * rstd)
        y = s.mul_(rstd[:, None]).mul_(w.double())
        assert torch.all((o["y"] - y).abs() <= (HALF_BF16 + 54 * U) * y.abs())
        step = torch.exp2(o["scales"].double() - 127).repeat_interleave(32, 1)[:, :C]
        got = o["codes"].view(torch.float8_e4m3fn).double() * step
        assert torch.all((got - y).abs() <= (2.0 ** -4 + 54 * U) * y.abs() + 2.0 ** -10 * step)
        part = _rmsnorm(x, w, shortcut, codes=False)
        assert torch.equal(part["y"], o["y"]) and torch.equal(part["rstd"], o["rstd"])


def test_rmsnorm_without_extras():
    """sum and rstd left out."""
    gen = torch.Generator().manual_seed(5)
    x, short, w = _normal(gen, 9, 136), _normal(gen, 9, 136), _normal(gen, 136, dtype=torch.float32)
    want = _rmsnorm(x, w, short)["y"]
    y = Guarded(9, 136, dtype=BF)
    mhc.mhc_rmsnorm(9, 136, x, w, y=y.t, shortcut=short)
    _checked(y)
    assert torch.equal(y.t, want)


def test_rmsnorm_borders():
    """Rows of zeros, of one value, with Inf and NaN, of the smallest and the largest numbers."""
    C = 96
    ramp = torch.linspace(-3, 5, C)
    rows = [torch.zeros(C), torch.full((C,), 1e-3), ramp, ramp.clone(), ramp.clone(), ramp * 1e15, ramp * 1e-30,
            torch.full((C,), 3.3895e38)]
    rows[3][7], rows[4][40] = float("inf"), float("nan")
    x = torch.stack(rows).to(BF).cuda()
    w = torch.ones(C, device="cuda")
    w[0], w[33] = 1e30, 0.0
    o = _rmsnorm(x, w, None)
    y, s = f64(o["y"]), f64(x)
    assert np.all(y[0] == 0) and torch.all(o["codes"][0] == 0) and torch.all(o["scales"][0] == 1)
    for r in (1, 2, 5, 6):
        want, rstd = experts.rmsnorm(s[r:r + 1], f64(w))
        _near(y[r:r + 1], want, (HALF_BF16 + 54 * U) * np.abs(want), r)
        _check_codes(o["codes"][r:r + 1], o["scales"][r:r + 1], want)
    # An infinity makes the root infinite: the row is zeros but for it.
    assert np.isnan(y[3, 7]) and np.all(np.delete(y[3], 7) == 0)
    assert np.isnan(y[4]).all()
    codes = o["codes"].cpu().numpy()
    assert codes[3, 7] & 0x7F == 0x7F and np.all(codes[4] & 0x7F == 0x7F)
    assert np.all(y[7] == 0)                                # its squares pass fp32's range
    assert np.isnan(f64(_rmsnorm(torch.zeros(1, C, dtype=BF, device="cuda"), None, None, eps=0.0)["y"])).all()


# Both sides of the row and channel counts at which one launch does it, and several rows a workgroup.
@pytest.mark.parametrize("B,C", NORM_SHAPES + [
    (1, 64), (9, 64), (301, 136), (512, 4104), (513, 4104), (512, 520), (255, 16384), (256, 16384), (2048, 384),
    (2048, 392), (768, 1024), (3000, 8), (2500, 24), (4100, 32), (2049, 40), (2100, 64), (2051, 136), (2060, 256), (2100, 264),
    (2049, 512), (5000, 504)])
def test_rmsnorm_bwd(B, C):
    _say(f"rmsnorm_bwd B={B} C={C}")
    gen = torch.Generator().manual_seed(B * 11 + C)
    s = (torch.randn(B, C, generator=gen) * torch.exp2(torch.randint(-6, 6, (B, 1), generator=gen))).to(BF).cuda()
    dy, dsum = _normal(gen, B, C, scale=1 / 64), _normal(gen, B, C, scale=1 / 64)
    w = 1 + _normal(gen, C, scale=0.3, dtype=torch.float32)
    rstd = (s.float().square().mean(1) + 1e-5).rsqrt()
    for weight in (None, w):
        for more in (None, dsum):
            dx, dw = Guarded(B, C, dtype=BF), Guarded(C)
            ws = Guarded(mhc.mhc_rmsnorm_bwd_workspace_size(B, C), dtype=torch.uint8, fill=0xFF)
            mhc.mhc_rmsnorm_bwd(B, C, s, weight, rstd, dy, dx.t, dweight=dw.t, workspace=ws.t, dsum=more)
            _checked(dx, dw, ws)
            want, want_w = experts.rmsnorm_bwd(f64(s), None if weight is None else f64(w), f64(rstd), f64(dy),
                                               None if more is None else f64(dsum))
            n, g = f64(s) * f64(rstd)[:, None], f64(dy) * (1.0 if weight is None else f64(w))
            A = np.sum(np.abs(g * n), axis=1, keepdims=True)
            mean = np.mean(g * n, axis=1, keepdims=True)
            e = f64(rstd)[:, None] * (np.abs(n) * 96 * U * A / C + 8 * U * (np.abs(g) + np.abs(n * mean)))
            e += U * np.abs(want)
            _near(dx.t, want, HALF_BF16 * (np.abs(want) + e) + e, "dx")
            _near(dw.t, want_w, (B + 40) * U * np.sum(np.abs(f64(dy) * n), axis=0), "dweight")
            alone = Guarded(B, C, dtype=BF)
            mhc.mhc_rmsnorm_bwd(B, C, s, weight, rstd, dy, alone.t, dsum=more)
            _checked(alone)
            assert torch.equal(alone.t, dx.t)


def test_rmsnorm_bwd_no_rows():
    dw = torch.full((40,), 7.0, device="cuda")
    none = torch.empty(0, 40, dtype=BF, device="cuda")
    mhc.mhc_rmsnorm_bwd(0, 40, none, None, torch.empty(0, device="cuda"), none, none, dweight=dw)
    assert torch.all(dw == 0)


# -- choice of experts ------------------------------------------------------------------------------

ROUTES = [  # B, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (3, 2, 1, 2, 1), (1, 256, 8, 8, 4), (130, 256, 8, 8, 4), (65, 100, 6, 1, 1), (33, 60, 10, 6, 3),
    (7, 1024, 32, 64, 5), (5, 1000, 32, 1, 1), (40, 64, 6, 64, 9), (9, 96, 32, 3, 2), (2, 512, 1, 16, 16),
    (66, 21, 12, 3, 2), (300, 8, 2, 1, 1), (17, 65, 4, 13, 1), (12, 160, 6, 8, 3), (10, 34, 3, 17, 2)]


def _route(logits, k, bias=None, **how):
    B, E = logits.shape
    ids, weights = Guarded(B, k, dtype=torch.int32), Guarded(B, k)
    mhc.mhc_route(B, E, k, logits, ids.t, weights.t, bias=bias, **how)
    _checked(ids, weights)
    return ids.t, weights.t


def _check_route(logits, k, bias=None, **how):
    ids, weights = _route(logits, k, bias, **how)
    x = f64(logits)
    want, want_w = experts.route(x, k, None if bias is None else f64(bias), **how)
    assert np.array_equal(ids.cpu().numpy(), want)
    x = experts.clean(x)
    at = np.maximum(want, 0)
    with np.errstate(invalid="ignore"):
        far = np.abs(np.take_along_axis(x, at, 1) - np.max(x, axis=1, keepdims=True))
    far = np.where((want >= 0) & np.isfinite(far), np.minimum(far, 1e6), 0.0)
    _near(weights, want_w, (32 + far) * U * np.abs(want_w), "weights")
    return ids, weights


@pytest.mark.parametrize("B,E,k,groups,top_groups", ROUTES)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("softmax", [False, True])
def test_route(B, E, k, groups, top_groups, dtype, softmax):
    _say(f"route B={B} E={E} k={k} groups={groups} top={top_groups} {dtype} softmax={softmax}")
    gen = torch.Generator().manual_seed(E * 100 + k)
    logits = _normal(gen, B, E, scale=2.0, dtype=dtype)
    bias = _normal(gen, E, scale=0.1, dtype=torch.float32)
    for b in (None, bias):
        for renorm in (False, True):
            _check_route(logits, k, b, groups=groups, top_groups=top_groups, softmax=softmax, renorm=renorm,
                         scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masked(softmax, biased):
    """Rows with few, one and no experts left, NaN, both infinities, the types' lowest and largest values,
    equal logits, groups that are all masked."""
    E, k = 24, 5
    gen = torch.Generator().manual_seed(9)
    bias = _normal(gen, E, scale=0.1, dtype=torch.float32) if biased else None
    for dtype in (torch.float32, BF):
        x = torch.randn(16, E, generator=gen).to(dtype)
        low, inf = torch.finfo(dtype).min, float("inf")
        x[1, 3:] = -inf
        x[2] = -inf
        x[2, 17] = 1.0
        x[3] = -inf
        x[4, 5] = float("nan")
        x[5] = float("nan")
        x[6, 2] = inf
        x[7, 4:9] = inf
        x[8] = low
        x[9, :12] = low
        x[10] = 0.0
        x[11] = -low
        x[12, 8:] = -inf
        x[13] = -120.0 + x[13]
        x[14] = 60.0 + x[14]
        x[15] = -0.0
        for renorm in (False, True):
            for groups, top in ((1, 1), (6, 3), (3, 2), (24, 7)):
                ids, _ = _check_route(x.cuda(), k, bias, groups=groups, top_groups=top, softmax=softmax, renorm=renorm)
                assert torch.all(ids[3] == -1) and torch.all(ids[5] == -1)


def test_route_bias_masks():
    """A bias of minus infinity or NaN takes an expert out, one of plus infinity brings it to the front."""
    gen = torch.Generator().manual_seed(4)
    x = _normal(gen, 20, 32, dtype=torch.float32)
    bias = torch.zeros(32)
    bias[3], bias[4], bias[20] = -float("inf"), float("nan"), float("inf")
    for softmax in (False, True):
        ids, _ = _check_route(x, 6, bias.cuda(), softmax=softmax, groups=4, top_groups=3)
        assert torch.all(ids[:, 0] == 20) and not torch.any((ids == 3) | (ids == 4))


@pytest.mark.parametrize("softmax", [False, True])
def test_route_near_ties(softmax):
    """Choices that a bias brings within 2^-25 of each other, and logits one rounding apart: the order is that of
    64-bit arithmetic."""
    gen = torch.Generator().manual_seed(11)
    B, E, k = 64, 96, 12
    x = torch.randn(1, E, generator=gen).expand(B, E).clone()
    x += (torch.randint(-2, 3, (B, E), generator=gen) * 2.0 ** -23) * x.abs()      # every row a few roundings off
    score = torch.softmax(x[0].double(), 0) if softmax else torch.sigmoid(x[0].double())
    bias = (0.75 - score).float()
    x, bias = x.cuda(), bias.cuda()
    for groups, top in ((1, 1), (8, 4)):
        _check_route(x, k, bias, softmax=softmax, groups=groups, top_groups=top)
    close = torch.full((B, E), 1.0)
    close += torch.randint(-3, 4, (B, E), generator=gen) * 2.0 ** -23
    _check_route(close.cuda(), k, softmax=softmax)
    _check_route((close * 15).cuda(), k, softmax=softmax, groups=8, top_groups=4)   # sigmoids next to 1
    _check_route((close * -15).cuda(), k, softmax=softmax)


def _crowded(B, E, gen):
    """Rows whose experts are all within 2^-33 of each other in the choice, or where 64-bit scores end: sigmoids next
    to 1, logits next to 0, scores that fall out of the type, scores of very different sizes."""
    at = torch.stack([torch.randperm(E, generator=gen) for _ in range(B)]).double()
    off = torch.rand(B, E, generator=gen).double()   # (sums of two are not equal by chance)
    kind = torch.arange(B).reshape(-1, 1) % 5
    return torch.where(kind == 0, 25 + at * 0.05,
                       torch.where(kind == 1, (at + 0.3 * off) * 1e-11,
                                   torch.where(kind == 2, -660 - at,
                                               torch.where(kind == 3, -0.5 * at, 30 + 0.0 * at)))).float()


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (40, 96, 12, 1, 1), (40, 96, 12, 8, 4), (35, 13, 3, 1, 1), (25, 96, 5, 48, 11), (20, 100, 32, 10, 7),
    (2565, 96, 12, 1, 1), (2563, 96, 8, 8, 4), (2561, 16, 4, 4, 2), (2570, 420, 8, 1, 1), (2560, 112, 7, 1, 1)])
def test_route_crowded(B, E, k, groups, top_groups):
    """More choices than k + 2 that 42 bits cannot tell apart: the order is still that of 64-bit arithmetic."""
    _say(f"route crowded B={B} E={E} k={k} groups={groups} top={top_groups}")
    gen = torch.Generator().manual_seed(B + E + k)
    x = _crowded(B, E, gen)
    if B > 40:
        x[2:9] = _normal(gen, 7, E, dtype=torch.float32).cpu()      # ordinary rows in the same wave
    rows = np.arange(B) if B <= 40 else _some_rows(B)
    for softmax in (False, True):
        for b in (torch.zeros(E), torch.full((E,), 0.25)):
            if groups == 1:
                b[E // 2] = -float("inf")
            how = dict(groups=groups, top_groups=top_groups, softmax=softmax)
            ids, _ = _route(x.cuda(), k, b.cuda(), **how)
            want, _ = experts.route(f64(x)[rows], k, f64(b), **how)
            got = ids.cpu().numpy()[rows]
            assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def _some_rows(B):
    """Rows to check of many: the first and the last ones, and some between."""
    return np.unique(np.concatenate([np.arange(6), np.arange(B - 9, B), np.linspace(0, B - 1, 60).astype(int)]))


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (2600, 16, 4, 1, 1), (2561, 30, 5, 3, 2), (2560, 64, 6, 8, 3), (2603, 128, 8, 1, 1), (2562, 100, 14, 4, 2),
    (2600, 256, 8, 8, 4), (2563, 256, 12, 16, 5), (2565, 200, 10, 1, 1), (2560, 11, 3, 11, 7), (2600, 255, 9, 15, 14),
    (2570, 300, 6, 1, 1), (2570, 64, 15, 1, 1), (2561, 512, 8, 8, 4), (2562, 270, 20, 30, 20), (2561, 513, 3, 1, 1),
    (2561, 30, 18, 1, 1), (2563, 32, 4, 32, 6), (2560, 60, 16, 1, 1), (2565, 96, 17, 24, 19), (2562, 128, 15, 1, 1),
    (2561, 200, 12, 25, 9), (2563, 256, 30, 32, 9), (1025, 512, 8, 8, 4), (2048, 100, 6, 1, 1), (2049, 256, 8, 8, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_route_many_rows(B, E, k, groups, top_groups, dtype):
    """Rows enough for several to share a wave, masked ones among them, and rows whose choices are nearly equal."""
    _say(f"route many B={B} E={E} k={k} groups={groups} top={top_groups} {dtype}")
    gen = torch.Generator().manual_seed(B + E)
    x = torch.randn(B, E, generator=gen) * 2
    x[torch.rand(B, E, generator=gen) < 0.05] = -float("inf")
    x[1], x[5, 1:], x[B - 2] = -float("inf"), -float("inf"), 0.25
    x[3, ::3], x[4, ::2] = float("nan"), float("inf")
    x[7] = torch.finfo(dtype).min
    x[B - 9:B - 4] = x[B - 9] + torch.randint(-1, 2, (5, E), generator=gen) * 2.0 ** -22
    x = x.to(dtype)
    bias = _normal(gen, E, scale=0.1, dtype=torch.float32)
    near = (0.5 - torch.sigmoid(x[B - 9].double())).float().nan_to_num(0.0).cuda()
    rows = _some_rows(B)
    x = x.cuda()
    for softmax in (False, True):
        for b in (None, bias, near):
            how = dict(groups=groups, top_groups=top_groups, softmax=softmax, renorm=b is not near)
            ids, weights = _route(x, k, b, **how)
            want, want_w = experts.route(f64(x)[rows], k, None if b is None else f64(b), **how)
            assert np.array_equal(ids.cpu().numpy()[rows], want)
            z = experts.clean(f64(x)[rows])
            with np.errstate(invalid="ignore"):
                far = np.abs(np.take_along_axis(z, np.maximum(want, 0), 1) - np.max(z, axis=1, keepdims=True))
            far = np.where((want >= 0) & np.isfinite(far), np.minimum(far, 1e6), 0.0)
            _near(f64(weights)[rows], want_w, (32 + far) * U * np.abs(want_w), "weights")
            # Every row as when it is on its own.
            for r in (0, B // 2, B - 1):
                one = _route(x[r:r + 1], k, b, **how)
                assert torch.equal(one[0][0], ids[r])


@pytest.mark.parametrize("B,E,k", [(1, 1, 1), (3, 2, 2), (130, 256, 8), (65, 100, 6), (7, 1024, 32), (5, 1000, 31),
                                   (300, 8, 2), (17, 65, 4), (9, 63, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd(B, E, k, dtype, softmax, renorm):
    _say(f"route_bwd B={B} E={E} k={k} {dtype} softmax={softmax} renorm={renorm}")
    gen = torch.Generator().manual_seed(E * 10 + k)
    logits = _normal(gen, B, E, scale=2.0, dtype=dtype)
    if B > 2 and E > 2:
        logits[1, :E // 2] = -float("inf")
        logits[2] = torch.finfo(dtype).min
    ids = torch.argsort(torch.rand(B, E, generator=gen), 1)[:, :k].to(torch.int32)
    if B > 4 and k > 1:
        ids[3, 1] = ids[3, 0]                       # the same expert twice
        ids[4, k // 2:] = -1
        ids[0, 0], ids[0, k - 1] = E, -2 ** 31
    _check_route_bwd(logits, ids.cuda(), _normal(gen, B, k, dtype=torch.float32), softmax, renorm)


def _check_route_bwd(logits, ids, dw, softmax, renorm, scale=1.5):
    (B, E), k = logits.shape, ids.shape[1]
    out = Guarded(B, E, dtype=logits.dtype)
    mhc.mhc_route_bwd(B, E, k, logits, ids, dw, out.t, softmax=softmax, renorm=renorm, scale=scale)
    _checked(out)
    x, at = experts.clean(f64(logits)), ids.cpu().numpy()
    want = experts.route_bwd(x, at, f64(dw), softmax, renorm, scale)
    # Magnitudes of the two terms that may cancel, each with its weight's error.
    size = np.zeros_like(want)
    for b in range(B):
        w = experts.weights_of(x[b], list(at[b]), softmax, renorm, scale)
        all_w = np.sum(np.abs(w * f64(dw)[b]))
        here = np.zeros(E)
        for j, e in enumerate(at[b]):
            if 0 <= e < E:
                s = 1.0 if softmax else experts.sigmoid(-x[b, e])
                here[e] += s * abs(w[j]) * (abs(f64(dw)[b, j]) + (all_w / scale if renorm else 0.0))
        if softmax and not renorm:
            here += experts._softmax(x[b]) * all_w / 1.0
        size[b] = here
    top = np.max(x, axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(x), np.minimum(np.abs(x - top), 1e4), 0.0)
    half = HALF_BF16 if logits.dtype == BF else 0.0
    e = (48 + far) * U * size
    _near(out.t, want, half * (np.abs(want) + e) + e, "dlogits")
    return out.t


@pytest.mark.parametrize("B,E,k", [(4096, 5, 2), (4099, 64, 6), (4097, 100, 6), (4100, 255, 16), (4096, 256, 8),
                                   (4098, 33, 1), (4099, 301, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_route_bwd_many_rows(B, E, k, dtype):
    _say(f"route_bwd many B={B} E={E} k={k} {dtype}")
    gen = torch.Generator().manual_seed(E + k)
    logits = _normal(gen, B, E, scale=2.0, dtype=dtype)
    logits[B - 2, :E // 2] = -float("inf")
    ids = torch.argsort(torch.rand(B, E, generator=gen), 1)[:, :k].to(torch.int32)
    if k > 1:
        ids[3, 1] = ids[3, 0]
        ids[B - 1, k // 2:] = -1
    rows = _some_rows(B)
    ids, dw = ids.cuda(), _normal(gen, B, k, dtype=torch.float32)
    for softmax in (False, True):
        for renorm in (False, True):
            out = Guarded(B, E, dtype=dtype)
            mhc.mhc_route_bwd(B, E, k, logits, ids, dw, out.t, softmax=softmax, renorm=renorm, scale=1.5)
            _checked(out)
            few = _check_route_bwd(logits[rows], ids[rows], dw[rows], softmax, renorm)
            # The same rows in a short call: within the roundings of two routes.
            off = (out.t[rows].double() - few.double()).abs()
            assert torch.all(off <= (2 * HALF_BF16 if dtype == BF else 96 * U) * few.double().abs().amax(1, True) + TINY)


def test_route_bwd_one_weight():
    """A single renormalised weight is constant: its gradient is zero, exactly."""
    gen = torch.Generator().manual_seed(3)
    x, dw = _normal(gen, 50, 40, dtype=torch.float32), _normal(gen, 50, 1, dtype=torch.float32)
    for softmax in (False, True):
        out = torch.full_like(x, 7.0)
        mhc.mhc_route_bwd(50, 40, 1, x, torch.zeros(50, 1, dtype=torch.int32, device="cuda"), dw, out, softmax=softmax)
        assert torch.all(out == 0)


def test_route_bwd_differences():
    """The gradient against differences of the library's own weights."""
    gen = torch.Generator().manual_seed(21)
    B, E, k, h = 16, 48, 6, 2.0 ** -7
    x, dw = _normal(gen, B, E, dtype=torch.float32), _normal(gen, B, k, dtype=torch.float32)
    d = torch.randint(0, 2, (B, E), generator=gen).float().cuda() * 2 - 1
    for softmax in (False, True):
        for renorm in (False, True):
            ids, w = _route(x, k, softmax=softmax, renorm=renorm)
            out = torch.empty_like(x)
            mhc.mhc_route_bwd(B, E, k, x, ids, dw, out, softmax=softmax, renorm=renorm)
            # The bias holds the choice while the logits move; the weights do not see it.
            bias = torch.zeros(B, E, device="cuda").scatter_(
                1, ids.long(), (10.0 - torch.arange(k, device="cuda").float()).expand(B, k))
            toll = []
            for sign in (1, -1):
                moved = [_route(x[b:b + 1] + sign * h * d[b:b + 1], k, bias[b], softmax=softmax, renorm=renorm)
                         for b in range(B)]
                assert all(torch.equal(m[0], ids[b:b + 1]) for b, m in enumerate(moved))
                toll.append(torch.cat([(m[1].double() * dw[b:b + 1]).sum(1) for b, m in enumerate(moved)]))
            got, want = (out.double() * d).sum(1), (toll[0] - toll[1]) / (2 * h)
            # h^2 / 6 of a third derivative that is at most 26 sums of |dw| (each weight's is), and the weights' own
            # rounding over 2 h
            tol = (h * h * 26 / 6 + 40 * U / (2 * h) + 64 * U * E) * dw.abs().double().sum(1)
            assert torch.all((got - want).abs() <= tol)


# -- the experts' order -----------------------------------------------------------------------------

ORDERS = [(1, 1, 1), (1, 8, 256), (5, 3, 2), (64, 8, 256), (65, 1, 7), (513, 4, 1024), (200, 32, 33), (1001, 6, 100),
          (3000, 8, 64), (20000, 8, 256), (40000, 5, 1000), (140001, 2, 3), (513, 8, 256), (4097, 8, 250),
          (6000, 8, 255), (12000, 8, 256), (2000, 7, 1024), (33000, 8, 31)]


def _order(ids, E):
    B, k = ids.shape
    slots, offsets = Guarded(B, k, dtype=torch.int32), Guarded(E + 1, dtype=torch.int32)
    ws = Guarded(mhc.mhc_experts_order_workspace_size(B, k, E), dtype=torch.uint8, fill=0xFF)
    mhc.mhc_experts_order(B, k, E, ids, slots.t, offsets.t, ws.t)
    _checked(slots, offsets, ws)
    return slots.t, offsets.t


def _order_torch(ids, E):
    """The same by a stable sort (the oracle is checked against it at small sizes)."""
    flat = ids.reshape(-1).long()
    real = (flat >= 0) & (flat < E)
    key = torch.where(real, flat, E)
    pairs = torch.sort(key, stable=True).indices
    slots = torch.empty_like(pairs)
    slots[pairs] = torch.arange(len(pairs), device=pairs.device)
    slots[~real] = -1
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:E].cumsum(0)])
    return slots.reshape(ids.shape).int(), offsets.int()


@pytest.mark.parametrize("B,k,E", ORDERS)
def test_order(B, k, E):
    _say(f"order B={B} k={k} E={E}")
    gen = torch.Generator().manual_seed(B + E)
    wide = torch.randint(-2, E + 2, (B, k), generator=gen)                          # some outside
    skew = (torch.rand(B, k, generator=gen) ** 6 * E).long()                        # few take most
    one = torch.full((B, k), E - 1)
    none = torch.full((B, k), -1)
    far = torch.randint(-2 ** 31, 2 ** 31, (B, k), generator=gen)
    for ids in (wide, skew, one, none, far):
        ids = ids.to(torch.int32).cuda()
        slots, offsets = _order(ids, E)
        want, first = _order_torch(ids, E)
        if B * k <= 4096:
            ref = experts.order(ids.cpu().numpy(), E)
            assert np.array_equal(want.cpu().numpy(), ref[0]) and np.array_equal(first.cpu().numpy(), ref[1])
        assert torch.equal(slots, want) and torch.equal(offsets, first)


def test_order_no_rows():
    offsets = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    mhc.mhc_experts_order(0, 4, 8, none, none, offsets, None)
    assert torch.all(offsets == 0)


# -- rows to their places and back ------------------------------------------------------------------

MOVES = [(1, 1, 8), (1, 8, 7168), (3, 2, 24), (5, 3, 40), (64, 8, 512), (33, 12, 1000), (130, 6, 264), (17, 32, 2056),
         (257, 1, 64), (9, 5, 8200), (1100, 4, 32), (70, 8, 1032)]


def _slots(gen, B, k, drop=True):
    """Places of B * k pairs in no order; some dropped."""
    slots = torch.randperm(B * k, generator=gen).reshape(B, k)
    if drop:
        slots[torch.rand(B, k, generator=gen) < 0.2] = -1
        if B > 2:
            slots[1] = -1                                    # a row without any
            slots[2, 0] = B * k                              # one behind the last
    return slots.to(torch.int32).cuda()


def _taken(slots, P):
    flat = slots.reshape(-1).long()
    mask = torch.zeros(P, dtype=torch.bool, device="cuda")
    mask[flat[(flat >= 0) & (flat < P)]] = True
    return mask


@pytest.mark.parametrize("B,k,C", MOVES)
def test_gather(B, k, C):
    _say(f"gather B={B} k={k} C={C}")
    gen = torch.Generator().manual_seed(B + k + C)
    P = B * k
    for drop in (False, True):
        slots = _slots(gen, B, k, drop)
        flat = slots.reshape(-1).long()
        ok = (flat >= 0) & (flat < P)
        for width, dtype, call in ((C, BF, "bf16"), (C, torch.uint8, "e4m3")):
            x = torch.randint(0, 256, (B, width * (2 if dtype == BF else 1)), generator=gen, dtype=torch.uint8).cuda()
            rows = Guarded(P, x.shape[1], dtype=torch.uint8)
            want = torch.full((P, x.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")
            want[flat[ok]] = x.repeat_interleave(k, 0)[ok]
            if call == "bf16":
                mhc.mhc_experts_gather(B, k, C, x, slots, rows.t)
                _checked(rows)
            else:
                blocks = -(-C // 32)
                scales = torch.randint(0, 256, (B, blocks), generator=gen, dtype=torch.uint8).cuda()
                more = Guarded(P, blocks, dtype=torch.uint8)
                mhc.mhc_experts_gather_ckpt(B, k, C, x, scales, slots, rows.t, more.t)
                _checked(rows, more)
                want_s = torch.full((P, blocks), 0x7F, dtype=torch.uint8, device="cuda")
                want_s[flat[ok]] = scales.repeat_interleave(k, 0)[ok]
                assert torch.equal(more.t, want_s)
            assert torch.equal(rows.t, want)                 # the rows that no slot names are as they were


@pytest.mark.parametrize("B,k,C", [(16384, 2, 32768), (2100, 8, 1040), (3000, 3, 24)])
def test_gather_many_rows(B, k, C):
    """More scales than the caches hold (they leave in a launch of their own), and rows of odd lengths."""
    _say(f"gather many B={B} k={k} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(B)
    P, blocks = B * k, -(-C // 32)
    slots = torch.randperm(P, generator=gen, device="cuda").reshape(B, k).to(torch.int32)
    slots[5] = -1
    codes = torch.randint(0, 256, (B, C), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0, 256, (B, blocks), generator=gen, device="cuda", dtype=torch.uint8)
    rows, more = Guarded(P, C, dtype=torch.uint8), Guarded(P, blocks, dtype=torch.uint8)
    mhc.mhc_experts_gather_ckpt(B, k, C, codes, scales, slots, rows.t, more.t)
    _checked(rows, more)
    for lo in range(0, B, 1024):
        at = slots[lo:lo + 1024].reshape(-1).long()
        ok = at >= 0
        assert torch.equal(rows.t[at[ok]], codes[lo:lo + 1024].repeat_interleave(k, 0)[ok])
        assert torch.equal(more.t[at[ok]], scales[lo:lo + 1024].repeat_interleave(k, 0)[ok])
    left = ~_taken(slots, P)
    assert int(left.sum()) == k and torch.all(rows.t[left] == 0x7F) and torch.all(more.t[left] == 0x7F)


@pytest.mark.parametrize("B,k,C", [
    (2100, 1, 1032), (1500, 2, 520), (900, 3, 264), (4000, 2, 40), (767, 1, 776), (768, 1, 776), (769, 2, 264),
    (700, 1, 256), (301, 3, 64), (90, 4, 8), (77, 9, 128), (41, 17, 200)])
def test_combine_bwd_many_rows(B, k, C):
    """One and two slots a row of many rows, on both sides of the choice of kernels."""
    _say(f"combine_bwd many B={B} k={k} C={C}")
    gen = torch.Generator().manual_seed(B)
    P, slots = B * k, _slots(gen, B, k)
    Y, g, w = _normal(gen, P, C), _normal(gen, B, C, scale=1 / 64), _normal(gen, B, k, dtype=torch.float32)
    taken = _taken(slots, P)
    Y[~taken] = float("nan")
    dY, dw = Guarded(P, C, dtype=BF, fill=0x3C), Guarded(B, k)
    before = dY.t.clone()
    mhc.mhc_experts_combine_bwd(B, k, C, Y, slots, w, g, dY.t, dw.t)
    _checked(dY, dw)
    want, want_w, A = experts.combine_bwd(f64(Y), slots.cpu().numpy(), f64(w), f64(g))
    t = taken.cpu().numpy()
    assert torch.equal(dY.t[~taken], before[~taken])
    _near(f64(dY.t)[t], want[t], (HALF_BF16 + 2 * U) * np.abs(want[t]), "dY")
    _near(dw.t, want_w, (C + 8) * U * A, "dweights")


@pytest.mark.parametrize("B,k,C", MOVES)
def test_combine(B, k, C):
    _say(f"combine B={B} k={k} C={C}")
    gen = torch.Generator().manual_seed(B * 3 + k + C)
    P = B * k
    for drop in (False, True):
        slots = _slots(gen, B, k, drop)
        Y, shared, w = _normal(gen, P, C), _normal(gen, B, C), _normal(gen, B, k, dtype=torch.float32)
        Y[~_taken(slots, P)] = float("nan")                  # not read
        w[(slots < 0) | (slots >= P)] = float("nan")
        for weights in (None, w):
            for s in (None, shared):
                out = Guarded(B, C, dtype=BF)
                mhc.mhc_experts_combine(B, k, C, Y, slots, weights, out.t, shared=s)
                _checked(out)
                want, A = experts.combine(f64(Y), slots.cpu().numpy(), None if weights is None else f64(w),
                                          None if s is None else f64(shared))
                _near(out.t, want, HALF_BF16 * np.abs(want) + (1 + HALF_BF16) * (k + 2) * U * A, "F_out")


@pytest.mark.parametrize("B,k,C", MOVES)
def test_combine_bwd(B, k, C):
    _say(f"combine_bwd B={B} k={k} C={C}")
    gen = torch.Generator().manual_seed(B * 5 + k + C)
    P = B * k
    for drop in (False, True):
        slots = _slots(gen, B, k, drop)
        Y, g, w = _normal(gen, P, C), _normal(gen, B, C, scale=1 / 64), _normal(gen, B, k, dtype=torch.float32)
        taken = _taken(slots, P)
        Y[~taken] = float("nan")
        w[(slots < 0) | (slots >= P)] = float("nan")
        dY, dw = Guarded(P, C, dtype=BF, fill=0x3C), Guarded(B, k)
        before = dY.t.clone()
        mhc.mhc_experts_combine_bwd(B, k, C, Y, slots, w, g, dY.t, dw.t)
        _checked(dY, dw)
        want, want_w, A = experts.combine_bwd(f64(Y), slots.cpu().numpy(), f64(w), f64(g))
        assert torch.equal(dY.t[~taken], before[~taken])     # left as they were
        t = taken.cpu().numpy()
        _near(f64(dY.t)[t], want[t], (HALF_BF16 + 2 * U) * np.abs(want[t]), "dY")
        _near(dw.t, want_w, (C + 8) * U * A, "dweights")


def test_more_than_2_32_bytes():
    """Rows past 2^32 bytes, to their places and back."""
    B, k, C = 40000, 8, 7168                                 # 4.6 GB of rows in the experts' order
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, C, generator=gen, device="cuda", dtype=BF)
    ids = torch.randint(0, 64, (B, k), generator=gen, device="cuda", dtype=torch.int32)
    slots, offsets = _order(ids, 64)
    rows = torch.empty(B * k, C, dtype=BF, device="cuda")
    mhc.mhc_experts_gather(B, k, C, x, slots, rows)
    for lo in range(0, B, 4000):
        assert torch.equal(rows[slots[lo:lo + 4000].reshape(-1).long()], x[lo:lo + 4000].repeat_interleave(k, 0))
    w = torch.full((B, k), 0.125, device="cuda")
    out, dw = torch.empty_like(x), torch.empty(B, k, device="cuda")
    mhc.mhc_experts_combine(B, k, C, rows, slots, w, out)
    assert torch.equal(out, x)                               # eight equal eighths
    dY = torch.empty_like(rows)
    mhc.mhc_experts_combine_bwd(B, k, C, rows, slots, w, x, dY, dw)
    assert torch.equal(dY, rows / 8)
    want = x.double().square().sum(1, keepdim=True)
    assert torch.all((dw - want).abs() <= (C + 8) * U * want)


def test_more_rows_than_workgroups():
    """Rows and pairs past what one grid takes: workgroups go on to the next."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    B, C = (1 << 21) + 5, 8
    _say("many rows: norm")
    x = torch.randn(B, C, generator=gen, device="cuda", dtype=BF)
    y, rstd = torch.empty_like(x), torch.empty(B, device="cuda")
    mhc.mhc_rmsnorm(B, C, x, None, y=y, rstd=rstd)
    want = 1 / (x.double().square().mean(1) + 1e-5).sqrt()
    assert torch.all((rstd - want).abs() <= 50 * U * want)
    n = x.double() * want[:, None]
    assert torch.all((y - n).abs() <= (HALF_BF16 + 54 * U) * n.abs())

    _say("many rows: order, gather, combine and its gradient")
    k, C, E = 8, 264, 5
    x = torch.randn(B, C, generator=gen, device="cuda", dtype=BF)
    ids = torch.randint(0, E, (B, k), generator=gen, device="cuda", dtype=torch.int32)
    slots, offsets = _order(ids, E)
    _, at = torch.sort(ids.reshape(-1), stable=True)
    assert torch.equal(slots.reshape(-1)[at], torch.arange(B * k, device="cuda", dtype=torch.int32))
    assert torch.equal(offsets[1:].long(), torch.bincount(ids.reshape(-1), minlength=E).cumsum(0))
    rows = torch.empty(B * k, C, dtype=BF, device="cuda")
    mhc.mhc_experts_gather(B, k, C, x, slots, rows)
    w = torch.full((B, k), 0.125, device="cuda")
    out, dY, dw = torch.empty_like(x), torch.empty_like(rows), torch.empty(B, k, device="cuda")
    mhc.mhc_experts_combine(B, k, C, rows, slots, w, out)
    mhc.mhc_experts_combine_bwd(B, k, C, rows, slots, w, x, dY, dw)
    assert torch.equal(out, x)                               # eight equal eighths
    for some in (slice(0, 3000), slice(B // 2, B // 2 + 3000), slice(B - 3000, B)):
        mine = slots[some].reshape(-1).long()
        assert torch.equal(rows[mine], x[some].repeat_interleave(k, 0))
        assert torch.equal(dY[mine], (x[some] / 8).repeat_interleave(k, 0))
    want = x.double().square().sum(1, keepdim=True)
    assert torch.all((dw - want).abs() <= (C + 8) * U * want)
    del x, rows, out, dY, dw, w, slots, ids, at, want

    _say("many rows: choice and its gradient")
    B = (1 << 26) + 17
    x = torch.randn(B, 2, generator=gen, device="cuda")
    ids, w = torch.empty(B, 1, device="cuda", dtype=torch.int32), torch.empty(B, 1, device="cuda")
    d = torch.empty_like(x)
    mhc.mhc_route(B, 2, 1, x, ids, w, renorm=False)
    assert torch.equal(ids[:, 0], (x[:, 1] > x[:, 0]).int())
    want = torch.sigmoid(x.double().amax(1))
    assert torch.all((w[:, 0] - want).abs() <= 32 * U * want)
    mhc.mhc_route_bwd(B, 2, 1, x, ids, w, d, renorm=False)
    best = x.double().amax(1, keepdim=True)
    want = torch.zeros_like(x, dtype=torch.float64).scatter_(1, ids.long(), best.sigmoid() * w * (-best).sigmoid())
    assert torch.all((d - want).abs() <= (48 + 2 * best.abs()) * U * want)


# -- streams, graphs --------------------------------------------------------------------------------

class _Layer:
    """One layer of experts between F_pre and F_out and its way back, by the library's calls; the experts are
    scalings, so that each step's own numbers can be checked."""

    def __init__(self, B, C, E, k, seed):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.C, self.E, self.k = B, C, E, k
        self.x, self.short, self.g = _normal(gen, B, C), _normal(gen, B, C), _normal(gen, B, C, scale=1 / 64)
        self.w = 1 + _normal(gen, C, scale=0.2, dtype=torch.float32)
        self.bias = _normal(gen, E, scale=0.05, dtype=torch.float32)
        self.logits = _normal(gen, B, E, scale=1.5, dtype=torch.float32)
        e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        f32, i32, u8 = torch.float32, torch.int32, torch.uint8
        self.o = {"sum": e(B, C), "y": e(B, C), "codes": e(B, C, dtype=u8), "scales": e(B, -(-C // 32), dtype=u8),
                  "rstd": e(B, dtype=f32), "ids": e(B, k, dtype=i32), "weights": e(B, k, dtype=f32),
                  "slots": e(B, k, dtype=i32), "offsets": e(E + 1, dtype=i32), "rows": e(B * k, C),
                  "row_codes": e(B * k, C, dtype=u8), "row_scales": e(B * k, -(-C // 32), dtype=u8),
                  "F_out": e(B, C), "dY": e(B * k, C), "dweights": e(B, k, dtype=f32), "dy": e(B, C),
                  "dlogits": e(B, E, dtype=f32), "dx": e(B, C), "dw": e(C, dtype=f32)}
        self.ws = (e(mhc.mhc_experts_order_workspace_size(B, k, E), dtype=u8),
                   e(mhc.mhc_rmsnorm_bwd_workspace_size(B, C), dtype=u8))

    def run(self, stream=None):
        B, C, E, k, o, s = self.B, self.C, self.E, self.k, self.o, {"stream": stream}
        mhc.mhc_rmsnorm(B, C, self.x, self.w, y=o["y"], codes=o["codes"], scales=o["scales"], shortcut=self.short,
                        sum=o["sum"], rstd=o["rstd"], **s)
        mhc.mhc_route(B, E, k, self.logits, o["ids"], o["weights"], bias=self.bias, **s)
        mhc.mhc_experts_order(B, k, E, o["ids"], o["slots"], o["offsets"], self.ws[0], **s)
        mhc.mhc_experts_gather(B, k, C, o["y"], o["slots"], o["rows"], **s)
        mhc.mhc_experts_gather_ckpt(B, k, C, o["codes"], o["scales"], o["slots"], o["row_codes"], o["row_scales"], **s)
        mhc.mhc_experts_combine(B, k, C, o["rows"], o["slots"], o["weights"], o["F_out"], shared=o["sum"], **s)
        mhc.mhc_experts_combine_bwd(B, k, C, o["rows"], o["slots"], o["weights"], self.g, o["dY"], o["dweights"], **s)
        mhc.mhc_experts_combine(B, k, C, o["dY"], o["slots"], None, o["dy"], **s)
        mhc.mhc_route_bwd(B, E, k, self.logits, o["ids"], o["dweights"], o["dlogits"], **s)
        mhc.mhc_rmsnorm_bwd(B, C, o["sum"], self.w, o["rstd"], o["dy"], o["dx"], dweight=o["dw"], workspace=self.ws[1],
                            dsum=self.g, **s)

    def blank(self):
        for t in self.o.values():
            t.view(torch.uint8).fill_(0x55)

    def bits(self):
        return {k: t.view(torch.uint8).clone() for k, t in self.o.items()}


def _same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("B,C,E,k", [(1, 264, 16, 4), (64, 512, 64, 8), (700, 1000, 100, 6)])
def test_graph_replays(B, C, E, k):
    """The layer captured and replayed several times, with other inputs and eager work in between."""
    _say(f"graph B={B} C={C} E={E} k={k}")
    a = _Layer(B, C, E, k, 1)
    a.run()
    torch.cuda.synchronize()
    want = a.bits()
    other = _Layer(B, C, E, k, 2)
    other.run()
    torch.cuda.synchronize()
    want_other = other.bits()
    keep = {n: getattr(a, n).clone() for n in ("x", "short", "g", "logits", "w", "bias")}
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.run()
    for turn in range(4):
        source = keep if turn % 2 == 0 else {n: getattr(other, n) for n in keep}
        for n, t in source.items():
            getattr(a, n).copy_(t)
        a.blank()
        graph.replay()
        torch.cuda.synchronize()
        _same(a.bits(), want if turn % 2 == 0 else want_other)
        other.run()                                          # eager, with its own workspaces
        torch.cuda.synchronize()
        _same(other.bits(), want_other)


def test_two_streams():
    """Two layers at once, each with its own workspaces, on streams that are not the current one."""
    layers = [_Layer(700, 520, 64, 8, 3), _Layer(300, 1000, 100, 6, 4)]
    want = []
    for layer in layers:
        layer.run()
        torch.cuda.synchronize()
        want.append(layer.bits())
        layer.blank()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.run(stream=s)
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        _same(layer.bits(), w)


def test_equal_bits():
    """Equal inputs, equal bits, many times over."""
    a = _Layer(900, 1032, 256, 8, 7)
    a.run()
    torch.cuda.synchronize()
    want = a.bits()
    for _ in range(10):
        a.blank()
        a.run()
        torch.cuda.synchronize()
        _same(a.bits(), want)


# -- a layer of experts in an mHC layer -------------------------------------------------------------

def test_layer_of_experts_in_the_stream():
    """mhc_pre, a whole layer of experts in 8 bits, mhc_post_res, and the way back, against the same steps in
    64 bits, step by step from the values the library's calls wrote.  Every product of the experts is torch's."""
    B, n, C, E, k, D = 48, 4, 256, 12, 3, 64
    gen = torch.Generator().manual_seed(31)
    X, H = _normal(gen, B, n * C), torch.rand(B, n * n + 2 * n, generator=gen).cuda()
    w, bias = 1 + _normal(gen, C, scale=0.2, dtype=torch.float32), _normal(gen, E, scale=0.05, dtype=torch.float32)
    router = _normal(gen, E, C, scale=C ** -0.5, dtype=torch.float32)
    up, down = (_normal(gen, E, *s, scale=0.1, dtype=torch.float32) for s in ((C, D), (D, C)))
    e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    f32, i32, u8, blocks = torch.float32, torch.int32, torch.uint8, C // 32

    # forward
    F_pre, y, codes, scales, rstd = e(B, C), e(B, C), e(B, C, dtype=u8), e(B, blocks, dtype=u8), e(B, dtype=f32)
    mhc.mhc_pre(B, n, C, X, H, F_pre)
    mhc.mhc_rmsnorm(B, C, F_pre, w, y=y, codes=codes, scales=scales, rstd=rstd)
    logits = y.float() @ router.t()
    ids, weights = e(B, k, dtype=i32), e(B, k, dtype=f32)
    mhc.mhc_route(B, E, k, logits, ids, weights, bias=bias, groups=4, top_groups=2, scale=1.5)
    slots, offsets = e(B, k, dtype=i32), e(E + 1, dtype=i32)
    ws = e(mhc.mhc_experts_order_workspace_size(B, k, E), dtype=u8)
    mhc.mhc_experts_order(B, k, E, ids, slots, offsets, ws)
    row_codes, row_scales, rows = e(B * k, C, dtype=u8), e(B * k, blocks, dtype=u8), e(B * k, C)
    mhc.mhc_experts_gather_ckpt(B, k, C, codes, scales, slots, row_codes, row_scales)
    mhc.mhc_ckpt_unpack(B * k, 1, C, row_codes, row_scales, rows)
    start = offsets.tolist()
    Y = e(B * k, C)
    hidden = torch.empty(B * k, D, device="cuda")
    for x in range(E):
        at = slice(start[x], start[x + 1])
        hidden[at] = torch.tanh(rows[at].float() @ up[x])
        Y[at] = (hidden[at] @ down[x]).to(BF)
    F_out, X_next = e(B, C), e(B, n * C)
    mhc.mhc_experts_combine(B, k, C, Y, slots, weights, F_out)
    mhc.mhc_post_res(B, n, C, X, F_out, H, X_next)
    torch.cuda.synchronize()

    want_y, want_rstd = experts.rmsnorm(f64(F_pre), f64(w))
    _near(y, want_y, (HALF_BF16 + 54 * U) * np.abs(want_y), "y")
    _check_codes(codes, scales, want_y)
    want_ids, want_w = experts.route(f64(logits), k, f64(bias), groups=4, top_groups=2, scale=1.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    _near(weights, want_w, 64 * U * want_w, "weights")
    want_slots, want_first = experts.order(want_ids, E)
    assert np.array_equal(slots.cpu().numpy(), want_slots) and start == want_first.tolist()
    held = backward.ckpt_decode(codes.cpu().numpy(), scales.cpu().numpy(), 1, C)
    assert np.array_equal(f64(rows)[want_slots.reshape(-1)], np.repeat(held, k, axis=0))
    want, A = experts.combine(f64(Y), want_slots, f64(weights))
    _near(F_out, want, HALF_BF16 * np.abs(want) + 6 * U * A, "F_out")

    # backward
    G = _normal(gen, B, n * C, scale=1 / 64)
    dF_out, dH = e(B, C), e(B, n * n + 2 * n, dtype=f32)
    mhc.mhc_post_res_bwd(B, n, C, X, F_out, H, G, dF_out, dH)
    dY, dweights, dlogits = e(B * k, C), e(B, k, dtype=f32), e(B, E, dtype=f32)
    mhc.mhc_experts_combine_bwd(B, k, C, Y, slots, weights, dF_out, dY, dweights)
    d_rows = e(B * k, C)
    for x in range(E):
        at = slice(start[x], start[x + 1])
        d_rows[at] = (((dY[at].float() @ down[x].t()) * (1 - hidden[at] ** 2)) @ up[x].t()).to(BF)
    dy = e(B, C)
    mhc.mhc_route_bwd(B, E, k, logits, ids, dweights, dlogits, scale=1.5)
    mhc.mhc_experts_combine(B, k, C, d_rows, slots, None, dy, shared=(dlogits @ router).to(BF))
    dF_pre, dw = e(B, C), e(C, dtype=f32)
    ws = e(mhc.mhc_rmsnorm_bwd_workspace_size(B, C), dtype=u8)
    mhc.mhc_rmsnorm_bwd(B, C, F_pre, w, rstd, dy, dF_pre, dweight=dw, workspace=ws)
    torch.cuda.synchronize()

    # The same by autograd in 64 bits, from F_pre to <F_out, dF_out>, the rounding to 8 bits passed as it is.
    p = F_pre.double().cpu().requires_grad_()
    wd = w.double().cpu().requires_grad_()
    norm = p * (p.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * wd
    l64 = norm @ router.double().cpu().t()
    chosen = torch.sigmoid(l64.gather(1, ids.long().cpu()))
    w64 = 1.5 * chosen / chosen.sum(1, keepdim=True)
    as_held = norm + (torch.from_numpy(held) - norm).detach()
    out = 0
    for j in range(k):
        u64, d64 = (t.double().cpu()[ids[:, j].long().cpu()] for t in (up, down))
        h64 = torch.tanh((as_held[:, None] @ u64))
        out = out + w64[:, j, None] * (h64 @ d64)[:, 0]
    grads = torch.autograd.grad((out * dF_out.double().cpu()).sum(), [p, wd])
    # Relative to the whole: the path rounds y, Y, dY, the experts' gradient, the router's, dy and dF_pre to bf16,
    # each by at most 2^-8 of its part, and fp32's roundings are far below: 8 * 2^-8 of the norm.
    for got, want in zip((dF_pre, dw), grads):
        off = (got.double().cpu() - want).norm() / want.norm()
        _say(f"gradient off by {off:.2e} of its norm")
        assert off <= 8 * HALF_BF16
