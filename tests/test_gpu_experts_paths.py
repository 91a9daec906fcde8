"""The calls around a layer of experts on the GPU, where tests/test_gpu_experts.py
does not reach: weights and gradients to their last roundings, kernels that
only some sizes take, and grids that are gone through more than once.

u = 2^-24; tolerances are derived at each test.
"""

import numpy as np
import pytest
import torch

import manifold_constrained_hyper_amd as mhc
from oracle import experts
from tests.test_gpu_experts import Guarded, U, _checked, _crowded, _normal, _route, _say, _some_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    mhc.load()
    yield


def _within(got, want, tol, what):
    """No more than tol off, without an allowance for small numbers."""
    off = np.abs((f64(got) if isinstance(got, torch.Tensor) else got) - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, at {np.argwhere(bad)[:3]}, by " \
                          f"{np.max(off[bad] / np.maximum(np.abs(want[bad]), 1e-300)):.2e} of the value"


# -- choice of experts ------------------------------------------------------------------------------

def _far_logits(B, E, gen, dtype):
    """Ordinary rows, and rows whose sigmoids or shares lie below fp32's normal numbers."""
    x = torch.randn(B, E, generator=gen) * 3
    x[1::4] = -90 - 10 * torch.rand(len(x[1::4]), E, generator=gen)
    x[2::4, ::2] = 88 + 14 * torch.rand(len(x[2::4]), len(range(0, E, 2)), generator=gen)
    x[3::4, 0] = 95.0
    return x.to(dtype).cuda()


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (40, 7, 7, 1, 1), (200, 64, 8, 8, 4), (60, 256, 16, 1, 1), (9, 1000, 32, 1, 1), (9, 1000, 8, 5, 3),
    (2600, 16, 14, 1, 1), (2603, 256, 8, 8, 4), (1100, 100, 6, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_weights_are_rounded_once(B, E, k, groups, top_groups, dtype):
    """Formed in 64 bits: exp to 2^-36, at most four of them in a weight, so 2^-33 = 2^-9 u before the one rounding
    of u (half a step of 2^-149 below the normal numbers): (1 + 2^-8) u."""
    _say(f"route weights B={B} E={E} k={k} {dtype}")
    gen = torch.Generator().manual_seed(E + k)
    x = _far_logits(B, E, gen, dtype)
    rows = np.arange(B) if B <= 200 else _some_rows(B)
    for bias in (None, _normal(gen, E, scale=0.1, dtype=torch.float32)):
        for softmax in (False, True):
            for renorm in (False, True):
                for scale in (2.5, 2.0 ** 60):
                    how = dict(groups=groups, top_groups=top_groups, softmax=softmax, renorm=renorm, scale=scale)
                    ids, weights = _route(x, k, bias, **how)
                    want, want_w = experts.route(f64(x)[rows], k, None if bias is None else f64(bias), **how)
                    assert np.array_equal(ids.cpu().numpy()[rows], want)
                    _within(f64(weights)[rows], want_w, (1 + 2.0 ** -8) * U * np.abs(want_w) + 2.0 ** -150,
                            f"weights softmax={softmax} renorm={renorm} scale={scale}")


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (5, 1000, 8, 5, 3), (5, 1000, 16, 5, 3), (9, 1023, 8, 33, 4), (7, 1023, 20, 33, 4), (3, 1020, 8, 3, 2),
    (6, 1020, 32, 17, 9), (70, 800, 8, 10, 4), (2600, 1015, 6, 5, 2), (5, 600, 24, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_many_experts_in_groups(B, E, k, groups, top_groups, dtype):
    """Groups that leave a lane up to 32 experts, with short and long lists of the best."""
    _say(f"route in groups B={B} E={E} k={k} groups={groups} top={top_groups} {dtype}")
    gen = torch.Generator().manual_seed(E * 10 + k + groups)
    x = torch.randn(B, E, generator=gen) * 2
    x[torch.rand(B, E, generator=gen) < 0.05] = -float("inf")
    x[1], x[2, 1:], x[0, ::7], x[min(3, B - 1), ::5] = -float("inf"), -float("inf"), float("nan"), float("inf")
    x = x.to(dtype).cuda()
    rows = np.arange(B) if B <= 100 else _some_rows(B)
    bias = _normal(gen, E, scale=0.1, dtype=torch.float32)
    for b in (None, bias):
        for softmax in (False, True):
            how = dict(groups=groups, top_groups=top_groups, softmax=softmax, renorm=b is None, scale=1.5)
            ids, weights = _route(x, k, b, **how)
            want, want_w = experts.route(f64(x)[rows], k, None if b is None else f64(b), **how)
            assert np.array_equal(ids.cpu().numpy()[rows], want)
            _within(f64(weights)[rows], want_w, (1 + 2.0 ** -8) * U * np.abs(want_w) + 2.0 ** -150, "weights")


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (20, 1000, 8, 5, 3), (15, 1000, 16, 5, 3), (15, 1023, 20, 33, 4), (20, 1000, 8, 1, 1), (15, 700, 20, 1, 1),
    (20, 512, 8, 1, 1), (15, 400, 20, 1, 1)])
def test_route_crowded_of_many_experts(B, E, k, groups, top_groups):
    """Choices that 42 bits cannot tell apart, with 8 to 32 experts a lane and a wave a row."""
    _say(f"route crowded B={B} E={E} k={k} groups={groups} top={top_groups}")
    gen = torch.Generator().manual_seed(B + E + k)
    x = _crowded(B, E, gen)
    x[7] = torch.randn(E, generator=gen)
    for softmax in (False, True):
        for b in (torch.zeros(E), torch.full((E,), 0.25)):
            b[E // 2] = -float("inf")
            how = dict(groups=groups, top_groups=top_groups, softmax=softmax)
            ids, _ = _route(x.cuda(), k, b.cuda(), **how)
            want, _ = experts.route(f64(x), k, f64(b), **how)
            assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:5]


@pytest.mark.parametrize("B,E,k", [(30, 64, 5), (12, 1000, 20), (4099, 50, 6), (4097, 200, 3)])
def test_route_bwd_of_small_shares(B, E, k):
    """The softmax's gradient where shares are far below the largest, to their own size.  Logits are multiples of 2^-6,
    so that x - top is exact; exp is off by 4 u, the sum of E <= 1024 terms by 4 and 22 more, its inverse by 1, the
    products of share and dw by 2: 33 u of a chosen one's p dw, and 2^-149 below the normal numbers.  The others' part
    takes the sum over the chosen (33 u and 5 for its own terms), the inverse once more (27 u), exp (4 u) and 2
    products: 72 u of p sum(p dw); its shares below 2^-126 count as 0."""
    _say(f"route_bwd small shares B={B} E={E} k={k}")
    gen = torch.Generator().manual_seed(B + E)
    x = -30 - torch.randint(0, 64 * 70, (B, E), generator=gen) / 64
    top = torch.randint(0, E, (B, 1), generator=gen)
    x.scatter_(1, top, 0.5)
    ids = torch.argsort(torch.rand(B, E, generator=gen).scatter_(1, top, 2.0), 1)[:, :k].int()   # far ones
    dw = torch.randn(B, k, generator=gen) * 2.0 ** 40
    out = Guarded(B, E)
    mhc.mhc_route_bwd(B, E, k, x.cuda(), ids.cuda(), dw.cuda(), out.t, softmax=True, renorm=False)
    _checked(out)
    p, d, at = torch.softmax(x.double(), 1), dw.double(), ids.long()
    part = torch.zeros_like(p).scatter_(1, at, p.gather(1, at) * d)
    along = part.sum(1, keepdim=True)
    size = part.abs().sum(1, keepdim=True)
    given = torch.zeros_like(p).scatter_(1, at, d.abs())
    tol = U * (34 * part.abs() + 72 * p * size) + 2.0 ** -148 * (given + p * given.sum(1, keepdim=True))
    tol += torch.where(p < 2.0 ** -125, 2.0 ** -125, 0.0) * size + 2.0 ** -149
    _within(out.t, (part - p * along).numpy(), tol.numpy(), "dlogits")


@pytest.mark.parametrize("B,E,k", [(40, 24, 4), (4100, 33, 6)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_of_far_sigmoids(B, E, k, renorm):
    """Sigmoids next to 0 and next to 1, whose gradients are below fp32's normal numbers but for dweights: exp is off by
    4 u (2^-148 there), a sigmoid by 3 more, a weight by 2 exps, sigmoid, sum of k <= 6 (its terms' 11 and 4) and
    division: 27 u; with products and difference 40 u of w sigmoid(-x) (|dw| + sum w |dw|)."""
    _say(f"route_bwd far sigmoids B={B} E={E} k={k} renorm={renorm}")
    gen = torch.Generator().manual_seed(B + k)
    x = _far_logits(B, E, gen, torch.float32).cpu()
    ids = torch.argsort(torch.rand(B, E, generator=gen), 1)[:, :k].int()
    dw = torch.randn(B, k, generator=gen) * 2.0 ** 70
    out = Guarded(B, E)
    mhc.mhc_route_bwd(B, E, k, x.cuda(), ids.cuda(), dw.cuda(), out.t, softmax=False, renorm=renorm, scale=1.5)
    _checked(out)
    rows = np.arange(B) if B < 100 else _some_rows(B)
    x, at, dw = f64(x)[rows], ids.numpy()[rows], f64(dw)[rows]
    want = experts.route_bwd(x, at, dw, False, renorm, 1.5)
    size, far = np.zeros_like(want), np.zeros_like(want)
    for b, z in enumerate(x):
        w = experts.weights_of(z, list(at[b]), False, renorm, 1.0)
        all_of = np.abs(1.5 * dw[b]) + (np.sum(np.abs(w * 1.5 * dw[b])) if renorm else 0.0)
        size[b, at[b]] = w * experts.sigmoid(-z[at[b]]) * all_of
        far[b, at[b]] = all_of                               # (two of the factors may be below the normal numbers)
    _within(f64(out.t)[rows], want, 40 * U * size + 2.0 ** -146 * far, "dlogits")


@pytest.mark.parametrize("B", [9, 4100])
def test_route_bwd_of_masked_ids(B):
    """An id whose logit is masked has no weight: what stands in its place of dweights changes nothing."""
    _say(f"route_bwd masked ids B={B}")
    gen = torch.Generator().manual_seed(B)
    E, k = 40, 5
    x, dw = _normal(gen, B, E, dtype=torch.float32), _normal(gen, B, k, dtype=torch.float32)
    ids = torch.argsort(torch.rand(B, E, generator=gen), 1)[:, :k].int().cuda()
    off = ids[:, 2:4].long()
    x.scatter_(1, off, torch.tensor([-float("inf"), float("nan")], device="cuda").expand(B, 2))
    for softmax in (False, True):
        for renorm in (False, True):
            got = []
            for value in (0.0, float("nan"), float("inf")):
                dw[:, 2:4] = value
                out = Guarded(B, E)
                mhc.mhc_route_bwd(B, E, k, x, ids, dw, out.t, softmax=softmax, renorm=renorm)
                _checked(out)
                got.append(out.t)
            assert torch.isfinite(got[0]).all() and torch.all(got[0].gather(1, off) == 0)
            assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# -- rows to their places ---------------------------------------------------------------------------

def _codes_and_slots(B, k, C, gen):
    P, blocks = B * k, -(-C // 32)
    slots = torch.randperm(P, generator=gen, device="cuda").reshape(B, k).to(torch.int32)
    slots[5], slots[B - 2, 0] = -1, P
    codes = torch.randint(0, 256, (B, C), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0, 256, (B * blocks,), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales, slots


@pytest.mark.parametrize("B,k,C", [
    (16640, 8, 7168), (16384, 7, 8192), (3900, 28, 8192), (14000, 8, 7168), (3700, 28, 8192),   # in 224 and 256 blocks
    (16640, 8, 7200), (16700, 8, 7176),                       # 225 blocks, which four does not divide
    (15000, 2, 32768)])                                       # 1024 blocks
def test_gather_scales_of_large_batches(B, k, C):
    """Rows in 8 bits, with scales that the caches hold together and more than they do (about 26 MB)."""
    _say(f"gather scales B={B} k={k} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(B)
    P, blocks = B * k, -(-C // 32)
    codes, scales, slots = _codes_and_slots(B, k, C, gen)
    scales = scales.view(B, blocks)
    rows, more = Guarded(P, C, dtype=torch.uint8), Guarded(P, blocks, dtype=torch.uint8)
    mhc.mhc_experts_gather_ckpt(B, k, C, codes, scales, slots, rows.t, more.t)
    _checked(rows, more)
    left = torch.ones(P, dtype=torch.bool, device="cuda")
    for lo in range(0, B, 1024):
        at = slots[lo:lo + 1024].reshape(-1).long()
        ok = (at >= 0) & (at < P)
        assert torch.equal(rows.t[at[ok]], codes[lo:lo + 1024].repeat_interleave(k, 0)[ok])
        assert torch.equal(more.t[at[ok]], scales[lo:lo + 1024].repeat_interleave(k, 0)[ok])
        left[at[ok]] = False
    assert int(left.sum()) == k + 1 and torch.all(rows.t[left] == 0x7F) and torch.all(more.t[left] == 0x7F)


@pytest.mark.parametrize("B,k,C", [(16640, 8, 7168), (300, 5, 2048), (40, 3, 256)])
@pytest.mark.parametrize("start", [1, 2])
def test_gather_scales_at_any_byte(B, k, C, start):
    """Scales are bytes, wherever they begin."""
    _say(f"gather scales at byte {start} B={B} k={k} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(B + start)
    P, blocks = B * k, C // 32
    codes, scales, slots = _codes_and_slots(B, k, C, gen)
    given = torch.empty(start + B * blocks, dtype=torch.uint8, device="cuda")
    given[start:] = scales
    rows, other = Guarded(P, C, dtype=torch.uint8), 3 - start
    more = torch.full((P * blocks + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    mhc.mhc_experts_gather_ckpt(B, k, C, codes, given[start:], slots, rows.t, more[other:other + P * blocks])
    _checked(rows)
    assert torch.all(more[:other] == 0xA5) and torch.all(more[other + P * blocks:] == 0xA5)
    more = more[other:other + P * blocks].view(P, blocks)
    at = slots.reshape(-1).long()
    ok = (at >= 0) & (at < P)
    assert torch.equal(more[at[ok]], scales.view(B, blocks).repeat_interleave(k, 0)[ok])


# -- norm -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,C", [(1030, 8200), (1030, 16384), (300, 16376), (2, 16392), (700, 24584), (700, 32768),
                                 (600, 32776), (520, 65536), (2050, 7168), (9000, 1000)])
def test_rmsnorm_bwd_several_rows_a_workgroup(B, C):
    """Every number of vectors a thread with several rows to a workgroup; bounds as in test_rmsnorm_bwd."""
    _say(f"rmsnorm_bwd several rows B={B} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(B + C)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    s = (normal(B, C) * torch.exp2(normal(B, 1))).bfloat16()
    dy, dsum, w = (normal(B, C) / 64).bfloat16(), (normal(B, C) / 64).bfloat16(), 1 + 0.3 * normal(C)
    rstd = (s.float().square().mean(1) + 1e-5).rsqrt()
    n = s.double() * rstd.double()[:, None]
    for weight in (None, w):
        g = dy.double() if weight is None else dy.double() * w.double()
        A = (g * n).abs().sum(1, keepdim=True)
        mean = (g * n).mean(1, keepdim=True)
        for more in (None, dsum):
            dx, dw = Guarded(B, C, dtype=torch.bfloat16), Guarded(C)
            ws = Guarded(mhc.mhc_rmsnorm_bwd_workspace_size(B, C), dtype=torch.uint8, fill=0xFF)
            mhc.mhc_rmsnorm_bwd(B, C, s, weight, rstd, dy, dx.t, dweight=dw.t, workspace=ws.t, dsum=more)
            _checked(dx, dw, ws)
            want = rstd.double()[:, None] * (g - n * mean)
            if more is not None:
                want = want + dsum.double()
            e = rstd.double()[:, None] * (n.abs() * 96 * U * A / C + 8 * U * (g.abs() + (n * mean).abs()))
            e += U * want.abs()
            assert torch.all((dx.t.double() - want).abs() <= 2.0 ** -8 * (want.abs() + e) + e)
            each = dy.double() * n
            assert torch.all((dw.t.double() - each.sum(0)).abs() <= (B + 40) * U * each.abs().sum(0))
            alone = Guarded(B, C, dtype=torch.bfloat16)
            mhc.mhc_rmsnorm_bwd(B, C, s, weight, rstd, dy, alone.t, dsum=more)
            _checked(alone)
            assert torch.equal(alone.t, dx.t)


# -- more work than one grid ------------------------------------------------------------------------

def test_rmsnorm_of_more_rows_than_workgroups():
    """Rows of a workgroup each, past 2^21 of them: workgroups go on to the next."""
    B, C = (1 << 21) + 5, 264
    _say(f"rmsnorm B={B} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.3 * torch.randn(C, generator=gen, device="cuda")
    o = {"y": Guarded(B, C, dtype=torch.bfloat16), "codes": Guarded(B, C, dtype=torch.uint8),
         "scales": Guarded(B, -(-C // 32), dtype=torch.uint8), "rstd": Guarded(B)}
    mhc.mhc_rmsnorm(B, C, x, w, **{k: v.t for k, v in o.items()})
    _checked(*o.values())
    for lo in range(0, B, 1 << 19):
        at = slice(lo, min(B, lo + (1 << 19)))
        s = x[at].double()
        rstd = 1 / (s.square().mean(1) + 1e-5).sqrt()
        assert torch.all((o["rstd"].t[at] - rstd).abs() <= 50 * U * rstd)
        y = s.mul_(rstd[:, None]).mul_(w.double())
        assert torch.all((o["y"].t[at] - y).abs() <= (2.0 ** -8 + 54 * U) * y.abs())
        step = torch.exp2(o["scales"].t[at].double() - 127).repeat_interleave(32, 1)[:, :C]
        got = o["codes"].t[at].view(torch.float8_e4m3fn).double() * step
        assert torch.all((got - y).abs() <= (2.0 ** -4 + 54 * U) * y.abs() + 2.0 ** -10 * step)


def test_combine_of_more_rows_than_waves():
    """Rows that a wave takes, past 2^24 of them, and 2^32 bytes."""
    B, C = (1 << 24) + 9, 264
    _say(f"combine B={B} C={C}")
    gen = torch.Generator(device="cuda").manual_seed(4)
    Y = torch.randint(-2 ** 31, 2 ** 31, (B, C // 2), generator=gen, device="cuda", dtype=torch.int32)
    Y &= ~0x40004000                                             # no NaN and no infinity: exponents below 128
    Y = Y.view(torch.bfloat16)
    slots = torch.arange(B - 1, -1, -1, device="cuda", dtype=torch.int32)
    slots[::1000003] = -1
    out = torch.full_like(Y, 7.0)
    mhc.mhc_experts_combine(B, 1, C, Y, slots, None, out)
    for lo in range(0, B, 1 << 21):
        hi = min(B, lo + (1 << 21))
        want = Y[B - hi:B - lo].flip(0)
        want[slots[lo:hi] < 0] = 0
        assert torch.all(out[lo:hi] == want)                     # (a zero's sign is lost in the sum)
