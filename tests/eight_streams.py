"""The gradient of the 20 normalisations at n = 8 in 32 bits: inputs, the
error that the arithmetic leaves, and the same arithmetic on the CPU.

Bound of one row's dz against the definition, u = 2^-24, M = max |dH_res| of
the row:

    (16 + 8 (1 + max |z|)) u M

16: the arithmetic itself.  Each of the 39 backward steps rounds a value of at
most M a few times, and the next step subtracts the mean of what it left along
its rows or columns, so most of it goes again; `emulated` below does the same
operations in the same order and stays under 2 u M from balanced matrices to
ones with a factor of e^20 between their elements (test_eight_streams.py), and
the hardware's exponential and reciprocal (an ulp each) are of that size too.

8 (1 + max |z|): z = alpha logit / r + b is rounded three times, at most 3 u
|z|, and the exponential adds an ulp or two, so z is off by 4 u (1 + |z|) at
most.  dz is linear in dH with factors made of the matrices' elements, all at
most 1; moving z by e moves it by no more than 2 e M (the second derivative of
<dH, H_res>; test_eight_streams.py tries random signs)."""

import numpy as np

from oracle import backward

N_STREAMS, ITERS = 8, 20
U = 2.0 ** -24
f32 = np.float32

# (what b_res has on its diagonal, standard deviation of z): a training start,
# matrices further from balanced, and some that 20 iterations do not balance.
SPREADS = [(2.0, 0.1), (2.0, 1.0), (0.0, 2.0), (0.0, 4.0), (4.0, 3.0)]
SLOW = [(0.0, 4.0), (4.0, 3.0)]     # where the 20th iteration still counts


def inputs(diag, spread, B, seed):
    """logits, r, b_res (alpha_res = 1) and dH of B rows, fp32, and z from them."""
    n = N_STREAMS
    rng = np.random.default_rng(seed)
    N = n * n + 2 * n
    logits = (spread * rng.standard_normal((B, N))).astype(f32)
    r = (0.5 + rng.random(B)).astype(f32)
    b = (diag * np.eye(n)).astype(f32).reshape(-1)
    dH = rng.standard_normal((B, N)).astype(f32)
    z = logits[:, 2 * n:].astype(np.float64) / r[:, None].astype(np.float64) + b
    return logits, r, b, dH, z.reshape(B, n, n)


def row_bound(z, dH_res):
    most = np.abs(dH_res).reshape(len(z), -1).max(1)
    return (16 + 8 * (1 + np.abs(z).reshape(len(z), -1).max(1))) * U * most


def exact(z, dH_res, iters=ITERS):
    return backward.sinkhorn_bwd(z, np.asarray(dH_res, np.float64).reshape(z.shape), iters)


def _axis_sum(x, axis):
    """Eight values in three levels of pairs, every level rounded."""
    y = np.moveaxis(x, axis, -1)
    for _ in range(3):
        y = (y[..., 0::2] + y[..., 1::2]).astype(f32)
    return np.moveaxis(y, -1, axis)


def emulated(z, dH_res):
    """dz with every operation rounded to fp32; every second matrix is rebuilt
    from the one before."""
    m0 = np.exp(z.astype(f32))
    m = (m0 / _axis_sum(m0, -1)).astype(f32)
    y, inv = [m], [None]
    for k in range(1, 2 * ITERS):
        inv.append((f32(1) / _axis_sum(m, -2 if k % 2 else -1)).astype(f32))
        m = (m * inv[k]).astype(f32)
        if k % 2 == 0:
            y.append(m)
    d = dH_res.reshape(z.shape).astype(f32)
    for k in range(2 * ITERS - 1, 0, -1):
        yk = (y[k // 2] * inv[k]).astype(f32) if k % 2 else y[k // 2]
        d = ((d - _axis_sum((d * yk).astype(f32), -2 if k % 2 else -1)).astype(f32) * inv[k]).astype(f32)
    return (y[0] * (d - _axis_sum((d * y[0]).astype(f32), -1)).astype(f32)).astype(f32)
