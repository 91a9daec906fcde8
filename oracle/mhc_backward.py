"""Plain, slow, fp64 gradients of the mHC residual-stream forward, the 8-bit
checkpoint of the stream, and the embedding lookup with its gradient.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see the package docstring).

The gradients are the derivatives of [mHC-cutile] section 2's formulas, by
hand; tests/test_oracle_backward_pins.py checks them against differences of
the forward oracle.  Inputs and outputs are numpy float64 unless said.
"""

import numpy as np

from . import fp8
from .mhc_oracle import SINKHORN_ITERS, sigmoid, split_h

CKPT_BLOCK = 32


def ckpt_encode(x, n, C):
    """Codes (uint8 [B, n*C]) and scale bytes (uint8 [B, n*ceil(C/32)]) of x
    [B, n*C]: per block of 32 channels of a stream the least s >= 1 with
    |x| <= 448 * 2^(s - 127) for its finite values; what is not finite is NaN.
    Codes under s = 247 stop at 240 (the next one, 2^128, is no bf16 number)."""
    x = np.asarray(x, np.float64).reshape(-1, n, C)
    B, blocks = x.shape[0], -(-C // CKPT_BLOCK)
    codes = np.zeros((B, n, C), np.uint8)
    scales = np.zeros((B, n, blocks), np.uint8)
    for k in range(blocks):
        v = x[:, :, k * CKPT_BLOCK:(k + 1) * CKPT_BLOCK]
        fine = np.isfinite(v)
        amax = np.max(np.where(fine, np.abs(v), 0.0), axis=2)
        s = np.ones(amax.shape, np.int64)
        for e in range(1, 255):
            s = np.where(amax > 448.0 * 2.0 ** (e - 127), e + 1, s)
        q = np.where(fine, v, 0.0) / np.exp2(s - 127.0)[:, :, None]
        most = np.where(s == 247, 240.0, 448.0)[:, :, None]
        c = fp8.e4m3_encode(np.clip(q, -most, most))
        codes[:, :, k * CKPT_BLOCK:(k + 1) * CKPT_BLOCK] = np.where(fine, c, 0x7F)
        scales[:, :, k] = s
    return codes.reshape(B, n * C), scales.reshape(B, n * blocks)


def ckpt_decode(codes, scales, n, C):
    """The values a checkpoint stands for, float64 [B, n*C]."""
    codes = np.asarray(codes, np.uint8)
    B, blocks = codes.shape[0], -(-C // CKPT_BLOCK)
    v = np.exp2(np.asarray(scales, np.float64).reshape(B, n, blocks) - 127.0)
    out = fp8.e4m3_decode(codes).reshape(B, n, C)
    for c in range(C):
        out[:, :, c] *= v[:, :, c // CKPT_BLOCK]
    return out.reshape(B, n * C)


def post_res_bwd(x, f_out, H, dx_next, n, C):
    """Gradients of step (4b) with respect to F_out and H: dF_out [B, C] and
    dH [B, N] (zeros in the pre block)."""
    x, g = (np.asarray(t, np.float64).reshape(-1, n, C) for t in (x, dx_next))
    f = np.asarray(f_out, np.float64)
    _, h_post, _ = split_h(H, n)
    dF = np.zeros_like(f)
    dH = np.zeros((x.shape[0], n * n + 2 * n))
    for i in range(n):
        dF += h_post[:, i:i + 1] * g[:, i]
        dH[:, n + i] = np.sum(g[:, i] * f, axis=1)
        for j in range(n):
            dH[:, 2 * n + i * n + j] = np.sum(g[:, i] * x[:, j], axis=1)
    return dF, dH


def sinkhorn_bwd(z, dm, iters=SINKHORN_ITERS):
    """Gradient of sinkhorn_knopp with respect to its argument.  z, dm [..., n, n]."""
    m = np.exp(np.asarray(z, np.float64))
    start, kept = m, []
    for _ in range(iters):
        for axis in (-1, -2):
            total = np.sum(m, axis=axis, keepdims=True)
            m = m / total
            kept.append((m, total, axis))
    d = np.asarray(dm, np.float64)
    for y, total, axis in kept[::-1]:
        d = (d - np.sum(d * y, axis=axis, keepdims=True)) / total
    return d * start


def coeffs_pre_bwd(x, phi, alphas, biases, logits, r, H, dx_next, dH, dF_pre, n, C):
    """Gradients of steps (1)-(4a) joined with the apply's path to X_t.

    alphas: (pre, post, res); biases: the three arrays.  Returns dict(dX [B, nC],
    dphi [nC, N], dalpha [3], db_pre, db_post, db_res, and dz, dlogits [B, N])."""
    x = np.asarray(x, np.float64).reshape(-1, n, C)
    g = np.asarray(dx_next, np.float64).reshape(-1, n, C)
    dF = np.asarray(dF_pre, np.float64)
    phi = np.asarray(phi, np.float64)
    logits, dH = np.asarray(logits, np.float64), np.asarray(dH, np.float64)
    r = np.asarray(r, np.float64).reshape(-1, 1)
    B, N = logits.shape
    h_pre, _, h_res = split_h(H, n)
    alpha = np.concatenate([np.full(n, alphas[0]), np.full(n, alphas[1]), np.full(n * n, alphas[2])])
    bias = np.concatenate([np.asarray(b, np.float64).reshape(-1) for b in biases])
    with np.errstate(invalid="ignore", divide="ignore"):
        z = alpha * logits / r + bias
    up = dH.copy()
    for i in range(n):
        up[:, i] = np.sum(x[:, i] * dF, axis=1)
    dz = np.zeros((B, N))
    s = sigmoid(z)
    dz[:, :n] = up[:, :n] * s[:, :n] * (1 - s[:, :n])
    dz[:, n:2 * n] = 2 * up[:, n:2 * n] * s[:, n:2 * n] * (1 - s[:, n:2 * n])
    with np.errstate(invalid="ignore", divide="ignore"):
        dz[:, 2 * n:] = sinkhorn_bwd(z[:, 2 * n:].reshape(B, n, n), up[:, 2 * n:].reshape(B, n, n)).reshape(B, n * n)
        dl = alpha * dz / r
        turn = -np.sum(dl * logits, axis=1, keepdims=True) / (n * C * r * r)
    dX = (dl @ phi.T).reshape(B, n, C) + turn[:, :, None] * x
    for j in range(n):
        dX[:, j] += h_pre[:, j:j + 1] * dF
        for i in range(n):
            dX[:, j] += h_res[:, i, j:j + 1] * g[:, i]
    with np.errstate(invalid="ignore", divide="ignore"):
        da = np.sum(dz * logits / r, axis=0)
    db = np.sum(dz, axis=0)
    return {"dX": dX.reshape(B, n * C), "dphi": x.reshape(B, n * C).T @ dl,
            "dalpha": np.array([da[:n].sum(), da[n:2 * n].sum(), da[2 * n:].sum()]),
            "db_pre": db[:n], "db_post": db[n:2 * n], "db_res": db[2 * n:], "dz": dz, "dlogits": dl}


def embed(tokens, table, scale, n):
    """X_0 [B, n*C] (not rounded): scale * table[token] in every stream, zeros
    for a token outside the table."""
    table = np.asarray(table, np.float64)
    out = np.zeros((len(tokens), n, table.shape[1]))
    for b, t in enumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[b] = scale * table[t]
    return out.reshape(len(tokens), -1)


def embed_bwd(tokens, dx0, scale, n, C, V):
    """dtable [V, C]."""
    g = np.asarray(dx0, np.float64).reshape(-1, n, C)
    out = np.zeros((V, C))
    for b, t in enumerate(tokens):
        if 0 <= t < V:
            out[t] += scale * g[b].sum(axis=0)
    return out
