"""A training step of the mHC calls in 64 bits that rounds what the step
stores (streams, F, their gradients: bf16; X_t as its checkpoint holds it)
where the step does, so that it can be compared with the step closely."""

import numpy as np
import torch

import oracle
from oracle import backward


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def step(p, B, n, C, ckpt, rounded=bf16):
    """p: tokens, table, scale, alphas, layers (phi, b_pre, b_post, b_res, w:
    float64 arrays), out [B, C].  Returns the gradients by name and, for each
    layer's small vectors, `noise`: sqrt(sum over rows of (the largest
    sqrt(sum_c (G_i X_j)^2, (G_i F)^2 or (dF_pre X_j)^2))^2)."""
    L = len(p["layers"])
    X, F, co, kept = [bf16(backward.embed(p["tokens"], p["table"], p["scale"], n))], [], [], []
    for q in p["layers"]:
        c = oracle.coefficients(X[-1], q["phi"], *p["alphas"], q["b_pre"], q["b_post"], q["b_res"], n, C)
        h_pre, h_post, h_res = oracle.split_h(c["H"], n)
        F.append(bf16(rounded(oracle.pre_mix(X[-1], h_pre, n, C)) * q["w"]))
        co.append(c)
        kept.append(backward.ckpt_decode(*backward.ckpt_encode(X[-1], n, C), n, C) if ckpt else X[-1])
        X.append(rounded(oracle.post_res(X[-1], F[-1], h_post, h_res, n, C)))
    G = np.repeat(p["out"][:, None], n, axis=1).reshape(B, n * C)
    got, noise = {}, {}
    for l in reversed(range(L)):
        q, c, x = p["layers"][l], co[l], kept[l]
        dF, dH = backward.post_res_bwd(x, F[l], c["H"], G, n, C)
        dFp = bf16(rounded(dF) * q["w"])
        d = backward.coeffs_pre_bwd(x, q["phi"], p["alphas"], (q["b_pre"], q["b_post"], q["b_res"]), c["logits"], c["r"],
                                    c["H"], G, dH, dFp, n, C)
        g2, x2 = (np.square(t).reshape(B, n, C) for t in (G, x))
        size = np.maximum(np.max(g2 @ x2.transpose(0, 2, 1), axis=(1, 2)),
                          np.maximum(np.max(g2 @ np.square(F[l])[:, :, None], axis=(1, 2)),
                                     np.max(x2 @ np.square(dFp)[:, :, None], axis=(1, 2))))
        noise[l] = float(np.sqrt(size.sum()))
        got.update({f"{k}{l}": d[k] for k in ("dphi", "dalpha", "db_pre", "db_post", "db_res")})
        G = rounded(d["dX"])
    got["dtable"] = backward.embed_bwd(p["tokens"], G, p["scale"], n, C, p["table"].shape[0])
    return got, noise
