"""What the operators around a layer of experts cost, and what they compute.

Between the layer input that the residual stream gives (F_pre) and the layer output that it takes back
(F_out) a layer of experts normalises its input, chooses each row's experts, brings the rows into the
experts' order, and joins what the experts made of them.  Three operators, each as a user's program calls
it (`own` true: the library's calls) and in a plain form of elementary torch operations (`own` false):

  rmsnorm   root-mean-square norm of a row with the shortcut's addition, to bf16 or to 8 bits (E4M3 codes
            and one power-of-two scale byte for 32 channels); "rmsnorm_bwd": its gradients
  route     the k experts of each row from its logits: sigmoid or softmax scores, a bias that only moves
            the choice, groups of experts, renormalised weights; "route_bwd": the logits' gradient
  experts   "gather": places of the (row, expert) pairs in the experts' order, and the rows copied there;
            "combine": the experts' outputs weighted and summed; "combine_bwd": its gradients

"out" and "x" say what a row is held in ("bf16", or "e4m3": codes and scale bytes).
"""

import math

import torch

own = False

BLOCK = 32            # channels that share one scale byte
EPS = 1e-5
GRAD = 2.0 ** -6      # size of the gradients that arrive from above
LARGEST = 3.4028234663852886e38   # fp32's: what a logit of plus infinity counts as


# -- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # A whole batch's layer input added to the shortcut, normalised into the 8-bit products' operand.
        {"name": "rmsnorm_large_e4m3", "op": "rmsnorm", "B": 16384, "C": 7168, "shortcut": True, "out": "e4m3"},
        # One token of a decoding step: latency.
        {"name": "rmsnorm_single", "op": "rmsnorm", "B": 1, "C": 7168, "shortcut": True, "out": "bf16"},
        # The same batch on its way back in a training step, with the shortcut's own gradient.
        {"name": "rmsnorm_bwd_large", "op": "rmsnorm_bwd", "B": 16384, "C": 7168, "shortcut": True},
        # A short ragged batch with a hidden size that ends inside a block of 32 channels.
        {"name": "rmsnorm_bwd_ragged", "op": "rmsnorm_bwd", "B": 1001, "C": 1000, "shortcut": False},
        # The whole batch's choice: sigmoid scores, balanced by a bias, half of eight groups.
        {"name": "route_large", "op": "route", "B": 16384, "E": 256, "k": 8, "groups": 8, "top_groups": 4,
         "softmax": False, "bias": True, "renorm": True, "scale": 2.5, "logits": "fp32", "off": 0},
        # One token's choice: latency.
        {"name": "route_single", "op": "route", "B": 1, "E": 256, "k": 8, "groups": 8, "top_groups": 4,
         "softmax": False, "bias": True, "renorm": True, "scale": 2.5, "logits": "fp32", "off": 0},
        # Softmax over an odd number of experts, as the weights stand: every logit has a gradient.
        {"name": "route_bwd_odd", "op": "route_bwd", "B": 16383, "E": 100, "k": 6, "softmax": True, "renorm": False,
         "scale": 1.0, "logits": "bf16", "off": 0},
        # The whole batch's normalised rows to their experts, in 8 bits.
        {"name": "gather_large_e4m3", "op": "gather", "B": 16384, "k": 8, "C": 7168, "E": 256, "x": "e4m3"},
        # A decoding step of 64 requests.
        {"name": "gather_few", "op": "gather", "B": 64, "k": 8, "C": 7168, "E": 256, "x": "bf16"},
        # The whole batch's expert outputs back into F_out.
        {"name": "combine_large", "op": "combine", "B": 16384, "k": 8, "C": 7168, "shared": True},
        # One token's.
        {"name": "combine_single", "op": "combine", "B": 1, "k": 8, "C": 7168, "shared": True},
        # And the way back: the gradients of the experts' outputs and of the weights.
        {"name": "combine_bwd_large", "op": "combine_bwd", "B": 16384, "k": 8, "C": 7168},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm", "rmsnorm_bwd", "route", "route", "route_bwd", "gather", "combine",
                     "combine_bwd"])
    if op in ("rmsnorm", "rmsnorm_bwd"):
        C = 8 * _log_uniform(rng, 4, 1024)
        case = {"op": op, "B": _log_uniform(rng, 1, min(65536, 16384 * 7168 // C)), "C": C,
                "shortcut": rng.random() < 0.6}
        if op == "rmsnorm":
            case["out"] = rng.choice(["bf16", "e4m3"])
        return case
    if op in ("route", "route_bwd"):
        E = _log_uniform(rng, 2, 512)
        case = {"op": op, "B": _log_uniform(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 16)),
                "softmax": rng.random() < 0.5, "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 1.0, 2.5]),
                "logits": rng.choice(["fp32", "bf16"]), "off": rng.choice([0, 0, 0, 1, E // 4])}
        if op == "route":
            groups = rng.choice([g for g in range(1, min(E, 16) + 1) if E % g == 0])
            case["groups"], case["top_groups"] = groups, rng.randint(1, groups)
            case["k"] = min(case["k"], case["top_groups"] * (E // groups))
            case["bias"] = rng.random() < 0.5
        elif case["renorm"]:        # weights that add up to a constant have a gradient from two on
            case["k"], case["off"] = max(2, case["k"]), min(case["off"], E - 2)
        return case
    k = rng.randint(1, 12)
    C = 8 * _log_uniform(rng, 4, 1024)
    case = {"op": op, "B": _log_uniform(rng, 1, min(16384, 16384 * 8 * 7168 // (k * C))), "k": k, "C": C}
    if op == "gather":
        case["E"] = _log_uniform(rng, k, 512)
        case["x"] = rng.choice(["bf16", "e4m3"])
        if case["x"] == "bf16":
            case["B"] = max(1, min(case["B"], 16384 * 4 * 7168 // (k * C)))
    elif op == "combine":
        case["shared"] = rng.random() < 0.5
    return case


def work(case):
    op, B = case["op"], case["B"]
    if op in ("rmsnorm", "rmsnorm_bwd"):
        C = case["C"]
        row = 2 * C                                       # a row in bf16
        held = C + -(-C // BLOCK)                         # in 8 bits
        if op == "rmsnorm":                               # x, shortcut in; sum, y, rstd out
            out = held if case["out"] == "e4m3" else row
            return {"bytes": B * (row + (2 * row if case["shortcut"] else 0) + out + 4) + 4 * C, "flops": 5 * B * C}
        # the normalised rows, dy, the shortcut's gradient, rstd in; dx, dweight out
        return {"bytes": B * (3 * row + (row if case["shortcut"] else 0) + 4) + 8 * C, "flops": 9 * B * C}
    if op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        one = 4 if case["logits"] == "fp32" else 2
        if op == "route":                                 # logits, bias in; ids, weights out
            return {"bytes": B * (one * E + 8 * k) + (4 * E if case["bias"] else 0), "flops": 6 * B * E}
        # the logits (the chosen ones where the others have no gradient), ids, dweights in; dlogits out
        every = case["softmax"] and not case["renorm"]
        return {"bytes": B * (one * (E if every else k) + 8 * k + one * E), "flops": B * (4 * E if every else 12 * k)}
    k, C = case["k"], case["C"]
    if op == "gather":                                    # rows, ids in; places, rows in the experts' order out
        row = 2 * C if case["x"] == "bf16" else C + -(-C // BLOCK)
        return {"bytes": B * (row + 4 * k + 4 * k + k * row) + 4 * (case["E"] + 1), "flops": B * k}
    if op == "combine":                                   # Y, places, weights, shared in; F_out out
        return {"bytes": B * (2 * k * C + 8 * k + (2 * C if case["shared"] else 0) + 2 * C), "flops": 2 * B * k * C}
    # Y, places, weights, dF_out in; dY, dweights out
    return {"bytes": B * (4 * k * C + 12 * k + 2 * C), "flops": 3 * B * k * C}


# -- inputs -----------------------------------------------------------------------------------------

def prepare(case, seed):
    op, B = case["op"], case["B"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}

    def normal(shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    if op in ("rmsnorm", "rmsnorm_bwd"):
        C = case["C"]
        size = torch.exp2(torch.randn((B, 1), generator=gen, device="cuda"))  # rows of different sizes
        x = torch.randn((B, C), generator=gen, device="cuda") * size
        x[:, ::61] *= 8                                                       # a few channels stand out
        s["x"] = x.to(torch.bfloat16)
        s["weight"] = 1 + normal(C, 0.1, torch.float32)
        if op == "rmsnorm":
            s["shortcut"] = normal((B, C)) if case["shortcut"] else None
        else:
            s["rstd"] = 1 / (s["x"].float().square().mean(1) + EPS).sqrt()
            s["dy"] = normal((B, C), GRAD)
            s["dsum"] = normal((B, C), GRAD) if case["shortcut"] else None
    elif op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        liked = torch.randn(E, generator=gen, device="cuda")                  # experts are not equally wanted
        logits = 1.5 * torch.randn((B, E), generator=gen, device="cuda") + liked
        if case["off"]:                                                       # experts out of service
            logits[:, torch.randperm(E, generator=gen, device="cuda")[:case["off"]]] = -math.inf
        s["logits"] = logits.to(torch.float32 if case["logits"] == "fp32" else torch.bfloat16)
        if op == "route":
            s["bias"] = -0.1 * liked + normal(E, 0.02, torch.float32) if case["bias"] else None
        else:
            s["ids"] = _choose(s["logits"].double(), k)
            s["dweights"] = normal((B, k), GRAD, torch.float32)
    else:
        k, C = case["k"], case["C"]
        E = case.get("E", 4 * k)
        liked = torch.randn((B, E), generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")
        ids = _choose(liked.double(), k)
        if op == "gather":
            x = normal((B, C))
            s["ids"] = ids
            if case["x"] == "bf16":
                s["x"] = x
            else:
                s["codes"], s["scales"] = _pack(x.float())
        else:
            s["slots"] = _order(ids, E)[0]
            s["Y"] = normal((B * k, C))
            s["weights"] = torch.rand((B, k), generator=gen, device="cuda") + 0.1
            s["weights"] /= s["weights"].sum(1, keepdim=True)
            if op == "combine":
                s["shared"] = normal((B, C)) if case["shared"] else None
            else:
                s["dF_out"] = normal((B, C), GRAD)
    if own:
        _buffers(s)
    return s


def _buffers(s):
    """What a user's program allocates once for these calls: outputs and workspaces."""
    import manifold_constrained_hyper_amd as mhc

    case = s["case"]
    op, B, k, C = case["op"], case["B"], case.get("k"), case.get("C")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "rmsnorm":
        s["rstd"] = empty(B)
        s["sum"] = empty(B, C, dtype=torch.bfloat16) if case["shortcut"] else None
        bf16 = case["out"] == "bf16"
        s["y"] = empty(B, C, dtype=torch.bfloat16) if bf16 else None
        s["codes"] = None if bf16 else empty(B, C, dtype=torch.uint8)
        s["scales"] = None if bf16 else empty(B, mhc.mhc_ckpt_scales_per_row(1, C), dtype=torch.uint8)
    elif op == "rmsnorm_bwd":
        s["dx"], s["dweight"] = empty(B, C, dtype=torch.bfloat16), empty(C)
        s["ws"] = empty(max(16, mhc.mhc_rmsnorm_bwd_workspace_size(B, C)), dtype=torch.uint8)
    elif op == "route":
        s["ids"], s["weights"] = empty(B, k, dtype=torch.int32), empty(B, k)
    elif op == "route_bwd":
        s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "gather":
        s["slots"], s["offsets"] = empty(B, k, dtype=torch.int32), empty(case["E"] + 1, dtype=torch.int32)
        s["ws"] = empty(max(16, mhc.mhc_experts_order_workspace_size(B, k, case["E"])), dtype=torch.uint8)
        if case["x"] == "bf16":
            s["rows"] = empty(B * k, C, dtype=torch.bfloat16)
        else:
            s["rows"] = empty(B * k, C, dtype=torch.uint8)
            s["rows_scales"] = empty(B * k, s["scales"].shape[1], dtype=torch.uint8)
    elif op == "combine":
        s["F_out"] = empty(B, C, dtype=torch.bfloat16)
    else:
        s["dY"], s["dweights"] = empty(B * k, C, dtype=torch.bfloat16), empty(B, k)


# -- one pass ---------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"rmsnorm": _rmsnorm, "rmsnorm_bwd": _rmsnorm_bwd, "route": _route, "route_bwd": _route_bwd,
            "gather": _gather, "combine": _combine, "combine_bwd": _combine_bwd}[s["case"]["op"]](s)


def _held(codes, scales):
    """Codes and scale bytes as the numbers that they are: E4M3, and powers of two."""
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _own(s):
    import manifold_constrained_hyper_amd as mhc

    case = s["case"]
    op, B, k, C, E = case["op"], case["B"], case.get("k"), case.get("C"), case.get("E")
    if op == "rmsnorm":
        mhc.mhc_rmsnorm(B, C, s["x"], s["weight"], y=s["y"], codes=s["codes"], scales=s["scales"],
                        shortcut=s["shortcut"], sum=s["sum"], rstd=s["rstd"], eps=EPS)
        out = {"rstd": s["rstd"], "sum": s["sum"], "y": s["y"]}
        if case["out"] == "e4m3":
            out["codes"], out["scales"] = _held(s["codes"], s["scales"])
        return out
    if op == "rmsnorm_bwd":
        mhc.mhc_rmsnorm_bwd(B, C, s["x"], s["weight"], s["rstd"], s["dy"], s["dx"], dweight=s["dweight"],
                            workspace=s["ws"], dsum=s["dsum"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "route":
        mhc.mhc_route(B, E, k, s["logits"], s["ids"], s["weights"], bias=s["bias"], groups=case["groups"],
                      top_groups=case["top_groups"], softmax=case["softmax"], renorm=case["renorm"],
                      scale=case["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if op == "route_bwd":
        mhc.mhc_route_bwd(B, E, k, s["logits"], s["ids"], s["dweights"], s["dlogits"], softmax=case["softmax"],
                          renorm=case["renorm"], scale=case["scale"])
        return {"dlogits": s["dlogits"]}
    if op == "gather":
        mhc.mhc_experts_order(B, k, E, s["ids"], s["slots"], s["offsets"], s["ws"])
        out = {"slots": s["slots"], "offsets": s["offsets"]}
        if case["x"] == "bf16":
            mhc.mhc_experts_gather(B, k, C, s["x"], s["slots"], s["rows"])
            out["rows"] = s["rows"]
        else:
            mhc.mhc_experts_gather_ckpt(B, k, C, s["codes"], s["scales"], s["slots"], s["rows"], s["rows_scales"])
            out["rows"], out["scales"] = _held(s["rows"], s["rows_scales"])
        return out
    if op == "combine":
        mhc.mhc_experts_combine(B, k, C, s["Y"], s["slots"], s["weights"], s["F_out"], shared=s["shared"])
        return {"F_out": s["F_out"]}
    mhc.mhc_experts_combine_bwd(B, k, C, s["Y"], s["slots"], s["weights"], s["dF_out"], s["dY"], s["dweights"])
    return {"dY": s["dY"], "dweights": s["dweights"]}


# -- plain forms ------------------------------------------------------------------------------------

def _pack(y):
    """E4M3 codes and scale bytes of rows in 32 bits: the least power of two 2^e >= 2^-126 with |y| <= 448 * 2^e
    in the block; the scale byte is e + 127."""
    B, C = y.shape
    blocks = -(-C // BLOCK)
    y = torch.nn.functional.pad(y, (0, blocks * BLOCK - C)).reshape(B, blocks, BLOCK)
    m, p = torch.frexp(y.abs().amax(2))
    e = torch.where(m > 0.875, p - 8, p - 9).clamp_(min=-126)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    q = (y * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(B, blocks * BLOCK)[:, :C].contiguous(), (e + 127).to(torch.uint8)


def _rmsnorm(s):
    x, out = s["x"].float(), {}
    if s["shortcut"] is not None:
        out["sum"] = (x + s["shortcut"].float()).to(torch.bfloat16)
        x = out["sum"].float()          # what is normalised is the sum that is kept
    rstd = 1 / (x.square().mean(1) + EPS).sqrt()
    y = x * rstd[:, None] * s["weight"]
    out["rstd"] = rstd
    if s["case"]["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["codes"], out["scales"] = _held(*_pack(y))
    return out


def _rmsnorm_bwd(s):
    n = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = (g - n * (g * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * n).sum(0)}


def _choose(score, k):
    """The k best of each row, the lowest index first where scores are equal; -1 where there are no more."""
    best, at = torch.sort(score, dim=1, descending=True, stable=True)
    return torch.where(best[:, :k] > -math.inf, at[:, :k], -1).to(torch.int32)


def _clean(logits, dtype):
    """Logits with NaN (no expert, as minus infinity) and plus infinity (the largest number) out of the way."""
    x = logits.to(dtype)
    return torch.where(x.isnan(), -math.inf, x).clamp(max=LARGEST)


def _softmax(x):
    """Over rows that may be all minus infinity: zeros there."""
    top = x.amax(1, keepdim=True)
    e = torch.where(x > -math.inf, (x - torch.where(top > -math.inf, top, 0)).exp(), 0)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1)


def _log_sigmoid(x):
    return x.clamp(max=0) - (-x.abs()).exp().log1p()


def _route(s):
    c = s["case"]
    B, E, k, groups = c["B"], c["E"], c["k"], c["groups"]
    x = _clean(s["logits"], torch.float64)      # in 64 bits: equal scores are equal, near ones in their order
    there = x > -math.inf
    score = _softmax(x) if c["softmax"] else 1 / (1 + (-x).exp())
    choice = torch.where(there, score if s["bias"] is None else score + s["bias"].double(), -math.inf)
    if c["top_groups"] < groups:
        best = torch.sort(choice.reshape(B, groups, E // groups), dim=2, descending=True).values
        rank = best[:, :, 0]
        if s["bias"] is not None and E > groups:
            rank = rank + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0)
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros(B, groups, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        choice = torch.where(mask.repeat_interleave(E // groups, 1), choice, -math.inf)
    ids = _choose(choice, k)
    at = ids.long().clamp(min=0)
    if c["renorm"]:
        chosen = torch.where(ids >= 0, x.gather(1, at), -math.inf)
        weights = _softmax(chosen if c["softmax"] else torch.where(ids >= 0, _log_sigmoid(x.gather(1, at)), -math.inf))
    else:
        weights = torch.where(ids >= 0, score.gather(1, at), 0)
    return {"ids": ids, "weights": (weights * c["scale"]).float()}


def _route_bwd(s):
    c = s["case"]
    x = _clean(s["logits"], torch.float32)
    there = s["ids"] >= 0
    at = s["ids"].long().clamp(min=0)
    dw = torch.where(there, s["dweights"] * c["scale"], 0)
    chosen = torch.where(there, x.gather(1, at), -math.inf)
    if c["softmax"] and not c["renorm"]:
        p = _softmax(x)
        d = -p * (p.gather(1, at) * dw).sum(1, keepdim=True)
        d = d.scatter_add_(1, at, p.gather(1, at) * dw)
    else:
        if c["renorm"]:
            w = _softmax(chosen if c["softmax"] else torch.where(there, _log_sigmoid(chosen), -math.inf))
            g = w * (dw - (w * dw).sum(1, keepdim=True))
        else:
            g = dw / (1 + (-chosen).exp())
        if not c["softmax"]:
            g = g / (1 + chosen.exp())
        d = torch.zeros_like(x).scatter_add_(1, at, torch.where(there, g, 0))
    return {"dlogits": d.to(s["logits"].dtype)}


def _order(ids, E):
    """Places of the (row, expert) pairs in the order of their experts, of equal ones in the order of the rows;
    the experts' first places; and the pairs in that order."""
    flat = ids.reshape(-1).long()
    pairs = torch.argsort(flat, stable=True)
    slots = torch.empty_like(pairs)
    slots[pairs] = torch.arange(len(pairs), device=pairs.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=pairs.device)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return slots.reshape(ids.shape).to(torch.int32), offsets.to(torch.int32), pairs


def _gather(s):
    c = s["case"]
    slots, offsets, pairs = _order(s["ids"], c["E"])
    out = {"slots": slots, "offsets": offsets}
    rows = pairs // c["k"]
    if c["x"] == "bf16":
        out["rows"] = s["x"][rows]
    else:
        out["rows"], out["scales"] = _held(s["codes"][rows], s["scales"][rows])
    return out


def _combine(s):
    out = (s["Y"][s["slots"].long()].float() * s["weights"][..., None]).sum(1)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return {"F_out": out.to(torch.bfloat16)}


def _combine_bwd(s):
    slots, d = s["slots"].long(), s["dF_out"].float()
    dY = torch.empty_like(s["Y"])
    dY[slots.reshape(-1)] = (s["weights"][..., None] * d[:, None]).to(torch.bfloat16).reshape(dY.shape)
    return {"dY": dY, "dweights": (s["Y"][slots].float() * d[:, None]).sum(2)}


# -- the definitions in 64 bits ---------------------------------------------------------------------

def _parts(rows, a_row):
    """Row ranges of about 2 GiB of 64-bit values each."""
    step = max(1, (1 << 28) // max(1, a_row))
    return [(lo, min(rows, lo + step)) for lo in range(0, rows, step)]


def _e4m3_64(v):
    """The E4M3 value nearest to v, ties to the even code: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    return {"rmsnorm": _exact_rmsnorm, "rmsnorm_bwd": _exact_rmsnorm_bwd, "route": _exact_route,
            "route_bwd": _exact_route_bwd, "gather": _exact_gather, "combine": _exact_combine,
            "combine_bwd": _exact_combine_bwd}[case["op"]](s)


def _exact_rmsnorm(s):
    c = s["case"]
    B, C = c["B"], c["C"]
    got = []
    for lo, hi in _parts(B, C):
        one = {}
        x = s["x"][lo:hi].double()
        if s["shortcut"] is not None:
            one["sum"] = x + s["shortcut"][lo:hi].double()
            x = one["sum"].to(torch.float32).to(torch.bfloat16).double()   # two bf16 values' sum, as it is kept
        norm = torch.linalg.vector_norm(x, dim=1)
        one["rstd"] = (norm * norm / C + EPS) ** -0.5
        y = s["weight"].double() * x * one["rstd"][:, None]
        if c["out"] == "bf16":
            one["y"] = y
        else:
            one["codes"] = torch.empty_like(y)
            one["scales"] = torch.empty(hi - lo, -(-C // BLOCK), dtype=torch.float64, device="cuda")
            for k, at in enumerate(range(0, C, BLOCK)):
                v = y[:, at:at + BLOCK]
                power = torch.ceil(torch.log2(v.abs().amax(1) / 448)).clamp(min=-126)
                one["scales"][:, k] = torch.exp2(power)
                one["codes"][:, at:at + BLOCK] = _e4m3_64(v / torch.exp2(power)[:, None])
        got.append(one)
    return {k: torch.cat([g[k] for g in got]) for k in got[0]}


def _exact_rmsnorm_bwd(s):
    c = s["case"]
    weight = s["weight"].double()
    dx, dweight = [], torch.zeros(c["C"], dtype=torch.float64, device="cuda")
    for lo, hi in _parts(c["B"], 2 * c["C"]):
        x, r, dy = s["x"][lo:hi].double(), s["rstd"][lo:hi, None].double(), s["dy"][lo:hi].double()
        # y_c = w_c x_c r with r = (mean x^2 + eps)^(-1/2), so dr/dx_c = -r^3 x_c / C
        along = (dy * weight * x).sum(1, keepdim=True)
        d = dy * weight * r - along * r ** 3 * x / c["C"]
        dx.append(d if s["dsum"] is None else d + s["dsum"][lo:hi].double())
        dweight += (dy * (x * r)).sum(0)
    return {"dx": torch.cat(dx), "dweight": dweight}


def _scores_64(x, softmax):
    """Scores of logits that may be minus infinity (no expert)."""
    if softmax:
        return torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
    return torch.sigmoid(x)


def _exact_route(s):
    """The weights of the experts that the scores choose, picked one after the other."""
    c = s["case"]
    B, E, k = c["B"], c["E"], c["k"]
    score = _scores_64(s["logits"].double(), c["softmax"])
    choice = score + (0 if s["bias"] is None else s["bias"].double())
    choice[s["logits"] == -math.inf] = -math.inf
    if c["top_groups"] < c["groups"]:
        each = choice.reshape(B, c["groups"], -1)
        first = each.amax(2)
        if s["bias"] is not None and each.shape[2] > 1:
            rest = each.clone().scatter_(2, each.argmax(2, keepdim=True), -math.inf).amax(2)
            first = first + rest.masked_fill(rest == -math.inf, 0.0)
        kept = torch.zeros_like(first, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            at = _first_best(first, kept)
            kept[torch.arange(B, device="cuda"), at] = True
        choice[~kept[:, :, None].expand_as(each).reshape(B, E)] = -math.inf
    taken = torch.zeros_like(choice, dtype=torch.bool)
    weights = torch.zeros(B, k, dtype=torch.float64, device="cuda")
    rows = torch.arange(B, device="cuda")
    for j in range(k):
        at = _first_best(choice, taken)
        real = choice[rows, at].gt(-math.inf) & ~taken[rows, at]
        weights[:, j] = torch.where(real, score[rows, at], 0.0)
        taken[rows, at] = True
    if c["renorm"]:
        total = weights.sum(1, keepdim=True)
        weights = weights / torch.where(total > 0, total, 1.0)
    return {"ids": None, "weights": c["scale"] * weights}


def _first_best(score, taken):
    """The lowest index of each row's largest score that is not taken."""
    left = score.masked_fill(taken, -math.inf)
    return (left == left.amax(1, keepdim=True)).to(torch.uint8).argmax(1)


def _exact_route_bwd(s):
    """The weights as a function of the logits, differentiated by autograd."""
    c = s["case"]
    x = s["logits"].double().requires_grad_()
    there = s["ids"] >= 0
    at = s["ids"].long().clamp(min=0)
    if c["softmax"]:
        off = s["logits"] == -math.inf
        e = (x - x.detach().amax(1, keepdim=True)).exp().masked_fill(off, 0.0)
        w = e.gather(1, at) / (1.0 if c["renorm"] else e.sum(1, keepdim=True))
    else:
        w = torch.sigmoid(x.gather(1, at))
    w = w.masked_fill(~there, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    toll = c["scale"] * (w * s["dweights"].double()).sum()
    return {"dlogits": torch.nan_to_num(torch.autograd.grad(toll, x)[0], nan=0.0)}


def _exact_gather(s):
    """A pair's place: the pairs of smaller experts, and the earlier ones of its own."""
    c = s["case"]
    k, E = c["k"], c["E"]
    flat = s["ids"].reshape(-1).long()
    hot = torch.nn.functional.one_hot(flat, E)
    before = hot.cumsum(0).gather(1, flat[:, None])[:, 0] - 1
    place = before + (hot.sum(0).cumsum(0) - hot.sum(0))[flat]
    del hot

    def moved(x):
        out = torch.empty(len(flat), x.shape[1], dtype=torch.float64, device="cuda")
        out[place] = x.repeat_interleave(k, 0)
        return out

    if c["x"] == "bf16":
        return {"slots": None, "offsets": None, "rows": moved(s["x"].double())}
    code = torch.arange(256, device="cuda")
    power, fraction = (code >> 3) & 15, (code & 7).double()
    value = torch.where(power == 0, fraction * 2.0 ** -9, (8 + fraction) * torch.exp2(power.double() - 10))
    value = torch.where(code >= 128, -value, value)
    return {"slots": None, "offsets": None, "rows": moved(value[s["codes"].int()]),
            "scales": moved(torch.exp2(s["scales"].double() - 127))}


def _exact_combine(s):
    c = s["case"]
    out = torch.zeros(c["B"], c["C"], dtype=torch.float64, device="cuda")
    if s["shared"] is not None:
        out += s["shared"]
    for j in range(c["k"]):
        out += s["weights"][:, j, None].double() * s["Y"].index_select(0, s["slots"][:, j])
    return {"F_out": out}


def _exact_combine_bwd(s):
    c = s["case"]
    d = s["dF_out"].double()
    dY = torch.empty(s["Y"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.empty(c["B"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        at = s["slots"][:, j].long()
        dY[at] = s["weights"][:, j, None].double() * d
        dweights[:, j] = (s["Y"][at].double() * d).sum(1)
    return {"dY": dY, "dweights": dweights}
