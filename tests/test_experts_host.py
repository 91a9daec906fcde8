"""Refusals and host functions of the calls around a layer of experts, without
a GPU (fake device addresses, nothing launched), as tests/test_train_host.py
does for the training calls."""

import pytest
import torch

import manifold_constrained_hyper_amd as mhc

pytestmark = pytest.mark.cpu

STEP = 1 << 38
OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = (mhc.MHC_OK, mhc.MHC_ERR_INVALID_ARG, mhc.MHC_ERR_UNSUPPORTED,
                                            mhc.MHC_ERR_WORKSPACE, mhc.MHC_ERR_HIP)
SIZE = {"B": 16, "C": 40, "E": 12, "k": 4}

# Each call: the sizes it takes, and its tensors: name, what it is, its
# alignment ("in?", "out?": may be left out).
CALLS = {
    "mhc_rmsnorm": ("B C", "x:in:16 shortcut:in?:16 weight:in?:16 sum:out?:16 y:out?:16 codes:out?:16 scales:out?:1 "
                           "rstd:out?:4"),
    "mhc_rmsnorm_bwd": ("B C", "sum:in:16 weight:in?:16 rstd:in:4 dy:in:16 dsum:in?:16 dx:out:16 dweight:out?:16 "
                               "workspace:out:16"),
    "mhc_route": ("B E k", "logits:in:4 bias:in?:4 ids:out:4 weights:out:4"),
    "mhc_route_bwd": ("B E k", "logits:in:4 ids:in:4 dweights:in:4 dlogits:out:4"),
    "mhc_experts_order": ("B k E", "ids:in:4 slots:out:4 offsets:out:4 workspace:out:16"),
    "mhc_experts_gather": ("B k C", "X:in:16 slots:in:4 rows:out:16"),
    "mhc_experts_gather_ckpt": ("B k C", "codes:in:16 scales:in:1 slots:in:4 row_codes:out:16 row_scales:out:1"),
    "mhc_experts_combine": ("B k C", "Y:in:16 slots:in:4 weights:in?:4 shared:in?:16 F_out:out:16"),
    "mhc_experts_combine_bwd": ("B k C", "Y:in:16 slots:in:4 weights:in:4 dF_out:in:16 dY:out:16 dweights:out:4"),
}


def _tensors(name):
    return [t.split(":") for t in CALLS[name][1].split()]


def _where(name):
    return {t: (1 << 44) + (i + 1) * STEP for i, (t, _, _) in enumerate(_tensors(name))}


def _workspace(name, s):
    if name == "mhc_rmsnorm_bwd":
        return mhc.mhc_rmsnorm_bwd_workspace_size(s["B"], s["C"])
    return mhc.mhc_experts_order_workspace_size(s["B"], s["k"], s["E"])


def _call(name, ws_bytes=None, **over):
    s = {**SIZE, **{k: over.pop(k) for k in list(over) if k in SIZE}}
    tensors = {**_where(name), **{k: over.pop(k) for k in list(over) if k in _where(name)}}
    if "workspace" in tensors:
        over["workspace_bytes"] = _workspace(name, s) if ws_bytes is None else ws_bytes
    return getattr(mhc, name)(*(s[k] for k in CALLS[name][0].split()), **tensors, **over, stream=0, check=False)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_shapes_and_pointers(name):
    assert _call(name, B=-1) == INVALID
    assert _call(name, B=1 << 31) == UNSUPPORTED
    takes = CALLS[name][0].split()
    if "C" in takes:
        assert _call(name, C=0) == INVALID
        assert _call(name, C=-8) == INVALID
        assert _call(name, C=12) == UNSUPPORTED
        assert _call(name, C=1 << 31) == UNSUPPORTED
        assert _call(name, B=1 << 26, C=1 << 16) == UNSUPPORTED
    if "E" in takes:
        assert _call(name, E=0) == INVALID
        assert _call(name, E=1025) == UNSUPPORTED
    if "k" in takes:
        assert _call(name, k=0) == INVALID
        assert _call(name, k=33, **({"E": 40} if "E" in takes else {})) == UNSUPPORTED
    if takes[1:2] == ["k"]:                       # pairs are counted in 32 bits
        assert _call(name, B=1 << 29, k=4) == UNSUPPORTED
    for what, kind, align in _tensors(name):
        at = _where(name)
        if not kind.endswith("?") and what != "workspace":
            assert _call(name, **{what: None}) == INVALID, what
        if int(align) > 1:
            assert _call(name, **{what: at[what] + int(align) // 2}) == UNSUPPORTED, what
        if kind.startswith("out"):                # an output over each other tensor
            for other in at:
                if other != what:
                    assert _call(name, **{what: at[other]}) == INVALID, (what, other)


def test_output_over_the_end_of_an_input():
    for name in sorted(CALLS):
        at, inputs = _where(name), [t for t in _tensors(name) if t[1].startswith("in")]
        big = {"B": 1 << 16}
        for what, kind, _ in _tensors(name):
            if not kind.startswith("out"):
                continue
            for other, _, _ in inputs:
                if other in ("weight", "bias"):   # as long as a row, whatever B
                    continue
                assert _call(name, **big, **{what: at[other] + 1024}) == INVALID, (name, what, other)


@pytest.mark.parametrize("name", ["mhc_rmsnorm_bwd", "mhc_experts_order"])
def test_workspace(name):
    size = _workspace(name, SIZE)
    assert size > 0
    assert _call(name, ws_bytes=size - 1) == WORKSPACE
    assert _call(name, ws_bytes=0) == WORKSPACE
    assert _call(name, workspace=None) == INVALID


def test_rmsnorm_outputs():
    none = {w: None for w in ("shortcut", "weight", "sum", "y", "codes", "scales", "rstd")}
    assert _call("mhc_rmsnorm", **none) == INVALID                       # nothing asked for
    assert _call("mhc_rmsnorm", y=None, codes=None) == INVALID           # scales without codes
    assert _call("mhc_rmsnorm", scales=None) == INVALID
    assert _call("mhc_rmsnorm", shortcut=None) == INVALID                # a sum of one
    for eps in (-1e-9, float("nan"), float("inf")):
        assert _call("mhc_rmsnorm", eps=eps) == INVALID
    assert _call("mhc_rmsnorm", C=65544) == UNSUPPORTED
    assert _call("mhc_rmsnorm_bwd", C=65544) == UNSUPPORTED


def test_route_choices():
    for bad in (dict(groups=0), dict(groups=5), dict(groups=-1), dict(groups=3, top_groups=4), dict(top_groups=0),
                dict(groups=6, top_groups=1), dict(k=13), dict(groups=24)):
        assert _call("mhc_route", **bad) == INVALID, bad
    assert _call("mhc_route", E=1024, groups=128, top_groups=128) == UNSUPPORTED
    lib = mhc.load()
    assert lib.mhc_route(16, 12, 4, 1, 1, 8, 1.0, 1 << 40, None, 1 << 41, 1 << 42, 0) == INVALID     # a flag of nothing
    assert lib.mhc_route_bwd(16, 12, 4, -1, 1.0, 1 << 40, 1 << 41, 1 << 42, 1 << 43, 0) == INVALID
    assert _call("mhc_route", bf16=True, logits=(1 << 44) + 1) == UNSUPPORTED
    assert _call("mhc_route_bwd", k=13) == INVALID


def test_no_rows():
    """B = 0: nothing to do and no pointer needed, except for what is zeros then."""
    for name in sorted(CALLS):
        none = {w: None for w, _, _ in _tensors(name)}
        if name == "mhc_experts_order":
            assert _call(name, B=0, **none) == INVALID
        else:
            assert _call(name, B=0, **none) == OK, name
    assert mhc.mhc_rmsnorm_bwd_workspace_size(0, 40) == 0
    assert mhc.mhc_rmsnorm_bwd_workspace_size(16, 41) == 0
    assert mhc.mhc_rmsnorm_bwd_workspace_size(16, 65544) == 0
    assert mhc.mhc_experts_order_workspace_size(0, 4, 12) == 0
    assert mhc.mhc_experts_order_workspace_size(16, 33, 12) == 0
    assert mhc.mhc_experts_order_workspace_size(16, 4, 1025) == 0


def test_binding_refuses_wrong_tensors():
    B, C, E, k = 4, 16, 8, 2
    x = torch.zeros(B, C, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: 64 bytes, the call needs 128"):
        mhc.mhc_rmsnorm(B, C, x[:2], None, y=1 << 40, stream=0)
    with pytest.raises(ValueError, match="weight: element size 2"):
        mhc.mhc_rmsnorm(B, C, 1 << 40, x[0], y=1 << 41, stream=0)
    with pytest.raises(ValueError, match="device tensors"):
        mhc.mhc_rmsnorm(B, C, x, None, y=1 << 41, stream=0)
    with pytest.raises(ValueError, match="dweight: 32 bytes, the call needs 64"):
        mhc.mhc_rmsnorm_bwd(B, C, 1 << 40, None, 1 << 41, 1 << 42, 1 << 43, dweight=torch.zeros(8), stream=0)
    with pytest.raises(ValueError, match="logits: torch.float16"):
        mhc.mhc_route(B, E, k, torch.zeros(B, E, dtype=torch.float16), 1 << 41, 1 << 42, stream=0)
    with pytest.raises(ValueError, match="ids: element size 8"):
        mhc.mhc_route(B, E, k, 1 << 40, torch.zeros(B, k, dtype=torch.int64), 1 << 42, stream=0)
    with pytest.raises(ValueError, match="dlogits: element size 4"):
        mhc.mhc_route_bwd(B, E, k, 1 << 40, 1 << 41, 1 << 42, torch.zeros(B, E), bf16=True, stream=0)
    with pytest.raises(ValueError, match="offsets: 32 bytes, the call needs 36"):
        mhc.mhc_experts_order(B, k, E, 1 << 40, 1 << 41, torch.zeros(E, dtype=torch.int32), 1 << 42, stream=0)
    with pytest.raises(ValueError, match="rows: 128 bytes, the call needs 256"):
        mhc.mhc_experts_gather(B, k, C, 1 << 40, 1 << 41, x, stream=0)
    with pytest.raises(ValueError, match="row_scales: 4 bytes, the call needs 8"):
        mhc.mhc_experts_gather_ckpt(B, k, C, 1 << 40, 1 << 41, 1 << 42, 1 << 43, torch.zeros(4, dtype=torch.uint8),
                                    stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        mhc.mhc_experts_combine(B, k, C, torch.zeros(4 * B, C, dtype=torch.bfloat16)[::2], 1 << 41, None, 1 << 42,
                                stream=0)
    with pytest.raises(ValueError, match="dweights: 16 bytes, the call needs 32"):
        mhc.mhc_experts_combine_bwd(B, k, C, 1 << 40, 1 << 41, 1 << 42, 1 << 43, 1 << 44, torch.zeros(4), stream=0)


# Types of the same size as each tensor's own, which hold other numbers.
OTHERS = {torch.bfloat16: (torch.float16,), torch.float32: (torch.int32,), torch.int32: (torch.float32,),
          "codes": (torch.float8_e5m2, torch.int8, torch.float8_e8m0fnu),
          "scales": (torch.float8_e4m3fn, torch.bool)}
TYPES = {torch.float32: "weight rstd dweight bias logits weights dweights dlogits".split(),
         torch.int32: "ids slots offsets".split(), "codes": ["codes"], "scales": ["scales"]}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_refuses_other_numbers(name):
    """A tensor of another type is refused, not read as what it is not; raw bytes and words are not, and a gather copies
    what it is given."""
    s = {"B": 4, "C": 32, "E": 8, "k": 2}
    for what, _, _ in _tensors(name):
        if what == "workspace" or "gather" in name and what != "slots":
            continue
        kind = next((k for k, names in TYPES.items() if what in names), torch.bfloat16)
        for dtype in OTHERS[kind]:
            with pytest.raises(ValueError, match=f"{what}: {dtype}"):
                _call(name, **s, **{what: torch.zeros(4096, dtype=dtype)})
        own = {"codes": torch.float8_e4m3fn, "scales": torch.float8_e8m0fnu}.get(kind, kind)
        for dtype in (own, torch.uint8, *([torch.int16] if own == torch.bfloat16 else [])):  # (but are on the host)
            with pytest.raises(ValueError, match="device tensors"):
                _call(name, **s, **{what: torch.zeros(4096 * 4, dtype=dtype)})


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a host without a HIP device (fake addresses)")
def test_no_device_is_mhc_err_hip():
    for name in sorted(CALLS):
        assert _call(name) == HIP, name
        optional = {w: None for w, kind, _ in _tensors(name) if kind.endswith("?") and w != "y"}
        assert _call(name, **optional) == HIP, name
    assert _call("mhc_rmsnorm", y=None) == HIP
    assert _call("mhc_rmsnorm_bwd", dweight=None, workspace=None, ws_bytes=0) == HIP
    assert _call("mhc_rmsnorm_bwd", B=0) == HIP and _call("mhc_experts_order", B=0) == HIP  # zeros
    assert _call("mhc_route", E=1024, k=32, groups=64, top_groups=2) == HIP
