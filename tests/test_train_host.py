"""Refusals and host functions of the training calls, without a GPU (fake
device addresses, nothing launched), as tests/test_abi_host.py does for the
forward."""

import pytest
import torch

import manifold_constrained_hyper_amd as mhc

pytestmark = pytest.mark.cpu

STEP = 1 << 38
OK, INVALID, UNSUPPORTED, WORKSPACE = (mhc.MHC_OK, mhc.MHC_ERR_INVALID_ARG, mhc.MHC_ERR_UNSUPPORTED,
                                       mhc.MHC_ERR_WORKSPACE)

# Each call's tensors in order: name, what it is ("in" or "out"), the
# alignment it needs, and the positions of host scalars between them.
POST = ["F_out:in:16", "H:in:4", "dX_next:in:16", "dF_out:out:16", "dH:out:4"]
COEF = ["phi:in:16", "=", "=", "=", "b_pre:in:4", "b_post:in:4", "b_res:in:4", "logits:in:4", "r:in:4", "H:in:4",
        "dX_next:in:16", "dH:in:4", "dF_pre:in:16", "dX_t:out:16", "dphi:out:16", "dalpha:out:4", "db_pre:out:4",
        "db_post:out:4", "db_res:out:4", "workspace:out:16"]
CALLS = {
    "mhc_ckpt_pack": ["X_t:in:16", "codes:out:16", "scales:out:1"],
    "mhc_ckpt_unpack": ["codes:in:16", "scales:in:1", "X_t:out:16"],
    "mhc_post_res_bwd": ["X_t:in:16"] + POST,
    "mhc_post_res_bwd_ckpt": ["codes:in:16", "scales:in:1"] + POST,
    "mhc_coeffs_pre_bwd": ["X_t:in:16"] + COEF,
    "mhc_coeffs_pre_bwd_ckpt": ["codes:in:16", "scales:in:1"] + COEF,
    "mhc_embed": ["=V", "tokens:in:8", "table:in:16", "=", "X_0:out:16"],
    "mhc_embed_bwd": ["=V", "tokens:in:8", "dX_0:in:16", "=", "dtable:out:16", "workspace:out:16"],
}


def _tensors(name):
    return [t.split(":") for t in CALLS[name] if not t.startswith("=")]


def _call(name, B=16, n=4, C=40, V=100, ws_bytes=None, **over):
    args, k = [], 0
    for t in CALLS[name]:
        if t.startswith("="):
            args.append(V if t == "=V" else 0.5)
        else:
            what = t.split(":")[0]
            k += 1
            args.append(over.get(what, (1 << 44) + k * STEP))
    kw = {}
    if "workspace:out:16" in CALLS[name]:
        size = (mhc.mhc_embed_bwd_workspace_size(B, n, C, V) if "embed" in name
                else mhc.mhc_coeffs_pre_bwd_workspace_size(B, n, C))
        kw["workspace_bytes"] = size if ws_bytes is None else ws_bytes
    return getattr(mhc, name)(B, n, C, *args, stream=0, check=False, **kw)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_shapes_and_pointers(name):
    assert _call(name, B=-1) == INVALID
    assert _call(name, n=0) == INVALID
    assert _call(name, C=0) == INVALID
    assert _call(name, n=3) == UNSUPPORTED
    assert _call(name, C=12) == UNSUPPORTED
    assert _call(name, B=1 << 31) == UNSUPPORTED
    assert _call(name, C=1 << 30) == UNSUPPORTED
    assert _call(name, B=1 << 30, C=1 << 12) == UNSUPPORTED
    at = {what: (1 << 44) + (k + 1) * STEP for k, (what, _, _) in enumerate(_tensors(name))}
    for what, kind, align in _tensors(name):
        assert _call(name, **{what: None}) == INVALID, what
        if int(align) > 1:
            assert _call(name, **{what: at[what] + int(align) // 2}) == UNSUPPORTED, what
        if kind == "out":          # an output over each other tensor, from either side
            for other in at:
                if other != what:
                    assert _call(name, **{what: at[other]}) == INVALID, (what, other)


@pytest.mark.parametrize("name", [c for c in sorted(CALLS) if "workspace:out:16" in CALLS[c]])
def test_workspace_size(name):
    size = (mhc.mhc_embed_bwd_workspace_size(16, 4, 40, 100) if "embed" in name
            else mhc.mhc_coeffs_pre_bwd_workspace_size(16, 4, 40))
    assert size > 0
    assert _call(name, ws_bytes=size - 1) == WORKSPACE
    assert _call(name, ws_bytes=0) == WORKSPACE


def test_no_rows():
    """B = 0: nothing to do and no pointer needed, except where the gradients
    of parameters are to be zeros."""
    none = {w: None for n in CALLS for w, _, _ in _tensors(n)}
    for name in ("mhc_ckpt_pack", "mhc_ckpt_unpack", "mhc_post_res_bwd", "mhc_post_res_bwd_ckpt", "mhc_embed"):
        assert _call(name, B=0, **none) == OK, name
    for name, outs in (("mhc_coeffs_pre_bwd", ("dphi", "dalpha", "db_pre", "db_post", "db_res")),
                       ("mhc_coeffs_pre_bwd_ckpt", ("dphi", "dalpha", "db_pre", "db_post", "db_res")),
                       ("mhc_embed_bwd", ("dtable",))):
        for what in outs:
            assert _call(name, B=0, **{what: None}) == INVALID, (name, what)
    assert mhc.mhc_embed_bwd(0, 4, 40, 10, None, None, 1.0, 1 << 44, None, accumulate=True, stream=0,
                             check=False) == OK          # nothing to add


def test_table_sizes():
    for name in ("mhc_embed", "mhc_embed_bwd"):
        assert _call(name, V=0) == INVALID
        assert _call(name, V=-5) == INVALID
        assert _call(name, V=1 << 31) == UNSUPPORTED
        assert _call(name, V=1 << 30, C=1 << 12, B=1) == UNSUPPORTED
        # a table that reaches into the output
        assert _call(name, V=1 << 24, C=1 << 14, B=1) == INVALID


def test_size_functions():
    assert mhc.mhc_ckpt_scales_per_row(4, 7168) == 4 * 224
    assert mhc.mhc_ckpt_scales_per_row(2, 40) == 4
    assert mhc.mhc_ckpt_scales_per_row(1, 8) == 1
    for n, C in ((3, 32), (4, 12), (0, 32), (4, 0), (4, -8)):
        assert mhc.mhc_ckpt_scales_per_row(n, C) == 0
    assert mhc.mhc_coeffs_pre_bwd_workspace_size(0, 4, 40) == 0
    assert mhc.mhc_coeffs_pre_bwd_workspace_size(16, 5, 40) == 0
    assert mhc.mhc_embed_bwd_workspace_size(0, 4, 40, 10) == 0
    assert mhc.mhc_embed_bwd_workspace_size(16, 4, 40, 0) == 0
    for B in (1, 5, 1000, 16384, 1 << 20):
        for n, C in ((1, 8), (4, 7168), (8, 4096)):
            N = n * n + 2 * n
            assert mhc.mhc_coeffs_pre_bwd_workspace_size(B, n, C) >= 4 * B * N   # dlogit at least
            assert mhc.mhc_embed_bwd_workspace_size(B, n, C, 1000) >= 8 * B


def test_binding_refuses_wrong_tensors():
    B, n, C = 4, 2, 16
    X = torch.zeros(B, n * C, dtype=torch.bfloat16)
    scales = torch.zeros(B, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="X_t: 128 bytes, the call needs 256"):
        mhc.mhc_ckpt_pack(B, n, C, X[:2], torch.zeros(B, n * C, dtype=torch.uint8), scales, stream=0)
    with pytest.raises(ValueError, match="codes: 64 bytes, the call needs 128"):
        mhc.mhc_ckpt_pack(B, n, C, 1 << 44, torch.zeros(2, n * C, dtype=torch.uint8), scales, stream=0)
    with pytest.raises(ValueError, match="scales: 4 bytes, the call needs 8"):
        mhc.mhc_ckpt_unpack(B, n, C, 1 << 44, scales[:2], X, stream=0)
    with pytest.raises(ValueError, match="codes: element size 2"):
        mhc.mhc_ckpt_unpack(B, n, C, X, scales, X, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        mhc.mhc_post_res_bwd(B, n, C, torch.zeros(2 * B, n * C, dtype=torch.bfloat16)[::2], 1 << 44, 1 << 45, 1 << 46,
                             1 << 47, 1 << 48, stream=0)
    with pytest.raises(ValueError, match="dH: element size 2"):
        mhc.mhc_post_res_bwd(B, n, C, 1 << 40, 1 << 41, 1 << 42, 1 << 43, 1 << 44,
                             torch.zeros(B, n * n + 2 * n, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="dalpha: 8 bytes, the call needs 12"):
        mhc.mhc_coeffs_pre_bwd(B, n, C, 1 << 40, 1 << 41, 0.1, 0.1, 0.1, *([1 << 42] * 9), 1 << 43, 1 << 44,
                               torch.zeros(2), 1 << 45, 1 << 46, 1 << 47, 1 << 48, 1 << 20, stream=0)
    with pytest.raises(ValueError, match="tokens: element size 4"):
        mhc.mhc_embed(B, n, C, 10, torch.zeros(B, dtype=torch.int32), 1 << 44, 1.0, 1 << 45, stream=0)
    with pytest.raises(ValueError, match="table: 288 bytes, the call needs 320"):
        mhc.mhc_embed(B, n, C, 10, 1 << 43, torch.zeros(9, C, dtype=torch.bfloat16), 1.0, 1 << 45, stream=0)
    with pytest.raises(ValueError, match="dtable: 576 bytes, the call needs 640"):
        mhc.mhc_embed_bwd(B, n, C, 10, 1 << 43, 1 << 44, 1.0, torch.zeros(9, C), 1 << 45, workspace_bytes=1 << 20,
                          stream=0)
    with pytest.raises(ValueError, match="device tensors"):
        mhc.mhc_embed_bwd(B, n, C, 10, 1 << 43, 1 << 44, 1.0, torch.zeros(10, C), 1 << 45, workspace_bytes=1 << 20,
                          stream=0)


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a host without a HIP device (fake addresses)")
def test_no_device_is_mhc_err_hip():
    for name in sorted(CALLS):
        assert _call(name) == mhc.MHC_ERR_HIP, name
    for name in ("mhc_coeffs_pre_bwd", "mhc_coeffs_pre_bwd_ckpt", "mhc_embed_bwd"):
        assert _call(name, B=0) == mhc.MHC_ERR_HIP, name  # the zeros of B = 0
