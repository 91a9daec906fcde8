"""The host code of the calls around a layer of experts under AddressSanitizer
and UndefinedBehaviorSanitizer: tests/host/experts_host_check.cpp drives their
refusals, the size functions and the workspace plans (test_train_sanitized.py
does the same for the training calls)."""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from tests.test_abi_sanitized import CLANG, CSRC, FLAGS, HIPCC, ROOT, SAN

pytestmark = pytest.mark.cpu

OUT = os.path.join(ROOT, "_build", "sanitized_experts")
SOURCES = ["mhc_experts_abi.hip", "mhc_experts.hip", "mhc_rmsnorm.hip", "mhc_route.hip", "mhc_coeffs_pre_bwd.hip"]


def _compile(src):
    obj = os.path.join(OUT, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, *SAN, *([] if src.endswith(".hip") else ["-x", "hip"]), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return obj


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(CLANG), reason="needs hipcc and clang++")
def test_calls_around_experts_under_asan_ubsan():
    os.makedirs(OUT, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "host", "experts_host_check.cpp")]
    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(_compile, srcs))
    exe = os.path.join(OUT, "experts_host_check")
    link = [CLANG, "-fsanitize=address,undefined", "-o", exe, *objs, "-L/opt/rocm/lib", "-lamdhip64",
            "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(link, capture_output=True, text=True)
    assert r.returncode == 0, f"{' '.join(link)}\n{r.stdout}\n{r.stderr}"
    no_device = torch.cuda.device_count() == 0
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "1" if no_device else "0"], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, f"driver failed ({r.returncode}):\n{r.stdout}\n{r.stderr[-4000:]}"
    assert "checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
