"""The host code of the dense products and of the few-token layer under AddressSanitizer and
UndefinedBehaviorSanitizer (host compilation only), driven by host_checks_linear_few.cpp."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import CSRC, HOST_SANITIZE, ROOT, _hipcc

SOURCES = ["moe_api.hip", "route.hip", "dispatch.hip", "gemm.hip", "combine.hip",
           "expert_choice.hip", "linear.hip", "few.hip"]


@pytest.mark.timeout(900)
def test_host_code_under_asan_and_ubsan(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not available")
    # device code is not looked at here: no optimisation
    flags = ["--offload-arch=gfx950", "-O0", "-g1", "-std=c++17", "-fno-omit-frame-pointer",
             "-Xarch_device", "-O1", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"), "-Wno-unused-command-line-argument",
             *HOST_SANITIZE]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([cc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    srcs.append(os.path.join(ROOT, "tests", "host_checks_linear_few.cpp"))
    with ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "host_checks")
    r = subprocess.run([cc, "--offload-arch=gfx950", *HOST_SANITIZE, *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert ", 0 failures" in r.stdout
