"""The host code of the plan, append and chunk calls under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_host_sanitizers.py
does for the others: objects built there are used if they are newer than the
sources."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import CLANG, CSRC, HIPCC, INCLUDE, OUT, ROCM, ROOT, _compile

DRIVER = os.path.join(ROOT, "tests", "host_sanitize", "tokens_driver.cpp")


def _object(src):
    obj = os.path.join(OUT, os.path.basename(src) + ".o")
    newest = max(os.path.getmtime(os.path.join(d, f)) for d in (CSRC, INCLUDE)
                 for f in os.listdir(d))
    return obj if os.path.exists(obj) and os.path.getmtime(obj) > newest else _compile(src)


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="host-only check; a GPU is present")
@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="ROCm compilers not installed")
def test_tokens_host_code_is_clean_under_asan_and_ubsan():
    os.makedirs(OUT, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_object, srcs))
    drv, exe = os.path.join(OUT, "tokens_driver.o"), os.path.join(OUT, "tokens_driver")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-fno-omit-frame-pointer"]
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", *san,
                        f"-I{INCLUDE}", f"-I{ROCM}/include", "-c", DRIVER, "-o", drv],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([CLANG, *san, drv, *objs, f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib",
                        "-lamdhip64", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "tokens driver ok" in r.stdout, (r.stdout, r.stderr[-4000:])
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
