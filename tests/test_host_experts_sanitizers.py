"""The entry points of the experts' choice, layer and adapters under
ThreadSanitizer, and under AddressSanitizer with UndefinedBehaviorSanitizer
(CPU only, on the stand-in device): tests/sanitize/experts.cpp linked against
the library's host sources built with the sanitizer.
"""
import os
import subprocess

import pytest

from gemm_autotuning_amd import build as b

from .test_host_sanitizers import CLANG, ROOT, SAN


@pytest.mark.parametrize("kind", sorted(SAN))
def test_experts_under_sanitizer(kind):
    out = os.path.join(b.BUILD, "san_experts_" + kind)
    os.makedirs(out, exist_ok=True)
    flags = [f for f in b.HOST_FLAGS if f != "-O2"] + ["-O1", "-g", "-fno-omit-frame-pointer"] + SAN[kind]
    objs, jobs = [], []
    for src in [os.path.join(b.CSRC, n) for n in b.HOST_SOURCES] + [os.path.join(ROOT, "tests", "sanitize", "experts.cpp")]:
        # both sources of that name have their own object
        obj = os.path.join(out, os.path.basename(os.path.dirname(src)) + "_" + os.path.basename(src) + ".o")
        objs.append(obj)
        jobs.append(subprocess.Popen([CLANG] + flags + ["-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj],
                                     stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for j in jobs:
        log, _ = j.communicate()
        assert j.returncode == 0, log
    exe = os.path.join(out, "experts")
    r = subprocess.run([CLANG] + SAN[kind] + ["-o", exe] + objs + b.kernel_objects() +
                       ["-L" + os.path.join(b.ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(b.ROCM, "lib"),
                        "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, TSAN_OPTIONS="halt_on_error=1", ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-6000:]
    assert "experts under sanitizer ok" in r.stdout and "runtime error" not in r.stderr
