"""The host code of the entry points of include/qw_mx.h under AddressSanitizer and
UndefinedBehaviorSanitizer, as tests/test_host_sanitizers.py does it for the
others (see abi_fuzz_mx.c).  Takes about a minute (the compile)."""

import os
import re
import subprocess

import pytest

from int8_int4_dequant_amd import build, qw
from tests.test_host_sanitizers import HOST_SAN, LLVM, ROOT


def test_every_entry_point_is_in_a_driver():
    with open(os.path.join(ROOT, "tests", "abi_fuzz_mx.c")) as f:
        called = set(re.findall(r"\b(qw_[a-z_]+)\(", f.read()))
    assert sorted(called & set(qw.EXPORTS_MX)) == sorted(qw.EXPORTS_MX)


@pytest.mark.timeout(600)
def test_mx_abi_under_host_sanitizers(tmp_path):
    if not (os.path.exists(build.HIPCC) and os.path.exists(os.path.join(LLVM, "clang"))):
        pytest.skip("hipcc / clang not installed")
    objs = build.compile_objects(str(tmp_path / "obj"), HOST_SAN)
    drv = str(tmp_path / "abi_fuzz_mx.o")
    san = "-fsanitize=address,undefined"
    subprocess.run([os.path.join(LLVM, "clang"), "-O1", "-g", san,
                    "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include"),
                    "-c", os.path.join(ROOT, "tests", "abi_fuzz_mx.c"), "-o", drv],
                   check=True, capture_output=True, text=True)
    exe = str(tmp_path / "abi_fuzz_mx")
    subprocess.run([os.path.join(LLVM, "clang++"), san, drv, *objs, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe],
                   check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe, "40000"], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    assert "abi_fuzz_mx:" in out and " 0 failures" in out, out[-4000:]
    print(out[-300:])
