"""The KV cache's host code under the address and undefined-behaviour
sanitizers, on the CPU: its sources are compiled host-only, linked with the
host-only HIP stand-in and driven through every entry point of
include/qcache.h by tests/sanitize/qcache_driver.cpp."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from compressed_gemv_amd import build as qbuild
from test_abi_sanitize import CLANG, HOST_SAN, SAN, _run

pytestmark = pytest.mark.skipif(not (os.path.exists(CLANG) and shutil.which("nm")), reason="clang++ or nm missing")


def test_kvcache_host_code_sanitized(tmp_path):
    sources = [s for s in qbuild.SOURCES if s.startswith("kvcache")]
    assert len(sources) == 4

    def compile_one(src):
        obj = str(tmp_path / src.replace(".hip", ".o"))
        _run([qbuild.hipcc(), "-O1", "-g", "-std=c++17", "-fPIC", "--offload-host-only", f"--offload-arch={qbuild.ARCH}",
              *HOST_SAN, "-Wno-unused-command-line-argument", "-I", qbuild.INCLUDE, "-I", qbuild.CSRC,
              "-c", os.path.join(qbuild.CSRC, src), "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, sources))
    names = {line.split()[-1] for o in objs for line in _run(["nm", "-u", o]).stdout.splitlines()
             if line.split()[-1].startswith("__hip_fatbin_")}
    stub = tmp_path / "images.cpp"
    stub.write_text("".join(f'extern "C" const char {n}[64] = {{0}};\n' for n in sorted(names)))
    exe = str(tmp_path / "qcache_driver")
    _run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
          "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", qbuild.INCLUDE, "-I", SAN,
          os.path.join(SAN, "fake_hip.cpp"), os.path.join(SAN, "qcache_driver.cpp"), str(stub), *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    print(r.stdout)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-8000:]
    assert " 0 failed" in r.stdout and "Sanitizer" not in r.stderr, r.stderr[-8000:]
