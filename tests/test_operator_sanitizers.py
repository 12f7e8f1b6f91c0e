"""The host code of the gradients and 4-bit operators under AddressSanitizer and
UndefinedBehaviorSanitizer.

``tests/sanitize/operator_checks.c`` calls each of their entry points with arguments its
host checks must reject, at and past the limits of every size, and checks the status
codes. All sources are rebuilt with both sanitizers on the host code only; every call ends
before any HIP runtime call, so no GPU is needed. (``test_host_sanitizers.py`` does the
same for the forward products.)
"""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import moe_ragged_grouped_amd.build as hb

CLANG = "/opt/rocm/llvm/bin/clang"
HERE = os.path.dirname(os.path.abspath(__file__))


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout + r.stderr


@pytest.mark.skipif(not (os.path.exists(hb.HIPCC) and os.path.exists(CLANG)), reason="no ROCm toolchain")
def test_operator_checks_clean_under_sanitizers(tmp_path):
    flags = [f for f in hb.FLAGS if f not in ("-shared", "-O3")] + [
        "-O1", "-g1", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
        "-Xarch_host", "-fno-sanitize-recover=all"]
    sources = hb.SOURCES + hb.OPERATOR_SOURCES
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in sources]
    with ThreadPoolExecutor(max_workers=len(sources)) as ex:
        list(ex.map(lambda so: _run([hb.HIPCC, *flags, "-c", "-o", so[1], so[0]]), zip(sources, objs)))
    lib = tmp_path / "libgg_san.so"
    _run([hb.HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", str(lib), *objs])
    exe = tmp_path / "operator_checks"
    _run([CLANG, "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
          os.path.join(hb.ROOT, "include"), os.path.join(HERE, "sanitize", "operator_checks.c"),
          "-L", str(tmp_path), "-lgg_san", "-Wl,-rpath," + str(tmp_path), "-o", str(exe)])
    # the HIP runtime itself is not instrumented; its allocations at load time are not
    # this library's leaks
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = _run([str(exe)], env=env)
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-3000:]
    assert "operator checks: 0 failure(s)" in out
