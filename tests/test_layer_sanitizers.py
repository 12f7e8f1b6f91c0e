"""The host checks of the row, norm and 8-bit block entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, no GPU)."""

import os
from concurrent.futures import ThreadPoolExecutor

import pytest

import moe_ragged_grouped_amd.build as hb
from tests.test_operator_sanitizers import CLANG, HERE, _run


@pytest.mark.skipif(not (os.path.exists(hb.HIPCC) and os.path.exists(CLANG)), reason="no ROCm toolchain")
def test_layer_checks_clean_under_sanitizers(tmp_path):
    flags = [f for f in hb.FLAGS if f not in ("-shared", "-O3")] + [
        "-O1", "-g1", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
        "-Xarch_host", "-fno-sanitize-recover=all"]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in hb.LAYER_SOURCES]
    with ThreadPoolExecutor(max_workers=len(objs)) as ex:
        list(ex.map(lambda so: _run([hb.HIPCC, *flags, "-c", "-o", so[1], so[0]]), zip(hb.LAYER_SOURCES, objs)))
    lib = tmp_path / "libgg_san.so"
    _run([hb.HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", str(lib), *objs])
    exe = tmp_path / "layer_checks"
    _run([CLANG, "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
          os.path.join(hb.ROOT, "include"), os.path.join(HERE, "sanitize", "layer_checks.c"),
          "-L", str(tmp_path), "-lgg_san", "-Wl,-rpath," + str(tmp_path), "-o", str(exe)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = _run([str(exe)], env=env)
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-3000:]
    assert "layer checks: 0 failure(s)" in out
