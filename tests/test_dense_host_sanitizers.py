"""Host code of the dense feed-forward operators under AddressSanitizer and
UndefinedBehaviourSanitizer (CPU only): dense.hip (validation) and
kernels_dense.hip (workspace sizes, choice of tile) compiled with both
sanitizers on the host side only, linked with the release objects of the other
files, and driven through their GPU-free paths
(tests/sanitize/dense_host_driver.c).  Any report aborts the driver."""
import os

import pytest

from test_host_sanitizers import CLANG, HIPCC, RELEASE_OBJ, ROOT, SAN, _run

OTHERS = ("kernels_route", "kernels_permute", "kernels_expert", "kernels_persistent", "abi", "batching")


@pytest.mark.skipif(not HIPCC.exists() or not CLANG.exists(), reason="ROCm toolchain not found")
def test_dense_host_code_under_address_and_ub_sanitizers(tmp_path):
    objs = [RELEASE_OBJ / f"{k}.o" for k in OTHERS]
    if not all(o.exists() for o in objs):
        pytest.skip("release objects not built (fp8_moe_layer_amd/build.py)")
    san_objs = []
    for src in ("dense", "kernels_dense"):
        o = tmp_path / f"{src}.o"
        # host-side sanitizers only: each -fsanitize= applies to the host pass
        _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-fno-omit-frame-pointer", "-Xclang", "-target-feature", "-Xclang",
              "-packed-fp32-ops", "-c", "-o", o, ROOT / "fp8_moe_layer_amd" / "csrc" / f"{src}.hip"])
        san_objs.append(o)
    lib = tmp_path / "libfp8moe_hostsan.so"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib, *san_objs, *objs])
    exe = tmp_path / "dense_host_driver"
    _run([CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-o", exe,
          SAN / "dense_host_driver.c", f"-L{tmp_path}", "-lfp8moe_hostsan", f"-Wl,-rpath,{tmp_path}"])
    res = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                               UBSAN_OPTIONS="print_stacktrace=1"))
    assert "dense host driver ok" in res.stdout
    assert "runtime error" not in res.stderr
