"""The host side of linear attention and of the norm with rotation under
AddressSanitizer and UndefinedBehaviorSanitizer.

Their argument checks, launch plans and launch sequences are built a second
time with instrumented host code (the device code as in the product build) and
linked against the product library for the rest, and their CPU tests run again
against that copy in a child interpreter with the sanitizer runtime
preloaded.  A report ends the child and fails this test.  Needs no GPU:
nothing is launched."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from selective_state_space_84_amd import build_lib
from test_abi_sanitize import REPO, SAN, _runtime

SOURCES = ["abi.hip", "linear_attn.hip", "linear_attn_bf16.hip", "linear_attn_update.hip", "qk_norm_rope.hip"]


@pytest.mark.skipif(_runtime() is None or not os.path.exists(build_lib.HIPCC),
                    reason="hipcc or the clang sanitizer runtime is missing")
def test_linear_attn_abi_clean_under_sanitizers(lib, tmp_path):
    def compile_one(src):
        obj = str(tmp_path / src.replace(".hip", ".o"))
        r = subprocess.run([build_lib.HIPCC, *build_lib.FLAGS, *SAN, "-c", os.path.join(build_lib.CSRC, src),
                            "-o", obj], capture_output=True, text=True, timeout=900)
        assert r.returncode == 0, src + "\n" + r.stdout[-2000:] + r.stderr[-2000:]
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    out = str(tmp_path / "libssm_scan_sanitized.so")
    subprocess.run([build_lib.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *SAN, "-shared-libsan", "-o", out,
                    *objs, build_lib.LIB, "-Wl,-rpath," + os.path.dirname(build_lib.LIB)],
                   check=True, capture_output=True, timeout=300)
    pre = os.environ.get("LD_PRELOAD", "")
    env = dict(os.environ, SSM_TEST_LIBRARY=out, LD_PRELOAD=(_runtime() + (" " + pre if pre else "")),
               ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:detect_odr_violation=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        *(os.path.join(REPO, "tests", f) for f in ("test_linear_attn_abi.py",
                                                                   "test_linear_attn_edges.py"))],
                       capture_output=True, text=True, timeout=600, env=env, cwd=REPO)
    text = r.stdout + r.stderr
    assert r.returncode == 0, text[-4000:]
    assert "ERROR: AddressSanitizer" not in text and "runtime error:" not in text, text[-4000:]
    assert " passed" in r.stdout
