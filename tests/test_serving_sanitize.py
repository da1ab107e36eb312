"""Sanitizer build (CPU only) of the serving library's host code: csrc/serve/serve_api.hip under
host-side AddressSanitizer and UndefinedBehaviorSanitizer (hipcc, each -fsanitize after
-Xarch_host), linked with the other sources' objects and driven by tests/serve_abi_check.c."""
import concurrent.futures as cf
import os

import pytest

from conftest import ROOT
from test_attention_sanitize import CLANG, HIPCC, SAN_ENV, run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not found")
def test_serving_host_code_under_asan_ubsan(tmp_path):
    import w4a8_codebook_gemm_amd.build as B
    srcs = B.serve_sources()
    api = [s for s in srcs if os.path.basename(s) == "serve_api.hip"]
    assert api
    rest = [s for s in srcs if s not in api]
    others = [str(tmp_path / (os.path.basename(s) + ".o")) for s in rest]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    api_obj = str(tmp_path / "serve_api_san.o")
    # the kernels do not run here: built as quickly as can be
    quick = [f for f in B.FLAGS if not f.startswith("-O")] + ["-O0"]
    with cf.ThreadPoolExecutor(max_workers=6) as ex:
        jobs = [ex.submit(run, [HIPCC, *B.FLAGS, "-O1", "-g", *san, "-c", api[0], "-o", api_obj])]
        jobs += [ex.submit(run, [HIPCC, *quick, "-c", s, "-o", o]) for s, o in zip(rest, others)]
        for j in jobs:
            j.result()
    run([HIPCC, f"--offload-arch={B.ARCH}", "-shared", "-fPIC", "-Xarch_host", "-fsanitize=address",
         "-Xarch_host", "-fsanitize=undefined", api_obj, *others, "-o", str(tmp_path / "libw4a8_serve_san.so")])
    exe = str(tmp_path / "serve_abi_check")
    run([CLANG, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", f"-I{os.path.join(ROOT, 'include')}",
         os.path.join(ROOT, "tests", "serve_abi_check.c"), f"-L{tmp_path}", "-lw4a8_serve_san", f"-Wl,-rpath,{tmp_path}",
         "-lm", "-o", exe])
    r = run([exe], env=SAN_ENV, timeout=300)
    assert r.stdout.strip().endswith("ok")
