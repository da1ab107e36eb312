"""Sanitizer build (CPU only) of the attention library's host code: csrc/attn/attn_api.hip under
host-side AddressSanitizer and UndefinedBehaviorSanitizer (hipcc, each -fsanitize after
-Xarch_host), linked with the other sources' objects and driven by tests/attn_abi_check.c."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from conftest import ROOT

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang"
SAN_ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")


def run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(map(str, cmd))}\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}"
    return r


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not found")
def test_attention_host_code_under_asan_ubsan(tmp_path):
    import w4a8_codebook_gemm_amd.build as B
    srcs = B.attn_sources()
    api = [s for s in srcs if os.path.basename(s) == "attn_api.hip"]
    assert api
    others = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs if s not in api]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    api_obj = str(tmp_path / "attn_api_san.o")
    # the kernels do not run here: built as quickly as can be
    quick = [f for f in B.FLAGS if not f.startswith("-O")] + ["-O0"]
    with cf.ThreadPoolExecutor(max_workers=5) as ex:
        jobs = [ex.submit(run, [HIPCC, *B.FLAGS, "-O1", "-g", *san, "-c", api[0], "-o", api_obj])]
        jobs += [ex.submit(run, [HIPCC, *quick, "-c", s, "-o", o]) for s, o in zip([s for s in srcs if s not in api], others)]
        for j in jobs:
            j.result()
    run([HIPCC, f"--offload-arch={B.ARCH}", "-shared", "-fPIC", "-Xarch_host", "-fsanitize=address",
         "-Xarch_host", "-fsanitize=undefined", api_obj, *others, "-o", str(tmp_path / "libw4a8_attn_san.so")])
    exe = str(tmp_path / "attn_abi_check")
    run([CLANG, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", f"-I{os.path.join(ROOT, 'include')}",
         os.path.join(ROOT, "tests", "attn_abi_check.c"), f"-L{tmp_path}", "-lw4a8_attn_san", f"-Wl,-rpath,{tmp_path}",
         "-lm", "-o", exe])
    r = run([exe], env=SAN_ENV, timeout=300)
    assert r.stdout.strip().endswith("ok")
