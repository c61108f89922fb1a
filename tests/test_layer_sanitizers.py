"""The host code of the norm, dropout and router calls under AddressSanitizer and
UndefinedBehaviorSanitizer, on the host side only (the kernels at -O1: none is launched)."""
import glob
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
from weight_merge_amd import build  # noqa: E402

ASAN_RT = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))


@pytest.mark.skipif(not ASAN_RT, reason="clang's AddressSanitizer runtime is not installed")
@pytest.mark.skipif(torch.cuda.is_available(), reason="the host tests pass fake pointers: run where no GPU is visible")
def test_layer_host_code_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    lib = str(tmp_path / "libadafuse_san.so")
    host_only = []
    for f in ("address", "undefined", "float-cast-overflow"):
        host_only += ["-Xarch_host", f"-fsanitize={f}"]
    host_only += ["-Xarch_host", "-fno-sanitize-recover=undefined,float-cast-overflow", "-Xarch_host",
                  "-fno-omit-frame-pointer"]
    flags = [f if f != "-O3" else "-O1" for f in build.FLAGS if f != "-shared"]
    paths = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(build.PKG, "csrc")]
    objects = [str(tmp_path / (os.path.basename(s) + ".o")) for s in build.sources()]
    runs = [subprocess.Popen([build.HIPCC, *flags, *host_only, *paths, "-c", s, "-o", o], stdout=subprocess.DEVNULL,
                             stderr=subprocess.PIPE, text=True) for s, o in zip(build.sources(), objects)]
    for run in runs:
        err = run.communicate()[1]
        assert run.returncode == 0, err[-3000:]
    res = subprocess.run([build.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *host_only, *objects, "-o", lib],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    syms = subprocess.run(["nm", "-D", "--undefined-only", lib], capture_output=True, text=True).stdout
    assert "__asan_" in syms and "__ubsan_" in syms, "the host code was not instrumented"
    driver = (
        "import sys, pytest\n"
        f"sys.path.insert(0, {ROOT!r})\n"
        "from weight_merge_amd import _lib\n"
        f"_lib.LIB_PATH = {lib!r}\n"
        f"sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', {os.path.join(ROOT, 'tests', 'test_layer_host.py')!r}]))\n"
    )
    env = dict(os.environ, LD_PRELOAD=ASAN_RT[-1], ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    run = subprocess.run([sys.executable, "-c", driver], capture_output=True, text=True, env=env, timeout=600)
    out = run.stdout + run.stderr
    assert run.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out and "failed" not in out
