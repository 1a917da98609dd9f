"""AddressSanitizer run of the host code of the chunk attention and the block
upkeep (CPU only, no GPU calls): their C-ABI source with the sanitizer on the
host side, the other objects as built, and a C driver through the rejection
paths and the workspace sizes."""
import os
import shutil
import subprocess
import tempfile

import pytest

from mixture_value_projection_amd import build
from test_asan_host import CLANG, CLANGXX, HERE, ROCM_LIB, _run


@pytest.fixture(scope="module")
def driver():
    if not (os.path.exists(build.HIPCC) and os.path.exists(CLANG) and os.path.exists(CLANGXX)):
        pytest.skip("ROCm compilers not found")
    os.makedirs(build.BUILDDIR, exist_ok=True)
    out = tempfile.mkdtemp(prefix="asan-", dir=build.BUILDDIR)
    others = [os.path.join(build.BUILDDIR, os.path.basename(s) + ".o") for s in build.sources()
              if not s.endswith("paged_api.hip")]
    if not all(os.path.exists(o) for o in others):
        build.build_library(verbose=False)
    obj = os.path.join(out, "paged_api.asan.o")
    _run([build.HIPCC, *build.COMMON, *build.DEVICE_FLAGS,
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer",
          "-c", os.path.join(build.CSRC, "paged_api.hip"), "-o", obj])
    _run([CLANGXX, "-shared", "-fPIC", "-fsanitize=address", "-o",
          os.path.join(out, "libmova_asan.so"), obj, *others, f"-L{ROCM_LIB}", "-lamdhip64"])
    exe = os.path.join(out, "chunk_asan_driver")
    _run([CLANG, "-fsanitize=address", "-fno-omit-frame-pointer", "-g", "-I",
          os.path.join(build.ROOT, "include"), os.path.join(HERE, "chunk_asan_driver.c"), "-o", exe,
          f"-L{out}", "-lmova_asan", f"-Wl,-rpath,{out}", f"-Wl,-rpath,{ROCM_LIB}"])
    yield exe
    shutil.rmtree(out, ignore_errors=True)


def test_host_paths_under_asan(driver):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0")
    r = subprocess.run([driver], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, f"driver failed:\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}"
    assert "chunk asan driver: ok" in r.stdout
    assert "ERROR: AddressSanitizer" not in r.stderr
