"""Host code of the operators around the scan under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only), as test_sanitizers.py does for the scan's: the
library's sources built with sanitized host code and driven by
tests/sanitize/mixer_driver.c, which makes only calls that are refused before a launch."""
import concurrent.futures as cf
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mamba2_ssd_chunked_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# sanitizers on the host compilation only: the device code is built as usual
HOST_SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
            "-Xarch_host", "-fno-sanitize-recover=all"]
SOURCES = ["mixer_api.cpp", "linattn.hip", "token_step.hip", "norm.hip"]

pytestmark = pytest.mark.slow


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r


def _env():
    return dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=86",
                UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=87")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_mixer_validation_under_sanitizers(tmp_path):
    common = ["--offload-arch=gfx950", "-O1", "-g", "-fPIC", "-std=c++17",
              "-I", os.path.join(ROOT, "include"), "-Xclang", "-target-feature", "-Xclang",
              "-packed-fp32-ops", "-Wno-unused-command-line-argument"] + HOST_SAN

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        _run([HIPCC] + common + lang + ["-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    drv = str(tmp_path / "mixer_driver.o")
    _run([HIPCC, "-g", "-O1", "-x", "c", "-I", os.path.join(ROOT, "include")] + HOST_SAN
         + ["-c", os.path.join(SAN, "mixer_driver.c"), "-o", drv])
    exe = str(tmp_path / "mixer_driver")
    _run([HIPCC, "--offload-arch=gfx950", "-o", exe, drv] + objs + HOST_SAN)
    r = _run([exe], env=_env())
    assert "0 failed checks" in r.stdout
