"""Host code of the layer's operators under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only), as test_mixer_sanitizers.py does for those around the scan: driven by
tests/sanitize/layer_driver.c, which makes only calls that are refused before a launch."""
import concurrent.futures as cf
import os

import pytest

from test_mixer_sanitizers import CSRC, HIPCC, HOST_SAN, ROOT, SAN, _env, _run

SOURCES = ["layer_api.cpp", "gdelta_fwd.hip", "gdelta_bwd.hip", "gdelta_step.hip", "block_norm.hip", "rope.hip"]
DEVICE = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]

pytestmark = pytest.mark.slow


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_layer_validation_under_sanitizers(tmp_path):
    common = ["--offload-arch=gfx950", "-O1", "-g", "-fPIC", "-std=c++17", "-I", os.path.join(ROOT, "include"),
              *DEVICE, "-Wno-unused-command-line-argument"] + HOST_SAN

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        _run([HIPCC] + common + lang + ["-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with cf.ThreadPoolExecutor(max_workers=6) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    drv = str(tmp_path / "layer_driver.o")
    _run([HIPCC, "-g", "-O1", "-x", "c", "-I", os.path.join(ROOT, "include")] + HOST_SAN
         + ["-c", os.path.join(SAN, "layer_driver.c"), "-o", drv])
    exe = str(tmp_path / "layer_driver")
    _run([HIPCC, "--offload-arch=gfx950", "-o", exe, drv] + objs + HOST_SAN)
    assert "0 failed checks" in _run([exe], env=_env()).stdout
