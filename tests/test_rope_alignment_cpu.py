"""The rotation's wide path takes tensors and token strides that are aligned to 16 bytes, so that none of its
accesses may claim more of the compiler.  From the LLVM IR of its kernels (CPU only)."""
import os
import re
import subprocess

import pytest

from mamba2_ssd_chunked_amd import build as B


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="needs hipcc")
def test_no_access_claims_more_than_16_bytes(tmp_path):
    out = str(tmp_path / "rope.ll")
    subprocess.run([B.HIPCC] + B.FLAGS + ["-x", "hip", "-S", "-emit-llvm", "--cuda-device-only",
                   os.path.join(B.CSRC, "rope.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    seen = [(line.strip(), int(m.group(1))) for line in text.split("\n")
            for m in [re.search(r"(?:load|store) .*(?:addrspace\(1\)|ptr) .*align (\d+)", line)]
            if m and "addrspace(4)" not in line and "addrspace(3)" not in line]
    assert any("<8 x float>" in s or "<4 x float>" in s for s, _ in seen)  # the wide accesses are there
    assert max(a for _, a in seen) <= 16, [s for s, a in seen if a > 16][:4]
