"""The built library holds the kernels that calls reach, and no more."""
import re
import shutil
import subprocess

import pytest


@pytest.fixture(scope="module")
def symbols():
    if shutil.which("nm") is None:
        pytest.skip("no nm")
    from block_quantized_dsq_b200 import build
    return subprocess.run(["nm", "-C", build.build()], capture_output=True, text=True, check=True).stdout


def test_fused_decode_kernels(symbols):
    """dsq_gemv_fused asks that its M tokens fit the shared memory kept for
    activations, and takes the tensor cores from 4 (Q8_0) or 5 (Q4_K) tokens on
    where 8 would fit: with 8 tokens always.  Fewer tokens of long rows stay on
    the CUDA cores, and so does an expert's single row."""
    found = {tuple(a.strip() for a in m[1].split(",")) for m in re.finditer(r"gemv_fused_kernel<([^>]*)>", symbols)}
    want = set()
    for qtype in ("8", "12"):
        for gated in ("false", "true"):
            want |= {(qtype, str(m), "false", "false", gated, "16" if m <= 2 else "8") for m in range(1, 8)}
            want |= {(qtype, "8", "true", "false", gated, "8"), (qtype, "1", "false", "true", gated, "16"),
                     (qtype, "8", "true", "true", gated, "8")}
            if qtype == "8":
                want.add((qtype, "8", "true", "true", gated, "16"))
    assert found == want
