"""Function attributes of kernels belong to the device that is current when they are set.  Set once for the process,
they are missing on every other device, where the launch then fails.  This machine may have no second device, so the
sources are looked at: no attribute is set in an initialiser of a static."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_sharding_affinity_gb300", "csrc")


def test_no_function_attribute_is_set_once_for_the_process():
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        seen += text.count("cudaFuncSetAttribute")
        for m in re.finditer(r"\bstatic\b[^;{}()]*=\s*\[[^\]]*\]\s*(?:\([^)]*\)\s*)?\{(.*?)\}\s*\(\s*\)\s*;", text, re.S):
            assert "cudaFuncSetAttribute" not in m.group(1), f"{os.path.basename(path)}: {m.group(0)[:80]}"
        assert "call_once" not in text or "cudaFuncSetAttribute" not in text
    assert seen
