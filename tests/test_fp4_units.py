"""The W4A4 sources are several translation units, each with device variables of its
own (the sticky error word, the wait limit): a header's host function that names one
must be each unit's own too, or the linker keeps one unit's for all."""
import os
import re
import shutil
import subprocess

import pytest

from w4a16_matmul_pack_b200 import build as B

NVCC = os.environ.get("NVCC", "nvcc")


@pytest.mark.skipif(shutil.which(NVCC) is None, reason="needs nvcc")
def test_functions_of_a_units_own_variables_are_its_own(tmp_path):
    """Not inlined (-O0), the reader of the error word is a local symbol."""
    src = tmp_path / "unit.cu"
    src.write_text('#include "%s/fp4_host.cuh"\nint use(int *o, int c) { return w4::take_device_error(o, c); }\n' % B.SRC_DIR)
    obj = tmp_path / "unit.o"
    subprocess.check_call([NVCC, "-O0", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-c", str(src), "-o", str(obj)])
    out = subprocess.run(["nm", "-C", str(obj)], capture_output=True, text=True, check=True).stdout
    kinds = [re.match(r"[0-9a-f]*\s+(\w) ", l).group(1)
             for l in out.splitlines() if "w4::take_device_error(" in l]
    assert kinds == ["t"], out


def test_no_shared_host_function_names_a_units_variable():
    names, found = set(), []
    text = {f: open(os.path.join(B.SRC_DIR, f)).read() for f in os.listdir(B.SRC_DIR) if f.endswith(".cuh")}
    for t in text.values():
        names |= set(re.findall(r"^__device__ [\w ]+ (g_\w+)\b", t, re.M))
    assert {"g_device_error", "g_wait_limit_ns"} <= names
    for f, t in text.items():
        for m in re.finditer(r"^inline [^\n;]*\{.*?^\}", t, re.M | re.S):
            found += [(f, m.group(0).split("(")[0]) for n in names if re.search(r"\b%s\b" % n, m.group(0))]
    assert not found
