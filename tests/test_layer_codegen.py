"""What the kernels of a layer's scans promise to the compiler (CPU only; hipcc cross-compiles)."""
import re
import subprocess

import pytest

from prefix_scan_stream_amd import build as b

PROBE = """#include "ls_elements.hpp"
namespace ls {
template <class E, int VEC, bool ONCE>
__global__ void probe(const char* from, char* to)
{
    Elements<E, VEC> v;
    v.template load<ONCE>(from + threadIdx.x * 48);
    v.template store<ONCE>(to + threadIdx.x * 48);
}
template __global__ void probe<%s, %d, %s>(const char*, char*);
}
"""


@pytest.mark.parametrize("element,vec,align", [("F32", 8, 16), ("F32", 4, 16), ("F32", 1, 4), ("F16", 8, 16), ("BF16", 8, 16), ("BF16", 1, 2)])
@pytest.mark.parametrize("once", ["false", "true"])
def test_elements_promise_no_more_than_16_bytes(tmp_path, element, vec, align, once):
    """A launcher asks for rows aligned to 16 bytes (or to an element), so a load or store of several elements
    is not to be compiled as one of memory aligned to more."""
    source, ir = tmp_path / "probe.hip", tmp_path / "probe.ll"
    source.write_text(PROBE % (element, vec, once))
    subprocess.check_call([b.HIPCC, "-x", "hip", *b.COMMON, *b.DEVICE, "-I", b.CSRC, "--cuda-device-only", "-emit-llvm", "-S",
                           str(source), "-o", str(ir)], stderr=subprocess.DEVNULL)
    body = ir.read_text().split("define ", 1)[1].split("\n}", 1)[0]
    found = [int(n) for n in re.findall(r"(?:load|store) (?!ptr).*addrspace\(1\).*align (\d+)", body)]
    assert len(found) >= 2 and set(found) == {align}
