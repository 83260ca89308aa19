"""What the 8-bit product's kernels rely on and no run shows while the compiler
happens to keep to it: seen in the assembly of code built here (host only)."""
import os
import re
import subprocess

import pytest

from speculative_sampling_verification_verify_amd import build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is missing")


def assembly(tmp_path, source):
    """The instructions and the compiler's remarks of a source file that sees the kernels."""
    src, out = tmp_path / "part.hip", tmp_path / "part.s"
    src.write_text('#include "sl_w4.h"\n#include "sl_f8.h"\n' + source)
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", "-I", os.path.dirname(build.SRC), str(src), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    return [line.strip() for line in out.read_text().splitlines()]


@pytest.mark.parametrize("form", ["1, 2, true", "2, 2, false"])
def test_results_through_lds_are_ordered(tmp_path, form):
    """A wavefront's lanes read in LDS what others wrote: a wavefront barrier lies between the writes of
    a row tile's results and the reads, and between these and the next row tile's writes."""
    code = assembly(tmp_path, f"template __global__ void sl::f8_tile_kernel<{form}>(sl::F8Args);\n")
    start = max(i for i, line in enumerate(code) if line.startswith("s_barrier"))   # behind the last product
    kinds = []
    for line in code[start:]:
        kind = "barrier" if "wave barrier" in line else "write" if line.startswith("ds_write") else \
            "read" if line.startswith("ds_read") else None
        if kind and (not kinds or kinds[-1] != kind):
            kinds.append(kind)
    assert kinds.count("write") >= 2 and kinds.count("read") >= 2
    for a, b in zip(kinds, kinds[1:]):
        assert (a, b) not in (("write", "read"), ("read", "write")), kinds


def test_loads_into_lds_leave_m0_to_the_compiler(tmp_path):
    """f8_to_lds and f8_word_to_lds write m0.  A load that the compiler itself sends to LDS behind them goes
    to its own address again."""
    code = assembly(tmp_path, """
__global__ void probe(const char* a, const char* b, char* out) {
  extern __shared__ __align__(16) char lds[];
  typedef __attribute__((address_space(3))) void* L;
  typedef __attribute__((address_space(1))) const void* G;
  __builtin_amdgcn_global_load_lds((G)(a + threadIdx.x * 16), (L)lds, 16, 0, 0);
  sl::f8_to_lds(b, threadIdx.x * 16, 4096);
  __builtin_amdgcn_global_load_lds((G)(a + threadIdx.x * 16), (L)lds, 16, 1024, 0);
  sl::f8_word_to_lds(b, threadIdx.x * 4, 8192);
  __builtin_amdgcn_global_load_lds((G)(a + threadIdx.x * 16), (L)lds, 16, 2048, 0);
  __syncthreads();
  out[threadIdx.x] = lds[threadIdx.x * 97];
}
""")
    seen = [("asm" if inside else "own", "m0" if re.match(r"s_mov_b32 m0\b", line) else "load")
            for line, inside in zip(code, _inside_asm(code)) if re.match(r"s_mov_b32 m0\b|global_load_lds", line)]
    assert seen == [("own", "m0"), ("own", "load"), ("asm", "m0"), ("asm", "load")] + \
        [("own", "m0"), ("own", "load"), ("asm", "m0"), ("asm", "load")] + [("own", "m0"), ("own", "load")], seen


def _inside_asm(code):
    """Of each line, whether it was written in inline assembly."""
    inside = False
    for line in code:
        inside = line == ";;#ASMSTART" or inside and line != ";;#ASMEND"
        yield inside
