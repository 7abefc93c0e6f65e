"""The direct loads to LDS from an address of every lane's own (dma16_lane,
dma4_lane of csrc/common.h): a wait state between the write of M0 and the load.
The device code of a small kernel is compiled for gfx950 and read, without a GPU."""
import os
import re
import subprocess

import pytest

from exact_lloyd_means_03_amd import build

SOURCE = """
#include "common.h"
__global__ void k(const char* base, const uint32_t* off, uint32_t* out) {
    __shared__ __attribute__((aligned(16))) char lds[4096];
    for (int i = 0; i < 2; ++i) km::LOAD(base + off[threadIdx.x + 64 * i], lds + i * 1024 + threadIdx.x / 64 * 256);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    out[threadIdx.x] = ((uint32_t*)lds)[threadIdx.x];
}
"""


@pytest.mark.parametrize("load", ["dma16_lane", "dma4_lane"])
def test_wait_states_before_a_load(tmp_path, load):
    src = tmp_path / "k.hip"
    src.write_text(SOURCE.replace("LOAD", load))
    out = tmp_path / "k.s"
    subprocess.run([build.HIPCC, *build.CFLAGS, "-I", build.CSRC, "--cuda-device-only", "-S", str(src), "-o", str(out)],
                   check=True, capture_output=True, env=dict(os.environ))
    code = [re.sub(r"\s+", " ", line.split(";")[0].strip()) for line in out.read_text().splitlines()]
    code = [c for c in code if c and not c.startswith((".", "_", "#")) and not c.endswith(":")]
    loads = [i for i, c in enumerate(code) if c.startswith("global_load_lds")]
    assert len(loads) == 2
    for i in loads:
        assert re.fullmatch(r"global_load_lds_dword(x4)? v\[\d+:\d+\], off", code[i])
        assert re.match(r"s_nop [1-9]", code[i - 1]), code[i - 1]
