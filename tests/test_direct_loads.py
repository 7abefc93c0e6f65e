"""The direct loads to LDS (dma16, dma2 of csrc/common.h) keep the wait states
that the hardware wants between the writes of their operands and the load: the
device code of a small kernel is compiled for gfx950 and read, without a GPU.
"""
import os
import re
import subprocess

import pytest

from exact_lloyd_means_03_amd import build

# the base of a load straight from two v_readfirstlane, and LDS addresses (M0) that change
SOURCE = """
#include "common.h"
__global__ void k(const uint64_t* base, const uint32_t* off, uint32_t* out) {
    __shared__ __attribute__((aligned(16))) char lds[4096];
    for (int i = 0; i < 2; ++i) {
        const uint64_t b = base[threadIdx.x / 64 + i];
        const uint64_t u = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32 |
                           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
        km::LOAD((const char*)u, off[threadIdx.x], lds + i * 1024);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    out[threadIdx.x] = ((uint32_t*)lds)[threadIdx.x];
}
"""


def _wait_states(code, at, reg):
    """Wait states before instruction `at` since the last write of `reg` (five if none is near)."""
    n = 0
    for ins in reversed(code[:at]):
        if n >= 5:
            break
        op, _, rest = ins.partition(" ")
        dst = rest.split(",")[0].strip()
        if dst == reg:
            return n, op
        pair = re.fullmatch(r"s\[(\d+):(\d+)\]", dst)
        if pair and re.fullmatch(r"s\d+", reg) and int(pair[1]) <= int(reg[1:]) <= int(pair[2]):
            return n, op
        n += int(rest, 0) + 1 if op == "s_nop" else 1
    return 5, None


@pytest.mark.parametrize("load", ["dma16", "dma2"])
def test_wait_states_before_a_direct_load(tmp_path, load):
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
        base = re.search(r"s\[(\d+):(\d+)\]", code[i])
        for reg in (f"s{base[1]}", f"s{base[2]}"):
            n, op = _wait_states(code, i, reg)
            assert n >= 5 or not op.startswith("v_"), f"{op} of {reg} {n} wait states before {code[i]}"
        n, op = _wait_states(code, i, "m0")
        assert n >= 1, f"{op} of m0 directly before {code[i]}"
