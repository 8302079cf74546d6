"""What the kernels of shared prefixes take addresses from, on the CPU (the library's own header, compiled for the
host): words that no kernel wrote lead nowhere."""
import os
import subprocess

import pytest

from adapter_linear_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>
#include "kv_internal.h"
using namespace lora;

int main()
{
    const int grid = 152;
    unsigned long long x = 88172645463325252ull;  // xorshift: any 64 bits
    int taken = 0;
    for (int i = 0; i < 2000000; ++i) {
        x ^= x << 13; x ^= x >> 7; x ^= x << 17;
        uint2 w = make_uint2((uint32_t)x, (uint32_t)(x >> 32));
        if (i & 1) w.x &= 0x00FF00FFu;             // numbers near the grid's
        if (i & 2) w.y &= 0x1FFu;                  // and near a block's rows
        const uint2 got = kv_where(w, grid);
        const int c0 = w.x & 0xFFFF, c1 = w.x >> 16;
        const bool fits = c0 <= c1 && c1 < grid && w.y < (uint32_t)kShareRows;
        if (got.y != w.y || got.x != (fits ? w.x : kJoined)) return 1;
        taken += fits;
    }
    if (taken < 1000) return 2;                    // (both outcomes were seen)
    // the ends of what is valid, and just beyond
    for (int c1 = 0; c1 < 2 * grid; ++c1)
        for (uint32_t row = 254; row < 258; ++row) {
            const bool fits = c1 < grid && row < 256;
            if ((kv_where(make_uint2((uint32_t)c1 << 16, row), grid).x != kJoined) != fits) return 3;
            if ((kv_where(make_uint2((uint32_t)c1 << 16 | c1, row), grid).x != kJoined) != fits) return 4;
            if (kv_where(make_uint2((uint32_t)c1 << 16 | (c1 + 1), row), grid).x != kJoined) return 5;
        }
    if (kv_where(make_uint2(kJoined, 0xFFFFFFFFu), grid).x != kJoined) return 6;
    puts("ok");
    return 0;
}
"""


def test_words_that_no_kernel_wrote_are_not_followed(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(cuda_build.nvcc())), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no CUDA headers")
    source, program = tmp_path / "where.cpp", tmp_path / "where"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", cuda, "-I", cuda_build.CSRC, str(source), "-o", str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0 and done.stdout == "ok\n"
