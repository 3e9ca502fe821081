"""A product's epilogue hands its results on by runs of a register array, whose bounds the compiler checks.

A read past such an array is undefined, and nothing at run time need show it.  So the kernel's own templates are
instantiated here: what its kinds ask for compiles, and one run further does not.
"""
import os
import shutil
import subprocess

import pytest

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="needs nvcc")

SOURCE = """
#include "rlk_fp8_gemm.cuh"
namespace rlk {
__global__ void probe(const __grid_constant__ Ext8Params p) {
    extern __shared__ unsigned char out[];
    float2 v[%d];
    for (float2& x : v) x = make_float2(1.f, 2.f);
    %s;
}
}
"""
STORE = "store_chunk<%s, %s, %d, %d>(dest_of(p, 32), out, (int)threadIdx.x, 0, 0, v)"
ADD = "add_residual<%s, %d>(p, out, (int)threadIdx.x, 0, 32, 0, v)"


def compile_probe(tmp_path, pairs, call):
    src = tmp_path / "probe.cu"
    src.write_text(SOURCE % (pairs, call))
    build = rlk._build
    return subprocess.run(["nvcc", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", build.INCLUDE,
                           "-I", build.CSRC, "-c", str(src), "-o", os.devnull], capture_output=True, text=True)


# the last run of each kind's array: 64 pairs of a whole tile, 32 of a half one, of which gated 16 are the gate's
@pytest.mark.parametrize("pairs,call", [(64, STORE % ("false", "true", 32, 32)), (64, STORE % ("true", "false", 48, 16)),
                                        (32, STORE % ("false", "false", 16, 16)), (32, STORE % ("true", "false", 0, 16)),
                                        (64, ADD % ("true", 32))])
def test_runs_inside_the_array(tmp_path, pairs, call):
    r = compile_probe(tmp_path, pairs, call)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("pairs,call", [(32, STORE % ("false", "false", 16, 32)), (64, STORE % ("true", "true", 56, 16)),
                                        (32, ADD % ("false", 16))])
def test_runs_past_the_array(tmp_path, pairs, call):
    r = compile_probe(tmp_path, pairs, call)
    assert r.returncode != 0 and "a chunk's pairs are the array's" in r.stderr, r.stderr
