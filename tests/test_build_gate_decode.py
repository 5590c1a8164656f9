"""Build gate on the register allocation of the decode-step kernels (CPU only: nvcc and ptxas, no
GPU), as tests/test_build_gate.py keeps the others': no kernel spills more than is listed here.

The shared prefix's kernel takes its scores and outputs from TMEM, by loads whose results must not
be stored before their wait; 25 warps leave a thread 72 registers.  tests/test_gpu_attention_range.py
runs it many times and compares the bits.  The cache write spills what 16 blocks an SM cost it (it
runs faster so), the attention kernel with 16 query rows what its second half's outputs cost it."""

import os
import re
import subprocess

import pytest

from conftest import ROOT

NVCC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")

# bytes of spill stores and loads, by what a kernel's mangled name holds; all others: none
BUDGET = {
    "attention.cu": {"attention_kernelILi128ELi16ELb0": (60, 64),
                     "attention_kernelILi128ELi16ELb1": (12, 12),
                     "attention_join_kernelILi64ELi8": (4, 4)},
    "attention_prefix.cu": {"prefix_kernel": (4, 8)},
    "kvcache.cu": {"kv_write_kernel": (32, 32)},
    "moe_decode.cu": {},
}


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no nvcc")
@pytest.mark.parametrize("src", BUDGET)
def test_spills_stay_within_budget(src):
    csrc = os.path.join(ROOT, "fp8_grouped_expert_gb300", "csrc")
    r = subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                        "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-Xptxas", "-v", "-c",
                        os.path.join(csrc, src), "-o", os.devnull], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    name, seen = None, 0
    for line in r.stderr.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            name = m.group(1)
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if not m or name is None:
            continue
        most = next((v for k, v in BUDGET[src].items() if k in name), (0, 0))
        assert int(m.group(1)) <= most[0] and int(m.group(2)) <= most[1], (name, line, most)
        name, seen = None, seen + 1
    assert seen, "ptxas reported no kernels"
