"""The whole C ABI in one place: what the headers declare, however a
declaration begins, is what the library exports and the binding knows."""
import os
import re
import shutil
import subprocess

import pytest

import nvfp4_post_quantization_amd as nq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ABI = {
    "nvfp4_status_string", "nvfp4_compute_scale2", "nvfp4_compute_scale2_batch", "nvfp4_hessian_workspace_bytes",
    "nvfp4_hessian_accum", "nvfp4_hessian_accum_noalloc", "nvfp4_hessian_accum_fq",
    "nvfp4_hessian_chunks_workspace_bytes", "nvfp4_hessian_accum_chunks", "nvfp4_hessian_accum_fq_chunks",
    "nvfp4_scale_sweep", "nvfp4_scale_sweep_ex", "nvfp4_scale_sweep_stats", "nvfp4_quantize_dynamic", "nvfp4_dequant",
    "mxfp4_to_nvfp4_cast", "fp8e4m3_compute_scale", "fp8e4m3_quantize", "fp8e4m3_dequant", "nvfp4_block_hadamard",
    "nvfp4_hessian_hadamard", "nvfp4_fakequant", "nvfp4_quantlinear_workspace_bytes", "nvfp4_quantlinear_forward",
    "nvfp4_probe_read", "nvfp4_probe_write", "nvfp4_probe_copy",
    "mxfp4_quantize", "mxfp4_dequant", "mxfp4_matmul_workspace_bytes", "mxfp4_matmul", "nvfp4_matmul_workspace_bytes",
    "nvfp4_matmul_w4a16", "nvfp4_matmul_w4a4", "nvfp4_moe_route", "nvfp4_moe_workspace_bytes", "nvfp4_moe_forward",
}


def test_headers_declare_the_abi():
    names = []
    for h in sorted(os.listdir(os.path.join(ROOT, "include"))):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h), encoding="utf-8").read(), flags=re.S)
        text = re.sub(r"^\s*#.*$", "", text, flags=re.M)
        names += re.findall(r"(\w+)\s*\([^(){};]*\)\s*;", text)
    assert len(names) == len(set(names)) and set(names) == ABI


def test_library_exports_the_abi():
    if not os.path.exists(nq.LIB_PATH):
        pytest.skip("libnvfp4mi.so not built")
    if not shutil.which("nm"):
        pytest.skip("no nm")
    out = subprocess.run(["nm", "-D", "--defined-only", nq.LIB_PATH], capture_output=True, text=True, check=True).stdout
    c_names = {l.split()[2] for l in out.splitlines() if l.split()[1] == "T" and not l.split()[2].startswith("_")}
    assert c_names == ABI


def test_binding_knows_the_abi():
    assert set(nq._SIGS) == ABI
