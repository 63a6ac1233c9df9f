"""The bounds-checked debug build covers every kernel file that stores through hand-computed indices, and reports the
counts of every translation unit."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//.*", "", fh.read())


def test_row_kernels_and_gemm_epilogues_check_their_indices():
    for name in ("rowwise.cu", "gemm_tc.cuh", "block_rows.cu", "gemm_block_pair.cuh", "gemm_block_few.cuh"):
        assert "TPMLP_IN_BOUNDS(" in source(name), name


def test_every_row_kernel_of_the_block_scaled_operators_checks():
    # the checks of a row's chunk and vectors are in chunk_ok / row_ok; every kernel has one check at least
    text = source("block_rows.cu")
    kernels = re.split(r"__global__", text)[1:]
    assert len(kernels) == 5
    for k in kernels:
        assert re.search(r"TPMLP_IN_BOUNDS\(|chunk_ok\(|row_ok\(", k), k[:120]


def test_counts_of_every_translation_unit_are_reported():
    defined = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        defined |= set(re.findall(r"^cudaError_t (\w+_bounds_status)\(", source(os.path.basename(path)), re.M))
    assert {"rowwise_bounds_status", "gemm_bounds_status", "block_rows_bounds_status", "gemm_block_bounds_status"} <= defined
    read = set(re.findall(r"\b(\w+_bounds_status)\(&c\[", source("abi.cu")))
    assert read == defined
