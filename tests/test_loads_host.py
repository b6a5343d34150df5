"""Kernels start before the one they depend on has ended (programmatic dependent launch), so none may read through the path for
data that nobody writes in a kernel's lifetime."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_kernel_reads_through_the_read_only_path():
    """By an intrinsic or instruction of that path, or, in a kernel that waits for the one before it, by a pointer that lets the
    compiler choose it."""
    files = glob.glob(os.path.join(ROOT, "sparse_long_context_gb300", "csrc", "*.cu*"))
    assert len(files) > 15
    found, kernels = [], 0
    for f in sorted(files):
        with open(f, encoding="utf-8") as src:
            text = re.sub(r"//[^\n]*", "", src.read())
        found += [(os.path.basename(f), m) for m in re.findall(r"__ldg\s*\(|\bld\.global(?:\.\w+)*\.nc\b", text)]
        for part in text.split("__global__")[1:]:
            name, args = re.search(r"(\w+)\s*\(((?:[^()]|\([^()]*\))*)\)\s*\{", re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)", "", part)).groups()
            kernels += "pdl_wait" in part
            if "pdl_wait" in part:
                found += [(name, a.strip()) for a in args.split(",") if "const" in a and "__restrict__" in a]
    assert kernels > 20 and not found, found
