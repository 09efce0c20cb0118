"""A rule of the kernels that are set up while the one before them drains, which no run can show: they read the
data of other kernels by plain loads.  A read-only load (ld.global.nc: __ldg, or a const __restrict__ pointer) needs
data that is constant for the kernel's whole life, the time before its grid_wait() included."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_embeddings_feature_gb300", "csrc")


def _code(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_kernels_that_wait_make_no_read_only_loads():
    early = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "launch_after(" in _code(p)]
    assert len(early) >= 4
    for path in early + [os.path.join(CSRC, "rows.cuh")]:
        code = _code(path)
        for word in ("__ldg", "__restrict__", ".nc"):
            lines = [line.strip() for line in code.splitlines() if word in line]
            assert not lines, (os.path.basename(path), lines)


def test_every_kernel_launched_early_waits():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        code = _code(path)
        if "launch_after(" not in code:
            continue
        for name, body in re.findall(r"__global__ void(?: __launch_bounds__\([^{;]*?\))? (\w+)\((?:[^{;]*)\) \{(.*?)\n\}", code,
                                     flags=re.S):
            assert "grid_wait();" in body, (os.path.basename(path), name)
