"""Kernels are launched while the kernel before them in the stream may still run, and wait
for it on the device.  Data that it writes is not read only for their whole life then,
which is what loads through the read-only path (ld.global.nc, which __ldg is) ask for: what
comes from memory is read by plain loads."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_blackwell_tiled_gb300", "csrc")


def _code(path):
    with open(path, encoding="utf-8") as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_load_through_the_read_only_path():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    assert len(files) > 10
    for path in files:
        found = re.findall(r"__ldg\b|ld\.global\.[\w.]*\bnc\b|ld\.global\.nc", _code(path))
        assert not found, f"{os.path.basename(path)}: {found}"
