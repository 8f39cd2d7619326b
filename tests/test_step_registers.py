"""A block of the one-token kernel of the delta rule holds its share of the
state in registers, for every head size that it takes: the largest forms (16
rows per thread) spill none, the others at most two values that are not the
state's (their occupancy is worth more)."""
import importlib.util
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_step_kernel_holds_its_state_in_registers(tmp_path):
    path = os.path.join(ROOT, "fft_convolution_gb300", "build.py")
    spec = importlib.util.spec_from_file_location("fft_convolution_gb300_build", path)
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    source = os.path.join(build.CSRC, "delta_step.cu")
    done = subprocess.run([build.nvcc()] + build.ARCH + build.NVCC_FLAGS +
                          ["-Xptxas", "-v", "-c", source, "-o", str(tmp_path / "delta_step.o")],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    rows = [int(n) for n in re.findall(r"entry function '\S*delta_step_kernelI\S*?Li(\d+)E", done.stderr)]
    spilled = [int(n) for n in re.findall(r"(\d+) bytes spill stores", done.stderr)]
    assert len(rows) == len(spilled) == 27  # three types, three row counts, three ways to load
    assert all(n <= (0 if r == 16 else 8) for r, n in zip(rows, spilled)), list(zip(rows, spilled))
