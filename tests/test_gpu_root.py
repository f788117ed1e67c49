"""The square root that 8-bit AdamW states are made with, against CUDA's for every float: their codes are the formula's
only as long as it is the IEEE root."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_every_float(mfsdp, tmp_path):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from matrix_optimizers_under_gb300 import _build
    exe = str(tmp_path / "root_sweep")
    build = subprocess.run([_build._nvcc()] + _build.NVCC_FLAGS + [os.path.join(ROOT, "tests", "c", "root_sweep.cu"), "-o",
                                                                   exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
