"""The norm's choice of threads and vectors for a row (norm_rows_form, csrc/mx_internal.h): a small host program compiled
against the header goes through every width that the entry point takes, for few rows and for many, and checks that the threads'
vectors cover the row, in whole warps and in a number that a kernel exists for.  No GPU is needed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "microscaled_precision_numerics_gb300", "csrc")

PROGRAM = r"""
#include "mx_internal.h"
#include "mxnum_layer.h"
#include <cstdio>

int main() {
    for (int64_t rows : {int64_t(1), int64_t(511), int64_t(512), int64_t(513), (int64_t(1) << 31) - 1})
        for (int64_t cols = 264; cols <= MX_RMSNORM_MAX_COLS; cols += 8) {
            const mxk::NormRowsForm f = mxk::norm_rows_form(rows, cols);
            const bool fits = f.nv == 1 || f.nv == 2 || f.nv == 4;
            if (!fits || f.threads <= 0 || f.threads % 32 || f.threads > mxk::NORM_ROWS_THREADS || (int64_t)f.nv * f.threads * 8 < cols) {
                std::printf("%lld rows of %lld columns: %d threads with %d vectors\n", (long long)rows, (long long)cols, f.threads, f.nv);
                return 1;
            }
        }
    std::printf("ok\n");
    return 0;
}
"""


def test_every_width_is_covered(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "forms.cu", tmp_path / "forms"
    src.write_text(PROGRAM)
    build = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2", "-I", CSRC, "-I",
                            os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
