"""Workspaces of the training-step operators without a GPU: a size of 256 bytes says that a call uses none, so no call
that uses some may report it, however little that is."""
import os
import shutil
import subprocess

import pytest

import orthogonalized_optimizer_step_amd as dion  # noqa: F401
from orthogonalized_optimizer_step_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "orthogonalized_optimizer_step_amd", "csrc")
lib = _lib.lib
BF16, FP32 = 0, 1
A, B, C, D, E, H = (0x10000000 * i for i in range(1, 7))   # far apart; nothing dereferences them
WORKSPACE, INVAL = -3, -1


# k in splits whose sums fit 256 bytes, and copies of a few unaligned rows
@pytest.mark.parametrize("m,n,k,b,ldb", [(1, 1, 7168, B, 7168), (1, 32, 7168, B, 7168), (2, 16, 7168, B, 7168),
                                         (16, 2, 7168, B, 7168), (1, 8, 14336, B, 14336), (1, 16, 14336, B, 14336),
                                         (17, 1, 128, B + 3, 128), (32, 4, 64, B + 1, 64), (17, 1, 128, B, 129)])
def test_little_scratch_of_a_product_is_asked_for_and_checked(m, n, k, b, ldb):
    need = lib.dion_int8_linear_workspace_size(A, k, b, ldb, m, n, k)
    assert need > 256

    def call(ws, have):
        return lib.dion_int8_linear(A, k, C, b, ldb, D, None, 0, E, n, m, n, k, BF16, ws, have, None)

    assert call(None, 0) == WORKSPACE and call(None, need) == WORKSPACE
    assert call(H, 0) == WORKSPACE and call(H, need - 1) == WORKSPACE and call(H + 16, need) == WORKSPACE
    assert call(A, need) == INVAL   # on top of an operand


# a few long rows in shares, whose parts fit 256 bytes
@pytest.mark.parametrize("rows,vocab,k,dt", [(1, 128256, 32, BF16), (1, 131072, 32, BF16), (2, 128256, 1, BF16),
                                             (1, 70001, 8, FP32)])
def test_little_scratch_of_a_distillation_step_is_asked_for_and_checked(rows, vocab, k, dt):
    need = lib.dion_distill_topk_workspace_size(rows, vocab, k, dt, 1)
    assert need > 256

    def call(ws, have):
        return lib.dion_distill_topk_step(A, vocab, B, C, None, D, E, vocab, rows, vocab, k, dt, BF16, 8, 1.0, ws, have,
                                          None)

    assert call(None, 0) == WORKSPACE and call(None, need) == WORKSPACE
    assert call(H, 0) == WORKSPACE and call(H, need - 1) == WORKSPACE and call(H + 16, need) == WORKSPACE
    assert call(A, need) == INVAL   # on top of the logits


def test_little_scratch_of_a_distillation_loss_is_asked_for_and_checked():
    rows, vocab, k = 1, 90000, 4
    need = lib.dion_distill_topk_workspace_size(rows, vocab, k, FP32, 0)
    assert need > 256

    def call(ws, have):
        return lib.dion_distill_topk(A, vocab, B, C, D, E, rows, vocab, k, FP32, BF16, 8, 1.0, ws, have, None)

    assert call(None, 0) == WORKSPACE and call(H, need - 1) == WORKSPACE and call(H + 16, need) == WORKSPACE
    assert call(A, need) == INVAL


def test_workspace_checks_for_any_scratch_under_asan_ubsan(tmp_path):
    """tests/host_check/train_workspace_check.cpp with train_api.cpp (sanitizers on the host compilation only)."""
    hipcc = "/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else shutil.which("hipcc")
    if not hipcc:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "train_workspace_check")
    cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip",
           os.path.join(CSRC, "train_api.cpp"), os.path.join(ROOT, "tests", "host_check", "train_workspace_check.cpp"),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "train workspace check:" in r.stdout
