"""The operators around the scan where a launch is large enough to choose its other forms: long
runs of the convolution.  The tests repeat the launch rule a
case is meant for, so that one which no longer reaches its form says so."""
import pytest

import test_gpu_layer as base

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu(gpu_available):
    if not gpu_available:
        pytest.skip("needs a GPU")


def cdiv(a, b):
    return -(-a // b)


# ---- convolution: tokens per run, forwards (at most 16, 4096 waves) and backwards (64, 2048) ----

def run_of(batch, L, C, V, longest, enough):
    cv = cdiv(C, V)
    lanes = min(64, 1 << (cv - 1).bit_length())
    run = longest
    while run > 4 and batch * cdiv(cv, lanes) * lanes * cdiv(L, run) < enough * 64:
        run //= 2
    return run


# a case of test_gpu_layer, then channels per thread, runs forwards and backwards.  197 tokens end
# inside a run and inside a group of rows of every length
CONV = [
    ((512, 197, (33,), 2, 0, "fp32", True, True), 1, 16, 64),
    ((512, 197, (33,), 3, 0, "fp32", True, True), 1, 16, 64),
    ((512, 197, (33,), 4, 0, "bf16", True, True), 1, 16, 64),
    ((512, 197, (100, 16, 16), 2, 4, "bf16", True, True), 4, 16, 64),
    ((512, 197, (100, 16, 16), 3, 4, "bf16", False, True), 4, 16, 64),
    ((512, 197, (100, 16, 16), 4, 4, "fp32", True, True), 4, 16, 64),
    ((700, 192, (132,), 4, 4, "bf16", True, False), 4, 16, 64),     # whole runs only
    ((300, 197, (100, 32), 4, 4, "bf16", True, True), 4, 8, 32),
    ((190, 197, (33,), 4, 0, "fp32", True, True), 1, 8, 16),
    ((96, 197, (132,), 4, 4, "bf16", True, True), 4, 4, 8),
]


@pytest.mark.parametrize("case,V,fwd,bwd", CONV, ids=str)
def test_conv_runs(case, V, fwd, bwd):
    batch, L, C = case[0], case[1], sum(case[2])
    assert run_of(batch, L, C, V, 16, 4096) == fwd and run_of(batch, L, C, V, 64, 2048) == bwd
    base.test_conv_fwd(case)
    base.test_conv_bwd(case)
