"""The operators around the scan where a launch is large enough to choose its other forms: long
runs of the convolution, several batches per lane of the token scan, one chunk for a whole prompt,
long chunks of the gradients, every number of pieces of the norm.  The tests repeat the launch
rule a case is meant for, so that one which no longer reaches its form says so."""
import numpy as np
import pytest

import state_space_sequence_03_amd as lib
import test_gpu_layer as base
from layer_util import within
from oracle import layer as ref

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


# ---- selective scan: batches per lane of the token form ----

# two from 16384 waves' worth of lanes on (RN lanes hold a channel); the odd batch is left alone
# in its lane
STEP = [
    (129, 2, 2050, 16, 2, "bf16", True, True, True, "softplus"),
    (129, 1, 2049, 13, 1, "fp32", False, True, True, "softplus"),      # no vector fits
    (129, 3, 1030, 19, 1, "bf16", True, True, False, "given"),
    (130, 1, 1024, 32, 1, "fp32", True, True, True, "clamped"),
    (131, 1, 520, 64, 2, "fp32", True, False, True, "softplus"),
]


@pytest.mark.parametrize("case", STEP, ids=str)
def test_token_scan_of_many_batches(case):
    batch, D, N = case[0], case[2], case[3]
    rn = 4 if N <= 16 else 8 if N <= 32 else 16
    assert batch * D * rn // 64 >= 2 * 8192
    base.test_scan_step(case)


# ---- selective scan: chunks ----

def scan_waves(batch, D, G, cw):
    return batch * G * cdiv(D // G, cw)


# prompts of more than 64 tokens in one chunk, from 720 waves of 64, 32 or 16 channels on
ONE_CHUNK = [
    (45, 133, 1030, 4, 1, "bf16", True, True, True, "softplus"),
    (46, 97, 512, 24, 1, "fp32", True, False, True, "softplus"),
    (46, 66, 510, 20, 2, "bf16", False, True, True, "given"),
    (45, 70, 260, 64, 1, "fp32", False, True, False, "clamped"),
]


@pytest.mark.parametrize("case", ONE_CHUNK, ids=str)
def test_prompts_in_one_chunk(case):
    batch, L, D, N, G = case[:5]
    assert scan_waves(batch, D, G, 64 if N <= 16 else 32 if N <= 32 else 16) >= 720 and L > 64
    base.test_scan_fwd(case)


# gradients in chunks of 32 tokens with more than 16 states, from 2048 waves on
LONG_CHUNKS = [
    (8, 263, 512, 32, 1, "bf16", True, True, True, "softplus"),
    (8, 263, 510, 19, 2, "fp32", False, True, False, "given"),
    (4, 263, 500, 64, 1, "fp32", True, False, True, "clamped"),
]


@pytest.mark.parametrize("case", LONG_CHUNKS, ids=str)
def test_gradients_in_long_chunks(case):
    batch, L, D, N, G = case[:5]
    assert scan_waves(batch, D, G, 16 if N <= 32 else 8) * cdiv(L, 32) >= 2048
    d, s, init, opt, ropt = base.scan_case(case)
    dy = d.normal(*s["x"].shape, dtype=s["x"].dtype)
    dfin = d.normal(batch, D, N) if init is not None else None
    got = lib.ssd_selscan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], init, dy, dfin,
                              want_dinit=True, want_ddt_bias=True, **opt)
    want = ref.selscan_bwd(**s, init=init, dy=dy, dfinal=dfin, **ropt)
    a = lambda t: None if t is None else np.abs(ref.f64(t))
    m = base.scan_mag(s)
    m["z"] = ref.f64(s["z"])
    mag = ref.selscan_bwd(**m, init=a(init), dy=a(dy), dfinal=a(dfin), mag=True, **ropt)
    count = 800 + 8 * L
    if s["z"] is not None:
        # The slope of SiLU, f = p (1 + z (1 - p)) with p = 1 / (1 + e^-z), is zero near -1.28,
        # where its roundings are not a part of itself: p is off by (2 |z| + 5) e of itself, which f
        # takes times |1 + z - 2 p z| <= 1.1 + |z|, and three more operations by p (1 + |z|) e each.
        # With |z| <= 6: 17 x 7.1 + 3 x 7 < 150 e, times |dy| and the terms of s.
        assert m["z"].max() <= 6 and m["z"].min() >= -6
        mag["dz"] = mag["dz"] + 150.0 / count * a(dy) * ref.selscan(**dict(m, z=None), init=a(init), **ropt)[2]
    for k, v in got.items():
        if v is not None:
            within(v, want[k], count, mag[k], k)


# ---- norm: pieces per thread ----

# a case of test_gpu_layer, then elements per piece, threads of a group, pieces per thread
NORM = [
    ((2, 5, 1500, 3, "fp32", True, 4, False), 4, 64, 2),
    ((2, 5, 1400, 2, "fp32", True, 0, True), 4, 64, 3),
    ((2, 5, 1000, 1, "fp32", True, 4, False), 4, 64, 4),
    ((1, 3, 2052, 1, "fp32", True, 4, False), 4, 192, 3),
    ((2, 5, 303, 3, "bf16", True, 1, False), 1, 64, 2),
    ((2, 5, 300, 2, "bf16", True, 0, True), 1, 64, 3),
    ((2, 5, 233, 1, "fp32", True, 3, False), 1, 64, 4),
    ((1, 3, 2049, 1, "bf16", True, 0, False), 1, 576, 4),
    ((2, 3, 2010, 2, "bf16", True, 0, False), 1, 256, 4),
]


@pytest.mark.parametrize("case,V,threads,pieces", NORM, ids=str)
def test_norm_pieces(case, V, threads, pieces):
    S = case[2] // case[3]
    n = cdiv(S, V)
    wide = 8 if V == 1 and n > 4096 else 2 if V == 8 else 4
    assert S % 8 != 0 or V == 4
    assert n > 64 and cdiv(n, 64 * wide) * 64 == threads and cdiv(n, threads) == pieces
    base.test_norm_fwd(case)
    base.test_norm_bwd(case)
