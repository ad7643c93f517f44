"""One token: the token strides of the operators around the scan then separate no rows, so any
value >= 0 is taken and none changes a result."""
import pytest
import torch

import state_space_sequence_03_amd as lib
from layer_util import Draw
from test_layer_boundary import BADVAL, SP, UNSUP, WS, scan_bwd, scan_fwd, so, st  # noqa: F401

FAR = 2 ** 27        # elements; 2^28 bytes of bf16, too far for several tokens


# ---- host checks, without a GPU ----

def test_a_far_stride_of_one_token_is_no_distance():
    # (no workspace: the call ends at the check after that of the strides)
    assert scan_bwd(SP(seqlen=1), dzs=st(64, FAR), n=0) == WS
    assert scan_bwd(SP(seqlen=1), dzs=st(64, 0), n=0) == WS
    assert scan_bwd(SP(), dzs=st(2 ** 40, FAR), n=0) == UNSUP     # two tokens are that far apart


def test_one_token_is_checked_all_the_same():
    assert scan_bwd(SP(seqlen=1), dzs=st(64, -1), n=0) == BADVAL
    assert scan_bwd(SP(seqlen=1), dzs=st(63, 0), n=0) == BADVAL   # batches overlap
    assert scan_fwd(SP(seqlen=1), zs=st(64, -1)) == BADVAL


# ---- results ----

on_gpu = pytest.mark.gpu
Bz, D, N = 3, 64, 16


@pytest.fixture
def draw(gpu_available):
    if not gpu_available:
        pytest.skip("needs a GPU")
    return Draw(61)


def at(t, token):
    """The one-token operand t at another token stride."""
    return t.as_strided(t.shape, (t.stride(0), token) + t.stride()[2:])


def odd_address(t):
    return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape).copy_(t)


def same(a, b):
    a, b = (list(v.values()) if isinstance(v, dict) else list(v) for v in (a, b))
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@on_gpu
@pytest.mark.parametrize("token", [0, 1, D // 2, FAR, 2 * FAR])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_token_strides_of_one_token(draw, token, io):
    n = lambda *s: draw.normal(*s, dtype=io)
    x, z, dy, dt = n(Bz, 1, D), n(Bz, 1, D), n(Bz, 1, D), draw.uniform(0.05, 0.3, Bz, 1, D, dtype=io)
    w, cw = draw.uniform(0.5, 1.5, D), draw.normal(D, 4)
    A, init = -draw.uniform(0.5, 2.0, D, N), draw.normal(Bz, D, N)
    B, C = n(Bz, 1, 1, N), n(Bz, 1, 1, N)
    out = lambda: at(torch.full_like(x, 7.0), token)
    # selective scan: z, B, C and dz
    want = lib.ssd_selscan_bwd(x, dt, A, B, C, None, z, init, dy, want_dinit=True)
    assert want["dz"].any(2).all()
    got = lib.ssd_selscan_bwd(x, dt, A, at(B, token), at(C, token), None, at(z, token), init, dy, want_dinit=True,
                              dz_out=out())
    assert same(got, want)
    assert same(lib.ssd_selscan_fwd(x, dt, A, at(B, token), at(C, token), None, at(z, token), init),
                lib.ssd_selscan_fwd(x, dt, A, B, C, None, z, init))
    a, b = init.clone(), init.clone()
    assert torch.equal(lib.ssd_selscan_step(a, x, dt, A, at(B, token), at(C, token), None, at(z, token)),
                       lib.ssd_selscan_step(b, x, dt, A, B, C, None, z)) and torch.equal(a, b)
    # convolution: x and dx
    assert same(lib.ssd_conv_fwd(at(x, token), cw, want_final_state=True), lib.ssd_conv_fwd(x, cw, want_final_state=True))
    assert same(lib.ssd_conv_bwd(at(x, token), cw, None, None, dy, dx_out=out()), lib.ssd_conv_bwd(x, cw, None, None, dy))
    # norm: z and dz.  An odd stride takes single elements, whose sums have another order, and
    # is compared with operands at an odd address, which do too
    like = odd_address if token % 2 else (lambda t: t)
    assert torch.equal(lib.ssd_gated_norm_fwd(x, at(z, token), w), lib.ssd_gated_norm_fwd(x, like(z), w))
    assert same(lib.ssd_gated_norm_bwd(x, at(z, token), w, dy, dz_out=out()),
                lib.ssd_gated_norm_bwd(x, like(z), w, dy, dz_out=like(torch.empty_like(z))))


@on_gpu
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_gradients_laid_out_like_an_x_of_one_token(draw, io):
    # [B, D, 1] transposed is contiguous, with a token stride of one element
    x = draw.normal(Bz, D, 1, dtype=io).transpose(1, 2)
    assert x.is_contiguous() and x.stride(1) == 1
    z, dy, dt = draw.normal(Bz, 1, D, dtype=io), draw.normal(Bz, 1, D, dtype=io), draw.uniform(0.05, 0.3, Bz, 1, D, dtype=io)
    A, B = -draw.uniform(0.5, 2.0, D, N), draw.normal(Bz, 1, 1, N, dtype=io)
    w, cw = draw.uniform(0.5, 1.5, D), draw.normal(D, 4)
    plain = torch.empty(Bz, 1, D, dtype=io, device="cuda").copy_(x)
    assert torch.empty_like(x).stride(1) == 1 and plain.stride(1) == D
    for call in (lambda x: lib.ssd_selscan_bwd(x, dt, A, B, B, None, z, None, dy),
                 lambda x: lib.ssd_conv_bwd(x, cw, None, None, dy),
                 lambda x: lib.ssd_gated_norm_bwd(x, z, w, dy)):
        assert same(call(x), call(plain))
