"""Inputs and error bounds shared by the tests of the operators around the scan.

Bounds.  With e = 2^-24 (half a step of fp32) an output may be off by the
rounding to its type, half a step of it relative to the value (bf16 2^-8, fp32
2^-24), and by the fp32 arithmetic before it, a count of e times the sum of
the magnitudes of the terms (`mag`).  The counts, from the formulas:
  conv      W fmas, a sigmoid of u (exp2 argument off by 2 |u| e, exp2 and
            reciprocal 1 ulp = 2 e each) and products; |u| < 12 in these tests:
            W + 2 + 24 + 8 -> 40.  Gradients: the slope of SiLU changes by up to
            half the error of u -> 64; sums of dweight run over at most 64
            tokens in a thread and 256 threads in fp32, then in 64 bits -> 400.
  selscan   a step size carries the rounding of dt + dt_bias (|bias| <= 8 against
            dt' ~ e^raw: 8 e) and a softplus (8 e) -> 16 e.  A term decayed by
            e^-v over time has its exponent off by (16 + 2) v e; terms with v > 20
            are below e of their undecayed size, which leaves 360 e; each of L
            steps rounds a and h twice, 4 L e; sums over states, channels and
            the gate 40 -> 400 + 4 L.  Sums over tokens or channels add at most
            64 + 256 fp32 roundings: gradients 800 + 8 L.
  norm      sums of positive terms over 32 additions at most, rsqrt, gate
            -> 100; gradients 200, dweight as conv.
"""
import numpy as np
import torch

E = 2.0 ** -24
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, count, mag, what, floor=1e-37):
    """|got - ref| <= half a step of got's type |ref| + count e mag + floor, where floor
    covers what falls below fp32's smallest normal value, 2^-126."""
    assert got is not None, what
    ref = np.asarray(ref)
    dtype, got = got.dtype, got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = half_step(dtype) * np.abs(ref) + 1.01 * count * E * np.asarray(mag) + floor
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d outside the bound, at %s: %r for %r (bound %.2g)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0], bound[bad][0])


class Draw:
    def __init__(self, seed, device="cuda"):
        self.g = torch.Generator().manual_seed(seed)
        self.device = device

    def normal(self, *shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=self.g) * std).to(dtype).to(self.device)

    def uniform(self, lo, hi, *shape, dtype=torch.float32):
        return (torch.rand(*shape, generator=self.g) * (hi - lo) + lo).to(dtype).to(self.device)

    def rows(self, *shape, pad=0, dtype=torch.float32, std=1.0):
        """A slice of rows that are `pad` elements longer at the front."""
        lead, last = shape[:2], int(np.prod(shape[2:]))
        t = self.normal(*lead, last + pad, dtype=dtype, std=std)[..., pad:]
        return t.unflatten(2, shape[2:]) if len(shape) > 3 else t


def cat(y):
    return y if isinstance(y, torch.Tensor) else torch.cat(list(y), 2)
