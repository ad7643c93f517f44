"""Error bounds of the operators of a residual block, beside layer_util's.

With e = 2^-24 (half a step of fp32):
  8 bits    a value v 448 / m that the arithmetic has to within a relative d may become any e4m3
            value between the nearest ones of (1 - d) and (1 + d) times it.  Values that are
            quantised as they are given carry the rounding of the product to fp32 and those of
            64-bit arithmetic: d = 1.01 e.  Behind the norm h and w enter exactly and r drops
            out: the same.  Behind a gate: sigmoid and its products as counted for
            the convolution (40 e), in v and in m: d = 100 e.
  scales    m / 448: given values, half a step of fp32; behind a norm the 100 e of a norm's output.
  norm      100 e, gradients 200 e of their terms, dweight 400 e (layer_util).
  products  fp32 results: sums of 128 products in fp32 (128 e), one scale product and fma for each
            block (3 e each, added over B blocks: B e) -> 132 + 2 B, of the terms' magnitudes.
            bf16 results: the 8-bit matrix instructions' sum of 128 products was measured at up to
            2^-16 of the sum of the magnitudes over 12800 results; four times that, 2^-14.
  clip      the norm is rounded once (its sum is 64-bit); a factor rounded to fp32 and a product
            rounded to the output's type.
"""
import numpy as np

from layer_util import E
from oracle import block as ref

HALF8 = 2.0 ** -4   # half a step of e4m3, relative


def in8(got, scaled, count, what):
    """got (e4m3) lies between the nearest values of scaled (1 - d) and (1 + d), d = 1.01 count e."""
    g = got.double().cpu().numpy().reshape(scaled.shape)
    d = 1.01 * count * E * np.abs(scaled)
    low, high = ref.nearest8(scaled - d), ref.nearest8(scaled + d)
    bad = ~((low <= g) & (g <= high))
    assert not bad.any(), "%s: %d of %d, at %s: %r for %r" % (what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0],
                                                             scaled[bad][0])


def matmul_count(depth):
    return 132 + 2 * (depth // 128)


ROUGH = 2.0 ** -14 / E   # the same as a count, for bf16 results
