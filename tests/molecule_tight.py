"""Tight error bounds of bf16 storage for the attention within molecules.

molecule_util's bounds leave room for weights and dS that enter a product rounded
to bf16 once.  Here they enter as a sum of two bf16 numbers: the first leaves half
a step, b = 2^-8, of the number, the second half a step of that, so P = 2^-16 of
every term.  What is left of b is the one rounding of each output:

* m, dh': P of the terms (the weights), then the output's rounding.
* dq: P of the terms of dS', which is taken from delta' = G . m with the stored m;
  delta' is off by up to b sum |G| |m| <= b sum_j a_ij |dP_ij| (terms in magnitude),
  and the sum that takes this out again holds the weights to b: b^2 = P.  3 P covers
  both, with delta' (1 + b) times its own size.
* dk: P of the terms of dS.
* An output's rounding acts on the number with its error: the factor 1 + b.
"""
import numpy as np

from tests.molecule_util import B, U, bounds

P = B * B


def tight(d, o):
    """Element-wise bounds of bf16 outputs, as molecule_util.bounds gives them."""
    out = bounds(d, o, "bf16")
    f32 = bounds(d, o, "f32")                  # the float32 arithmetic alone
    for x, planes in (("m", 1), ("dhp", 1), ("dq", 3), ("dk", 3)):
        if x in o:
            out[x] = (f32[x] + planes * P * o["abs_" + x]) * (1 + B) + B * np.abs(o[x])
    return out


def packed_bytes(shape):
    """Workspace of the forward pass where it takes the tcgen05 kernels: keys, values and positions in blocks of
    64 rows of a head, queries in blocks of 128, a block for every slot that a row tile can have."""
    up = lambda x, m: (x + m - 1) // m * m
    dv, ks = shape.D * shape.C // shape.H, 2 if shape.dk > 16 else 1
    key = 64 * 16 * (2 * ks + up(dv // 8, 2) + 1)
    slots = lambda n, rows: n // rows + shape.n_mol + 2
    return up(slots(shape.nk, 64) * shape.H * key, 256) + up(slots(shape.nq, 128) * shape.H * 2 * ks * 128 * 16, 256)
