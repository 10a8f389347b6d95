"""Inputs and error bounds shared by the tests of the attention within molecules.

The bounds follow the arithmetic.  With u = 2^-24 (half a float32 step) and, for
bf16 storage, b = 2^-8 (half a bf16 step):

* A score is a float32 sum of dk products, a scaling, a tanh right to a few
  roundings of itself, a distance (differences, squares, their sum, an
  approximate root: below 8 u) and its product with the slope, all in base 2:
  below (dk + 16) u score + 16 u dist, score and dist as the oracle gives
  them.  Its weight carries that twice (numerator and normaliser), the
  exponential's own error (2 x 4 u), the normaliser's n additions (n u) and,
  in the backward pass, the stored lse's rounding (2 (score + dist + 16) u):
  WEIGHT below.
* m sums n terms: (n + 8) u of its terms' magnitudes.  On bf16 the weights may
  enter the products rounded once (b) and the result is rounded once (b).
* dP is a float32 sum of dv products, delta one of n terms of them; dS carries
  the weight's error twice.  From a stored bf16 m, delta carries 2 b of its
  terms.  On bf16, dS may enter the products rounded once (b); outputs are
  rounded once (b).
* f'(x) = 1 - tanh^2(x / cap) of a capped score: d ln f' / dx = -2 tanh / cap,
  so the (dk + 8) u score of x (and of the exponential's argument) moves f' by
  up to 2 (dk + 8) u score / cap of itself, which dq and dk carry.
"""
import numpy as np
import torch

from oracle.storage import round_bf16

U, B = 2.0 ** -24, 2.0 ** -8


def ptr_of(lengths, front=0):
    p = [front]
    for n in lengths:
        p.append(p[-1] + n)
    return p


def make(dtype, lmax, C, H, dk, lengths, queries=None, cap=0.0, bias=True, seed=0, front=0, behind=0, scale=1.5):
    """numpy inputs (already rounded to the storage type) of molecules with these lengths; ``queries``:
    query rows per molecule (None: the self form); front, behind: rows of no molecule."""
    r = np.random.default_rng(seed)
    st = round_bf16 if dtype == "bf16" else lambda a: np.asarray(a, np.float32).astype(np.float64)
    kp = ptr_of(lengths, front)
    qp = kp if queries is None else ptr_of(queries, front)
    nk, nq, D = kp[-1] + behind, qp[-1] + behind, (lmax + 1) ** 2
    d = dict(q=st(r.normal(size=(nq, H, dk)) * scale), k=st(r.normal(size=(nk, H, dk)) * scale),
             hp=st(r.normal(size=(nk, D, C))), q_ptr=qp, k_ptr=None if queries is None else kp, cap=cap)
    f32 = lambda a: np.asarray(a, np.float32).astype(np.float64)
    if bias:
        side = (10.0 * max(1, max(lengths, default=1))) ** (1 / 3)
        d["pos_q"] = f32((r.random((nq, 3)) - 0.5) * side)
        d["pos_k"] = None if queries is None else f32((r.random((nk, 3)) - 0.5) * side)
        d["slope"] = f32(2.0 ** (-6.0 * (np.arange(H) + 1) / H) * np.where(np.arange(H) % 5 == 4, -0.2, 1.0))
    g = st(r.normal(size=(nq, D, C)))
    return d, g


def shape_of(d, dtype):
    from equivariant_graph_attention_b200 import egat
    nq, H, dk = d["q"].shape
    nk, D, C = d["hp"].shape
    return egat.MoleculeShape(nq=nq, nk=nk, n_mol=len(d["q_ptr"]) - 1, lmax=int(round(D ** 0.5)) - 1, C=C, H=H,
                              dk=dk, dtype=dtype, cap=d["cap"])


def on_gpu(d, dtype):
    T = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = {}
    for n, a in d.items():
        if n == "cap":
            continue
        if a is None:
            out[n] = None
        elif n.endswith("ptr"):
            out[n] = torch.tensor(a, dtype=torch.int32, device="cuda")
        else:
            out[n] = torch.from_numpy(np.ascontiguousarray(a)).to("cuda", T if n in ("q", "k", "hp") else torch.float32)
    return out


def bounds(d, o, dtype):
    """Element-wise bounds of |got - oracle| for m, lse and every gradient in o."""
    b = B if dtype == "bf16" else 0.0
    dk, dv = d["q"].shape[2], d["hp"].shape[1] * d["hp"].shape[2] // d["q"].shape[1]
    kp = d["k_ptr"] if d["k_ptr"] is not None else d["q_ptr"]
    n = max([1] + [y - x for x, y in zip(kp, kp[1:])] + [y - x for x, y in zip(d["q_ptr"], d["q_ptr"][1:])])
    score = ((dk + 16) * o["score"] + 16 * o["dist"]) * U
    weight = 2 * score + (8 + n) * U + 2 * (o["score"] + o["dist"] + 16) * U
    ds = 3 * weight + (dv + 2 * n + 32) * U
    lse = np.where(np.isfinite(o["lse"]), o["lse"], 0.0)
    out = {"m": (weight + (n + 8) * U + b) * o["abs_m"] + b * np.abs(o["m"]),
           "lse": score + (n + 16) * U + 4 * U * np.abs(lse)}
    if "dq" in o:
        out["dhp"] = (weight + (n + 8) * U + b) * o["abs_dhp"] + b * np.abs(o["dhp"])
        for x in ("dq", "dk"):
            fx = 2 * (dk + 8) * U * o["score"] / d["cap"] if d["cap"] else 0.0
            out[x] = (ds + fx + (n + 8) * U + 3 * b) * o["abs_" + x] + b * np.abs(o[x])
        for x in ("dpos_q", "dpos_k", "dslope"):
            if x in o:
                out[x] = (ds + (2 * n + len(d["q_ptr"]) + 64) * U) * o["abs_" + x]
    return {x: v + 1e-30 for x, v in out.items()}


def close(got, want, bound, what=""):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    bad = ~(off <= bound) & ~((got == want))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(off / bound):.3g} of the "
                           f"bound at {np.unravel_index(np.nanargmax(off / bound), off.shape)}")
