"""Cases for the attention within each molecule and the layer norm: inputs, plain forms, exact forms and sizes.

A molecule of the batch is a run of consecutive rows, given by row pointers.  Every query row attends to all
key rows of its own molecule:

    s_ij = f(q_i.k_j / sqrt(dk)) - slope |r_i - r_j|,   f(x) = x, or cap tanh(x / cap)
    m_i  = sum_j softmax_j(s_ij) h'_j

Ops: ``attention`` (forward), ``attention_train`` (forward and gradients), ``norm`` and ``norm_train`` (layer norm
of the degree-0 channels inside rows of irreps, or of dense rows).
"""
import math
import random

import torch

own = False

EPS = 1e-5


def _attention(name, op="attention", dtype="bf16", lmax=2, C=128, H=16, dk=16, molecules=1, shortest=64,
               longest=64, queries=0, cap=0.0, bias=True, positions=False):
    c = dict(op=op, dtype=dtype, lmax=lmax, C=C, H=H, dk=dk, molecules=molecules, shortest=shortest,
             longest=longest, queries=queries, cap=cap, bias=bias, positions=positions)
    return dict(c, name=name) if name else c


def _norm(name, op="norm_train", dtype="bf16", rows=1, width=128, degrees=1):
    c = dict(op=op, dtype=dtype, rows=rows, width=width, degrees=degrees)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the tiny float32 system: one call's latency
        _attention("tiny_f32", dtype="f32", lmax=1, C=16, H=2, dk=8),
        # inference over a batch of drug-sized molecules, hydrogens included
        _attention("batch_512", molecules=512, shortest=5, longest=120),
        # the 216-water box in float32
        _attention("water_f32", dtype="f32", shortest=648, longest=648),
        # one condensed system with capped logits and decay over distance
        _attention("system_4096_capped", shortest=4096, longest=4096, cap=20.0),
        # the largest: degree-3 values, plain softmax
        _attention("system_8191_l3", lmax=3, shortest=8191, longest=8191, bias=False),
        # one probe atom against a long system (insertion energies): the single-row form
        _attention("probe_1", queries=1, shortest=32768, longest=32768),
        # a few probes in each of several systems of uneven size
        _attention("probes_8x7", molecules=8, queries=7, shortest=900, longest=9000, cap=20.0),
        # a training step over a batch of molecules with forces
        _attention("train_batch_256", op="attention_train", molecules=256, shortest=5, longest=120, positions=True),
        # a training step on one system of 4,096 atoms, positions fixed
        _attention("train_4096_capped", op="attention_train", shortest=4096, longest=4096, cap=20.0),
        # a float32 training step on small molecules, forces wanted
        _attention("train_f32", op="attention_train", dtype="f32", lmax=1, C=32, H=4, dk=8, molecules=24,
                   shortest=9, longest=150, positions=True),
        # the degree-0 scalars of 32,768 atoms, read in place from rows of nine components
        _norm("norm_scalars_32768", rows=32768, width=128, degrees=9),
        # wide dense rows of a large batch, forward alone
        _norm("norm_100000x1000", op="norm", rows=100000, width=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        op, dtype = rng.choice(["norm", "norm_train"]), rng.choice(["f32", "bf16"])
        if rng.random() < 0.5:
            return _norm(None, op=op, dtype=dtype, rows=_log(rng, 1, 60000), width=rng.choice([16, 32, 64, 128]),
                         degrees=rng.choice([1, 4, 9, 16]))
        width = _log(rng, 8, 4096)
        return _norm(None, op=op, dtype=dtype, rows=_log(rng, 1, max(2, 40_000_000 // width)), width=width)
    lmax = rng.choice([0, 1, 2, 2, 3])
    C, H, dk = rng.choice([(16, 2, 8), (32, 4, 8), (64, 8, 16), (128, 16, 16), (128, 16, 16), (128, 16, 16), (128, 8, 32),
                           (64, 4, 16)])
    kw = dict(dtype=rng.choice(["f32", "bf16", "bf16"]), lmax=lmax, C=C, H=H, dk=dk, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
              bias=rng.random() < 0.7)
    kind = rng.choice(["batch", "system", "probes"])
    if kind == "probes":
        return _attention(None, molecules=rng.choice([1, 1, 3, 8]), queries=_log(rng, 1, 64),
                          shortest=_log(rng, 200, 2000), longest=_log(rng, 2000, 12000), **kw)
    if rng.random() < 0.45:
        kw.update(op="attention_train", positions=kw["bias"] and rng.random() < 0.5)
    train = "op" in kw
    if kind == "batch":
        longest = _log(rng, 20, 200)
        return _attention(None, molecules=_log(rng, 4, 256 if train else 600), shortest=rng.randint(1, 12), longest=longest, **kw)
    n = _log(rng, 100, 2600 if train else 4200)
    return _attention(None, shortest=n, longest=n, **kw)


# ---- inputs

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lengths(c):
    """Atoms per molecule, from the case alone."""
    r = random.Random(c["molecules"] * 1000003 + c["shortest"] * 1009 + c["longest"])
    n = [r.randint(c["shortest"], max(c["shortest"], c["longest"])) for _ in range(c["molecules"])]
    return n, ([c["queries"]] * len(n) if c["queries"] else n)


def _ptr(lengths):
    p = [0]
    for n in lengths:
        p.append(p[-1] + n)
    return p


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, type=T):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(type)

    if case["op"].startswith("norm"):
        n, W, D = case["rows"], case["width"], case["degrees"]
        h = (torch.randn((n, D, W), generator=g, device="cuda") * 1.5 + 0.25).to(T)
        s = dict(case=case, x=h[:, 0, :], weight=1.0 + 0.1 * normal(W, type=torch.float32),
                 bias=0.1 * normal(W, type=torch.float32))
        if case["op"] == "norm_train":
            s["grad"] = normal(n, W)
        return s
    nk, nq = _lengths(case)
    kp, qp = _ptr(nk), _ptr(nq)
    H, dk, D, C = case["H"], case["dk"], (case["lmax"] + 1) ** 2, case["C"]
    wide = 2.0 if case["cap"] else 1.0  # capped logits are those that grow
    s = dict(case=case, longest_q=max(nq), longest_k=max(nk), q=normal(qp[-1], H, dk, scale=wide),
             k=normal(kp[-1], H, dk, scale=wide), hp=normal(kp[-1], D, C),
             q_ptr=torch.tensor(qp, dtype=torch.int32, device="cuda"))
    s["k_ptr"] = torch.tensor(kp, dtype=torch.int32, device="cuda") if case["queries"] else None
    if case["bias"]:
        # 0.1 atoms per cubic Angstrom, each molecule centred

        def atoms(lengths):
            side = torch.tensor([(10.0 * n) ** (1 / 3) for n in nk], device="cuda")
            side = torch.repeat_interleave(side, torch.tensor(lengths, device="cuda"))
            return (torch.rand((sum(lengths), 3), generator=g, device="cuda") - 0.5) * side[:, None]

        s["pos_q"] = atoms(nq)
        s["pos_k"] = atoms(nk) if case["queries"] else None
        s["slope"] = torch.tensor([2.0 ** (-6.0 * (h + 1) / H) for h in range(H)], device="cuda")
    if case["op"] == "attention_train":
        s["grad"] = normal(qp[-1], D, C)
    return s


# ---- one pass

def run(state):
    if own:
        return _own(state)
    return _plain_norm(state) if state["case"]["op"].startswith("norm") else _plain_attention(state)


def _own(s):
    from equivariant_graph_attention_b200 import egat
    c = s["case"]
    if c["op"].startswith("norm"):
        if c["op"] == "norm":
            return {"y": egat.egat_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)[0]}
        y, stats = egat.egat_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, want_stats=True)
        dx, dw, db = egat.egat_layer_norm_backward(s["x"], s["weight"], stats, s["grad"])
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    q, k, hp = s["q"], s["k"], s["hp"]
    shape = egat.MoleculeShape(nq=q.shape[0], nk=k.shape[0], n_mol=c["molecules"], lmax=c["lmax"], C=c["C"], H=c["H"],
                               dk=c["dk"], dtype=c["dtype"], cap=c["cap"])
    bias = dict(pos_q=s.get("pos_q"), pos_k=s.get("pos_k"), slope=s.get("slope"))
    train = c["op"] == "attention_train"
    m, lse = egat.egat_molecule_attention(shape, q, k, hp, s["q_ptr"], s["k_ptr"], want_lse=train, **bias)
    if not train:
        return {"m": m}
    dq, dk, dhp, dpos, _, dslope = egat.egat_molecule_attention_backward(
        shape, q, k, hp, s["q_ptr"], m, lse, s["grad"], s["k_ptr"], positions=c["positions"], **bias)
    out = {"m": m, "dq": dq, "dk": dk, "dhp": dhp}
    if c["positions"]:
        out.update(dpos=dpos, dslope=dslope)
    return out


def _plain_norm(s):
    x = s["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    xh = d * rstd
    y = (xh * s["weight"] + s["bias"]).to(s["x"].dtype)
    if "grad" not in s:
        return {"y": y}
    g = s["grad"].float()
    t = g * s["weight"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype), "dweight": (g * xh).sum(0, dtype=torch.float64).float(),
            "dbias": g.sum(0, dtype=torch.float64).float()}


def _rows(ptr, n, longest):
    """Rows of each molecule, padded to the longest, and which of them are there; each row's place in that table."""
    a = torch.arange(longest, device="cuda")
    start, end = ptr[:-1, None].long(), ptr[1:, None].long()
    at = torch.arange(n, device="cuda")
    b = torch.searchsorted(ptr.long(), at, right=True) - 1
    return (start + a).clamp(max=n - 1), start + a < end, (b, at - ptr.long()[b])


def _plain_attention(s):
    c = s["case"]
    T, H, dk, cap = s["q"].dtype, c["H"], c["dk"], c["cap"]
    D, ch = (c["lmax"] + 1) ** 2, c["C"] // c["H"]
    nq, nk = s["q"].shape[0], s["k"].shape[0]
    qi, q_there, q_at = _rows(s["q_ptr"], nq, s["longest_q"])
    ki, k_there, k_at = _rows(s["k_ptr"] if s["k_ptr"] is not None else s["q_ptr"], nk, s["longest_k"])

    def split(x):  # [n, D, C] -> [molecules, H, rows, D * C / H]
        b, m = x.shape[:2]
        return x.float().view(b, m, D, H, ch).permute(0, 3, 1, 2, 4).reshape(b, H, m, D * ch)

    def join(x, at):  # and back, the padding left out
        b, _, m, _ = x.shape
        x = x.view(b, H, m, D, ch).permute(0, 2, 3, 1, 4).reshape(b, m, D, c["C"])
        return x[at].to(T)

    Q, K, V = s["q"][qi].float().transpose(1, 2), s["k"][ki].float().transpose(1, 2), split(s["hp"][ki])
    x = Q @ K.transpose(2, 3)
    x *= dk ** -0.5
    t = None
    if cap:
        t = torch.tanh(x / cap)
        x = cap * t
    if c["bias"]:
        xk = s["pos_k"] if s["pos_k"] is not None else s["pos_q"]
        diff = s["pos_q"][qi][:, :, None] - xk[ki][:, None]
        dist = diff.square().sum(-1).sqrt()
        x = x - s["slope"][:, None, None] * dist[:, None]
    x = x.masked_fill(~k_there[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp_()
    p /= p.sum(-1, keepdim=True)
    out = {"m": join(p @ V, q_at)}
    if "grad" not in s:
        return out
    G = split(s["grad"][qi]) * q_there[:, None, :, None]
    dS = G @ V.transpose(2, 3)
    dS -= (dS * p).sum(-1, keepdim=True)
    dS *= p
    out["dhp"] = join(p.transpose(2, 3) @ G, k_at)
    if c["positions"]:
        out["dslope"] = -(dS * dist[:, None]).sum((0, 2, 3), dtype=torch.float64).float()
        w = -(dS * s["slope"][:, None, None]).sum(1)
        w = torch.where(dist > 0, w / dist, 0.0)[..., None] * diff
        out["dpos"] = w.sum(2)[q_at] - w.sum(1)[k_at]
    if cap:
        dS *= 1 - t * t
    dS *= dk ** -0.5
    out["dq"] = (dS @ K).transpose(1, 2)[q_at].to(T)
    out["dk"] = (dS.transpose(2, 3) @ Q).transpose(1, 2)[k_at].to(T)
    return out


# ---- the definition in 64 bits, one molecule and some rows at a time

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_attention(s, case)


def _exact_norm(s):
    W = s["x"].shape[1]
    keep, dw, db = {"y": [], "dx": []}, 0.0, 0.0
    w = s["weight"].double()
    for r in range(0, s["x"].shape[0], 20000):
        x = s["x"][r:r + 20000].double()
        mu = x.sum(1, keepdim=True) / W
        sd = (((x - mu) ** 2).sum(1, keepdim=True) / W + EPS) ** 0.5
        z = (x - mu) / sd
        keep["y"].append(z * w + s["bias"].double())
        if "grad" in s:
            g = s["grad"][r:r + 20000].double()
            dw, db = dw + (g * z).sum(0), db + g.sum(0)
            g = g * w
            keep["dx"].append((g - (g.sum(1, keepdim=True) + z * (g * z).sum(1, keepdim=True)) / W) / sd)
    out = {"y": torch.cat(keep["y"])}
    return out if "grad" not in s else dict(out, dx=torch.cat(keep["dx"]), dweight=dw, dbias=db)


def _exact_attention(s, c):
    H, dk, cap, C, D = c["H"], c["dk"], c["cap"], c["C"], (c["lmax"] + 1) ** 2
    nk, nq = _lengths(c)
    train = "grad" in s
    q, k, hp = s["q"].double(), s["k"].double(), s["hp"].double()
    m = torch.zeros(q.shape[0], D, C, dtype=torch.float64, device="cuda")
    dq, dkk, dhp = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(hp)
    if c["bias"]:
        rq = s["pos_q"].double()
        rk = rq if s["pos_k"] is None else s["pos_k"].double()
        slope = s["slope"].double()
        dpos, dslope = torch.zeros_like(rq), torch.zeros_like(slope)
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        K = k[k0:k0 + b]
        V = hp[k0:k0 + b].view(b, D, H, C // H)
        step = max(1, 60_000_000 // (b * H))
        for r in range(0, a, step):
            rows = slice(q0 + r, q0 + min(a, r + step))
            logit = torch.einsum("ihd,jhd->hij", q[rows], K) / math.sqrt(dk)
            score = cap * torch.tanh(logit / cap) if cap else logit
            if c["bias"]:
                d = torch.linalg.vector_norm(rq[rows, None] - rk[None, k0:k0 + b], dim=2)
                score = score - slope[:, None, None] * d
            w = torch.softmax(score, 2)
            m[rows] = torch.einsum("hij,jdhc->idhc", w, V).reshape(-1, D, C)
            if not train:
                continue
            G = s["grad"][rows].double().view(-1, D, H, C // H)
            dw = torch.einsum("idhc,jdhc->hij", G, V)
            dhp[k0:k0 + b] += torch.einsum("hij,idhc->jdhc", w, G).reshape(b, D, C)
            ds = w * (dw - (w * dw).sum(2, keepdim=True))
            if c["positions"]:
                dslope -= (ds * d).sum((1, 2))
                u = -(ds * slope[:, None, None]).sum(0) / torch.where(d > 0, d, torch.inf)
                dpos[rows] += u.sum(1, keepdim=True) * rq[rows] - u @ rk[k0:k0 + b]
                dpos[k0:k0 + b] += u.sum(0)[:, None] * rk[k0:k0 + b] - u.T @ rq[rows]
            if cap:
                ds = ds / torch.cosh(logit / cap) ** 2
            dq[rows] = torch.einsum("hij,jhd->ihd", ds, K) / math.sqrt(dk)
            dkk[k0:k0 + b] += torch.einsum("hij,ihd->jhd", ds, q[rows]) / math.sqrt(dk)
        q0, k0 = q0 + a, k0 + b
    if not train:
        return {"m": m}
    out = {"m": m, "dq": dq, "dk": dkk, "dhp": dhp}
    return dict(out, dpos=dpos, dslope=dslope) if c["positions"] else out


# ---- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n = case["rows"] * case["width"]
        train = case["op"] == "norm_train"
        return {"bytes": n * e * (4 if train else 2) + 8 * case["width"] * (2 if train else 1), "flops": n * (20 if train else 8)}
    nk, nq = _lengths(case)
    pairs, H, dk, D, C = sum(a * b for a, b in zip(nq, nk)), case["H"], case["dk"], (case["lmax"] + 1) ** 2, case["C"]
    Nq, Nk, dv = sum(nq), sum(nk), D * C // H
    b = e * ((Nq + Nk) * H * dk + (Nq + Nk) * D * C)
    f = 2 * pairs * H * (dk + dv)
    if case["bias"]:
        b += 12 * (Nq + (Nk if case["queries"] else 0))
    if case["op"] == "attention_train":
        b += e * ((Nq + Nk) * H * dk + (Nq + Nk) * D * C) + (12 * Nq if case["positions"] else 0)
        f += 2 * pairs * H * (2 * dk + 2 * dv)
    return {"bytes": b, "flops": f}
