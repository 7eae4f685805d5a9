"""Cases for the library's gated expert block and its gradient, and for the
orthogonalised update of expert weights, in a plain form and through the
library.

Operators:
  gated          z = act(x W_gate^T) * (x W_up^T) over segments of rows, one
                 expert each, and the sums h before the activation, which a
                 training step keeps
  gated_grad     from the gradient dy of the block's output: dh, that of h,
                 through the down projection and the activation, and z again
                 for the gradient of the down projection's weights
  orthogonalize  five Newton-Schulz steps on every expert's matrix

With ``own`` false ``run`` computes them from elementary torch operations in
fp32; with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
# of each of the five steps: X <- a X + b (X X^T) X + c (X X^T)^2 X
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


# ------------------------------------------------------------------- cases
# recipe: the activation is SiLU(g) u, or with it g' sigmoid(1.702 g') (u' + 1) of
# values clamped at 7 (g from above, u on both sides)
def listed():
    return [
        # a few routed rows on a small layer in training: launch latency; odd
        # segments, outputs and inputs that end inside a tile
        dict(name="gated_tiny", op="gated", dtype="float16", rows=37, inter=264, hidden=520,
             experts=8, skew=1.0, keep=True, recipe=False),
        # one token, top-2, of a Mixtral-shaped layer: two experts' weights
        dict(name="gated_token", op="gated", dtype="bfloat16", rows=2, inter=14336, hidden=4096,
             experts=8, skew=0.0, keep=False, recipe=False),
        # 64 tokens, top-2, the same layer: bound by all the weights
        dict(name="gated_decode", op="gated", dtype="bfloat16", rows=128, inter=14336,
             hidden=4096, experts=8, skew=0.3, keep=False, recipe=False),
        # a training step of 4096 tokens, top-2: bound by the tensor cores
        dict(name="gated_prefill", op="gated", dtype="bfloat16", rows=8192, inter=14336,
             hidden=4096, experts=8, skew=0.0, keep=True, recipe=False),
        # 2048 tokens, top-8 over 256 experts, the clamped activation: few rows an
        # expert, so the weights count
        dict(name="gated_many_experts", op="gated", dtype="bfloat16", rows=16384, inter=2048,
             hidden=7168, experts=256, skew=0.5, keep=False, recipe=True),
        # fine-tuning step on a small layer: ragged everywhere
        dict(name="grad_small", op="gated_grad", dtype="float16", rows=515, inter=520,
             hidden=776, experts=16, skew=1.0, recipe=False),
        # 4096 tokens, top-2, the Mixtral-shaped layer
        dict(name="grad_prefill", op="gated_grad", dtype="bfloat16", rows=8192, inter=14336,
             hidden=4096, experts=8, skew=0.0, recipe=False),
        # 2048 tokens, top-8 over 256 experts, the clamped activation
        dict(name="grad_many_experts", op="gated_grad", dtype="bfloat16", rows=16384, inter=2048,
             hidden=7168, experts=256, skew=0.5, recipe=True),
        # fp32 momentum of a small layer's gate/up weights: many short products
        dict(name="ortho_small", op="orthogonalize", dtype="float32", experts=8, n=512, k=256),
        # sizes that no tile, vector or copy divides
        dict(name="ortho_odd", op="orthogonalize", dtype="bfloat16", experts=16, n=1031, k=517),
        # 16 of 256 experts (one GPU's share), down projection: more rows than columns
        dict(name="ortho_tall", op="orthogonalize", dtype="bfloat16", experts=16, n=7168, k=2048),
        # two experts of the Mixtral-shaped down projection, fp32 momentum
        dict(name="ortho_wide", op="orthogonalize", dtype="float32", experts=2, n=4096, k=14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "orthogonalize",
                     "orthogonalize"])
    if op == "orthogonalize":
        experts, n, k = _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 1, 8192)
        # at most the largest listed case's products
        experts = max(1, min(experts, int(4.8e11 / (min(n, k) ** 2 * max(n, k)))))
        if min(n, k) ** 2 * max(n, k) > 4.8e11:
            n = 4096
        return dict(op=op, dtype=rng.choice(["bfloat16", "float16", "float32"]),
                    experts=experts, n=n, k=k)
    experts = _log(rng, 1, 256)
    inter, hidden = 8 * _log(rng, 1, 1792), 8 * _log(rng, 1, 1024)
    hidden = min(hidden, max(8, 450000000 // (experts * inter) // 8 * 8))
    case = dict(op=op, dtype=rng.choice(["bfloat16", "float16"]), rows=_log(rng, 1, 8192),
                inter=inter, hidden=hidden, experts=experts, skew=rng.choice([0.0, 0.5, 1.0]),
                recipe=rng.choice([False, True]))
    if op == "gated":
        case["keep"] = rng.choice([False, True])
    return case


# ------------------------------------------------------------------ inputs
def _generator(seed, device):
    return torch.Generator(device=device).manual_seed(int(seed) * 7919 + 29)


def _segments(case, seed):
    """Rows of each expert: every routed row picks one by preferences of the
    stated spread, so small cases have experts without rows."""
    g = _generator(seed, "cpu")
    prefs = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g), 0)
    picks = torch.multinomial(prefs, case["rows"], replacement=True, generator=g)
    counts = torch.bincount(picks, minlength=case["experts"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]), int(counts.max())


def _normal(shape, scale, dtype, g):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=g)
    return t


def prepare(case, seed):
    g = _generator(seed, "cuda")
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if op == "orthogonalize":
        experts, n, k = case["experts"], case["n"], case["k"]
        # a gradient's spectrum: one strong direction over a broad rest
        s["g"] = _normal((experts, n, k), 0.01, dt, g)
        s["g"] += 0.02 * _normal((experts, n, 1), 1.0, dt, g) * _normal((experts, 1, k), 1.0, dt, g)
        return s
    offsets, s["longest"] = _segments(case, seed)
    s["offsets"] = offsets.to(device="cuda", dtype=torch.int32)
    rows, inter, hidden, experts = (case[v] for v in ("rows", "inter", "hidden", "experts"))
    if op == "gated":
        s["x"] = _normal((rows, hidden), 1.0, dt, g)
        # sums of a spread of about 1.5, or 3 for the clamped activation
        s["w13"] = _normal((experts, 2 * inter, hidden),
                           (3.0 if case["recipe"] else 1.5) / math.sqrt(hidden), dt, g)
        return s
    s["dy"] = _normal((rows, hidden), 1.0, dt, g)
    s["w2"] = _normal((experts, hidden, inter), 0.02, dt, g)
    s["h"] = _normal((rows, 2 * inter), 3.0 if case["recipe"] else 1.5, dt, g)
    return s


# -------------------------------------------------------------- plain forms
def _rows_to_blocks(s, t):
    """[R, C] rows as [E, longest, C] fp32, zeros behind each segment."""
    off = s["offsets"].long()
    at = torch.arange(s["longest"], device="cuda")
    inside = at < (off[1:] - off[:-1])[:, None]
    rows = (off[:-1, None] + at).clamp(max=t.shape[0] - 1)
    return torch.where(inside[..., None], t[rows].float(), 0.0)


def _blocks_to_rows(s, blocks, rows):
    off = s["offsets"].long()
    r = torch.arange(rows, device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return blocks[e, r - off[e]]


def _parameters(case):
    """alpha, beta and limit of the activation."""
    return (1.702, 1.0, 7.0) if case["recipe"] else (1.0, 0.0, math.inf)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "orthogonalize":
        a, b, c = COEFFICIENTS
        x = s["g"].float()
        if case["n"] > case["k"]:
            x = x.transpose(1, 2)
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
        for _ in range(STEPS):
            gram = x @ x.transpose(1, 2)
            x = a * x + (b * gram + c * (gram @ gram)) @ x
        if case["n"] > case["k"]:
            x = x.transpose(1, 2)
        return x.to(torch.bfloat16, memory_format=torch.contiguous_format)
    rows, inter, dt = case["rows"], case["inter"], DTYPES[case["dtype"]]
    alpha, beta, limit = _parameters(case)
    if op == "gated":
        h = torch.bmm(_rows_to_blocks(s, s["x"]), s["w13"].float().transpose(1, 2))
        h = _blocks_to_rows(s, h, rows)
        g, u = h[:, :inter], h[:, inter:]
        gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
        z = (gc / (1.0 + torch.exp(-alpha * gc)) * (uc + beta)).to(dt)
        return {"z": z, "h": h.to(dt)} if case["keep"] else {"z": z}
    dz = _blocks_to_rows(s, torch.bmm(_rows_to_blocks(s, s["dy"]), s["w2"].float()), rows)
    g, u = s["h"][:, :inter].float(), s["h"][:, inter:].float()
    gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    sig = 1.0 / (1.0 + torch.exp(-alpha * gc))
    act = gc * sig
    dg = dz * (uc + beta) * sig * (1.0 + alpha * gc * (1.0 - sig)) * (g <= limit)
    du = dz * act * (u.abs() <= limit)
    return {"dh": torch.cat([dg, du], 1).to(dt), "z": (act * (uc + beta)).to(dt)}


# ------------------------------------------------------- the library's calls
def _run_own(s):
    import mixture_experts_ffn_align_gb300 as moe

    case, op = s["case"], s["case"]["op"]

    def kept(name, make):   # workspace and output buffers that a program keeps
        if name not in s:
            s[name] = make()
        return s[name]

    def bytes_of(n):
        return torch.empty(max(int(n), 1), dtype=torch.uint8, device="cuda")

    if op == "orthogonalize":
        g = s["g"]
        out = kept("out", lambda: torch.empty(g.shape, dtype=torch.bfloat16, device="cuda"))
        ws = kept("ws", lambda: bytes_of(moe.moe_orthogonalize_workspace_bytes(*g.shape)))
        moe.moe_orthogonalize(g, out, ws, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return out
    rows, inter, hidden, dt = case["rows"], case["inter"], case["hidden"], DTYPES[case["dtype"]]
    off = s["offsets"]

    def buffer(name, *shape):
        return kept(name, lambda: torch.empty(*shape, dtype=dt, device="cuda"))

    act = dict(alpha=1.702, beta=1.0, limit=7.0) if case["recipe"] else {}
    z = buffer("z", rows, inter)
    if op == "gated":
        p = kept("plan", lambda: moe.Ragged(R=rows, N=2 * inter, K=hidden, E=case["experts"],
                                            dtype=case["dtype"]))
        ws = kept("ws", lambda: bytes_of(moe.moe_ragged_workspace_bytes(p)))
        h = buffer("h", rows, 2 * inter) if case["keep"] else None
        moe.ragged_gated(p, s["x"], s["w13"], off, z, ws, h=h, **act)
        return {"z": z, "h": h} if case["keep"] else {"z": z}
    p = kept("plan", lambda: moe.Ragged(R=rows, N=hidden, K=inter, E=case["experts"],
                                        dtype=case["dtype"]))
    ws = kept("ws", lambda: bytes_of(moe.moe_ragged_workspace_bytes(p)))
    dh = buffer("dh", rows, 2 * inter)
    moe.ragged_gated_dgrad(p, s["dy"], s["w2"], s["h"], off, dh, ws, z=z, **act)
    return {"dh": dh, "z": z}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- definition, 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "orthogonalize":
        small, large = sorted((case["n"], case["k"]))
        # fp64 products at about 1 TFLOP/s
        if case["experts"] * STEPS * 2.0 * small * small * (2 * large + small) > 1.3e13:
            return None
        s = prepare(case, seed)
        out = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
        for i, m in enumerate(s["g"]):
            x = m.double() if case["n"] <= case["k"] else m.double().T
            x = x / (torch.linalg.vector_norm(x) + EPS)
            eye = torch.eye(x.shape[0], dtype=torch.float64, device="cuda")
            for _ in range(STEPS):
                gram = x @ x.T
                # Horner's form of the polynomial in the Gram matrix
                x = (COEFFICIENTS[0] * eye
                     + gram @ (COEFFICIENTS[1] * eye + COEFFICIENTS[2] * gram)) @ x
            out[i] = x if case["n"] <= case["k"] else x.T
        return out
    s = prepare(case, seed)
    off = s["offsets"].tolist()
    rows, inter = case["rows"], case["inter"]
    alpha, beta, limit = _parameters(case)

    def gate(g):           # value and slope of g' sigmoid(alpha g') at g' = min(g, limit)
        c = torch.minimum(g, torch.full_like(g, limit))
        p = torch.special.expit(alpha * c)
        slope = p + alpha * c * p * torch.special.expit(-alpha * c)
        return c * p, torch.where(g > limit, torch.zeros_like(slope), slope)

    def up(u):
        return torch.where(u > limit, limit, torch.where(u < -limit, -limit, u)) + beta

    z = torch.zeros(rows, inter, dtype=torch.float64, device="cuda")
    h = torch.zeros(rows, 2 * inter, dtype=torch.float64, device="cuda")
    for i in range(case["experts"]):
        at = slice(off[i], off[i + 1])
        if off[i] == off[i + 1]:
            continue
        if op == "gated":
            h[at] = s["x"][at].double() @ s["w13"][i].double().T
            z[at] = gate(h[at, :inter])[0] * up(h[at, inter:])
        else:
            g, u = s["h"][at, :inter].double(), s["h"][at, inter:].double()
            dz = s["dy"][at].double() @ s["w2"][i].double()
            value, slope = gate(g)
            z[at] = value * up(u)
            h[at, :inter] = dz * slope * up(u)
            h[at, inter:] = torch.where((u > limit) | (u < -limit), torch.zeros_like(u),
                                        dz * value)
    if op == "gated_grad":
        return {"dh": h, "z": z}
    return {"z": z, "h": h} if case["keep"] else {"z": z}


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "orthogonalize":
        small, large = sorted((case["n"], case["k"]))
        each = case["n"] * case["k"] * case["experts"]
        # both Gram products are symmetric: half of each has to be computed
        step = small * (small + 1.0) * (large + small) + 2.0 * small * small * large
        return {"bytes": each * ((4 if case["dtype"] == "float32" else 2) + 2.0),
                "flops": STEPS * case["experts"] * step}
    rows, inter, hidden = case["rows"], case["inter"], case["hidden"]
    some = min(case["experts"], rows)   # experts that can have rows
    if op == "gated":
        values = rows * (hidden + inter * (3 if case["keep"] else 1)) + some * 2 * inter * hidden
        return {"bytes": 2.0 * values, "flops": 4.0 * rows * inter * hidden}
    # dy, w2 and h read, dh and z written
    return {"bytes": 2.0 * (rows * (hidden + 5 * inter) + some * inter * hidden),
            "flops": 2.0 * rows * inter * hidden}
