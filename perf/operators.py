"""Cases for the library's training and 4-bit operators, in a plain form and
through the library.

Operators:
  forward    ragged grouped product y[r] = W_e x[r] over segments of rows
  backward   its gradients: dx[r] = W_e^T dy[r] and dW_e = sum_r dy[r] x[r]^T
  quantize   E2M1 codes with one power-of-two scale per 32 values, and back
  product    grouped product of 4-bit activations (quantised in the call) with
             4-bit weights
  clip       global norm over many gradient tensors, and clipping

With ``own`` false ``run`` computes them from elementary torch operations in
fp32; with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few routed rows on a small layer: launch latency; odd segments, N and K
        # that end inside a tile
        dict(name="forward_tiny", op="forward", dtype="float16", rows=37, n=520, k=264,
             experts=8, skew=1.0),
        # 64 tokens, top-2, Mixtral-shaped gate/up product: bound by the weights
        dict(name="forward_decode", op="forward", dtype="bfloat16", rows=128, n=28672, k=4096,
             experts=8, skew=0.3),
        # 4096 tokens, top-2, the same layer: bound by the tensor cores
        dict(name="forward_prefill", op="forward", dtype="bfloat16", rows=8192, n=28672, k=4096,
             experts=8, skew=0.0),
        # fine-tuning step on a small layer: ragged everywhere
        dict(name="backward_small", op="backward", dtype="float16", rows=515, n=1032, k=776,
             experts=16, skew=1.0),
        # 4096 tokens, top-2, down projection of the Mixtral-shaped layer
        dict(name="backward_prefill", op="backward", dtype="bfloat16", rows=8192, n=4096,
             k=14336, experts=8, skew=0.0),
        # 2048 tokens, top-8 over 256 experts: few rows an expert, so the weights
        # (read) and their gradient (written) count
        dict(name="backward_many_experts", op="backward", dtype="bfloat16", rows=16384, n=7168,
             k=2048, experts=256, skew=0.5),
        # activations of a decode step
        dict(name="quantize_tokens", op="quantize", dtype="bfloat16", rows=64, k=7168),
        # the gate/up weights of a Mixtral-shaped layer, at load time
        dict(name="quantize_weights", op="quantize", dtype="bfloat16", rows=229376, k=4096),
        # 64 tokens, top-8 over 256 experts: bound by the 4-bit weights
        dict(name="product_decode", op="product", dtype="bfloat16", rows=512, n=4096, k=7168,
             experts=256, skew=0.0),
        # 4096 tokens, top-2, Mixtral-shaped gate/up product: bound by the tensor cores
        dict(name="product_prefill", op="product", dtype="bfloat16", rows=8192, n=28672, k=4096,
             experts=8, skew=0.0),
        # adapters and routers: many small tensors of all types
        dict(name="clip_small", op="clip", tensors=60, total=300007, max_norm=1.0),
        # every gradient of a Mixtral-shaped expert layer and a few small ones
        dict(name="clip_layer", op="clip", tensors=24, total=1400000003, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "quantize", "product",
                     "product", "clip"])
    if op == "quantize":
        k = 32 * _log(rng, 1, 512)
        return dict(op=op, dtype=rng.choice(["bfloat16", "float16", "float32"]),
                    rows=_log(rng, 1, min(229376, 900000000 // k)), k=k)
    if op == "clip":
        tensors = _log(rng, 1, 60)
        return dict(op=op, tensors=tensors, total=_log(rng, 64 * tensors, 1000000000),
                    max_norm=rng.choice([0.1, 1.0, 1e6]))
    step = 128 if op == "product" else 8
    experts = _log(rng, 1, 256)
    n = step * _log(rng, 1, 16384 // step)
    k = step * _log(rng, 1, 16384 // step)
    k = min(k, max(step, 900000000 // (experts * n) // step * step))
    rows = _log(rng, 1, 8192)
    dtype = "bfloat16" if op == "product" else rng.choice(["bfloat16", "float16"])
    return dict(op=op, dtype=dtype, rows=rows, n=n, k=k, experts=experts,
                skew=rng.choice([0.0, 0.5, 1.0]))


# ------------------------------------------------------------------ inputs
def _generator(seed, device):
    return torch.Generator(device=device).manual_seed(int(seed) * 7919 + 17)


def _segments(case, seed):
    """Rows of each expert: every routed row picks one by preferences of the
    stated spread, so small cases have experts without rows."""
    g = _generator(seed, "cpu")
    prefs = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g), 0)
    picks = torch.multinomial(prefs, case["rows"], replacement=True, generator=g)
    counts = torch.bincount(picks, minlength=case["experts"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]), int(counts.max())


def _sizes(case):
    """Lengths of the gradient tensors: a geometric spread of the total."""
    n, total = case["tensors"], case["total"]
    share = [0.8 ** min(i, 60) for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    sizes[0] += total - sum(sizes)
    return sizes


def _normal(shape, scale, dtype, g):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=g)
    return t


def prepare(case, seed):
    g = _generator(seed, "cuda")
    op = case["op"]
    s = dict(case=case)
    if op == "clip":
        types = [torch.bfloat16, torch.float32, torch.float16]
        # the largest gradients are bf16, as the weights'; the small ones are of all types
        s["grads"] = [_normal(n, 0.02, types[0] if n > 50000000 else types[i % 3], g)
                      for i, n in enumerate(_sizes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        return s
    dt = DTYPES[case["dtype"]]
    if op == "quantize":
        x = _normal((case["rows"], case["k"]), 1.0, dt, g)
        # magnitudes differ from channel group to channel group, as activations' do
        x *= torch.exp2(torch.randint(-6, 3, (case["k"] // 32,), generator=g, device="cuda")
                        .to(dt)).repeat_interleave(32)
        x[0, :32] = 0
        s["x"] = x
        return s
    offsets, s["longest"] = _segments(case, seed)
    s["offsets"] = offsets.to(device="cuda", dtype=torch.int32)
    rows, n, k, experts = (case[v] for v in ("rows", "n", "k", "experts"))
    s["x"] = _normal((rows, k), 1.0, dt, g)
    if op == "product":
        s["w_codes"] = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8,
                                     generator=g, device="cuda")
        s["w_scales"] = torch.randint(120, 126, (experts, n, k // 32), dtype=torch.uint8,
                                      generator=g, device="cuda")
        # the layout that the library's load-time packing gives: blocks of 128 rows x
        # 128 columns, byte 16 l + 4 c + j the scale of row 32 c + l, chunk j
        s["w_packed"] = (s["w_scales"].view(experts, n // 128, 4, 32, k // 128, 4)
                         .permute(0, 4, 1, 3, 2, 5).contiguous())
        return s
    s["w"] = _normal((experts, n, k), 0.02, dt, g)
    if op == "backward":
        s["dy"] = _normal((rows, n), 1.0, dt, g)
    return s


# -------------------------------------------------------------- plain forms
def _rows_to_blocks(s, t):
    """[R, C] rows as [E, longest, C] fp32, zeros behind each segment."""
    off = s["offsets"].long()
    at = torch.arange(s["longest"], device="cuda")
    inside = at < (off[1:] - off[:-1])[:, None]
    rows = (off[:-1, None] + at).clamp(max=t.shape[0] - 1)
    return torch.where(inside[..., None], t[rows].float(), 0.0)


def _blocks_to_rows(s, blocks, rows, dtype):
    off = s["offsets"].long()
    r = torch.arange(rows, device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return blocks[e, r - off[e]].to(dtype)


def _power(e):
    """2^e in fp32, from the bits of the fp64 value: exact."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _quantize_plain(x):
    """E2M1 magnitudes' values (fp32, signed) per 32 and the scales' exponents."""
    v = x.float().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    # exponent of the largest magnitude less that of 6, the largest E2M1 value
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2, -127).clamp(-127, 127)
    a = v.abs() * _power(-e)
    one = ((a >= 0.75).float() + (a > 0.25).float() + (a > 1.25).float() + (a >= 1.75).float()) * 0.5
    q = one + (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float()
    return torch.where(v < 0, -q, q), e


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "clip":
        total = torch.stack([t.float().square().sum() for t in s["grads"]]).sum()
        norm = total.sqrt()
        c = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
        return {"norm": norm, "grads": [(t.float() * c).to(t.dtype) for t in s["grads"]]}
    if op == "quantize":
        q, e = _quantize_plain(s["x"])
        return {"values": (q * _power(e)).flatten(-2).to(torch.bfloat16),
                "scales": (e.squeeze(-1) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}
    rows = case["rows"]
    if op == "product":
        q, e = _quantize_plain(s["x"])
        x = _rows_to_blocks(s, (q * _power(e)).flatten(-2))
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        grid = torch.cat([grid, -grid])
        c = s["w_codes"]
        w = torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], -1).flatten(-2)
        scale = _power(s["w_scales"].int() - 127)
        w = (w.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
        return _blocks_to_rows(s, torch.bmm(x, w.transpose(1, 2)), rows, torch.bfloat16)
    dt = s["x"].dtype
    if op == "forward":
        y = torch.bmm(_rows_to_blocks(s, s["x"]), s["w"].float().transpose(1, 2))
        return _blocks_to_rows(s, y, rows, dt)
    x, dy = _rows_to_blocks(s, s["x"]), _rows_to_blocks(s, s["dy"])
    dw = torch.bmm(dy.transpose(1, 2), x).to(dt)
    return {"dx": _blocks_to_rows(s, torch.bmm(dy, s["w"].float()), rows, dt), "dw": dw}


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

    if op == "clip":
        norm = kept("norm", lambda: torch.empty((), device="cuda"))
        ws = kept("ws", lambda: bytes_of(moe.moe_clip_workspace_bytes()))
        moe.moe_clip_grad_norm(s["grads"], case["max_norm"], norm, ws, out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    if op == "quantize":
        x = s["x"]
        codes = kept("codes", lambda: bytes_of(x.numel() // 2).view(x.shape[0], -1))
        scales = kept("scales", lambda: bytes_of(x.numel() // 32).view(x.shape[0], -1))
        values = kept("values", lambda: torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"))
        moe.moe_mxfp4_quantize(x, codes, scales)
        moe.moe_mxfp4_dequantize(codes, scales, values)
        return {"values": values, "scales": scales.view(torch.float8_e8m0fnu)}
    x, off = s["x"], s["offsets"]
    p = kept("plan", lambda: moe.Ragged(R=case["rows"], N=case["n"], K=case["k"],
                                        E=case["experts"], dtype=case["dtype"]))
    ws = kept("ws", lambda: bytes_of(moe.moe_ragged_workspace_bytes(p)))
    if op == "product":
        codes = kept("codes", lambda: bytes_of(x.numel() // 2).view(x.shape[0], -1))
        scales = kept("scales", lambda: bytes_of(x.numel() // 32).view(x.shape[0], -1))
        y = kept("y", lambda: torch.empty(case["rows"], case["n"], dtype=x.dtype, device="cuda"))
        moe.moe_mxfp4_quantize(x, codes, scales)
        moe.ragged_gemm_mxfp4(p, codes, scales, s["w_codes"], s["w_packed"], off, y, ws)
        return y
    if op == "forward":
        y = kept("y", lambda: torch.empty(case["rows"], case["n"], dtype=x.dtype, device="cuda"))
        moe.ragged_gemm(p, x, s["w"], off, y, ws)
        return y
    dx = kept("dx", lambda: torch.empty_like(x))
    dw = kept("dw", lambda: torch.empty_like(s["w"]))
    moe.ragged_gemm_dgrad(p, s["dy"], s["w"], off, dx, ws)
    moe.ragged_gemm_wgrad(p, s["dy"], x, off, dw, ws)
    return {"dx": dx, "dw": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- definition, 64 bits
def _floor_log2(a):
    """Exponent field of fp64 magnitudes (every fp32 value is a normal one)."""
    return (a.view(torch.int64) >> 52) - 1023


def _pow2(e):
    return ((e + 1023) << 52).view(torch.float64)


def _quantize_exact(x):
    """Values of the 4-bit form in fp64: the quantum of each magnitude's binade
    (at least that of 1), nearest multiple, ties to the even one."""
    v = x.double().unflatten(-1, (-1, 32))
    e = _floor_log2(v.abs().amax(-1, keepdim=True)).clamp(min=-125) - 2
    a = v / _pow2(e)
    quantum = 0.5 * _pow2(_floor_log2(a.abs().clamp(min=1.0)))
    return (torch.round(a / quantum) * quantum).clamp(-6.0, 6.0), _pow2(e)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "grads": [t.double() * c for t in s["grads"]]}
    if op == "quantize":
        q, e = _quantize_exact(s["x"])
        return {"values": (q * e).flatten(-2), "scales": e.squeeze(-1)}
    off = s["offsets"].tolist()
    rows, n, k = case["rows"], case["n"], case["k"]
    if op == "product":
        q, e = _quantize_exact(s["x"])
        x = (q * e).flatten(-2)
    else:
        x = s["x"].double()
    if op == "backward":
        dx = torch.zeros(rows, k, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device="cuda")
        for i in range(case["experts"]):
            at = slice(off[i], off[i + 1])
            dy = s["dy"][at].double()
            dx[at] = dy @ s["w"][i].double()
            dw[i] = dy.T @ x[at]
        return {"dx": dx, "dw": dw}
    y = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for i in range(case["experts"]):
        at = slice(off[i], off[i + 1])
        if off[i] == off[i + 1]:
            continue
        if op == "product":
            c = s["w_codes"][i].long()
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
            sign, ef, m = 1.0 - 2.0 * (c >> 3).double(), (c >> 1) & 3, (c & 1).double()
            w = sign * torch.where(ef == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(ef.double() - 1.0))
            w = (w.unflatten(-1, (-1, 32))
                 * _pow2(s["w_scales"][i].long() - 127)[..., None]).flatten(-2)
        else:
            w = s["w"][i].double()
        y[at] = x[at] @ w.T
    return y


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _sizes(case)
        size = [2 if n > 50000000 else (2, 4, 2)[i % 3] for i, n in enumerate(sizes)]
        total = sum(n * b for n, b in zip(sizes, size))
        return {"bytes": 2.0 * total, "flops": 3.0 * case["total"]}
    if op == "quantize":
        n = case["rows"] * case["k"]
        wide = 4 if case["dtype"] == "float32" else 2
        # read once; the codes and scales written; the bf16 values written
        return {"bytes": n * (wide + 0.5 + 1.0 / 32.0 + 2.0), "flops": 4.0 * n}
    rows, n, k = case["rows"], case["n"], case["k"]
    some = min(case["experts"], rows)   # experts that can have rows
    if op == "product":
        return {"bytes": rows * (k + n) * 2.0 + some * n * k * (0.5 + 1.0 / 32.0),
                "flops": 2.0 * rows * n * k}
    if op == "forward":
        return {"bytes": 2.0 * (rows * (k + n) + some * n * k), "flops": 2.0 * rows * n * k}
    # x, dy and w read, dx and every expert's dw written
    return {"bytes": 2.0 * (rows * (2 * k + n) + (some + case["experts"]) * n * k),
            "flops": 4.0 * rows * n * k}
