"""The 8-bit operators and what they are measured on.

Four operators of an 8-bit layer (W8A8: int8 weights with a scale per output
channel, int8 activations with a scale per token):

    int8_quantize           rows of x -> codes and a scale per row
    rmsnorm_int8_quantize   residual addition, root-mean-square norm, codes and scales
    silu_mul_int8_quantize  silu(gate) * up, codes and scales
    int8_gemm               y = (xq . wq^T) * x_scale * w_scale + bias

Codes are whole numbers in -127..127: the integer nearest to 127 p / max|p| of
the row, ties to even, decided on the exact quotient. That quotient is taken
in 64 bits below, so that a value next to a rounding border falls on the same
side everywhere.

`own` False: elementary torch operations. `own` True: the library's calls,
into outputs that the caller holds, as a serving loop makes them.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token's activations before a product that no norm feeds (the attention's output projection)
        dict(name="quantize_token", op="quantize", rows=1, k=4096, dtype="bf16"),
        # a weight matrix quantized per output channel when a model is loaded
        dict(name="quantize_weights", op="quantize", rows=14336, k=4096, dtype="bf16"),
        # one decode step of one sequence: the norm before the projections, residual updated
        dict(name="norm_token", op="norm", rows=1, k=4096, dtype="bf16", residual=True),
        # a prompt of 8192 tokens
        dict(name="norm_prompt", op="norm", rows=8192, k=4096, dtype="bf16", residual=True),
        # fp32 activations at a width that is no power of two, an odd number of rows, no residual (first layer)
        dict(name="norm_f32_odd", op="norm", rows=777, k=2880, dtype="f32", residual=False),
        # a batch of 16 decoding sequences between the two products of the MLP
        dict(name="act_batch16", op="act", rows=16, k=14336, dtype="bf16"),
        # the same for a prompt of 2048 tokens
        dict(name="act_prompt", op="act", rows=2048, k=14336, dtype="bf16"),
        # one token through the MLP's up projection: the weights' bytes bound it
        dict(name="gemm_b1", op="gemm", m=1, n=14336, k=4096, dtype="bf16", bias=False),
        # 16 tokens through the down projection
        dict(name="gemm_b16", op="gemm", m=16, n=4096, k=14336, dtype="bf16", bias=False),
        # a ragged batch of drafted tokens or a short prompt, with a bias
        dict(name="gemm_m130", op="gemm", m=130, n=4096, k=4096, dtype="bf16", bias=True),
        # sizes that fill no tile, fp32 out, a bias
        dict(name="gemm_f32_odd", op="gemm", m=515, n=2881, k=2896, dtype="f32", bias=True),
        # a prompt of 2048 tokens through gate and up: the matrix cores bound it
        dict(name="gemm_prompt", op="gemm", m=2048, n=28672, k=4096, dtype="bf16", bias=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["quantize", "norm", "act", "gemm", "gemm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        while True:
            m = _spread(rng, 1, 8192)
            n = _spread(rng, 64, 32768)
            k = _spread(rng, 64, 16384, 16)   # every row of codes is a whole number of 16-byte blocks
            if m * n * k <= 2048 * 28672 * 4096 and m * k + n * k + 4 * m * n <= 1 << 29:
                return dict(op=op, m=m, n=n, k=k, dtype=dtype, bias=rng.random() < 0.5)
    most = 14336 * 4096 if op == "quantize" else 8192 * 4096
    if dtype == "f32":
        most //= 2
    while True:
        rows = _spread(rng, 1, 16384)
        k = _spread(rng, 64, 32768, 16)
        if rows * k <= most // (2 if op == "act" else 1):
            break
    case = dict(op=op, rows=rows, k=k, dtype=dtype)
    if op == "norm":
        case["residual"] = rng.random() < 0.7
    return case


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, k, dtype, g):
    """Normal values of a different size in every row, and a few columns that are 20 times the rest, as residual streams have."""
    x = torch.randn(rows, k, device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), device="cuda", generator=g).float())
    at = torch.randint(0, k, (3,), device="cuda", generator=g)
    x[:, at] *= 20.0
    return x.to(dtype)


def _codes(rows, k, g):
    """int8 codes as quantized normal rows have them (largest magnitude 127), in blocks to bound the memory."""
    out = torch.empty(rows, k, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // k)
    for r in range(0, rows, step):
        x = torch.randn(min(step, rows - r), k, device="cuda", generator=g)
        out[r:r + step] = (x * (127.0 / x.abs().amax(1, keepdim=True))).round_()
    return out


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _codes(m, k, g)
        s["w"] = _codes(n, k, g)
        s["xs"] = torch.rand(m, device="cuda", generator=g) * 0.05 + 0.01
        s["ws"] = torch.rand(n, device="cuda", generator=g) * 5e-4 + 2e-4
        s["b"] = torch.randn(n, device="cuda", generator=g) if case["bias"] else None
        s["y"] = torch.empty(m, n, dtype=dt, device="cuda")
        return s
    rows, k = case["rows"], case["k"]
    s["x"] = _activations(rows, 2 * k if case["op"] == "act" else k, dt, g)
    if case["op"] == "norm":
        s["w"] = (1.0 + 0.2 * torch.randn(k, device="cuda", generator=g)).to(dt)
        s["res"] = _activations(rows, k, dt, g) if case["residual"] else None
        s["h"] = torch.empty(rows, k, dtype=dt, device="cuda") if case["residual"] else None
    s["out"] = (torch.empty(rows, k, dtype=torch.int8, device="cuda"),
                torch.empty(rows, dtype=torch.float32, device="cuda"))
    return s


def _plain_codes(p):
    """Codes of rows p (values in 32 or 64 bits) and the rows' largest magnitudes, in 64 bits."""
    p = p.double()
    top = p.abs().amax(1, keepdim=True)
    q = torch.round(p * 127.0 / top)
    q = torch.where(top > 0, q, torch.zeros_like(q))
    return q.to(torch.int8), top[:, 0]


def run(state):
    s = state
    if own:
        import gemm_e2m1_lut_amd as g
        if s["op"] == "gemm":
            return g.int8_gemm(s["x"], s["xs"], s["w"], s["ws"], bias=s["b"], out=s["y"], out_dtype=DT[s["dtype"]])
        if s["op"] == "quantize":
            return g.int8_quantize(s["x"], out=s["out"])
        if s["op"] == "act":
            return g.silu_mul_int8_quantize(s["x"], out=s["out"])
        return g.rmsnorm_int8_quantize(s["x"], s["w"], EPS, residual=s["res"], residual_out=s["h"], out=s["out"])
    if s["op"] == "gemm":
        y = s["x"].float() @ s["w"].float().t()
        y = y * s["xs"][:, None] * s["ws"]
        if s["b"] is not None:
            y = y + s["b"]
        return y.to(DT[s["dtype"]])
    if s["op"] == "quantize":
        q, top = _plain_codes(s["x"])
        return q, (top / 127.0).float()
    if s["op"] == "act":
        k = s["k"]
        gate, up = s["x"][:, :k].double(), s["x"][:, k:].double()
        q, top = _plain_codes(gate / (1.0 + torch.exp(-gate)) * up)
        return q, (top / 127.0).float()
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    q, top = _plain_codes(h * s["w"].float())
    mean = h.double().square().mean(1)
    scale = (top / (127.0 * torch.sqrt(mean + EPS))).float()
    return (q, scale) if s["res"] is None else (q, scale, h.to(DT[s["dtype"]]))


def work(case):
    o = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + (4 * n if case["bias"] else 0) + o * m * n, "flops": 2 * m * n * k}
    rows, k = case["rows"], case["k"]
    out = rows * k + 4 * rows
    if case["op"] == "quantize":
        return {"bytes": o * rows * k + out, "flops": 3 * rows * k}
    if case["op"] == "act":
        return {"bytes": 2 * o * rows * k + out, "flops": 9 * rows * k}
    return {"bytes": (3 if case["residual"] else 1) * o * rows * k + o * k + out, "flops": 7 * rows * k}


def exact(case, seed):
    """From the definitions, in 64 bits: row by row sums as dot products, codes from scaled rows."""
    s = prepare(case, seed)
    one = torch.float64
    if case["op"] == "gemm":
        acc = torch.mm(s["x"].to(one), s["w"].to(one).t().contiguous())
        y = torch.einsum("mn,m,n->mn", acc, s["xs"].to(one), s["ws"].to(one))
        return y if s["b"] is None else y.add_(s["b"].to(one))
    k = case["k"]
    if case["op"] == "quantize":
        p, div = s["x"].to(one), None
    elif case["op"] == "act":
        gate = s["x"].narrow(1, 0, k).to(one)
        p, div = s["x"].narrow(1, k, k).to(one).mul_(gate).mul_(torch.sigmoid(gate)), None
    else:
        # the residual's sum is defined in 32 bits, and so is its product with the weight
        h = s["x"].to(torch.float32)
        if s["res"] is not None:
            h = torch.add(h, s["res"].to(torch.float32))
        p = torch.mul(h, s["w"].to(torch.float32)).to(one)
        h = h.to(one)
        div = torch.linalg.vector_norm(h, dim=1).square().div(k).add(EPS).sqrt()
    unit = p.abs().max(dim=1).values / 127.0
    q = torch.div(p, torch.where(unit > 0, unit, torch.ones_like(unit)).unsqueeze(1)).round()
    scale = unit if div is None else unit / div
    if case["op"] == "norm" and case["residual"]:
        return None, scale, h
    return None, scale
