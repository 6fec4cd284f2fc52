"""What is measured of the products of a feed-forward layer: the gated block
act(x Wg^T) * (x Wu^T) and its gradients, the product in 8-bit integers with a
scale for each token and each output channel (with the tokens' quantization
where the activations come in 16 bits), and the orthogonalized update of a
weight by Newton-Schulz products.

With `own` false, `run` computes them from elementary torch operations in 32
bits; with `own` true it makes the calls of dense_gemm_nt_amd that a user makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# the odd quintic a s + b s^3 + c s^5, applied to every singular value s
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


def listed():
    return [
        # one token of one request through the block's first half: pure latency
        {"name": "gated_token", "op": "gated", "M": 1, "F": 14336, "K": 4096, "act": "silu",
         "dtype": "bf16"},
        # a decode step of 64 requests on a large model's block
        {"name": "gated_decode", "op": "gated", "M": 64, "F": 28672, "K": 8192, "act": "silu",
         "dtype": "bf16"},
        # a prefill batch, an odd number of tokens
        {"name": "gated_prefill", "op": "gated", "M": 5001, "F": 14336, "K": 4096, "act": "gelu",
         "dtype": "fp16"},
        # a fine-tuning step of a small model, ragged
        {"name": "gated_train_small", "op": "gated_grad", "M": 777, "F": 1408, "K": 2048,
         "act": "gelu", "dtype": "fp16"},
        # a short batch of a large model, a hidden size that no tile divides
        {"name": "gated_train_odd", "op": "gated_grad", "M": 1500, "F": 5461, "K": 4096,
         "act": "silu", "dtype": "bf16"},
        # a training step's full batch
        {"name": "gated_train", "op": "gated_grad", "M": 8192, "F": 8192, "K": 4096,
         "act": "silu", "dtype": "bf16"},
        # one token, quantized on the way in, through a projection held in 8 bits
        {"name": "int8_token", "op": "int8", "M": 1, "N": 8192, "K": 8192, "dynamic": True,
         "dtype": "bf16"},
        # a decode batch whose producer has quantized its output already
        {"name": "int8_decode", "op": "int8", "M": 200, "N": 10240, "K": 8192, "dynamic": False,
         "dtype": "bf16"},
        # a prefill batch, quantized on the way in, odd sizes
        {"name": "int8_prefill", "op": "int8", "M": 8111, "N": 8200, "K": 8192, "dynamic": True,
         "dtype": "fp16"},
        # the update of a small layer's weight, ragged
        {"name": "ortho_small", "op": "ortho", "B": 1, "m": 1000, "n": 2047, "dtype": "fp32"},
        # the weights of one kind of many small layers, stacked
        {"name": "ortho_stack", "op": "ortho", "B": 12, "m": 2048, "n": 768, "dtype": "bf16"},
        # a large layer's weight
        {"name": "ortho_large", "op": "ortho", "B": 1, "m": 4096, "n": 8192, "dtype": "fp32"},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "int8", "int8", "ortho"])
    if op in ("gated", "gated_grad"):
        while True:
            c = {"op": op, "M": _log(rng, 1 if op == "gated" else 16, 8192), "F": _log(rng, 512, 28672),
                 "K": _log(rng, 512, 8192, 8), "act": rng.choice(["silu", "gelu", "relu"]),
                 "dtype": rng.choice(["bf16", "fp16"])}
            if c["M"] * c["F"] * c["K"] <= (1 << 38):
                return c
    if op == "int8":
        while True:
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 28672), "K": _log(rng, 512, 8192, 16),
                 "dynamic": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp16"])}
            if c["M"] * c["N"] * c["K"] <= (1 << 39):
                return c
    while True:
        c = {"op": op, "B": rng.choice([1, 1, 1, 2, 5, 12]), "m": _log(rng, 64, 4096), "n": _log(rng, 64, 8192),
             "dtype": rng.choice(["fp32", "bf16"])}
        least = min(c["m"], c["n"])
        if c["B"] * least * c["m"] * c["n"] <= (1 << 35):
            return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantize(x):
    """Codes and scales of each row: the scale is the row's largest magnitude over
    127, a code the nearest integer (even at a tie) to the 32-bit quotient."""
    x = x.float()
    scale = x.abs().max(1).values / 127.0
    some = torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(1)
    return torch.round(x / some).clamp(-127.0, 127.0), scale


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    st = {"case": case}
    if case["op"] in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        st.update(x=normal(M, K).to(dt), Wg=normal(F, K, std=0.02).to(dt), Wu=normal(F, K, std=0.02).to(dt))
        if case["op"] == "gated_grad":
            st["dh"] = normal(M, F, std=0.05).to(dt)
    elif case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        # tokens of uneven size with a few large features, as activations are
        large = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        x = normal(M, K) * large * (0.5 + torch.rand(M, 1, generator=g, device="cuda"))
        W, st["scale_w"] = _quantize(normal(N, K, std=0.02))
        st["W"] = W.to(torch.int8)
        if case["dynamic"]:
            st["x"] = x.to(dt)
        else:
            codes, st["scale_x"] = _quantize(x)
            st["x"] = codes.to(torch.int8)
    else:
        B, m, n = case["B"], case["m"], case["n"]
        # a gradient as it comes from tokens with a few shared directions
        r = max(1, min(m, n) // 8)
        size = torch.exp(0.5 * normal(B, m, 1))
        shared = torch.matmul(normal(B, m, r), normal(B, r, n, std=0.3 * r ** -0.5))
        G = ((normal(B, m, n) + shared) * size * 1e-3).to(dt)
        st["G"] = G[0] if B == 1 else G
    return st


# ---------------------------------------------------------------- plain forms

def _activation(v, act):
    """act(v) and act'(v)."""
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).to(v.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return v * s, s * (1.0 + v * (1.0 - s))
    phi = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v * phi, phi + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def _plain_gated(st):
    x, Wg, Wu = st["x"].float(), st["Wg"].float(), st["Wu"].float()
    a, _ = _activation(x @ Wg.t(), st["case"]["act"])
    return {"h": (a * (x @ Wu.t())).to(st["x"].dtype)}


def _plain_gated_grad(st):
    dt = st["x"].dtype
    x, Wg, Wu, dh = st["x"].float(), st["Wg"].float(), st["Wu"].float(), st["dh"].float()
    a, slope = _activation(x @ Wg.t(), st["case"]["act"])
    dg = dh * (x @ Wu.t()) * slope
    du = dh * a
    return {"dx": (dg @ Wg + du @ Wu).to(dt), "dWg": (dg.t() @ x).to(dt), "dWu": (du.t() @ x).to(dt)}


def _plain_int8(st):
    codes, scale = _quantize(st["x"]) if st["case"]["dynamic"] else (st["x"].float(), st["scale_x"])
    y = (codes @ st["W"].float().t()) * scale.unsqueeze(1) * st["scale_w"]
    return {"y": y.to(DTYPES[st["case"]["dtype"]])}


def _plain_ortho(st):
    a, b, c = COEFFICIENTS
    X = st["G"].float()
    X = X if X.dim() == 3 else X.unsqueeze(0)
    wide = X.shape[1] <= X.shape[2]
    X = X if wide else X.transpose(1, 2).contiguous()      # the smaller square of the two
    X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + EPS)
    for _ in range(STEPS):
        A = torch.matmul(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    X = X if wide else X.transpose(1, 2)
    return {"update": X.reshape(st["G"].shape).to(torch.bfloat16)}


# ------------------------------------------------------------ the framework's

def _own(st):
    import dense_gemm_nt_amd as g
    case = st["case"]
    if case["op"] == "gated":
        return {"h": g.gemm_gated(st["x"], st["Wg"], st["Wu"], activation=case["act"])}
    if case["op"] == "gated_grad":
        dx, dWg, dWu = g.gemm_gated_backward(st["dh"], st["x"], st["Wg"], st["Wu"], activation=case["act"])
        return {"dx": dx, "dWg": dWg, "dWu": dWu}
    if case["op"] == "int8":
        codes, scale = g.quantize_int8(st["x"]) if case["dynamic"] else (st["x"], st["scale_x"])
        return {"y": g.gemm_int8(codes, st["W"], scale, st["scale_w"], out_dtype=DTYPES[case["dtype"]])}
    return {"update": g.orthogonalize(st["G"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}


def run(state):
    if own:
        return _own(state)
    return {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "int8": _plain_int8,
            "ortho": _plain_ortho}[state["case"]["op"]](state)


def work(case):
    sz = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        if case["op"] == "gated":
            return {"bytes": sz * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
        # both projections again, then the gradients in x and in both weights
        return {"bytes": sz * (M * K + 2 * F * K + M * F) + sz * (M * K + 2 * F * K), "flops": 12 * M * F * K}
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (sz if case["dynamic"] else 1) * M * K + N * K + sz * M * N + 4 * N
                + (0 if case["dynamic"] else 4 * M), "flops": 2 * M * N * K}
    B, m, n = case["B"], case["m"], case["n"]
    r, k = min(m, n), max(m, n)
    # two symmetric squares, of which half has to be computed, and one product a step
    return {"bytes": B * m * n * (sz + 2), "flops": STEPS * B * (r * r * k + r * r * r + 2 * r * r * k)}


# ----------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    wide = torch.float64
    if case["op"] in ("gated", "gated_grad"):
        x, Wg, Wu = st["x"].to(wide), st["Wg"].to(wide), st["Wu"].to(wide)
        gate, up = torch.matmul(x, Wg.t()), torch.matmul(x, Wu.t())
        if case["act"] == "silu":
            sg = torch.sigmoid(gate)
            value, slope = gate * sg, sg + gate * sg * torch.sigmoid(-gate)
        elif case["act"] == "gelu":
            cdf = 0.5 * torch.special.erfc(-gate / math.sqrt(2.0))
            value, slope = gate * cdf, cdf + gate * torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
        else:
            value, slope = gate.clamp(min=0), torch.heaviside(gate, torch.zeros_like(gate))
        if case["op"] == "gated":
            return {"h": value * up}
        dh = st["dh"].to(wide)
        d_up, d_gate = dh * value, dh * up * slope
        return {"dx": torch.matmul(d_gate, Wg) + torch.matmul(d_up, Wu),
                "dWg": torch.matmul(d_gate.t(), x), "dWu": torch.matmul(d_up.t(), x)}
    if case["op"] == "int8":
        if case["dynamic"]:
            # (the scale and the quotient are 32-bit numbers by definition)
            x = st["x"].to(wide)
            top = x.abs().amax(1)
            scale = (top / 127.0).to(torch.float32).to(wide)
            safe = torch.where(top > 0, scale, torch.ones_like(scale))
            codes = (x / safe[:, None]).to(torch.float32).to(wide).round().clamp(-127, 127)
        else:
            codes, scale = st["x"].to(wide), st["scale_x"].to(wide)
        return {"y": torch.matmul(codes, st["W"].to(wide).t()) * scale[:, None] * st["scale_w"].to(wide)[None, :]}
    a, b, c = COEFFICIENTS
    G = st["G"].to(wide)
    G = G.reshape(-1, case["m"], case["n"])
    out = []
    for X in G:                             # one matrix at a time, on its smaller side
        flip = X.shape[0] > X.shape[1]
        X = X.t() if flip else X
        X = X / (torch.linalg.matrix_norm(X) + EPS)
        eye = torch.eye(X.shape[0], dtype=wide, device=X.device)
        for _ in range(STEPS):
            S = X @ X.t()
            X = (a * eye + S @ (b * eye + c * S)) @ X
        out.append(X.t() if flip else X)
    return {"update": torch.stack(out).reshape(st["G"].shape)}
