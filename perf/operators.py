"""What is measured of the operators whose weight is chosen per row: a shared
projection with low-rank adapters (forward and backward), the top-k router with
its balance loss and per-expert counts (forward and backward), and the experts'
products over rows sorted by expert (forward, input gradient, weight gradient).

With `own` false, `run` computes them from elementary torch operations in 32
bits; with `own` true it makes the calls of dense_gemm_nt_amd that a user makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request through an adapted projection: pure latency
        {"name": "lora_token", "op": "lora", "M": 1, "N": 4096, "K": 4096, "R": 16, "L": 8,
         "rows": "mixed", "dtype": "bf16"},
        # a decode step of 64 requests, nearly every one with an adapter of its own
        {"name": "lora_decode", "op": "lora", "M": 64, "N": 10240, "K": 8192, "R": 16, "L": 48,
         "rows": "mixed", "dtype": "bf16"},
        # a prefill batch of four adapters' prompts, an odd number of tokens
        {"name": "lora_prefill", "op": "lora", "M": 5001, "N": 8192, "K": 8192, "R": 64, "L": 4,
         "rows": "runs", "dtype": "fp16"},
        # one fine-tuning step of three small adapters at once, ragged
        {"name": "lora_train_small", "op": "lora_grad", "M": 777, "N": 4096, "K": 2048, "R": 8,
         "L": 3, "rows": "mixed", "dtype": "fp16"},
        # one fine-tuning step of one adapter on a full batch
        {"name": "lora_train", "op": "lora_grad", "M": 8192, "N": 8192, "K": 4096, "R": 32, "L": 1,
         "rows": "runs", "dtype": "bf16"},
        # routing of one decode step
        {"name": "route_decode", "op": "route", "T": 16, "E": 64, "k": 8, "dtype": "fp32",
         "renorm": True, "grad": False},
        # a training micro-batch with 16-bit logits (many ties), padded tokens
        {"name": "route_train_small", "op": "route", "T": 4099, "E": 60, "k": 4, "dtype": "bf16",
         "renorm": False, "grad": True},
        # a large training batch with many experts
        {"name": "route_train", "op": "route", "T": 65536, "E": 256, "k": 8, "dtype": "fp32",
         "renorm": True, "grad": True},
        # the experts' up projection in a decode step: 64 tokens to 8 experts each
        {"name": "routed_decode", "op": "routed", "S": 512, "E": 64, "N": 2048, "K": 7168,
         "dtype": "bf16", "grad": False},
        # the same weights' kind in a prefill: uneven experts, odd sizes
        {"name": "routed_prefill", "op": "routed", "S": 16411, "E": 16, "N": 4100, "K": 4096,
         "dtype": "bf16", "grad": False},
        # gradients of a small expert layer
        {"name": "routed_train_small", "op": "routed", "S": 1000, "E": 8, "N": 1408, "K": 2048,
         "dtype": "fp16", "grad": True},
        # gradients of a large one
        {"name": "routed_train", "op": "routed", "S": 16384, "E": 32, "N": 2048, "K": 4096,
         "dtype": "bf16", "grad": True},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_grad", "route", "routed", "routed"])
    if op in ("lora", "lora_grad"):
        while True:
            c = {"op": op, "M": _log(rng, 1 if op == "lora" else 16, 8192),
                 "N": _log(rng, 512, 10240, 1 if op == "lora" else 8), "K": _log(rng, 512, 8192, 8),
                 "R": rng.choice([8, 16, 24, 32, 64]), "L": _log(rng, 1, 64 if op == "lora" else 8),
                 "rows": rng.choice(["mixed", "runs"]), "dtype": rng.choice(["bf16", "fp16"])}
            # many adapters at once are what decode steps bring
            if c["L"] * c["M"] <= 65536 and c["M"] * c["N"] * c["K"] <= (1 << 38):
                return c
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 65536), "E": _log(rng, 8, 256), "k": rng.randint(1, 8),
                "dtype": rng.choice(["fp32", "bf16"]), "renorm": rng.random() < 0.5,
                "grad": rng.random() < 0.5}
    while True:
        c = {"op": op, "S": _log(rng, 8, 16384), "E": _log(rng, 4, 64), "N": _log(rng, 512, 4096, 4),
             "K": _log(rng, 512, 7168, 8), "dtype": rng.choice(["bf16", "fp16"]),
             "grad": rng.random() < 0.4}
        if c["grad"]:
            c["N"] = c["N"] // 8 * 8
        if c["S"] * c["N"] * c["K"] <= (1 << 37) and c["E"] * c["N"] * c["K"] <= (1 << 30):
            return c


def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def _row_ids(M, L, kind, g):
    """Adapter of each row: "mixed" deals the adapters out in random order, with
    one row in eight left without one; "runs" gives each adapter one run of
    rows of uneven length (prompts packed one after another)."""
    if kind == "mixed":
        ids = torch.randperm(M, generator=g, device="cuda") % L
        bare = torch.rand(M, generator=g, device="cuda") < 0.125
        if M > 1:
            ids = torch.where(bare, torch.full_like(ids, -1), ids)
    else:
        cuts = torch.rand(L - 1, generator=g, device="cuda").sort().values * M
        ids = (torch.arange(M, device="cuda").unsqueeze(1) >= cuts.unsqueeze(0)).sum(1)
    return ids.to(torch.int32)


def _expert_rows(S, E, g):
    """Uneven rows per expert, an empty expert now and then, and a few rows
    behind the last expert's that belong to none."""
    share = torch.rand(E, generator=g, device="cuda") ** 2
    share = torch.where(torch.rand(E, generator=g, device="cuda") < 0.05, torch.zeros_like(share), share)
    share[0] += 0.01
    ends = (share.cumsum(0) / share.sum() * (S - S // 64)).floor().to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    if case["op"] in ("lora", "lora_grad"):
        M, N, K, R, L = (case[n] for n in "MNKRL")
        st = {"x": normal(M, K), "W": normal(N, K, std=0.02), "A": normal(L, R, K, std=K ** -0.5),
              "B": normal(L, N, R, std=0.02), "ids": _row_ids(M, L, case["rows"], g),
              "scale": 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")}
        if case["op"] == "lora_grad":
            st["dy"] = normal(M, N, std=0.1)
    elif case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        lean = torch.randn(E, generator=g, device="cuda") * 0.5      # favoured experts
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5 + lean
        off = torch.rand(T, E, generator=g, device="cuda") < 0.01    # experts closed to a token
        st = {"logits": logits.masked_fill(off, float("-inf")).to(dt),
              "mask": torch.rand(T, generator=g, device="cuda") < 0.95}
        if case["grad"]:
            st["grad_weights"] = torch.randn(T, k, generator=g, device="cuda")
            st["grad_loss"] = torch.full((), 0.01 * T, device="cuda")
    else:
        S, E, N, K = (case[n] for n in "SENK")
        st = {"x": normal(S, K), "W": normal(E, N, K, std=0.02), "offsets": _expert_rows(S, E, g)}
        st["bounds"] = st["offsets"].tolist()
        if case["grad"]:
            st["dy"] = normal(S, N, std=0.1)
    st["case"] = case
    return st


# ---------------------------------------------------------------- plain forms

def _adapter_columns(st, wide):
    """The adapters side by side: A [L R, K], B [N, L R], and each row's scale
    on its own adapter's columns (zero elsewhere) [M, L R]."""
    A, B = st["A"].to(wide), st["B"].to(wide)
    L, R, K = A.shape
    pick = (st["ids"].unsqueeze(1) == torch.arange(L, device=A.device).unsqueeze(0)).to(wide)
    pick = (pick * st["scale"].to(wide)).repeat_interleave(R, dim=1)
    return A.reshape(L * R, K), B.permute(1, 0, 2).reshape(B.shape[1], L * R), pick


def _plain_lora(st):
    x, W = st["x"].float(), st["W"].float()
    A, B, pick = _adapter_columns(st, torch.float32)
    y = x @ W.t() + ((x @ A.t()) * pick) @ B.t()
    return {"y": y.to(st["x"].dtype)}


def _plain_lora_grad(st):
    x, W, dy = st["x"].float(), st["W"].float(), st["dy"].float()
    A, B, pick = _adapter_columns(st, torch.float32)
    L, R, K = st["A"].shape
    t, u = (x @ A.t()) * pick, (dy @ B) * pick
    dB = (dy.t() @ t).reshape(-1, L, R).permute(1, 0, 2).contiguous()
    return {"dx": (dy @ W + u @ A).to(st["x"].dtype), "dA": (u.t() @ x).reshape(L, R, K), "dB": dB}


def _route(st, wide):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    dev = st["logits"].device
    x = st["logits"].to(wide).masked_fill(~st["mask"].unsqueeze(1), float("-inf"))
    top = x.max(1, keepdim=True).values
    live = top > float("-inf")
    e = torch.where(live, torch.exp(x - torch.where(live, top, torch.zeros_like(top))), torch.zeros_like(x))
    p = e / torch.where(live, e.sum(1, keepdim=True), torch.ones_like(top))
    column = torch.arange(E, device=dev).unsqueeze(0)
    left, ids, w = x.clone(), [], []
    for _ in range(k):                                    # the largest left, the first of equals
        best = left.max(1, keepdim=True).values
        i = torch.where(left == best, column, torch.full_like(column, E)).min(1, keepdim=True).values
        found = best > float("-inf")
        ids.append(torch.where(found, i, torch.full_like(i, -1)))
        w.append(torch.where(found, p.gather(1, i), torch.zeros_like(best)))
        left.scatter_(1, i, float("-inf"))
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    total = w.sum(1, keepdim=True)
    if case["renorm"]:
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    key = torch.where(ids >= 0, ids, torch.full_like(ids, E)).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=dev).scatter_add_(0, key, torch.ones_like(key))[:E]
    n = live.sum()
    nz = n.clamp(min=1).to(wide)
    f = counts.to(wide) / (nz * k)
    loss = (E * (f * (p.sum(0) / nz)).sum()).to(torch.float32)
    out = {"ids": ids.to(torch.int32), "weights": w.to(torch.float32), "counts": counts.to(torch.int32),
           "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32),
           "order": torch.sort(key, stable=True).indices.to(torch.int32), "loss": loss}
    if case["grad"]:
        gw = st["grad_weights"].to(wide)
        if case["renorm"]:
            gw = (gw - (gw * w).sum(1, keepdim=True)) / torch.where(total > 0, total, torch.ones_like(total))
        dp = (st["grad_loss"].to(wide) * E / nz * f).unsqueeze(0).expand(T, E).clone()
        dp.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, gw, torch.zeros_like(gw)))
        out["dlogits"] = (p * (dp - (p * dp).sum(1, keepdim=True))).to(st["logits"].dtype)
    return out


def _plain_routed(st):
    x, W, b = st["x"], st["W"], st["bounds"]
    y = torch.zeros(x.shape[0], W.shape[1], device=x.device)
    for e in range(W.shape[0]):
        y[b[e]:b[e + 1]] = x[b[e]:b[e + 1]].float() @ W[e].float().t()
    out = {"y": y.to(x.dtype)}
    if st["case"]["grad"]:
        dy = st["dy"]
        dx = torch.zeros(x.shape, device=x.device)
        dW = torch.empty(W.shape, device=x.device)
        for e in range(W.shape[0]):
            r = slice(b[e], b[e + 1])
            dx[r] = dy[r].float() @ W[e].float()
            dW[e] = dy[r].float().t() @ x[r].float()
        out = {"dx": dx.to(x.dtype), "dW": dW}
    return out


# ------------------------------------------------------------ the framework's

def _own(st):
    import dense_gemm_nt_amd as g
    case = st["case"]
    if case["op"] == "lora":
        return {"y": g.gemm_lora(st["x"], st["W"], st["A"], st["B"], st["ids"], st["scale"])}
    if case["op"] == "lora_grad":
        dx, dA, dB = g.gemm_lora_backward(st["dy"], st["x"], st["W"], st["A"], st["B"], st["ids"],
                                          st["scale"])
        return {"dx": dx, "dA": dA, "dB": dB}
    if case["op"] == "route":
        r = g.route_topk(st["logits"], case["k"], mask=st["mask"], renormalize=case["renorm"])
        out = {"ids": r.ids, "weights": r.weights, "counts": r.counts, "offsets": r.offsets,
               "order": r.order, "loss": r.loss}
        if case["grad"]:
            out["dlogits"] = g.route_topk_backward(st["logits"], r, grad_weights=st["grad_weights"],
                                                   grad_loss=st["grad_loss"])
        return out
    if case["grad"]:
        return {"dx": g.gemm_routed(st["dy"], st["W"].transpose(1, 2), st["offsets"]),
                "dW": g.gemm_routed_wgrad(st["dy"], st["x"], st["offsets"], out_dtype=torch.float32)}
    return {"y": g.gemm_routed(st["x"], st["W"], st["offsets"])}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "lora":
        return _plain_lora(state)
    if op == "lora_grad":
        return _plain_lora_grad(state)
    return _route(state, torch.float32) if op == "route" else _plain_routed(state)


def work(case):
    sz = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("lora", "lora_grad"):
        M, N, K, R = (case[n] for n in "MNKR")
        used = min(case["L"], M)
        read = sz * (M * K + N * K + used * R * (K + N)) + 4 * M
        if case["op"] == "lora":
            return {"bytes": read + sz * M * N, "flops": 2 * M * N * K + 2 * M * R * (K + N)}
        return {"bytes": read + sz * M * (N + K) + 4 * case["L"] * R * (K + N),
                "flops": 2 * M * N * K + 2 * M * R * (3 * K + 2 * N)}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        nbytes = T * E * sz + T + T * k * 12 + 4 * (2 * E + 2)
        flops = T * E * (6 + k)
        if case["grad"]:
            nbytes += T * E * sz + T * k * 4
            flops += T * E * 6
        return {"bytes": nbytes, "flops": flops}
    S, E, N, K = (case[n] for n in "SENK")
    live = min(E, S)
    if case["grad"]:
        return {"bytes": sz * (S * (N + 2 * K) + live * N * K) + 4 * E * N * K,
                "flops": 4 * S * N * K}
    return {"bytes": sz * (S * (N + K) + live * N * K), "flops": 2 * S * N * K}


# ----------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    wide = torch.float64
    if case["op"] in ("lora", "lora_grad"):
        x, W, scale = st["x"].to(wide), st["W"].to(wide), st["scale"].to(wide)
        if case["op"] == "lora":
            y = x @ W.t()
        else:
            dy = st["dy"].to(wide)
            dx = dy @ W
            dA = torch.zeros(st["A"].shape, dtype=wide, device="cuda")
            dB = torch.zeros(st["B"].shape, dtype=wide, device="cuda")
        for a in range(case["L"]):                      # one adapter's rows at a time
            r = (st["ids"] == a).nonzero().squeeze(1)
            if not len(r):
                continue
            Aa, Ba = st["A"][a].to(wide), st["B"][a].to(wide)
            low = x[r] @ Aa.t()
            if case["op"] == "lora":
                y[r] += scale[a] * (low @ Ba.t())
            else:
                back = scale[a] * (dy[r] @ Ba)
                dx[r] += back @ Aa
                dA[a] = back.t() @ x[r]
                dB[a] = scale[a] * (dy[r].t() @ low)
        return {"y": y} if case["op"] == "lora" else {"dx": dx, "dA": dA, "dB": dB}
    if case["op"] == "route":
        return _exact_route(case, st)
    S, N = case["S"], case["N"]
    seen = torch.arange(S, device="cuda")
    expert = torch.bucketize(seen, st["offsets"][1:].long(), right=True)   # E: no expert
    if case["grad"]:
        dx = torch.zeros(S, case["K"], dtype=wide, device="cuda")
        dW = torch.zeros(case["E"], N, case["K"], dtype=wide, device="cuda")
    y = torch.zeros(S, N, dtype=wide, device="cuda")
    for e in range(case["E"]):
        r = (expert == e).nonzero().squeeze(1)
        if not len(r):
            continue
        W = st["W"][e].to(wide)
        if case["grad"]:
            d = st["dy"][r].to(wide)
            dx[r] = d @ W
            dW[e] = d.t() @ st["x"][r].to(wide)
        else:
            y[r] = st["x"][r].to(wide) @ W.t()
    return {"dx": dx, "dW": dW} if case["grad"] else {"y": y}


def _exact_route(case, st):
    wide = torch.float64
    T, E, k = case["T"], case["E"], case["k"]
    x = st["logits"].to(wide)
    x[~st["mask"]] = float("-inf")
    live = (x > float("-inf")).any(1)
    p = torch.zeros(T, E, dtype=wide, device="cuda")
    z = x[live]
    p[live] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    # a stable descending sort keeps equal logits in the order of their index
    vals, idx = torch.sort(x, dim=1, descending=True, stable=True)
    kk = min(k, E)
    ids = torch.where(vals[:, :kk] > float("-inf"), idx[:, :kk], torch.full_like(idx[:, :kk], -1))
    if kk < k:
        ids = torch.cat([ids, ids.new_full((T, k - kk), -1)], 1)
    chosen = ids >= 0
    raw = torch.where(chosen, p.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=wide, device="cuda"))
    total = raw.sum(1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    w = raw / safe if case["renorm"] else raw
    counts = torch.bincount(ids[chosen], minlength=E)
    n = int(live.sum())
    f = counts.to(wide) / max(1, n * k)
    loss = E * (f * p.sum(0) / max(1, n)).sum()
    group = torch.where(chosen, ids, torch.full_like(ids, E)).reshape(-1)
    order = torch.argsort(group * (T * k) + torch.arange(T * k, device="cuda"))
    out = {"ids": ids.to(torch.int32), "weights": w, "counts": counts.to(torch.int32),
           "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32),
           "order": order.to(torch.int32), "loss": loss}
    if case["grad"]:
        gw = torch.where(chosen, st["grad_weights"].to(wide), torch.zeros((), dtype=wide, device="cuda"))
        if case["renorm"]:
            gw = torch.where(chosen, (gw - (gw * w).sum(1, keepdim=True)) / safe, torch.zeros_like(gw))
        dp = torch.zeros(T, E, dtype=wide, device="cuda")
        for j in range(k):
            dp.scatter_add_(1, ids[:, j:j + 1].clamp(min=0), gw[:, j:j + 1])
        dp += st["grad_loss"].to(wide) * E * f / max(1, n)
        out["dlogits"] = p * (dp - (p * dp).sum(1, keepdim=True))
    return out
