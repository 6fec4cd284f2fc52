"""Plain 64-bit forms of the products whose weight depends on the row, written
from their definitions, one row, adapter or expert at a time (float64 torch
tensors on the CPU).  Gradients are the formulas'; tests pin them by differences of
the forward forms here.  Where a caller needs error bounds, the sums of absolute
values come with the result."""
from __future__ import annotations

import torch

F64 = torch.float64


def lora(x, W, A, B, ids, scale):
    """y and the sums of absolute products (of the projection, of the adapters)."""
    x, W, A, B, scale = (t.to(F64) for t in (x, W, A, B, scale))
    y = x @ W.t()
    s_base = x.abs() @ W.abs().t()
    s_low = torch.zeros_like(y)
    for m, a in enumerate(ids.tolist()):
        if 0 <= a < A.shape[0]:
            y[m] += scale[a] * (B[a] @ (A[a] @ x[m]))
            s_low[m] = scale[a].abs() * (B[a].abs() @ (A[a].abs() @ x[m].abs()))
    return y, s_base, s_low


def lora_backward(dy, x, W, A, B, ids, scale):
    """{name: (gradient, sum of absolute products of the projection, of the
    adapters)} for dx, dA, dB."""
    dy, x, W, A, B, scale = (t.to(F64) for t in (dy, x, W, A, B, scale))
    dx, s_dx = dy @ W, dy.abs() @ W.abs()
    l_dx = torch.zeros_like(dx)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    s_dA, s_dB = torch.zeros_like(A), torch.zeros_like(B)
    for m, a in enumerate(ids.tolist()):
        if not 0 <= a < A.shape[0]:
            continue
        u, low = scale[a] * (dy[m] @ B[a]), scale[a] * (A[a] @ x[m])
        ua, la = scale[a].abs() * (dy[m].abs() @ B[a].abs()), scale[a].abs() * (A[a].abs() @ x[m].abs())
        dx[m] += u @ A[a]
        l_dx[m] = ua @ A[a].abs()
        dA[a] += torch.outer(u, x[m])
        s_dA[a] += torch.outer(ua, x[m].abs())
        dB[a] += torch.outer(dy[m], low)
        s_dB[a] += torch.outer(dy[m].abs(), la)
    return {"dx": (dx, s_dx, l_dx), "dA": (dA, torch.zeros_like(s_dA), s_dA),
            "dB": (dB, torch.zeros_like(s_dB), s_dB)}


def route(logits, k, mask=None, renormalize=True):
    """ids, weights, counts, offsets, order, tokens, loss and p (zeros for tokens
    that are not routed), as a dict.  NaN ranks as the lowest finite float32."""
    x = logits.to(F64)
    T, E = x.shape
    ids = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=F64)
    p = torch.zeros(T, E, dtype=F64)
    routed = 0
    for t in range(T):
        if mask is not None and not bool(mask[t]):
            continue
        key = [(-3.402823466e38 if v != v else v) for v in x[t].tolist()]
        if max(key) == float("-inf"):
            continue
        routed += 1
        e = torch.exp(x[t] - max(key))
        p[t] = e / e.sum()
        best = sorted((e for e in range(E) if key[e] > float("-inf")), key=lambda e: (-key[e], e))[:k]
        ids[t, :len(best)] = torch.tensor(best)
        w[t, :len(best)] = p[t, best]
        if renormalize:
            w[t] /= w[t].sum()
    flat = ids.reshape(-1).tolist()
    counts = [flat.count(e) for e in range(E)]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    order = sorted(range(T * k), key=lambda i: (flat[i] if flat[i] >= 0 else E, i))
    n = routed
    loss = torch.zeros((), dtype=F64)
    if n:
        f = torch.tensor(counts, dtype=F64) / (n * k)
        loss = E * (f * (p.sum(0) / n)).sum()
    return {"ids": ids, "weights": w, "counts": torch.tensor(counts), "offsets": torch.tensor(offsets),
            "order": torch.tensor(order, dtype=torch.int64), "tokens": n, "loss": loss, "p": p}


def route_backward(logits, r, renormalize, grad_weights=None, grad_loss=None):
    """The gradient of a route() result `r` in the logits (counts are constants)."""
    T, E = logits.shape
    k = r["ids"].shape[1]
    d = torch.zeros(T, E, dtype=F64)
    n = r["tokens"]
    for t in range(T):
        chosen = [(j, e) for j, e in enumerate(r["ids"][t].tolist()) if e >= 0]
        if not chosen:
            continue
        p = r["p"][t]
        dp = torch.zeros(E, dtype=F64)
        if grad_loss is not None:
            dp += float(grad_loss) * E * r["counts"].to(F64) / (n * k) / n
        if grad_weights is not None:
            g = grad_weights[t].to(F64)
            total = sum(p[e] for _, e in chosen)
            mean = sum(g[j] * r["weights"][t, j] for j, _ in chosen)
            for j, e in chosen:
                dp[e] += (g[j] - mean) / total if renormalize else g[j]
        d[t] = p * (dp - (p * dp).sum())
    return d


def segments(offsets, rows):
    """The row range of each expert, as the device reads any offsets: clamped to
    [0, rows] and to their running maximum; and where the last one ends."""
    top, out = 0, []
    o = [min(max(v, 0), rows) for v in offsets]
    top = o[0]
    for hi in o[1:]:
        start, top = top, max(top, hi)
        out.append((start, top))
    return out, top


def routed(x, W, offsets):
    """C [rows, N] with NaN in rows of no expert, and the sums of absolute products."""
    x, W = x.to(F64), W.to(F64)
    C = torch.full((x.shape[0], W.shape[1]), float("nan"), dtype=F64)
    S = torch.zeros_like(C)
    for e, (a, b) in enumerate(segments(offsets.tolist(), x.shape[0])[0]):
        C[a:b] = x[a:b] @ W[e].t()
        S[a:b] = x[a:b].abs() @ W[e].abs().t()
    return C, S


def routed_wgrad(dy, x, offsets):
    dy, x = dy.to(F64), x.to(F64)
    seg = segments(offsets.tolist(), x.shape[0])[0]
    dW = torch.zeros(len(seg), dy.shape[1], x.shape[1], dtype=F64)
    S = torch.zeros_like(dW)
    for e, (a, b) in enumerate(seg):
        dW[e] = dy[a:b].t() @ x[a:b]
        S[e] = dy[a:b].abs().t() @ x[a:b].abs()
    return dW, S
