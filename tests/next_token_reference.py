"""The operators between two attentions and after the last in 64 bits, from their formulas."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative to the value


def act(v, kind):
    """In 64 bits."""
    if kind == "relu":
        return torch.where(v < 0, 0.0, v)
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def linear(x, w, bias, kind, res):
    """y, and the sum of the absolute products behind every value."""
    x, w = x.double(), w.double()
    v = x @ w.T
    spread = x.abs() @ w.abs().T
    if bias is not None:
        v = v + bias.double()
        spread = spread + bias.double().abs()
    y = act(v, kind)
    return (y if res is None else y + res.double()), spread


def norm(v, kind, gain, bias, eps):
    if kind in (None, "none"):
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if gain is not None:
        v = v * gain.double()
    if bias is not None and kind == "layer":
        v = v + bias.double()
    return v


def block_norm(h, u, gate, gate_act, post, pre, skip, scale, eps):
    """post, pre: (kind, gain, bias).  h', y."""
    r = skip * h.double()
    if u is not None:
        v = norm(u.double(), *post, eps)
        if gate is not None:
            v = v * act(gate.double(), gate_act)
        r = r + scale * v
    return r, norm(r, *pre, eps)


def sample_row(logits, u, T=1.0, k=0, p=1.0, m=0.0):
    """One row in plain Python steps over a sorted list: (token, logprob, kept)."""
    l = logits.double().cpu()  # noqa: E741
    inf = float("inf")
    ids = torch.nonzero(l > -inf)[:, 0]  # NaN compares false
    if len(ids) == 0:
        return -1, -inf, 0
    if bool((l[ids] == inf).any()):
        ids = ids[l[ids] == inf]
        l = torch.where(l == inf, 0.0, -inf)  # noqa: E741
    ids = ids[torch.sort(l[ids] + 0.0, descending=True, stable=True)[1]]
    if not T >= 1e-5:
        k, T = 1, 1.0
    if k > 0:
        ids = ids[:k]
    w = torch.exp((l[ids] - l[ids[0]]) / T)
    if p < 1:
        total, run, n = math.fsum(w.tolist()), torch.cumsum(w, 0), 0
        n = int((run < p * total).sum()) + 1
        ids, w = ids[:n], w[:n]
    if m > 0:
        n = max(1, int((w >= m).sum()))
        ids, w = ids[:n], w[:n]
    n = len(ids)
    ids, back = torch.sort(ids)
    w = w[back]
    run, total = torch.cumsum(w, 0), math.fsum(w.tolist())
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    at = int((run <= u * total).sum())
    return int(ids[at]), math.log(float(w[at]) / total), n
