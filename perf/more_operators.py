"""Cases for the operators between two attentions and at the end of a step: the linear
layer with bias, activation and residual in its epilogue, the norms before and after a
block fused with its gate and residual, and the sampling of the next token.

Each operator has its plain form here (elementary torch operations in 32 bits, and in 64
for the sampling, whose sums decide between tokens) and the call that a user makes of the
library.  ``own`` selects between them.  A case is a dict of plain values; the values of
its tensors follow from the seed given to prepare().
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
GREEDY_BELOW = 1e-5  # a temperature below this takes the highest logit


def _cases():
    return [
        # --- y = act(x W^T + bias) + residual ---
        # one user's token through the query down-projection (7168 -> 1536): the smallest call
        dict(name="linear_one_token", op="linear", M=1, K=7168, N=1536, act=None, bias=False, res=False, f32=False,
             out32=False),
        # the output projection of a decode batch, added to the residual stream: the weight's stream
        dict(name="linear_decode_64", op="linear", M=64, K=16384, N=7168, act=None, bias=False, res=True, f32=False,
             out32=False),
        # fp32 logits of a decode batch over a large vocabulary
        dict(name="linear_logits", op="linear", M=17, K=7168, N=131072, act=None, bias=False, res=False, f32=False,
             out32=True),
        # a prompt chunk through the output projection, added to the residual stream
        dict(name="linear_prompt", op="linear", M=4096, K=16384, N=7168, act=None, bias=False, res=True, f32=False,
             out32=False),
        # an odd batch through a biased layer with an activation whose rows do not start on 16 bytes
        dict(name="linear_odd_gelu", op="linear", M=777, K=2047, N=5001, act="gelu", bias=True, res=False, f32=False,
             out32=False),
        # a layer kept in fp32 (a router or a small head)
        dict(name="linear_fp32", op="linear", M=500, K=1536, N=260, act="silu", bias=True, res=False, f32=True,
             out32=True),
        # --- h' = skip h + scale act(gate) norm(u),  y = norm(h') ---
        # a decode batch of 64 users: residual add and the next block's norm
        dict(name="norm_decode", op="norm", N=64, D=7168, post=None, pre="rms", gate=None, gate_act=None, h32=False,
             f32=False, scale=1.0),
        # a prompt with a norm on both sides of the block and a sigmoid gate for each value
        dict(name="norm_prompt_gated", op="norm", N=8192, D=7168, post="rms", pre="rms", gate="full",
             gate_act="sigmoid", h32=False, f32=False, scale=0.5),
        # an fp32 residual stream of odd width under bf16 blocks, layer norm, one gate row for all tokens
        dict(name="norm_odd_layer", op="norm", N=3001, D=2049, post=None, pre="layer", gate="row", gate_act=None,
             h32=True, f32=False, scale=1.0),
        # --- the next token ---
        # one user, nucleus sampling: latency
        dict(name="sample_one", op="sample", R=1, V=131072, f32=True, k=False, p=True, m=False, masked=False),
        # a batch with its own settings in every row
        dict(name="sample_batch", op="sample", R=256, V=131072, f32=True, k=True, p=True, m=True, masked=False),
        # bf16 logits (many equal values) of an odd vocabulary under a grammar's mask
        dict(name="sample_bf16_masked", op="sample", R=67, V=50001, f32=False, k=True, p=True, m=False, masked=True),
    ]


def listed():
    return _cases()


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["linear", "linear", "norm", "sample"])
    if op == "linear":
        f32 = rng.random() < 0.15
        even = 1 if rng.random() < 0.25 else 64
        K = max(1, _log(rng, 32, 16384) // even) * even
        N = _log(rng, 1, 40000) if even == 1 else max(1, _log(rng, 8, 131072) // 8) * 8
        return dict(op=op, M=_log(rng, 1, 8192), K=K, N=N, act=rng.choice([None, None, "relu", "silu", "gelu", "gelu_tanh"]),
                    bias=rng.random() < 0.5, res=rng.random() < 0.5, f32=f32, out32=f32 or rng.random() < 0.3)
    if op == "norm":
        f32 = rng.random() < 0.2
        gate = rng.choice([None, None, "full", "row"])
        D = _log(rng, 64, 16384)
        return dict(op=op, N=_log(rng, 1, 16384), D=D if rng.random() < 0.25 else max(1, D // 64) * 64,
                    post=rng.choice([None, None, "rms", "layer"]), pre=rng.choice(["rms", "rms", "layer"]), gate=gate,
                    gate_act=rng.choice([None, "sigmoid", "silu"]) if gate else None, h32=f32 or rng.random() < 0.3,
                    f32=f32, scale=rng.choice([1.0, 1.0, 0.5, 0.22]))
    return dict(op=op, R=_log(rng, 1, 256), V=_log(rng, 1000, 131072), f32=rng.random() < 0.6, k=rng.random() < 0.5,
                p=rng.random() < 0.6, m=rng.random() < 0.3, masked=rng.random() < 0.3)


def draw(rng):
    """One more case; its work stays under that of the largest listed case of the same operator."""
    while True:
        c = _draw(rng)
        w = work(c)
        cap = [work(x) for x in _cases() if x["op"] == c["op"]]
        if w["bytes"] <= max(x["bytes"] for x in cap) and w["flops"] <= max(x["flops"] for x in cap):
            return c


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    s = dict(c)
    if c["op"] == "linear":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["out"] = torch.float32 if c["out32"] else torch.bfloat16
        s["x"] = torch.randn(c["M"], c["K"], dtype=dt, **dev)
        s["W"] = torch.randn(c["N"], c["K"], dtype=dt, **dev).mul_(1 / math.sqrt(c["K"]))
        s["b"] = 0.1 * torch.randn(c["N"], **dev) if c["bias"] else None
        s["r"] = torch.randn(c["M"], c["N"], dtype=s["out"], **dev) if c["res"] else None
    elif c["op"] == "norm":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["h"] = 3 * torch.randn(c["N"], c["D"], dtype=torch.float32 if c["h32"] else dt, **dev)
        s["u"] = torch.randn(c["N"], c["D"], dtype=dt, **dev)
        s["g"] = None
        if c["gate"]:
            s["g"] = torch.randn(c["N"] if c["gate"] == "full" else 1, c["D"], dtype=dt, **dev)
        for n in ("pre", "post"):
            s[n + "_gain"] = 1 + 0.1 * torch.randn(c["D"], **dev) if c[n] else None
            s[n + "_bias"] = 0.1 * torch.randn(c["D"], **dev) if c[n] == "layer" else None
    else:
        R, V = c["R"], c["V"]
        # a broad bulk and some tokens that stand out, as a language model's logits have
        x = 1.8 * torch.randn(R, V, **dev)
        at = torch.randint(0, V, (R, 40), **dev)
        x.scatter_add_(1, at, 4 + 3 * torch.randn(R, 40, **dev).abs())
        if c["masked"]:
            x.masked_fill_(torch.rand(R, V, **dev) < 0.9, float("-inf"))
        s["logits"] = x if c["f32"] else x.bfloat16()
        s["u"] = torch.rand(R, **dev)

        def pick(values, dt):
            return torch.tensor(values, dtype=dt, device="cuda")[torch.randint(0, len(values), (R,), **dev)]

        s["T"] = pick([0.6, 0.7, 0.8, 1.0, 1.0, 1.2, 0.0], torch.float32)
        s["k_"] = pick([0, 20, 50, 200, 1000], torch.int32) if c["k"] else None
        s["p_"] = pick([0.7, 0.9, 0.95, 0.95, 1.0], torch.float32) if c["p"] else None
        s["m_"] = pick([0.0, 0.02, 0.05, 0.1], torch.float32) if c["m"] else None
    return s


# ---------------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------------
def _act(v, kind):
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s):
    y = s["x"].float() @ s["W"].float().t()
    if s["b"] is not None:
        y += s["b"]
    y = _act(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["out"])


def _norm(x, kind, gain, bias):
    if kind is None:
        return x
    if kind == "rms":
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    d = x - x.mean(-1, keepdim=True)
    return d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS) * gain + bias


def _plain_norm(s):
    v = _norm(s["u"].float(), s["post"], s["post_gain"], s["post_bias"])
    if s["g"] is not None:
        v = v * _act(s["g"].float(), s["gate_act"])
    h = s["h"].float() + s["scale"] * v
    y = _norm(h, s["pre"], s["pre_gain"], s["pre_bias"])
    return h.to(s["h"].dtype), y.to(s["u"].dtype)


def _plain_sample(s):
    l = s["logits"].double()  # noqa: E741
    V = l.shape[1]
    top = l.amax(1, keepdim=True)
    T = s["T"].double()[:, None]
    greedy = T < GREEDY_BELOW
    w = torch.exp((l - top) / torch.where(greedy, 1.0, T))
    l, order = torch.sort(l, dim=1, descending=True, stable=True)
    w = w.gather(1, order)
    rank = torch.arange(V, device=l.device)[None]
    keep = l > float("-inf")
    if s["k_"] is not None:
        keep &= (rank < s["k_"][:, None]) | (s["k_"][:, None] <= 0)
    keep &= (rank == 0) | ~greedy
    if s["p_"] is not None:
        p = s["p_"].double()[:, None]
        cum = torch.cumsum(w * keep, 1)
        before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
        keep &= (before < p * cum[:, -1:]) | (p >= 1)
    if s["m_"] is not None:
        keep &= (w >= s["m_"].double()[:, None]) | (rank == 0)
    kept = torch.zeros_like(w).scatter_(1, order, w * keep)  # in the vocabulary's order again
    cum = torch.cumsum(kept, 1)
    token = (cum > s["u"].double()[:, None] * cum[:, -1:]).int().argmax(1)
    logprob = torch.log(kept.gather(1, token[:, None])[:, 0] / cum[:, -1])
    return token.int(), logprob.float(), keep.sum(1).int()


# ---------------------------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import sparse_latent_attention_indexer_gb300 as dsa

    if s["op"] == "linear":
        return dsa.dsa_linear(s["x"], s["W"], bias=s["b"], act=s["act"], residual=s["r"], dtype=s["out"])
    if s["op"] == "norm":
        post = dsa.Norm(s["post"], s["post_gain"], s["post_bias"]) if s["post"] else None
        pre = dsa.Norm(s["pre"], s["pre_gain"], s["pre_bias"])
        return dsa.dsa_block_norm(s["h"], pre, u=s["u"], post=post, gate=s["g"], gate_act=s["gate_act"],
                                  scale=s["scale"], eps=EPS)
    return dsa.dsa_sample(s["logits"], s["u"], temperature=s["T"], top_k=s["k_"], top_p=s["p_"], min_p=s["m_"],
                          want_kept=True)


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "norm": _plain_norm, "sample": _plain_sample}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        item, out = 4 if c["f32"] else 2, 4 if c["out32"] else 2
        return {"bytes": item * (M * K + N * K) + out * M * N * (2 if c["res"] else 1) + (4 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "norm":
        n = c["N"] * c["D"]
        item = 4 if c["f32"] else 2
        h = 4 if c["h32"] else item
        gate = item * (n if c["gate"] == "full" else c["D"] if c["gate"] else 0)
        return {"bytes": n * (2 * h + 2 * item) + gate, "flops": n * 12}
    n = c["R"] * c["V"]
    return {"bytes": n * (4 if c["f32"] else 2) + c["R"] * 32, "flops": n * 4}


def _exact_linear(s):
    if work(s)["flops"] > 2e12:
        return None
    x, parts = s["x"].double(), []
    step = max(1, (1 << 28) // s["K"])
    for n in range(0, s["N"], step):
        z = torch.einsum("mk,nk->mn", x, s["W"][n:n + step].double())
        if s["b"] is not None:
            z = z + s["b"][n:n + step].double()
        if s["act"] == "relu":
            z = torch.maximum(z, torch.zeros_like(z))
        elif s["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif s["act"] == "gelu":  # z times the normal distribution's function at z
            z = z * 0.5 * torch.erfc(-z / math.sqrt(2))
        elif s["act"] == "gelu_tanh":  # (1 + tanh t) / 2 = sigmoid(2 t)
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        if s["r"] is not None:
            z = z + s["r"][:, n:n + step].double()
        parts.append(z)
    return torch.cat(parts, 1)


def _exact_norm(s):
    def normed(v, n):
        if s[n] is None:
            return v
        if s[n] == "layer":
            v = v - v.sum(-1, keepdim=True) / s["D"]
        v = v / ((v ** 2).sum(-1, keepdim=True) / s["D"] + EPS).sqrt()
        v = v * s[n + "_gain"].double()
        return v + s[n + "_bias"].double() if s[n] == "layer" else v

    v = normed(s["u"].double(), "post")
    if s["g"] is not None:
        gate = s["g"].double()
        v = v * (torch.sigmoid(gate) if s["gate_act"] == "sigmoid" else gate * torch.sigmoid(gate)
                 if s["gate_act"] == "silu" else gate)
    h = s["h"].double() + s["scale"] * v
    return h, normed(h, "pre")


def _exact_sample(s):
    """Row by row: the tokens in their order, cut by each rule in turn, then the draw over what is left."""
    token, logprob, kept = [], [], []
    for r in range(s["R"]):
        row = s["logits"][r].double()
        ids = torch.nonzero(row > float("-inf"))[:, 0]
        ids = ids[torch.sort(row[ids], descending=True, stable=True)[1]]
        T = float(s["T"][r])
        k = int(s["k_"][r]) if s["k_"] is not None else 0
        if T < GREEDY_BELOW:
            k, T = 1, 1.0
        if k > 0:
            ids = ids[:k]
        w = ((row[ids] - row[ids[0]]) / T).exp()
        if s["p_"] is not None and float(s["p_"][r]) < 1:
            sums = w.cumsum(0)
            n = int((sums < float(s["p_"][r]) * sums[-1]).sum()) + 1
            ids, w = ids[:n], w[:n]
        if s["m_"] is not None:
            n = max(1, int((w >= float(s["m_"][r])).sum()))
            ids, w = ids[:n], w[:n]
        kept.append(len(ids))
        ids, back = torch.sort(ids)
        sums = w[back].cumsum(0)
        n = int((sums <= float(s["u"][r]) * sums[-1]).sum())
        token.append(int(ids[n]))
        logprob.append(float((w[back][n] / sums[-1]).log()))
    dev = s["logits"].device
    return (torch.tensor(token, dtype=torch.int32, device=dev), torch.tensor(logprob, dtype=torch.float64, device=dev),
            torch.tensor(kept, dtype=torch.int32, device=dev))


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "norm": _exact_norm, "sample": _exact_sample}[s["op"]](s)
