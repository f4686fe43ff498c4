"""Cases for the operators of speculative decoding over a latent cache: writing
and reading back a (quantised, paged) cache, attention of a tree of drafted
tokens over it, and the per-head norm and position rotation of queries and keys.

Each operator has its plain form here (elementary torch operations in 32 bits)
and the call that a user makes of the library.  ``own`` selects between them.
A case is a dict of plain values; the ragged lengths of a case follow from its
``lens`` number, the values of its tensors from the seed given to prepare().
"""
from __future__ import annotations

import math
import random

import torch

own = False

D_N, D_R, D_C, D_V = 128, 64, 512, 128  # head widths of the 671B configuration
SCALE = 1.0 / math.sqrt(D_N + D_R)
EPS = 1e-6


def _cases():
    return [
        # --- attention of drafted tokens over the cache ---
        # one user, one token, a short context: the latency of a single decode step
        dict(name="tree_one_token", op="tree", B=1, T=1, P=777, H=128, page=64, fp8=False, tree=False, lens=1),
        # a decode batch with long contexts over the FP8 cache: the cache stream
        dict(name="tree_decode_fp8", op="tree", B=32, T=1, P=65536, H=128, page=64, fp8=True, tree=False, lens=2),
        # draft trees of up to 32 nodes on ragged contexts, bf16 cache
        dict(name="tree_32_nodes", op="tree", B=16, T=32, P=12288, H=128, page=64, fp8=False, tree=True, lens=3),
        # one eighth of the heads (a tensor-parallel share), small pages, larger trees, FP8 cache
        dict(name="tree_16_heads_fp8", op="tree", B=8, T=60, P=32768, H=16, page=16, fp8=True, tree=True, lens=4),
        # a prompt chunk (causal chain) on a contiguous bf16 cache, half the heads, odd lengths
        dict(name="chain_chunk", op="tree", B=3, T=301, P=5001, H=64, page=0, fp8=False, tree=False, lens=5),
        # --- writing the cache ---
        # the new tokens of a decode step of 64 users, quantised into their pages
        dict(name="write_decode_fp8", op="write", B=64, T=1, P=8192, page=64, fp8=True, f32=False, lens=6),
        # prompts written at once, quantised from the fp32 projection
        dict(name="write_prompts_fp8", op="write", B=5, T=24576, P=100, page=64, fp8=True, f32=True, lens=7),
        # --- reading it back ---
        # the accepted paths of 64 draft trees
        dict(name="read_path_fp8", op="read", B=64, T=5, P=4096, page=64, fp8=True, pos=True, lens=8),
        # whole prefixes, as bf16 rows for a prompt's continuation
        dict(name="read_prefix_fp8", op="read", B=6, T=24576, P=0, page=32, fp8=True, pos=False, lens=9),
        # --- norm and rotation of queries and keys ---
        # a decode step of 64 users: 128 query heads of 192 and one key head
        dict(name="heads_decode", op="heads", B=64, T=1, P=30000, Hq=128, Hk=1, D=192, rope="pairs", norm="rms",
             split=True, f32=False, lens=10),
        # a prompt of one user, queries and keys of every head
        dict(name="heads_prompt", op="heads", B=1, T=4096, P=0, Hq=128, Hk=1, D=192, rope="pairs", norm="rms",
             split=True, f32=False, lens=11),
        # the indexer's heads (64 x 128 and one key), layer norm, halves rotated in place, at given positions
        dict(name="heads_index", op="heads", B=7, T=999, P=4000, Hq=64, Hk=1, D=128, rope="halves", norm="layer",
             split=False, f32=True, lens=12),
    ]


def listed():
    return _cases()


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["tree", "tree", "tree", "write", "read", "heads"])
    lens = rng.randrange(1 << 30)
    if op == "tree":
        tree = rng.random() < 0.6
        return dict(op=op, B=_log(rng, 1, 32), T=_log(rng, 1, 64 if tree else 400), P=_log(rng, 1, 65536),
                    H=rng.choice([16, 32, 64, 128, 128]), page=rng.choice([0, 16, 32, 64, 128]),
                    fp8=rng.random() < 0.5, tree=tree, lens=lens)
    if op == "write":
        return dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 24576), P=_log(rng, 1, 8192),
                    page=rng.choice([0, 16, 64, 128]), fp8=rng.random() < 0.7, f32=rng.random() < 0.5, lens=lens)
    if op == "read":
        pos = rng.random() < 0.5
        return dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 200 if pos else 24576), P=_log(rng, 1, 8192),
                    page=rng.choice([0, 16, 64, 128]), fp8=rng.random() < 0.7, pos=pos, lens=lens)
    return dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 4096), P=_log(rng, 1, 30000), Hq=rng.choice([16, 64, 128]),
                Hk=rng.choice([0, 1, 1, 8]), D=rng.choice([128, 192, 192]), rope=rng.choice(["pairs", "halves"]),
                norm=rng.choice(["rms", "layer", "none"]), split=rng.random() < 0.5, f32=rng.random() < 0.3, lens=lens)


def draw(rng):
    """One more case; its work stays under that of the largest listed case of the same operator."""
    while True:
        c = _draw(rng)
        w = work(c)
        cap = [work(x) for x in _cases() if x["op"] == c["op"]]
        if w["bytes"] <= max(x["bytes"] for x in cap) and w["flops"] <= max(x["flops"] for x in cap):
            return c


# ---------------------------------------------------------------------------------------------------------------
# Lengths, trees, pages
# ---------------------------------------------------------------------------------------------------------------
def _lengths(c):
    """Nodes and cached tokens of every sequence: the first has the most of both, the others fewer."""
    r = random.Random(c["lens"])
    T = [c["T"]] + [r.randint((c["T"] + 1) // 2, c["T"]) for _ in range(c["B"] - 1)]
    P = [c["P"]] + [r.randint(c["P"] // 4, c["P"]) for _ in range(c["B"] - 1)]
    return T, P


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _ancestors(T, r):
    """The visible nodes of every node of a random tree, as integers of T bits: its ancestors and itself."""
    rows = []
    for t in range(T):
        up = r.randint(max(-1, t - 6), t - 1)  # its parent; -1: the last cached token
        rows.append((1 << t) | (rows[up] if up >= 0 else 0))
    return rows


def _quantise(x):
    """e4m3 codes and the power-of-two scale of every 128 values: the smallest 2^e with amax <= 448 * 2^e."""
    blocks = x.reshape(*x.shape[:-1], -1, 128)
    m, e = torch.frexp(blocks.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m == 0, 0, e).clamp(-127, 127)
    codes = (blocks * torch.ldexp(torch.ones_like(m), -e)).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape), torch.ldexp(torch.ones_like(m), e)[..., 0]


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _pages(s, c, S, g):
    """The cache's rows and, with pages, a block table of pages in no order, with pages nobody uses between."""
    s["page"], s["table"] = c["page"], None
    if not c["page"]:
        s["rows"] = sum(S)
        return
    per = [-(-x // c["page"]) for x in S]
    n = sum(per) + 3
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    s["table"], s["rows"] = table, n * c["page"]


def _cache(s, c, g):
    """A cache that holds normal latents (unit mean square) and rotary keys in every row."""
    rows = s["rows"]
    lat = _rms(torch.randn(rows, D_C, generator=g, device="cuda"))
    if c["fp8"]:
        codes, s["scale"] = _quantise(lat)
        s["kv"] = codes.view(torch.uint8)
        s["pe"] = torch.randn(rows, D_R, generator=g, device="cuda").bfloat16()
    else:  # one packed row a token
        buf = torch.cat([lat, torch.randn(rows, D_R, generator=g, device="cuda")], 1).bfloat16()
        s["kv"], s["pe"], s["scale"] = buf[:, :D_C], buf[:, D_C:], None


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    T, P = _lengths(c)
    S = [a + b for a, b in zip(T, P)]
    dev = dict(device="cuda")
    s = dict(c, cu_q=_cum(T), cu_k=_cum(S), start=P, N=sum(T), Tmax=max(T), Smax=max(S))
    # what the plain forms index with
    s["first"] = torch.tensor(s["cu_q"][:-1], **dev)
    s["base"] = torch.tensor(s["cu_k"][:-1], **dev)
    s["count"], s["before"] = torch.tensor(T, **dev), torch.tensor(P, **dev)
    s["seq"] = torch.repeat_interleave(torch.arange(c["B"], **dev), s["count"])
    s["node"] = torch.arange(s["N"], **dev) - s["first"][s["seq"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, **dev)

    if c["op"] == "heads":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["q"] = normal(s["N"], c["Hq"], c["D"]).to(dt)
        s["k"] = normal(s["N"], c["Hk"], c["D"]).to(dt) if c["Hk"] else None
        for n in ("q", "k"):
            s[n + "_gain"] = 1 + 0.1 * normal(c["D"]) if c["norm"] != "none" else None
            s[n + "_bias"] = 0.1 * normal(c["D"]) if c["norm"] == "layer" else None
        n_pos = max(S) + 1
        ang = torch.arange(n_pos, **dev, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(D_R // 2, **dev, dtype=torch.float64) / (D_R // 2))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        # a node sits at the depth of its ancestors, not at its row
        depth = torch.tensor([r.randint(0, t) for n in T for t in range(n)], **dev)
        s["pos"] = (s["before"][s["seq"]] + depth).to(torch.int32)
        return s
    _pages(s, c, S, g)
    _cache(s, c, g)
    if c["op"] == "write":
        x = torch.cat([_rms(normal(s["N"], D_C)), normal(s["N"], D_R)], 1).to(torch.float32 if c["f32"] else torch.bfloat16)
        s["c_new"], s["pe_new"] = x[:, :D_C], x[:, D_C:]
    elif c["op"] == "read":
        s["at"] = None
        if c["pos"]:  # positions of an accepted path: any of the sequence, in rising order
            at = [p for a, b in zip(T, S) for p in sorted(r.sample(range(b), a))]
            s["at"] = torch.tensor(at, dtype=torch.int32, **dev)
    else:
        s["q_nope"], s["q_pe"] = normal(s["N"], c["H"], D_N).bfloat16(), normal(s["N"], c["H"], D_R).bfloat16()
        s["W_UK"] = (normal(c["H"], D_N, D_C) / math.sqrt(D_C)).bfloat16()
        s["W_UV"] = (normal(c["H"], D_C, D_V) / math.sqrt(D_C)).bfloat16()
        s["mask"] = None
        if c["tree"]:
            words = (c["T"] + 63) // 64
            bits = [row for n in T for row in _ancestors(n, r)]
            sign = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
            s["mask"] = torch.tensor([[sign(v >> (64 * w) & (1 << 64) - 1) for w in range(words)] for v in bits], **dev)
    return s


# ---------------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------------
def _rows_of(s, seq, pos):
    """Cache rows of positions of sequences."""
    if s["table"] is None:
        return s["base"][seq] + pos
    return s["table"][seq, pos // s["page"]].long() * s["page"] + pos % s["page"]


def _values(s, rows):
    """Latents and rotary keys of cache rows, in 32 bits."""
    lat = s["kv"][rows]
    if s["scale"] is not None:
        lat = lat.view(torch.float8_e4m3fn).float() * s["scale"][rows].repeat_interleave(128, -1)
    return lat.float(), s["pe"][rows].float()


def _plain_tree(s):
    dev = s["q_nope"].device
    B, H = s["B"], s["H"]
    node, pos = torch.arange(s["Tmax"], device=dev), torch.arange(s["Smax"], device=dev)
    row = s["first"][:, None] + node.minimum(s["count"][:, None] - 1)  # [B, Tmax], padded
    length = s["before"] + s["count"]
    at = pos[None].minimum(length[:, None] - 1)                                             # [B, Smax], padded
    c, pe = _values(s, _rows_of(s, torch.arange(B, device=dev)[:, None], at))
    qt = torch.einsum("bthd,hdc->bthc", s["q_nope"][row].float(), s["W_UK"].float())
    z = torch.bmm(qt.reshape(B, -1, D_C), c.transpose(1, 2))
    z += torch.bmm(s["q_pe"][row].float().reshape(B, -1, D_R), pe.transpose(1, 2))
    rel = pos[None] - s["before"][:, None]                                                  # [B, Smax]
    if s["mask"] is None:
        see = rel[:, None] <= node[None, :, None]
    else:
        m = s["mask"][row]                                                                  # [B, Tmax, words]
        word = (rel.clamp(min=0) >> 6).clamp(max=m.shape[2] - 1)[:, None].expand(-1, s["Tmax"], -1)
        see = (rel < 0)[:, None] | ((m.gather(2, word) >> (rel & 63)[:, None]) & 1).bool()
    see = see & (pos[None] < length[:, None])[:, None]
    z = (z * SCALE).view(B, s["Tmax"], H, -1).masked_fill_(~see[:, :, None], float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, -1, s["Smax"])
    o = torch.bmm(p, c).view(B, s["Tmax"], H, D_C)[s["seq"], s["node"]]
    return torch.einsum("nhc,hcv->nhv", o, s["W_UV"].float()).bfloat16()


def _plain_write(s):
    rows = _rows_of(s, s["seq"], s["before"][s["seq"]] + s["node"])
    if s["scale"] is not None:
        codes, s["scale"][rows] = _quantise(s["c_new"].float())
        s["kv"][rows] = codes.view(torch.uint8)
    else:
        s["kv"][rows] = s["c_new"].to(s["kv"].dtype)
    s["pe"][rows] = s["pe_new"].to(s["pe"].dtype)
    return _held(s)


def _held(s):
    """The whole cache; codes as the e4m3 numbers they are."""
    if s["scale"] is None:
        return {"kv": s["kv"], "pe": s["pe"]}
    return {"kv": s["kv"].view(torch.float8_e4m3fn), "scale": s["scale"], "pe": s["pe"]}


def _plain_read(s):
    pos = s["before"][s["seq"]] + s["node"] if s["at"] is None else s["at"].long()
    lat, pe = _values(s, _rows_of(s, s["seq"], pos))
    return lat.bfloat16(), pe.bfloat16()


def _norm(x, kind, gain, bias, eps):
    if kind == "none":
        return x
    if kind == "rms":
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain
    d = x - x.mean(-1, keepdim=True)
    return d * torch.rsqrt((d * d).mean(-1, keepdim=True) + eps) * gain + bias


def _plain_heads(s):
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]

    def one(x, gain, bias):
        if x is None:
            return None
        y = _norm(x.float(), s["norm"], gain, bias, EPS)
        keep, turn = y[..., :-D_R], y[..., -D_R:]
        a, b = (turn[..., ::2], turn[..., 1::2]) if s["rope"] == "pairs" else (turn[..., :D_R // 2], turn[..., D_R // 2:])
        turn = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        if s["split"]:
            return keep.to(x.dtype), turn.to(x.dtype)
        return torch.cat([keep, turn], -1).to(x.dtype)

    return one(s["q"], s["q_gain"], s["q_bias"]), one(s["k"], s["k_gain"], s["k_bias"])


# ---------------------------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import sparse_latent_attention_indexer_gb300 as dsa

    seqs = dsa.Seqs(s["cu_q"], s["cu_k"], s["start"])
    if s["op"] == "heads":
        def heads(n):
            return None if s[n] is None else dsa.Heads(s[n], norm=s["norm"], gain=s[n + "_gain"], bias=s[n + "_bias"])

        return dsa.dsa_head_norm_rope(heads("q"), heads("k"), s["cos"], s["sin"], seqs, pos=s["pos"], rope=s["rope"],
                                      eps=EPS, split=s["split"])
    cache = dsa.LatentCache(s["kv"], s["pe"], s["scale"])
    pages = None if s["table"] is None else dsa.Pages(s["table"], s["page"], s["rows"] // s["page"])
    if s["op"] == "write":
        dsa.dsa_latent_cache_write(s["c_new"], s["pe_new"], cache, seqs, pages=pages)
        return _held(s)
    if s["op"] == "read":
        return dsa.dsa_latent_cache_read(cache, seqs, pages=pages, pos=s["at"], dtype=torch.bfloat16)
    out, _ = dsa.dsa_tree_mla_fwd(s["q_nope"], s["q_pe"], cache, s["W_UK"], s["W_UV"], seqs, SCALE,
                                  tree_mask=s["mask"], pages=pages, want_lse=False)
    return out


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "write": _plain_write, "read": _plain_read, "heads": _plain_heads}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    T, P = _lengths(c)
    N = sum(T)
    if c["op"] == "heads":
        item = 4 if c["f32"] else 2
        heads = c["Hq"] + c["Hk"]
        n = N * heads * c["D"]
        return {"bytes": 2 * n * item + N * (4 + D_R * 4), "flops": 8 * n}
    row = D_C + D_C // 128 * 4 + D_R * 2 if c["fp8"] else (D_C + D_R) * 2
    if c["op"] == "write":
        return {"bytes": N * ((D_C + D_R) * (4 if c["f32"] else 2) + row), "flops": 3 * N * D_C}
    if c["op"] == "read":
        return {"bytes": N * (row + (D_C + D_R) * 2), "flops": N * D_C}
    if c["tree"]:  # the cached tokens and the node itself (its ancestors are few)
        pairs = sum(t * p + t for t, p in zip(T, P))
    else:
        pairs = sum(t * p + t * (t + 1) // 2 for t, p in zip(T, P))
    H = c["H"]
    return {"bytes": sum(t + p for t, p in zip(T, P)) * row + N * H * (D_N + D_R + D_V) * 2 + H * D_C * (D_N + D_V) * 2,
            "flops": 2 * H * pairs * (2 * D_C + D_R) + 2 * N * H * D_C * (D_N + D_V)}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, sequence by sequence and token by token where that is how
    the definition goes; None where it would take too long."""
    c = case
    s = prepare(c, seed)
    T, P = _lengths(c)
    if c["op"] == "heads":
        i = torch.arange(D_R // 2, device="cuda")
        p = s["pos"].long()
        turn = torch.complex(s["cos"][p].double(), s["sin"][p].double())[:, None]
        first = c["D"] - D_R

        def one(n):
            x = s[n]
            if x is None:
                return None
            x = x.double()
            if c["norm"] == "rms":
                x = x / ((x ** 2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * s[n + "_gain"].double()
            elif c["norm"] == "layer":
                x = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
                x = x * s[n + "_gain"].double() + s[n + "_bias"].double()
            if c["rope"] == "pairs":
                z = torch.complex(x[..., first + 2 * i], x[..., first + 2 * i + 1]) * turn
            else:
                z = torch.complex(x[..., first + i], x[..., first + D_R // 2 + i]) * turn
            rot = torch.cat([z.real, z.imag], -1)
            return (x[..., :first], rot) if c["split"] else torch.cat([x[..., :first], rot], -1)

        return one("q"), one("k")

    def row_list(b, pos):
        if s["table"] is None:
            return s["cu_k"][b] + pos
        return s["table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]

    def kept(rows):
        v = s["kv"][rows]
        if s["scale"] is None:
            return v.double(), s["pe"][rows].double()
        v = v.view(torch.float8_e4m3fn).to(torch.float64).view(-1, D_C // 128, 128)
        return (v * s["scale"][rows].double()[..., None]).reshape(-1, D_C), s["pe"][rows].double()

    if c["op"] == "write":
        scale = None if s["scale"] is None else s["scale"].double()
        kv = s["kv"].double() if scale is None else s["kv"].view(torch.float8_e4m3fn).double()
        pe = s["pe"].double()
        for b in range(c["B"]):
            n0, n1 = s["cu_q"][b], s["cu_q"][b + 1]
            at = row_list(b, P[b] + torch.arange(T[b], device="cuda"))
            x = s["c_new"][n0:n1].double()
            if scale is not None:
                top = x.view(-1, D_C // 128, 128).abs().amax(-1)
                e = torch.ceil(torch.log2(top / 448))
                e = e + (top > 448 * 2.0 ** e).double() - (top <= 448 * 2.0 ** (e - 1)).double()
                scale[at] = 2.0 ** e
                x = x / (2.0 ** e).repeat_interleave(128, 1)
            kv[at], pe[at] = x, s["pe_new"][n0:n1].double()
        return {"kv": kv, "pe": pe} if scale is None else {"kv": kv, "scale": scale, "pe": pe}
    if c["op"] == "read":
        got = []
        for b in range(c["B"]):
            n0, n1 = s["cu_q"][b], s["cu_q"][b + 1]
            pos = P[b] + torch.arange(T[b], device="cuda") if s["at"] is None else s["at"][n0:n1].long()
            got.append(kept(row_list(b, pos)))
        return torch.cat([x for x, _ in got]), torch.cat([x for _, x in got])
    if work(c)["flops"] > 4e12:
        return None
    out = []
    for b in range(c["B"]):
        n0, n1 = s["cu_q"][b], s["cu_q"][b + 1]
        lat, pe = kept(row_list(b, torch.arange(P[b] + T[b], device="cuda")))
        sees = torch.ones(T[b], P[b] + T[b], dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            sees[:, P[b]:] = torch.ones(T[b], T[b], dtype=torch.bool, device="cuda").tril()
        else:
            bit = torch.arange(64, device="cuda")
            sees[:, P[b]:] = ((s["mask"][n0:n1, :, None] >> bit) & 1).bool().flatten(1)[:, :T[b]]
        heads = []
        for h in range(c["H"]):
            qn, qp = s["q_nope"][n0:n1, h].double(), s["q_pe"][n0:n1, h].double()
            z = ((qn @ s["W_UK"][h].double()) @ lat.T + qp @ pe.T) * SCALE
            p = torch.softmax(z.masked_fill(~sees, float("-inf")), -1)
            heads.append((p @ lat) @ s["W_UV"][h].double())
        out.append(torch.stack(heads, 1))
    return torch.cat(out)
