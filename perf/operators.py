"""Workloads of the operators around a verification step: the logits adjustment,
the 4-bit LM head and the attention of draft rows over a shared prefix.

Each case is a dict of plain values.  ``prepare`` makes a case's inputs from a
seed, ``run`` takes one pass through the operator: in its plain form (torch
operations in float32) or, with ``own`` set, through this package's call.
``exact`` gives the same outputs in float64 from the definitions.
"""
import math

import torch

own = False
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
NEG_INF = float("-inf")


def listed():
    return [
        # -- logits adjustment ------------------------------------------------
        # target rows of the B=256 gamma=8 window: penalties over a chat history, out of place
        {"name": "adjust_window_b256", "op": "adjust", "B": 256, "R": 9, "tree": "", "V": 128256, "dtype": "bf16",
         "hist": 2048, "bias": 32, "mask": "none", "allow": 1.0, "inplace": False},
        # tree (4, 3, 2) with a grammar state per node (odd vocabulary)
        {"name": "adjust_tree_b4", "op": "adjust", "B": 4, "R": 41, "tree": "4,3,2", "V": 50257, "dtype": "f16",
         "hist": 700, "bias": 8, "mask": "row", "allow": 0.25, "inplace": False},
        # one token of one sequence: the draft model's own step, latency only
        {"name": "adjust_single_b1", "op": "adjust", "B": 1, "R": 1, "tree": "", "V": 32000, "dtype": "f32",
         "hist": 300, "bias": 0, "mask": "none", "allow": 1.0, "inplace": False},
        # grammar mask alone, in place on the logits buffer of a window, a state per row
        {"name": "adjust_mask_inplace_b32", "op": "adjust", "B": 32, "R": 9, "tree": "", "V": 128256, "dtype": "bf16",
         "hist": 0, "bias": 0, "mask": "row", "allow": 0.02, "inplace": True},
        # -- 4-bit LM head ----------------------------------------------------
        # one token of a small draft model
        {"name": "head_m1_v32000", "op": "head", "M": 1, "K": 2048, "V": 32000, "G": 64, "dtype": "f16", "zeros": False, "out": "f32"},
        # a draft step of 8 sequences, weights with zero points
        {"name": "head_m8_v128256", "op": "head", "M": 8, "K": 4096, "V": 128256, "G": 128, "dtype": "bf16", "zeros": True, "out": "f32"},
        # the window of 8 sequences (gamma = 8) through a quantised target head
        {"name": "head_m72_v128256", "op": "head", "M": 72, "K": 4096, "V": 128256, "G": 128, "dtype": "bf16", "zeros": False, "out": "bf16"},
        # a draft step of 256 sequences, odd vocabulary
        {"name": "head_m256_v50257", "op": "head", "M": 256, "K": 4096, "V": 50257, "G": 32, "dtype": "bf16", "zeros": True, "out": "f32"},
        # -- attention over a shared prefix -----------------------------------
        # one token of one sequence behind a short system prompt, latency only
        {"name": "attend_single_b1", "op": "attend", "B": 1, "R": 1, "tree": "", "Hq": 32, "Hkv": 8, "D": 128, "P": 333, "ctx": 700, "dtype": "bf16"},
        # tree (4, 3, 2) of four sequences, 20 heads of 64 without grouping, no prefix
        {"name": "attend_tree_b4", "op": "attend", "B": 4, "R": 41, "tree": "4,3,2", "Hq": 20, "Hkv": 20, "D": 64, "P": 0, "ctx": 983, "dtype": "f16"},
        # windows of 64 sequences behind one long prompt: the prefix is matrix work
        {"name": "attend_window_b64", "op": "attend", "B": 64, "R": 9, "tree": "", "Hq": 32, "Hkv": 8, "D": 128, "P": 8192, "ctx": 1024, "dtype": "bf16"},
        # single tokens of 128 sequences with long caches of their own: the caches are the traffic
        {"name": "attend_decode_b128", "op": "attend", "B": 128, "R": 1, "tree": "", "Hq": 32, "Hkv": 8, "D": 128, "P": 2048, "ctx": 4000, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_int0(rng, lo, hi):
    """0 in one case out of four, else log-spread over [lo, hi]."""
    return 0 if rng.random() < 0.25 else _log_int(rng, lo, hi)


def draw(rng):
    op = rng.choice(["adjust", "head", "attend"])
    if op == "adjust":
        V = _log_int(rng, 1000, 131072)
        tree = rng.choice(["", "", "4,3,2", "2,2,2", "3,1,1"])
        R = len(_parents(tree)) if tree else rng.randint(1, 17)
        B = _log_int(rng, 1, 256)
        B = max(1, min(B, 256 * 9 * 128256 // (R * V)))
        mask = rng.choice(["none", "row", "seq"])
        return {"op": op, "B": B, "R": R, "tree": tree, "V": V, "dtype": rng.choice(["f32", "bf16", "f16"]) if B * R * V < 1 << 27 else "bf16",
                "hist": _log_int0(rng, 8, 8192), "bias": rng.choice([0, 1, 32, 300]), "mask": mask,
                "allow": 1.0 if mask == "none" else rng.choice([0.02, 0.5, 0.95]), "inplace": False}
    if op == "head":
        G = rng.choice([32, 64, 128])
        unit = max(G, 64)
        K = unit * _log_int(rng, 512 // unit, 8192 // unit)
        V = _log_int(rng, 1000, 131072)
        M = max(1, min(_log_int(rng, 1, 256), 256 * 4096 * 50257 // (K * V)))
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "M": M, "K": K, "V": V, "G": G, "dtype": dtype, "zeros": rng.random() < 0.5, "out": rng.choice(["f32", dtype])}
    tree = rng.choice(["", "", "4,3,2", "2,2,2"])
    R = len(_parents(tree)) if tree else rng.randint(1, 17)
    Hkv, D = rng.choice([1, 2, 4, 8, 20]), rng.choice([64, 128])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    P, ctx = _log_int0(rng, 16, 8192), _log_int0(rng, 16, 4000)
    B = _log_int(rng, 1, 128)
    B = max(1, min(B, 64 * 9 * 32 * 128 * 9000 // (R * Hq * D * (P + ctx + R)), 128 * 4000 * 8 * 128 // ((ctx + R) * Hkv * D)))
    return {"op": op, "B": B, "R": R, "tree": tree, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "ctx": ctx, "dtype": rng.choice(["bf16", "f16"])}


# -- the rows of a step ----------------------------------------------------------
def _parents(tree):
    """Parent array of a tree given by its branching factors, breadth first."""
    parent, level = [-1], [0]
    for f in (int(x) for x in tree.split(",")):
        level = [len(parent) + i for i in range(len(level) * f)]
        parent += [p for p in range(level[0] - len(level) // f, level[0]) for _ in range(f)]
    return parent


def _row_parents(c):
    return _parents(c["tree"]) if c["tree"] else list(range(-1, c["R"] - 1))


def _ancestors(parent):
    """anc[v][w]: w is v or an ancestor of v."""
    R = len(parent)
    anc = torch.zeros(R, R, dtype=torch.bool)
    for v, p in enumerate(parent):
        if p >= 0:
            anc[v] = anc[p]
        anc[v, v] = True
    return anc


def _lens(lo, hi, B, g):
    """B lengths spread evenly over [lo, hi], in an order of the seed's."""
    at = torch.randperm(B, generator=g, device=DEV)
    return (lo + (hi - lo) * (at + 1) // B).to(torch.int32)


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _tokens(shape, V, g):
    """Token ids as text has them: few frequent ones, a long tail."""
    return (torch.rand(shape, generator=g, device=DEV) ** 4 * V).long().clamp_(max=V - 1).to(torch.int32)


def prepare(c, seed):
    g = _generator(seed)
    parent = _row_parents(c) if c["op"] != "head" else None
    return {"adjust": _prepare_adjust, "head": _prepare_head, "attend": _prepare_attend}[c["op"]](c, g, parent)


def _prepare_adjust(c, g, parent):
    B, R, V = c["B"], c["R"], c["V"]
    x = torch.empty(B, R, V, dtype=DTYPES[c["dtype"]], device=DEV)
    for b in range(0, B, 16):
        x[b:b + 16] = torch.randn(min(16, B - b), R, V, generator=g, device=DEV) * 3
    s = {"c": c, "x": x, "parent": parent if c["tree"] else None, "allowed": None}
    # window row i follows drafts 0..i-1 (tokens[i-1] is row i's own node); a tree's node v carries tokens[v]
    s["tokens"] = _tokens((B, R if c["tree"] else max(R - 1, 1)), V, g)
    anc = _ancestors(parent).to(DEV)
    anc[:, 0] = False
    s["anc"] = anc
    s["history"] = s["history_len"] = s["prompt_len"] = None
    s["repetition"] = s["presence"] = s["frequency"] = s["bias_tokens"] = s["bias_values"] = None
    if not c["inplace"]:
        s["repetition"] = 1 + 0.3 * torch.rand(B, generator=g, device=DEV)
        s["presence"] = 0.5 * torch.rand(B, generator=g, device=DEV)
        s["frequency"] = 0.3 * torch.rand(B, generator=g, device=DEV)
    if c["hist"]:
        s["history"] = _tokens((B, c["hist"]), V, g)
        s["history_len"] = _lens(c["hist"] // 4, c["hist"], B, g)
        s["prompt_len"] = (s["history_len"] // 2).to(torch.int32)
    if c["bias"]:
        s["bias_tokens"] = _tokens((B, c["bias"]), V, g)
        s["bias_values"] = torch.randn(B, c["bias"], generator=g, device=DEV) * 5
    if c["mask"] != "none":
        rows, W = R if c["mask"] == "row" else 1, (V + 31) // 32
        words = torch.empty(B, rows, W, dtype=torch.int32, device=DEV)
        weight = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
        for b in range(0, B, 4):
            bits = torch.rand(min(4, B - b), rows, W, 32, generator=g, device=DEV) < c["allow"]
            w = (bits * weight).sum(-1)
            words[b:b + 4] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
        s["allowed"] = words.expand(B, R, W)
    return s


def _prepare_head(c, g, parent):
    M, K, V, G, t = c["M"], c["K"], c["V"], c["G"], DTYPES[c["dtype"]]
    h = torch.randn(M, K, generator=g, device=DEV)
    h[:, torch.randint(0, K, (4,), generator=g, device=DEV)] *= 8  # a few channels stand out
    s = {"c": c, "h": h.to(t)}
    s["wq"] = torch.randint(0, 256, (V, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand(V, K // G, generator=g, device=DEV)) * 0.01).to(t)
    s["zeros"] = torch.randint(4, 12, (V, K // G), generator=g, device=DEV, dtype=torch.uint8) if c["zeros"] else None
    return s


def _prepare_attend(c, g, parent):
    B, R, Hq, Hkv, D, P, t = c["B"], c["R"], c["Hq"], c["Hkv"], c["D"], c["P"], DTYPES[c["dtype"]]
    cap = c["ctx"] + R + 7
    s = {"c": c, "parent": parent if c["tree"] else None, "anc": _ancestors(parent).to(DEV)}
    s["q"] = (1.5 * torch.randn(B, R, Hq, D, generator=g, device=DEV)).to(t)
    s["len"] = _lens(c["ctx"] // 4, c["ctx"], B, g)
    s["pk"] = torch.randn(P, Hkv, D, generator=g, device=DEV).to(t) if P else None
    s["pv"] = torch.randn(P, Hkv, D, generator=g, device=DEV).to(t) if P else None
    for n in ("k", "v"):
        s[n] = torch.empty(B, cap, Hkv, D, dtype=t, device=DEV)
        for b in range(B):
            s[n][b] = torch.randn(cap, Hkv, D, generator=g, device=DEV)
    return s


def run(s):
    return {"adjust": _run_adjust, "head": _run_head, "attend": _run_attend}[s["c"]["op"]](s)


def _run_adjust(s):
    c, x = s["c"], s["x"]
    if own:
        import draft_token_verification_06_amd as sv
        return sv.adjust_logits(x, tokens=s["tokens"], parent=s["parent"], history=s["history"], history_len=s["history_len"],
                                prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                                frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                                allowed=s["allowed"], out=x if c["inplace"] else None)
    B, R, V = x.shape
    y = x.float()
    if s["repetition"] is not None:
        # occurrences: the history's (dead entries go to column V), then each row's path
        count = torch.zeros(B, R, V + 1, dtype=torch.int32, device=DEV)
        prompt = torch.zeros(B, 1, V + 1, dtype=torch.int32, device=DEV)
        if s["history"] is not None:
            h, at = s["history"].long(), torch.arange(s["history"].shape[1], device=DEV)
            dead = torch.full_like(h, V)
            said = torch.where((at >= s["prompt_len"][:, None]) & (at < s["history_len"][:, None]), h, dead)
            told = torch.where(at < s["prompt_len"][:, None], h, dead)
            base = torch.zeros(B, V + 1, dtype=torch.int32, device=DEV).scatter_add_(1, said, torch.ones_like(said, dtype=torch.int32))
            prompt = prompt.scatter_(2, told[:, None], 1)
            count += base[:, None]
        if R > 1:
            node = torch.zeros(B, R, dtype=torch.int64, device=DEV)
            node[:, 1:] = s["tokens"][:, 1:] if s["parent"] is not None else s["tokens"][:, :R - 1]
            path = torch.where(s["anc"], node[:, None, :].expand(B, R, R), V)
            count.scatter_add_(2, path, torch.ones_like(path, dtype=torch.int32))
        count, prompt = count[..., :V], prompt[..., :V]
        rho = s["repetition"][:, None, None]
        y = torch.where((count > 0) | (prompt > 0), torch.where(y > 0, y / rho, y * rho), y)
        y = y - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_tokens"] is not None:
        # of the entries that name one token the last one counts
        n = s["bias_tokens"].shape[1]
        which = torch.zeros(B, V, dtype=torch.int64, device=DEV)
        which.scatter_reduce_(1, s["bias_tokens"].long(), torch.arange(1, n + 1, device=DEV).expand(B, n), "amax")
        values = torch.cat([torch.zeros(B, 1, device=DEV), s["bias_values"]], 1)
        y = y + torch.gather(values, 1, which)[:, None]
    if s["allowed"] is not None:
        bits = (s["allowed"][..., None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        y = torch.where(bits.reshape(B, R, -1)[..., :V] != 0, y, NEG_INF)
    if c["inplace"]:
        return x.copy_(y)
    return y.to(x.dtype)


def _nibbles(wq):
    """4-bit values (rows, K) of packed rows: the even k in the low half of byte k / 2."""
    return torch.stack([wq & 15, wq >> 4], -1).reshape(wq.shape[0], -1)


def _run_head(s):
    c = s["c"]
    if own:
        import draft_token_verification_06_amd as sv
        return sv.lmhead_quant(s["h"], s["wq"], s["scales"], s["zeros"], out_dtype=DTYPES[c["out"]])
    V, G = c["V"], c["G"]
    q = _nibbles(s["wq"]).float().view(V, -1, G)
    w = (q - (s["zeros"].float()[..., None] if s["zeros"] is not None else 8.0)) * s["scales"].float()[..., None]
    return (s["h"].float() @ w.view(V, -1).t()).to(DTYPES[c["out"]])


def _run_attend(s):
    c, q = s["c"], s["q"]
    B, R, Hq, D = q.shape
    Hkv, P, scale = c["Hkv"], c["P"], 1 / math.sqrt(D)
    if own:
        import draft_token_verification_06_amd as sv
        r = sv.attention(q, s["k"], s["v"], s["len"], prefix_k=s["pk"], prefix_v=s["pv"], parent=s["parent"], scale=scale,
                         return_lse=True)
        return r.out, r.lse
    n = Hq // Hkv
    # rows (b, r, head of the group) of each kv head
    x = q.float().view(B, R, Hkv, n, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * n, D)
    k, v = s["k"].float().permute(0, 2, 1, 3).contiguous(), s["v"].float().permute(0, 2, 1, 3).contiguous()
    L = k.shape[2]
    score = torch.matmul(x, k.transpose(2, 3).contiguous()) * scale
    rel = torch.arange(L, device=DEV) - s["len"][:, None]
    seen = torch.zeros(B, R, L, dtype=torch.bool, device=DEV) | (rel < 0)[:, None]
    draft = ((rel >= 0) & (rel < R))[:, None].expand(B, R, L)
    seen |= draft & torch.gather(s["anc"].expand(B, R, R), 2, rel.clamp(0, R - 1)[:, None].expand(B, R, L))
    score = score.masked_fill_(~seen.repeat_interleave(n, 1)[:, None], NEG_INF)
    if P:
        pk, pv = (s[i].float().permute(1, 0, 2).contiguous() for i in ("pk", "pv"))
        xp = x.permute(1, 0, 2, 3).reshape(Hkv, B * R * n, D)
        before = torch.matmul(xp, pk.transpose(1, 2).contiguous()) * scale
        score = torch.cat([before.view(Hkv, B, R * n, P).transpose(0, 1), score], 3)
    top = score.amax(3, keepdim=True)
    e = (score - top).exp_()
    total = e.sum(3, keepdim=True)
    o = torch.matmul(e[..., P:], v)
    if P:
        before = e[..., :P].transpose(0, 1).reshape(Hkv, B * R * n, P)
        o += torch.matmul(before, pv).view(Hkv, B, R * n, D).transpose(0, 1)
    o = (o / total).view(B, Hkv, R, n, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(q.dtype)
    lse = (top + total.log()).view(B, Hkv, R, n).permute(0, 2, 1, 3).reshape(B, R, Hq)
    return o, lse


def work(c):
    e = BYTES[c["dtype"]]
    if c["op"] == "adjust":
        rows, V = c["B"] * c["R"], c["V"]
        masks = {"none": 0, "row": rows, "seq": c["B"]}[c["mask"]] * V / 8
        if c["inplace"]:  # what the mask forbids is written, the rest stays
            return {"bytes": masks + rows * V * e * (1 - c["allow"]), "flops": 0}
        small = c["B"] * (4 * c["hist"] * 5 / 8 + 8 * c["bias"])
        return {"bytes": rows * V * e * (1 + c["allow"]) + masks + small, "flops": rows * V}
    if c["op"] == "head":
        M, K, V, groups = c["M"], c["K"], c["V"], c["K"] // c["G"]
        return {"bytes": V * K / 2 + V * groups * (e + bool(c["zeros"])) + M * K * e + M * V * BYTES[c["out"]], "flops": 2 * M * K * V}
    B, R, Hq, Hkv, D, P = c["B"], c["R"], c["Hq"], c["Hkv"], c["D"], c["P"]
    lo, hi = c["ctx"] // 4, c["ctx"]
    own_keys = sum(lo + (hi - lo) * (i + 1) // B for i in range(B))
    pairs = B * R * P + R * own_keys + B * int(_ancestors(_row_parents(c)).sum())
    return {"bytes": 2 * B * R * Hq * D * e + 4 * B * R * Hq + 2 * Hkv * D * e * (P + own_keys + B * R), "flops": 4 * D * Hq * pairs}


# -- the definitions in 64 bits --------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return {"adjust": _exact_adjust, "head": _exact_head, "attend": _exact_attend}[c["op"]](c, s)


def _exact_adjust(c, s):
    B, R, V = s["x"].shape
    if B * R * V > 1 << 29:  # larger calls take too long row by row
        return None
    out = torch.empty(B, R, V, dtype=torch.float64, device=DEV)
    parent = _row_parents(c)
    shifts = torch.arange(32, device=DEV)
    for b in range(B):
        said = torch.zeros(V, dtype=torch.float64, device=DEV)
        told = torch.zeros(V, dtype=torch.bool, device=DEV)
        if s["history"] is not None:
            n, p = int(s["history_len"][b]), int(s["prompt_len"][b])
            said += torch.bincount(s["history"][b, p:n].long(), minlength=V)
            told[s["history"][b, :p].long()] = True
        bias = torch.zeros(V, dtype=torch.float64, device=DEV)
        if s["bias_tokens"] is not None:
            last = dict(zip(s["bias_tokens"][b].tolist(), s["bias_values"][b].double().tolist()))
            bias[torch.tensor(list(last), device=DEV)] = torch.tensor(list(last.values()), dtype=torch.float64, device=DEV)
        node = s["tokens"][b].tolist()
        node = node if s["parent"] is not None else [-1] + node
        for r in range(R):
            y = s["x"][b, r].double()
            if s["repetition"] is not None:
                count, v = said.clone(), r
                while v > 0:
                    count[node[v]] += 1
                    v = parent[v]
                rho = s["repetition"][b].double()
                y = torch.where((count > 0) | told, torch.where(y > 0, y / rho, y * rho), y)
                y = y - s["frequency"][b].double() * count - s["presence"][b].double() * (count > 0).double()
            y = y + bias
            if s["allowed"] is not None:
                bits = ((s["allowed"][b, r].long()[:, None] >> shifts) & 1).reshape(-1)[:V]
                y[bits == 0] = NEG_INF
            out[b, r] = y
    return out


def _exact_head(c, s):
    V, G = c["V"], c["G"]
    h, out = s["h"].double(), torch.empty(c["M"], c["V"], dtype=torch.float64, device=DEV)
    for v in range(0, V, 8192):
        q = torch.empty(min(8192, V - v), c["K"], dtype=torch.float64, device=DEV)
        q[:, 0::2], q[:, 1::2] = (s["wq"][v:v + 8192] % 16).double(), (s["wq"][v:v + 8192] // 16).double()
        z = s["zeros"][v:v + 8192].double() if s["zeros"] is not None else torch.full_like(s["scales"][v:v + 8192], 8).double()
        w = (q - z.repeat_interleave(G, 1)) * s["scales"][v:v + 8192].double().repeat_interleave(G, 1)
        out[:, v:v + 8192] = h @ w.t().contiguous()
    return out


def _exact_attend(c, s):
    B, R, Hq, Hkv, D, P = c["B"], c["R"], c["Hq"], c["Hkv"], c["D"], c["P"]
    o = torch.empty(B, R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, R, Hq, dtype=torch.float64, device=DEV)
    n = Hq // Hkv
    for b in range(B):
        L = int(s["len"][b])
        k, v = s["k"][b, :L + R].double(), s["v"][b, :L + R].double()
        if P:
            k, v = torch.cat([s["pk"].double(), k]), torch.cat([s["pv"].double(), v])
        ok = torch.ones(R, P + L + R, dtype=torch.bool, device=DEV)
        ok[:, P + L:] = s["anc"]
        for h in range(Hkv):
            q = s["q"][b, :, h * n:(h + 1) * n].double().reshape(R * n, D)
            a = (q @ k[:, h].t().contiguous()) / math.sqrt(D)
            a[~ok.repeat_interleave(n, 0)] = NEG_INF
            z = torch.logsumexp(a, 1)
            lse[b, :, h * n:(h + 1) * n] = z.view(R, n)
            o[b, :, h * n:(h + 1) * n] = ((a - z[:, None]).exp() @ v[:, h]).view(R, n, D)
    return o, lse
