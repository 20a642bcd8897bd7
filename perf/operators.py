"""Performance cases of the rotated paged append, the shared-prefix decode and the attention with shaped scores.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits) or, where ``own`` is true, through the library's entry
points.  ``exact`` evaluates the same definition in 64 bits.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # One decoding step of 64 sequences far into their streams: one new token each is rotated and
        # enters its page.
        {"name": "rope step 64 seqs", "op": "rope", "B": 64, "len_lo": 1, "len_hi": 1, "H": 32, "Hkv": 8,
         "D": 128, "rot": 128, "interleaved": False, "page": 256, "pos_lo": 4096, "pos_hi": 131072,
         "packed": True},
        # Eight ragged prompts prefilled together, q / k / v being slices of one fused projection.
        {"name": "rope ragged prompts", "op": "rope", "B": 8, "len_lo": 301, "len_hi": 1749, "H": 32,
         "Hkv": 8, "D": 128, "rot": 128, "interleaved": False, "page": 64, "pos_lo": 0, "pos_hi": 4096,
         "packed": True},
        # Short chunks of many streams with small heads, adjacent pairs, only half of the head rotated.
        {"name": "rope half head pairs", "op": "rope", "B": 37, "len_lo": 1, "len_hi": 91, "H": 16,
         "Hkv": 16, "D": 64, "rot": 32, "interleaved": True, "page": 64, "pos_lo": 0, "pos_hi": 16384,
         "packed": False},
        # 64 answers grow from one long instruction, still short.
        {"name": "shared prompt 8192", "op": "shared", "B": 64, "H": 32, "Hkv": 8, "D": 128, "page": 256,
         "prefix": 8192, "W": 4096, "tail_lo": 1, "tail_hi": 256, "cap": 0.0, "bias": False, "keep": True},
        # A handful of candidates behind a short odd prompt; small heads, capped and biased scores.
        {"name": "shared prompt 300", "op": "shared", "B": 5, "H": 12, "Hkv": 12, "D": 64, "page": 64,
         "prefix": 300, "W": 256, "tail_lo": 1, "tail_hi": 40, "cap": 30.0, "bias": True, "keep": False},
        # Many answers over one long document, capped scores.
        {"name": "shared document 32k", "op": "shared", "B": 128, "H": 32, "Hkv": 8, "D": 128, "page": 256,
         "prefix": 32741, "W": 4096, "tail_lo": 100, "tail_hi": 700, "cap": 50.0, "bias": False,
         "keep": True},
        # Prefill of a packed row of documents, causal window of 4096, capped scores, padded end.
        {"name": "forward packed capped", "op": "forward", "B": 1, "N": 8192, "H": 32, "Hkv": 8, "D": 128,
         "L": 4095, "R": 0, "cap": 50.0, "bias": False, "docs": 7, "pad": 77, "prefix": False},
        # A bidirectional encoder with a distance bias over whole sequences.
        {"name": "forward biased encoder", "op": "forward", "B": 4, "N": 4096, "H": 12, "Hkv": 12, "D": 64,
         "L": 256, "R": 256, "cap": 0.0, "bias": True, "docs": 0, "pad": 0, "prefix": False},
        # A few short documents whose beginnings see themselves in both directions.
        {"name": "forward prefix masks", "op": "forward", "B": 2, "N": 517, "H": 8, "Hkv": 2, "D": 128,
         "L": -1, "R": 0, "cap": 0.0, "bias": False, "docs": 3, "pad": 20, "prefix": True},
        # A training step on packed documents with capped scores.
        {"name": "train packed capped", "op": "train", "B": 1, "N": 4096, "H": 32, "Hkv": 8, "D": 128,
         "L": 4095, "R": 0, "cap": 50.0, "bias": False, "docs": 4, "pad": 33, "prefix": False},
        # A training step with small heads and everything on: odd length, window, cap, bias, prefixes.
        {"name": "train small heads", "op": "train", "B": 2, "N": 1003, "H": 16, "Hkv": 16, "D": 64,
         "L": 128, "R": 0, "cap": 20.0, "bias": True, "docs": 3, "pad": 50, "prefix": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = ((32, 8), (8, 2), (12, 12), (16, 16), (16, 2), (6, 2), (4, 1), (10, 2))


def draw(rng):
    op = rng.choice(("rope", "shared", "forward", "train"))
    H, Hkv = rng.choice(HEADS)
    D = rng.choice((64, 128))
    if op == "rope":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 8192 // B))
        return {"op": op, "B": B, "len_lo": rng.randint(1, hi), "len_hi": hi, "H": H, "Hkv": Hkv, "D": D,
                "rot": rng.choice((D, D // 2, D // 4)), "interleaved": rng.random() < 0.4,
                "page": rng.choice((64, 128, 256)), "pos_lo": 0, "pos_hi": _log(rng, 1, 131072),
                "packed": rng.random() < 0.5}
    if op == "shared":
        B = _log(rng, 1, 128)
        lo = _log(rng, 1, 400)
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "D": D, "page": rng.choice((64, 128, 256)),
                "prefix": _log(rng, 64, 32000 if Hkv <= 8 else 12000), "W": _log(rng, 64, 8192), "tail_lo": lo,
                "tail_hi": lo + _log(rng, 1, 300), "cap": rng.choice((0.0, 20.0, 50.0)),
                "bias": rng.random() < 0.3, "keep": rng.random() < 0.7}
    N = _log(rng, 40, 6000 if op == "forward" else 3000)
    docs = rng.choice((0, 1, 2, 4, 7))
    R = rng.choice((0, 0, _log(rng, 1, 512)))
    return {"op": op, "B": rng.randint(1, min(4, 8000 // N)), "N": N, "H": H, "Hkv": Hkv, "D": D,
            "L": rng.choice((-1, _log(rng, 16, 4096))), "R": R, "cap": rng.choice((0.0, 20.0, 50.0)),
            "bias": rng.random() < 0.4, "docs": docs, "pad": rng.randint(0, N // 8) if docs else 0,
            "prefix": bool(docs) and rng.random() < 0.4}


# ------------------------------------------------------------------ what a case holds, apart from values
def _spread(n, lo, hi, salt):
    """n lengths in [lo, hi], unevenly spread, the same for every seed."""
    return [lo + (salt + 7919 * (i + 1) * (i + 3)) % (hi - lo + 1) for i in range(n)]


def _bounds(c):
    """Per row of the batch the documents' boundaries [docs + 1], and the prefix lengths [docs]."""
    cu, pre = [], []
    for b in range(c["B"]):
        w = [100 + x for x in _spread(c["docs"], 0, 400, 31 * b + c["N"])]
        end, at, edges = c["N"] - c["pad"], 0, [0]
        for m in range(c["docs"]):
            at += w[m]
            edges.append(end * at // sum(w))
        cu.append(edges)
        pre.append([(y - x) // (2 + m % 3) for m, (x, y) in enumerate(zip(edges, edges[1:]))])
    return cu, pre


def _pairs(c):
    """Query-key pairs of one head."""
    i = torch.arange(c["N"])
    total = 0
    cu, pre = _bounds(c) if c["docs"] else ([[0, c["N"]]] * c["B"], [[0]] * c["B"])
    for e, f in zip(cu, pre):
        for x, y, n in zip(e, e[1:], f):
            r = i[x:y]
            lo = r.clone().fill_(x) if c["L"] < 0 else (r - c["L"]).clamp(min=x)
            hi = r.clone().fill_(y - 1) if c["R"] < 0 else (r + c["R"]).clamp(max=y - 1)
            if c["prefix"]:
                hi = hi.clamp(min=x + n - 1)
            total += int((hi - lo + 1).sum())
    return total


def work(case):
    c = case
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        T = sum(_spread(c["B"], c["len_lo"], c["len_hi"], c["H"]))
        return {"bytes": 4 * T * (H + 2 * Hkv) * D, "flops": 3 * T * (H + Hkv) * c["rot"]}
    if c["op"] == "shared":
        tails = _spread(c["B"], c["tail_lo"], c["tail_hi"], c["prefix"])
        seen = [min(t, c["W"]) for t in tails]
        pre = [c["prefix"] if c["keep"] else min(c["prefix"], max(0, c["W"] - t)) for t in tails]
        return {"bytes": 4 * (max(pre) + sum(seen)) * Hkv * D + 4 * c["B"] * H * D,
                "flops": 4 * H * D * (sum(pre) + sum(seen))}
    rows = c["B"] * c["N"] * D * 2
    p = _pairs(c)
    if c["op"] == "forward":
        return {"bytes": rows * (2 * H + 2 * Hkv), "flops": 4 * H * D * p}
    return {"bytes": rows * (6 * H + 6 * Hkv), "flops": 14 * H * D * p}


# ------------------------------------------------------------------ inputs
def _pages(g, counts, first, columns, n):
    """A table [B, columns] that gives each sequence its pages, counts[b] from logical page first[b] on, in
    a random order of a pool of n pages."""
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(counts), columns), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, (k, f) in enumerate(zip(counts, first)):
        table[b, f:f + k] = order[at:at + k]
        at += k
    return table


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, D = c["H"], c["Hkv"], c["D"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

    s = {"c": c}
    if c["op"] == "rope":
        lens = _spread(c["B"], c["len_lo"], c["len_hi"], H)
        T = sum(lens)
        pos0 = torch.randint(c["pos_lo"], c["pos_hi"] + 1, (c["B"],), generator=g, device="cuda")
        at = [int(p) for p in pos0.cpu()]
        first = [p // c["page"] for p in at]
        counts = [(p + n - 1) // c["page"] - f + 1 for p, n, f in zip(at, lens, first)]
        n = sum((x + 2 * c["page"] - 2) // c["page"] for x in lens)  # as many as any positions need
        s["table"] = _pages(g, counts, first, max(f + k for f, k in zip(first, counts)), n)
        if c["packed"]:
            qkv = normal(T, (H + 2 * Hkv) * D)
            q, k, v = qkv.split((H * D, Hkv * D, Hkv * D), 1)
            s["q"], s["k"], s["v"] = q.unflatten(1, (H, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
        else:
            s["q"], s["k"], s["v"] = normal(T, H, D), normal(T, Hkv, D), normal(T, Hkv, D)
        s["k_pages"], s["v_pages"] = normal(n * c["page"], Hkv, D), normal(n * c["page"], Hkv, D)
        s["q_out"] = torch.empty(T, H, D, dtype=BF16, device="cuda")
        s["pos0"] = pos0
        edges = [0]
        for n in lens:
            edges.append(edges[-1] + n)
        s["cu"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
        i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / c["rot"])).float()
        return s
    if c["bias"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    else:
        s["slopes"] = None
    if c["op"] == "shared":
        P, page, B = c["prefix"], c["page"], c["B"]
        tails = _spread(B, c["tail_lo"], c["tail_hi"], P)
        shared = -(-P // page)
        first = [P // page] * B
        counts = [(P + t - 1) // page - P // page + 1 for t in tails]
        n = shared + sum(counts)
        table = _pages(g, [shared] + counts, [0] + first, max(shared, max(f + k for f, k in zip(first, counts))), n)
        s["prefix_table"], s["table"] = table[0, :shared].contiguous(), table[1:].contiguous()
        s["k_pages"], s["v_pages"] = normal(n * page, Hkv, D), normal(n * page, Hkv, D)
        s["q"] = normal(B, H, D, std=2.0)
        s["pos"] = torch.tensor([P + t - 1 for t in tails], dtype=torch.int64, device="cuda")
        s["longest"] = max(tails)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, device="cuda")
        return s
    B, N = c["B"], c["N"]
    s["q"], s["k"], s["v"] = normal(B, N, H, D, std=2.0), normal(B, N, Hkv, D), normal(B, N, Hkv, D)
    if c["op"] == "train":
        s["dout"] = normal(B, N, H, D)
    cu, pre = _bounds(c)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if c["docs"] else None
    s["pre"] = torch.tensor(pre, dtype=torch.int32, device="cuda") if c["prefix"] else None
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1).to(BF16)


def _rope_plain(s):
    c = s["c"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    pos = s["pos0"][b] + t - s["cu"][b]
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    row = s["table"][b, pos // c["page"]].long() * c["page"] + pos % c["page"]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
    s["k_pages"][row] = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])
    s["v_pages"][row] = s["v"]
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _shared_plain(s):
    c, pos = s["c"], s["pos"]
    P, page, H, Hkv, D = c["prefix"], c["page"], c["H"], c["Hkv"], c["D"]
    q = s["q"].float().unflatten(1, (Hkv, H // Hkv))
    j = torch.arange(P, device="cuda")
    row = s["prefix_table"][j // page].long() * page + j % page
    kp, vp = s["k_pages"][row].float(), s["v_pages"][row].float()
    o = torch.arange(P, P + s["longest"], device="cuda")
    row = s["table"][:, o // page].clamp(min=0).long() * page + o % page
    ko, vo = s["k_pages"][row].float(), s["v_pages"][row].float()
    x = torch.cat((torch.einsum("bgid,pgd->bgip", q, kp), torch.einsum("bgid,bpgd->bgip", q, ko)), -1)
    x = x / math.sqrt(D)
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j = torch.cat((j, o))
    far = pos[:, None] - j
    if c["bias"]:
        x = x - s["slopes"].view(1, Hkv, -1, 1) * far[:, None, None, :].float()
    keep = (far >= 0) & (far < c["W"])
    if c["keep"]:
        keep = keep | ((j < P) & (far >= 0))
    x = x.masked_fill(~keep[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    y = torch.einsum("bgip,pgd->bgid", p[..., :P], vp) + torch.einsum("bgip,bpgd->bgid", p[..., P:], vo)
    return {"out": (y / l).flatten(1, 2).to(BF16), "lse": (m + torch.log(l)).flatten(1)}


def _keys(s):
    """First and last key of each row, [B, N] each (last < first: none)."""
    c = s["c"]
    i = torch.arange(c["N"], device="cuda").expand(c["B"], -1)
    start, end, pre = torch.zeros_like(i), torch.full_like(i, c["N"]), torch.zeros_like(i)
    if s["cu"] is not None:
        cu = s["cu"].long()
        m = (i[:, :, None] >= cu[:, None, 1:]).sum(-1)
        inside = m < c["docs"]
        m = m.clamp(max=c["docs"] - 1)
        start = cu[:, :-1].gather(1, m)
        end = torch.where(inside, cu[:, 1:].gather(1, m), start)
        if s["pre"] is not None:
            pre = s["pre"].long().gather(1, m)
    lo = start if c["L"] < 0 else torch.maximum(start, i - c["L"])
    hi = end - 1 if c["R"] < 0 else torch.minimum(end - 1, torch.maximum(i + c["R"], start + pre - 1))
    return torch.where(end > start, lo, 1), torch.where(end > start, hi, 0)


def _attend_plain(s):
    """out and lse in 32 bits, and what the gradients need."""
    c = s["c"]
    q = s["q"].float().unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    k, v = s["k"].float().permute(0, 2, 1, 3)[:, :, None], s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    x = q @ k.transpose(-1, -2) * s["scale"]
    slope = None
    if c["cap"] > 0:
        t = torch.tanh(x / c["cap"])
        slope = 1.0 - t * t if c["op"] == "train" else None
        x = c["cap"] * t
        del t
    i = torch.arange(c["N"], device="cuda")
    if c["bias"]:
        x = x - s["slopes"].view(1, c["Hkv"], -1, 1, 1) * (i[:, None] - i).abs().float()
    lo, hi = _keys(s)
    keep = (i >= lo[:, :, None]) & (i <= hi[:, :, None])
    x = x.masked_fill_(~keep[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).squeeze(-1).flatten(1, 2)
    p = p.mul_(torch.where(l > 0, 1.0 / l, 0.0))
    return q, k, v, p, slope, p @ v, lse


def _rows(x):
    """[B, Hkv, G, N, D] -> [B, N, H, D], rounded."""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3).to(BF16)


def _forward_plain(s):
    _, _, _, _, _, y, lse = _attend_plain(s)
    return {"out": _rows(y), "lse": lse}


def _train_plain(s):
    q, k, v, p, slope, y, lse = _attend_plain(s)
    do = s["dout"].float().unflatten(2, (s["c"]["Hkv"], -1)).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    ds = (do @ v.transpose(-1, -2)).sub_((do * y).sum(-1, keepdim=True)).mul_(p)
    if slope is not None:
        ds = ds.mul_(slope)
    dq = ds @ k * s["scale"]
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True) * s["scale"]
    return {"out": _rows(y), "lse": lse, "dq": _rows(dq), "dk": _rows(dk), "dv": _rows(dv)}


# ------------------------------------------------------------------ the library's entry points
def _own(s):
    import sliding_window_attention_fwd_b200 as swa

    c = s["c"]
    if c["op"] == "rope":
        swa.swa_rope_append_paged(s["q"], s["k"], s["v"], s["inv_freq"], s["cu"], s["pos0"], s["table"],
                                  s["k_pages"], s["v_pages"], c["page"], q_out=s["q_out"],
                                  interleaved=c["interleaved"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "shared":
        swa.swa_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], c["prefix"], s["table"],
                              s["pos"], c["page"], c["W"], out=s["out"], lse=s["lse"],
                              keep_prefix=c["keep"], max_tail=s["longest"], softcap=c["cap"],
                              slopes=s["slopes"])
        return {"out": s["out"], "lse": s["lse"]}
    lse = torch.empty(c["B"], c["H"], c["N"], device="cuda")
    shape = {"win_left": c["L"], "win_right": c["R"], "softcap": c["cap"], "slopes": s["slopes"],
             "cu_docs": s["cu"], "prefix": s["pre"]}
    out = swa.swa_forward_scored(s["q"], s["k"], s["v"], lse=lse, **shape)
    if c["op"] == "forward":
        return {"out": out, "lse": lse}
    dq, dk, dv = swa.swa_backward_scored(s["q"], s["k"], s["v"], out, s["dout"], lse, **shape)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope_plain, "shared": _shared_plain, "forward": _forward_plain,
            "train": _train_plain}[state["c"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _turn(x, pos, inv_freq, rot, interleaved):
    """Multiplies the pairs of x [n, heads, D], as complex numbers, by exp(i pos inv_freq)."""
    x = x.double()
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * inv_freq.double())
    half = x[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    half = half if interleaved else half.transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(half.contiguous()) * w[:, None])
    y = (y if interleaved else y.transpose(-1, -2)).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _rope_exact(s):
    c = s["c"]
    q, kp, vp = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), s["k_pages"].double(), s["v_pages"].double()
    cu, pos0, table = s["cu"].tolist(), s["pos0"].tolist(), s["table"].cpu()
    for b in range(c["B"]):
        x, y = cu[b], cu[b + 1]
        pos = torch.arange(pos0[b], pos0[b] + y - x)
        row = (table[b, pos // c["page"]].long() * c["page"] + pos % c["page"]).cuda()
        q[x:y] = _turn(s["q"][x:y], pos.cuda(), s["inv_freq"], c["rot"], c["interleaved"])
        kp[row] = _turn(s["k"][x:y], pos.cuda(), s["inv_freq"], c["rot"], c["interleaved"])
        vp[row] = s["v"][x:y].double()
    return {"q": q, "k_pages": kp, "v_pages": vp}


def _shared_exact(s):
    c = s["c"]
    P, page, H, Hkv, D = c["prefix"], c["page"], c["H"], c["Hkv"], c["D"]
    out = torch.empty(c["B"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["B"], H, dtype=torch.float64, device="cuda")
    ptab, table, grp = s["prefix_table"].cpu(), s["table"].cpu(), H // Hkv
    for b, p in enumerate(s["pos"].tolist()):
        j = torch.tensor([x for x in range(p + 1) if x > p - c["W"] or (c["keep"] and x < P)])
        page_of = torch.where(j < P, ptab[(j // page).clamp(max=len(ptab) - 1)], table[b, j // page])
        row = (page_of.long() * page + j % page).cuda()
        k, v = s["k_pages"][row].double(), s["v_pages"][row].double()
        x = torch.einsum("gid,jgd->gij", s["q"][b].double().view(Hkv, grp, D), k) / math.sqrt(D)
        if c["cap"] > 0:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if c["bias"]:
            x = x - s["slopes"].double().view(Hkv, grp, 1) * (p - j).cuda().double()
        out[b] = torch.einsum("gij,jgd->gid", torch.softmax(x, -1), v).reshape(H, D)
        lse[b] = torch.logsumexp(x, -1).view(H)
    return {"out": out, "lse": lse}


def _seen(c, b):
    """Which keys [N, N] the rows of sequence b see, from the definition, document by document."""
    seen = torch.zeros(c["N"], c["N"], dtype=torch.bool, device="cuda")
    cu, pre = _bounds(c) if c["docs"] else ([[0, c["N"]]] * c["B"], [[0]] * c["B"])
    for x, y, n in zip(cu[b], cu[b][1:], pre[b]):
        i = torch.arange(y - x, device="cuda")
        back = i[:, None] - i[None, :]
        ahead = torch.ones_like(back, dtype=torch.bool) if c["R"] < 0 else back >= -c["R"]
        if c["prefix"]:
            ahead |= (i < n)[:, None] & (i < n)[None, :]
        seen[x:y, x:y] = ahead if c["L"] < 0 else ahead & (back <= c["L"])
    return seen


def _attend_exact(s, train):
    c = s["c"]
    B, N, H, Hkv, D = c["B"], c["N"], c["H"], c["Hkv"], c["D"]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    got = {"out": new(B, N, H, D), "lse": new(B, H, N)}
    if train:
        got |= {"dq": new(B, N, H, D), "dk": new(B, N, Hkv, D), "dv": new(B, N, Hkv, D)}
    i = torch.arange(N, device="cuda")
    dist = (i[:, None] - i).abs().double()
    for b in range(B):
        seen = _seen(c, b)
        some = seen.any(1)
        for h in range(H):
            g = h // (H // Hkv)
            q, k, v = (t.double().clone().requires_grad_(train) for t in (s["q"][b, :, h], s["k"][b, :, g], s["v"][b, :, g]))
            x = q @ k.T / math.sqrt(D)
            if c["cap"] > 0:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if c["bias"]:
                x = x - s["slopes"][h].double() * dist
            x = torch.where(seen, x, -math.inf)[some]
            y = torch.softmax(x, -1) @ v
            got["out"][b, some, h] = y.detach()
            got["lse"][b, h] = -math.inf
            got["lse"][b, h, some] = torch.logsumexp(x.detach(), -1)
            if train:
                dq, dk, dv = torch.autograd.grad(y, (q, k, v), s["dout"][b, :, h].double()[some])
                got["dq"][b, :, h] = dq
                got["dk"][b, :, g] += dk
                got["dv"][b, :, g] += dv
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s)
    if case["op"] == "shared":
        return _shared_exact(s)
    return _attend_exact(s, case["op"] == "train")
