"""Cases of the prompt-side operators: the rotation table of positions with several axes
(spec_rope_table_axes), the append of a chunk's rotated keys and values to the paged cache
(spec_kv_append_paged) and the attention of a chunk of new tokens over that cache
(spec_chunk_attention_paged).

Every case is one call: `run` computes it in elementary torch operations, or with `own` set through
the library.  Row counts and context lengths of a batch follow from the case alone (`lengths`).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 128      # keys per cache page
D = 128         # head size of the cache
THETA = 1e6

_ws = None      # the program's one workspace (own only)


# --------------------------------------------------------------------------- cases
def _attn(name, Hq, Hkv, B, rows, ctx, ones=0, lens=1):
    return {"name": name, "op": "attention", "Hq": Hq, "Hkv": Hkv, "B": B, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ones": ones, "lens": lens}


def _append(name, Hq, Hkv, B, rows, ctx, ones=0, lens=1, rotate=True):
    return {"name": name, "op": "append", "Hq": Hq, "Hkv": Hkv, "B": B, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ones": ones, "lens": lens, "rotate": rotate}


def _table(name, rows, t, h, w, interleaved):
    return {"name": name, "op": "table", "rows": rows, "t": t, "h": h, "w": w, "interleaved": interleaved}


def listed():
    return [
        # a few sequences one token at a time in short contexts: launch and latency
        _attn("attn 4 x 1 token", 32, 8, 4, (1, 1), (300, 1000)),
        # one chunk of a prompt behind what earlier chunks left in the cache
        _attn("attn chunk 512 at 7680", 32, 8, 1, (512, 512), (7680, 7680)),
        # a whole long prompt at once, nothing cached
        _attn("attn prompt 8192", 32, 8, 1, (8192, 8192), (0, 0)),
        # a serving step: most sequences decode, a few bring chunks of odd sizes
        _attn("attn mixed 24", 32, 8, 24, (97, 333), (0, 4096), ones=18, lens=2),
        # short prompts of the draft stack (2 query heads per kv head), ragged
        _attn("attn draft prompts", 16, 8, 8, (100, 1900), (0, 0), lens=3),
        # a short question behind a very long document
        _attn("attn 61 rows at 131000", 32, 8, 1, (61, 61), (131000, 131000)),
        # the appends that go with them: single tokens, a whole prompt, a ragged serving step
        _append("append 8 x 1 token", 32, 8, 8, (1, 1), (100, 2000)),
        _append("append prompt 8192", 32, 8, 1, (8192, 8192), (0, 0)),
        _append("append mixed 24", 16, 8, 24, (97, 999), (0, 4096), ones=12, lens=4),
        # keys already rotated by the projection: a plain append
        _append("append rotated keys", 32, 8, 6, (300, 900), (1, 1500), lens=5, rotate=False),
        # positions of a small image's tokens, and of a video's
        _table("table 77 rows", 77, 16, 24, 24, False),
        _table("table 16000 rows", 16000, 24, 20, 20, True),
    ]


def lengths(case):
    """Rows and cached tokens of each sequence: `ones` sequences bring one row, the others a chunk."""
    r = random.Random(case["lens"])
    rows = [1 if b < case["ones"] else r.randint(case["rows_lo"], case["rows_hi"]) for b in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    order = list(range(case["B"]))
    r.shuffle(order)
    return [rows[b] for b in order], [ctx[b] for b in order]


HEADS = [(32, 8), (16, 8), (8, 8), (32, 4), (28, 4), (12, 4), (16, 1), (5, 1), (40, 8)]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_batch(rng, rows_max, ctx_max):
    while True:
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, rows_max)
        lo = rng.randint(1, hi)
        chi = _log_int(rng, 1, ctx_max) if rng.random() < 0.85 else 0
        c = {"B": B, "rows_lo": lo, "rows_hi": hi, "ctx_lo": rng.randint(0, chi), "ctx_hi": chi,
             "ones": rng.randint(0, B - 1) if rng.random() < 0.4 else 0, "lens": rng.randrange(1 << 20)}
        rows, ctx = lengths(c)
        keys = max(m + n for m, n in zip(rows, ctx))
        if sum(rows) <= 16384 and B * keys <= 140000:
            return c, rows, keys


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "table"])
    if op == "table":
        half, a = D // 2, rng.choice([1, 2, 3])
        t, h = (half, 0) if a == 1 else (rng.randint(8, 48), 0)
        h = half - t if a == 2 else (rng.randint(4, half - t - 4) if a == 3 else 0)
        il = a == 3 and rng.random() < 0.5
        if il:      # the interleaved order gives an axis at most every third frequency
            h = min(h, 20)
            w = rng.randint(1, 20)
            t = half - h - w
        else:
            w = half - t - h
        return {"op": op, "rows": _log_int(rng, 1, 16000), "t": t, "h": h, "w": w, "interleaved": il}
    Hq, Hkv = rng.choice(HEADS)
    if op == "append":
        while True:
            c, rows, _ = _draw_batch(rng, 8192, 16384)
            if sum(rows) * (2 * Hq + 4 * Hkv) <= 8192 * (2 * 32 + 4 * 8):
                return {"op": op, "Hq": Hq, "Hkv": Hkv, **c, "rotate": rng.random() < 0.8}
    most = max(work(c)["flops"] for c in listed())
    while True:
        c, rows, keys = _draw_batch(rng, 8192, 131072)
        c = {"op": op, "Hq": Hq, "Hkv": Hkv, **c}
        if work(c)["flops"] <= most and c["B"] * max(rows) * keys * Hq <= 8192 * 8192 * 32:
            return c


def work(case):
    if case["op"] == "table":
        M = case["rows"]
        axes = 1 + (case["h"] > 0) + (case["w"] > 0)
        return {"bytes": M * (4 * axes + D // 2 * 8), "flops": 0}
    rows, ctx = lengths(case)
    M, B, Hq, Hkv = sum(rows), case["B"], case["Hq"], case["Hkv"]
    pages = sum((m + n + PAGE - 1) // PAGE for m, n in zip(rows, ctx))
    index = 4 * (2 * B + 1)
    if case["op"] == "append":
        heads = 2 * Hkv + (Hq if case["rotate"] else 0)
        # the table entries of the pages that get rows
        touched = sum((n + m - 1) // PAGE - n // PAGE + 1 for m, n in zip(rows, ctx))
        return {"bytes": 2 * M * heads * D * 2 + (M * D // 2 * 8 if case["rotate"] else 0) + index + 4 * touched,
                "flops": 3 * M * (Hq + Hkv) * D if case["rotate"] else 0}
    pairs = sum(m * n + m * (m + 1) // 2 for m, n in zip(rows, ctx))
    keys = sum(m + n for m, n in zip(rows, ctx))
    return {"bytes": 2 * M * Hq * D * 2 + 2 * keys * Hkv * D * 2 + index + 4 * pages, "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _batch(case, seed, g, extra):
    """Ragged batch over a paged cache whose pages lie in a random order among `extra` others."""
    rows, ctx = lengths(case)
    need = [(m + n + PAGE - 1) // PAGE for m, n in zip(rows, ctx)]
    num_pages, max_pages = sum(need) + extra, max(need)
    perm = np.random.RandomState(seed % (1 << 31)).permutation(num_pages).astype(np.int32)
    table = np.zeros((case["B"], max_pages), np.int32)
    used = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[used:used + n]
        used += n
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    Hkv = case["Hkv"]
    return {"case": case, "M": int(cu[-1]), "max_rows": max(rows), "Hq": case["Hq"], "Hkv": Hkv,
            "cu": torch.from_numpy(cu).cuda(), "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
            "table": torch.from_numpy(table).cuda(),
            "kpool": _normal(g, (Hkv, num_pages, PAGE, D)), "vpool": _normal(g, (Hkv, num_pages, PAGE, D))}


def _positions(case, seed):
    """Positions of text, then of a grid of patches whose axes advance separately, then of text."""
    r = random.Random(seed)
    axes = 1 + (case["h"] > 0) + (case["w"] > 0)
    M = case["rows"]
    lead = r.randint(0, max(0, M // 4))
    width, height = r.randint(5, 40), r.randint(5, 40)
    base = r.randint(0, 30000)
    i = torch.arange(M, device="cuda")
    j = (i - lead).clamp(min=0)
    grid = torch.stack([j // (width * height), j // width % height, j % width])[:axes] + base + lead
    return torch.where(i[None, :] < lead, (base + i)[None, :], grid).to(torch.int32).contiguous()


def prepare(case, seed):
    if case["op"] == "table":
        sections = [s for s in (case["t"], case["h"], case["w"]) if s > 0]
        return {"case": case, "op": "table", "pos": _positions(case, seed), "sections": sections}
    g = _gen(seed)
    s = _batch(case, seed, g, 5)
    s["op"] = case["op"]
    M, hq, hk = s["M"], s["Hq"] * D, s["Hkv"] * D
    if case["op"] == "attention":
        # queries as a norm and a trained scale leave them: logits of a few units
        s["q"] = _normal(g, (M, hq), 2.0)
        return s
    s["qkv"] = _normal(g, (M, hq + 2 * hk))      # the fused projection's rows
    if case["rotate"]:
        s["qrot"] = torch.empty((M, hq), dtype=torch.bfloat16, device="cuda")
        pos = _row_positions(s)[1].double()
        ang = pos[:, None] * torch.tensor([THETA ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64,
                                          device="cuda")
        s["cs"] = torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()
    return s


def _row_positions(s):
    """(sequence, position) of each packed row."""
    r = torch.arange(s["M"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], r, right=True) - 1
    return b, s["ctx"][b] + r - s["cu"][b]


# --------------------------------------------------------------------------- one pass
def _axis_of(sections, interleaved):
    """Axis of each frequency: consecutive sections, or every third one up to the section's length."""
    n, half = len(sections), D // 2
    i = torch.arange(half, device="cuda")
    if interleaved:
        length = torch.tensor([half] + [n * s for s in sections[1:]], device="cuda")
        a = i % n
        return torch.where(i < length[a], a, torch.zeros_like(a))
    ends = torch.tensor(sections, device="cuda").cumsum(0)
    return torch.searchsorted(ends, i, right=True)


def _plain_table(s):
    axis = _axis_of(s["sections"], s["case"]["interleaved"])
    inv = THETA ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    ang = s["pos"][axis].double().t() * inv
    return torch.stack([ang.cos(), ang.sin()], dim=-1).float()


def _rotate(x, heads, cs):
    x = x.float().view(x.shape[0], heads, 2, D // 2)
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[:, :, 0], x[:, :, 1]
    return torch.stack([a * c - b * sn, b * c + a * sn], dim=2).reshape(x.shape[0], heads, D).to(torch.bfloat16)


def _plain_append(s):
    M, Hq, Hkv = s["M"], s["Hq"], s["Hkv"]
    q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], dim=1)
    b, p = _row_positions(s)
    page = s["table"][b, p // PAGE].long()
    if s["case"]["rotate"]:
        s["qrot"].copy_(_rotate(q, Hq, s["cs"]).view(M, Hq * D))
        k = _rotate(k, Hkv, s["cs"])
    s["kpool"][:, page, (p % PAGE).long()] = k.reshape(M, Hkv, D).transpose(0, 1)
    s["vpool"][:, page, (p % PAGE).long()] = v.reshape(M, Hkv, D).transpose(0, 1)


def _plain_attention(s):
    Hq, Hkv, B = s["Hq"], s["Hkv"], s["case"]["B"]
    G, R, L = Hq // Hkv, s["max_rows"], s["table"].shape[1] * PAGE
    k = s["kpool"][:, s["table"].long()].view(Hkv, B, L, D).float()
    v = s["vpool"][:, s["table"].long()].view(Hkv, B, L, D).float()
    j = torch.arange(R, device="cuda")
    row = (s["cu"][:-1, None] + j).clamp(max=s["M"] - 1)                        # [B, R], padded
    q = s["q"].view(s["M"], Hkv, G, D)[row].permute(2, 0, 3, 1, 4).float()       # [Hkv, B, G, R, D]
    x = torch.matmul(q.reshape(Hkv, B, G * R, D), k.transpose(2, 3)).view(Hkv, B, G, R, L)
    hidden = torch.arange(L, device="cuda") > (s["ctx"][:, None] + j)[..., None]  # [B, R, L]
    x.mul_(1.0 / math.sqrt(D)).masked_fill_(hidden[None, :, None], float("-inf"))
    x.sub_(x.amax(dim=-1, keepdim=True)).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(Hkv, B, G * R, L), v).view(Hkv, B, G, R, D).div_(total)
    b, p = _row_positions(s)
    o = o.permute(1, 3, 0, 2, 4)[b, (p - s["ctx"][b]).long()]                    # [M, Hkv, G, D]
    return o.reshape(s["M"], Hq * D).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        global _ws
        from speculative_decoding_verify_05_gb300 import binding as S
        if s["op"] == "table":
            return S.spec_rope_table_axes(s["pos"], s["sections"], D, THETA, interleaved=s["case"]["interleaved"])
        hq, hk = s["Hq"] * D, s["Hkv"] * D
        if s["op"] == "append":
            x, turn = s["qkv"], s["case"]["rotate"]
            S.spec_kv_append_paged(x[:, hq:hq + hk], x[:, hq + hk:], s["cu"], s["ctx"], s["kpool"], s["vpool"],
                                   s["table"], cs=s["cs"] if turn else None, Q=x[:, :hq] if turn else None,
                                   Qrot=s["qrot"] if turn else None)
        else:
            if _ws is None:
                _ws = S.Workspace("cuda")
            return S.spec_chunk_attention_paged(s["q"], s["cu"], s["ctx"], s["kpool"], s["vpool"], s["table"], ws=_ws)
    elif s["op"] == "table":
        return _plain_table(s)
    elif s["op"] == "append":
        _plain_append(s)
    else:
        return _plain_attention(s)
    out = {"k": s["kpool"], "v": s["vpool"]}
    if s["case"]["rotate"]:
        out["q"] = s["qrot"]
    return out


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "table":
        pos = s["pos"].cpu().numpy().astype(np.float64)
        out = np.empty((case["rows"], D // 2, 2))
        sections, n = s["sections"], len(s["sections"])
        for i in range(D // 2):
            axis = 0
            if case["interleaved"]:
                if i < n * sections[i % n]:
                    axis = i % n
            else:
                while i >= sum(sections[:axis + 1]):
                    axis += 1
            ang = pos[axis] * THETA ** (-2.0 * i / D)
            out[:, i, 0], out[:, i, 1] = np.cos(ang), np.sin(ang)
        return out
    rows, ctx = lengths(case)
    table = s["table"].cpu().numpy()
    Hq, Hkv = case["Hq"], case["Hkv"]
    G, first = Hq // Hkv, 0
    if case["op"] == "append":
        kp, vp = s["kpool"].double(), s["vpool"].double()
        x = s["qkv"].double().view(s["M"], Hq + 2 * Hkv, D)
        if case["rotate"]:
            w = torch.complex(s["cs"][..., 0].double(), s["cs"][..., 1].double())[:, None]
            z = torch.complex(x[:, :Hq + Hkv, :D // 2], x[:, :Hq + Hkv, D // 2:]) * w
            x[:, :Hq + Hkv] = torch.cat([z.real, z.imag], dim=-1)
        for b in range(case["B"]):
            for t in range(ctx[b] // PAGE, (ctx[b] + rows[b] - 1) // PAGE + 1):
                lo, hi = max(ctx[b], t * PAGE), min(ctx[b] + rows[b], (t + 1) * PAGE)
                src = x[first + lo - ctx[b]:first + hi - ctx[b]].transpose(0, 1)
                kp[:, table[b, t], lo - t * PAGE:hi - t * PAGE] = src[Hq:Hq + Hkv]
                vp[:, table[b, t], lo - t * PAGE:hi - t * PAGE] = src[Hq + Hkv:]
            first += rows[b]
        out = {"k": kp, "v": vp}
        if case["rotate"]:
            out["q"] = x[:, :Hq].reshape(s["M"], Hq * D)
        return out
    if work(case)["flops"] > 1.3e12:      # (64-bit products run at about a teraflop per second)
        return None
    out = torch.empty((s["M"], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n = ctx[b] + rows[b]
        pages = torch.from_numpy(table[b, :(n + PAGE - 1) // PAGE]).long().cuda()
        for h in range(Hkv):
            k = s["kpool"][h, pages].reshape(-1, D)[:n].double()
            v = s["vpool"][h, pages].reshape(-1, D)[:n].double()
            for j0 in range(0, rows[b], 1024):      # a block of rows at a time, over the keys it can see
                j1 = min(rows[b], j0 + 1024)
                m = ctx[b] + j1
                q = s["q"].view(s["M"], Hq, D)[first + j0:first + j1, h * G:(h + 1) * G].double()
                x = torch.einsum("jgd,kd->jgk", q, k[:m]) / math.sqrt(D)
                late = torch.arange(m, device="cuda")[None, :] > torch.arange(ctx[b] + j0, m, device="cuda")[:, None]
                x.masked_fill_(late[:, None], float("-inf"))
                out[first + j0:first + j1, h * G:(h + 1) * G] = torch.einsum("jgk,kd->jgd", torch.softmax(x, -1), v[:m])
        first += rows[b]
    return out.reshape(s["M"], Hq * D)
