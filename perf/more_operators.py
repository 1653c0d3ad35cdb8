"""Cases of the paged cache held in 4 bits: the norms of queries and keys with their rotation
(spec_qk_norm_rope), the append that quantises a chunk's keys and values (spec_kv_append_paged_q4), the
read of cached keys and values (spec_kv_read_paged_q4) and the attention of a chunk's rows over
that cache (spec_chunk_attention_paged_q4).

A value in the cache is a whole number n of -7 .. 7 times the scale of its 32 neighbouring dims of one key, an 8-bit
float of 5 exponent and 3 mantissa bits without a sign: byte c stands for (1 + (c & 7) / 8) 2^((c >> 3) - 20).  A page
holds 128 keys of one kv head in 8704 bytes: 4 planes of 128 rows of 16 bytes, then 512 scales.
  keys    plane q, row k: dims 32 q .. 32 q + 31 of key k;  scale of dims 32 g .. of key k at 4 k + g
  values  plane q, row d: keys 32 q .. 32 q + 31 of dim d;  scale of dims 32 g .. of key k at 128 g + k
A row's 16 bytes are 4 words of 8 entries: n + 8 of entries 0, 2, 4, 6, 1, 3, 5, 7 from the low bits up.

Row counts and context lengths of a batch follow from the case alone (`lengths`).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 128      # keys per cache page
D = 128         # head size of the cache
PAGE_BYTES = 8704
GROUP = 32      # dims that share a scale
THETA = 1e6
EPS = 1e-6
TOP = 3840.0    # the largest scale
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]     # entry of each nibble of a word

_ws = None      # the program's one workspace (own only)


# --------------------------------------------------------------------------- cases
def _attn(name, Hq, Hkv, B, rows, ctx, ones=0, lens=1):
    return {"name": name, "op": "attention", "Hq": Hq, "Hkv": Hkv, "B": B, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ones": ones, "lens": lens}


def _append(name, Hq, Hkv, B, rows, ctx, ones=0, lens=1, norm=True, rotate=True):
    return {"name": name, "op": "append", "Hq": Hq, "Hkv": Hkv, "B": B, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "ones": ones, "lens": lens, "norm": norm, "rotate": rotate}


def _read(name, Hkv, B, rows, first, lens=1):
    return {"name": name, "op": "read", "Hq": Hkv, "Hkv": Hkv, "B": B, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": first[0], "ctx_hi": first[1], "ones": 0, "lens": lens}


def _norm(name, Hq, Hkv, rows, rotate=True):
    return {"name": name, "op": "norm", "Hq": Hq, "Hkv": Hkv, "rows": rows, "rotate": rotate}


def listed():
    return [
        # a few sequences one token at a time in short contexts: launch and latency
        _attn("attn 4 x 1 token", 32, 8, 4, (1, 1), (300, 1000)),
        # a verify round: 64 sequences with 1 to 10 drafts each, contexts up to 8192
        _attn("attn verify 64", 32, 8, 64, (2, 11), (128, 8192)),
        # a decode step over long contexts
        _attn("attn 16 x 1 at 30000", 32, 8, 16, (1, 1), (20000, 40000), lens=2),
        # a whole long prompt at once, nothing cached
        _attn("attn prompt 8192", 32, 8, 1, (8192, 8192), (0, 0)),
        # a serving step: most sequences decode, a few bring chunks of odd sizes
        _attn("attn mixed 24", 32, 8, 24, (97, 333), (0, 4096), ones=18, lens=2),
        # written and read back: single tokens, a whole prompt, a ragged serving step of rotated keys
        _append("append 8 x 1 token", 32, 8, 8, (1, 1), (100, 2000)),
        _append("append prompt 8192", 32, 8, 1, (8192, 8192), (0, 0)),
        _append("append rotated mixed 24", 16, 8, 24, (97, 999), (0, 4096), ones=12, lens=4, norm=False, rotate=False),
        # cached keys and values read back: one sequence's short prefix, the contexts of a whole batch
        _read("read 77 keys", 8, 1, (77, 77), (301, 301)),
        _read("read 32 contexts", 8, 32, (500, 4000), (0, 100), lens=3),
        # queries and keys of a verify round of few rows, and of a prompt's chunk
        _norm("norm 9 rows", 32, 8, 9),
        _norm("norm 8192 rows", 32, 8, 8192),
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
        if sum(rows) <= 16384 and B * keys <= 300000:
            return c, rows, keys


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "attention", "append", "append", "read", "norm"])
    Hq, Hkv = rng.choice(HEADS)
    cap = {o: max(work(c)["bytes"] for c in listed() if c["op"] == o) for o in ("append", "read", "norm")}
    while True:
        if op == "norm":
            c = {"op": op, "Hq": Hq, "Hkv": Hkv, "rows": _log_int(rng, 1, 16000), "rotate": rng.random() < 0.8}
        elif op == "read":
            c = {"op": op, "Hq": Hkv, "Hkv": Hkv, **_draw_batch(rng, 8192, 32768)[0]}
        elif op == "append":
            c = {"op": op, "Hq": Hq, "Hkv": Hkv, **_draw_batch(rng, 8192, 16384)[0], "norm": rng.random() < 0.6,
                 "rotate": rng.random() < 0.8}
        else:
            # half of the batches bring the few rows of decode steps and verify rounds
            c, rows, keys = _draw_batch(rng, 12 if rng.random() < 0.5 else 8192, 131072)
            c = {"op": op, "Hq": Hq, "Hkv": Hkv, **c}
            most = max(work(x)["flops"] for x in listed())
            if work(c)["flops"] <= most and c["B"] * max(rows) * keys * Hq <= 8192 * 8192 * 32:
                return c
            continue
        if work(c)["bytes"] <= cap[op]:
            return c


def work(case):
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "norm":
        M = case["rows"]
        return {"bytes": 2 * M * (Hq + Hkv) * D * 2 + (M * D // 2 * 8 if case["rotate"] else 0) + 4 * D,
                "flops": (4 + (3 if case["rotate"] else 0)) * M * (Hq + Hkv) * D}
    rows, ctx = lengths(case)
    M, B = sum(rows), case["B"]
    index = 4 * (2 * B + 1)
    key = PAGE_BYTES // PAGE * 2 * Hkv           # bytes of a key and its value in the cache, all heads
    # the table entries of the pages that hold the rows
    touched = sum((n + m - 1) // PAGE - n // PAGE + 1 for m, n in zip(rows, ctx))
    if case["op"] == "read":
        return {"bytes": M * key + 2 * M * Hkv * D * 2 + index + 4 * touched, "flops": 2 * M * Hkv * D}
    if case["op"] == "append":
        # the rows in, the turned queries out, 4-bit keys and values written and read once, the rows read back out
        turned = case["norm"] or case["rotate"]
        bytes_ = (2 * M * (2 * Hkv + (2 * Hq if turned else 0)) * D + (M * D // 2 * 8 if case["rotate"] else 0)
                  + 2 * M * key + 2 * M * Hkv * D * 2 + index + 4 * touched)
        per = (4 if case["norm"] else 0) + (3 if case["rotate"] else 0)
        return {"bytes": bytes_, "flops": per * M * (Hq + Hkv) * D + 5 * M * 2 * Hkv * D}
    pairs = sum(m * n + m * (m + 1) // 2 for m, n in zip(rows, ctx))
    keys = sum(m + n for m, n in zip(rows, ctx))
    pages = sum((m + n + PAGE - 1) // PAGE for m, n in zip(rows, ctx))
    return {"bytes": 2 * M * Hq * D * 2 + keys * key + index + 4 * pages, "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------- the cache's format
def _seven(x):
    """(By a plain number a GPU multiplies with its reciprocal, which is off where the quotient lies on a border.)"""
    return torch.full((1,), 7.0, dtype=x.dtype, device=x.device)


def _quantise(x):
    """Whole numbers (float) and scales of fp32 values [.., D]: the nearest of 8 scales per power of two to a seventh of
    the group's largest magnitude, and each value over its scale to the nearest, halves to even."""
    g = x.reshape(*x.shape[:-1], D // GROUP, GROUP)
    t = (g.abs().amax(dim=-1) / _seven(g)).clamp(min=2.0 ** -20, max=TOP)
    i = t.view(torch.int32)
    s = ((i + 0x7FFFF + ((i >> 20) & 1)) & -0x100000).view(torch.float32)
    n = torch.round(g / s[..., None]).clamp_(-7, 7)
    return n.reshape(x.shape), s


def _codes(s):
    return (s.contiguous().view(torch.int32) >> 20) - 107 * 8


def _scales(c):
    return ((c.int() + 107 * 8) << 20).view(torch.float32)


def _pack(n):
    """[.., 32] whole numbers -> [.., 16] bytes."""
    u = (n + 8).to(torch.uint8).reshape(*n.shape[:-1], 4, 8)[..., ORDER].reshape(*n.shape[:-1], 16, 2)
    return u[..., 0] | (u[..., 1] << 4)


def _unpack(p):
    """[.., 16] bytes -> [.., 32] whole numbers (float)."""
    u = torch.stack([p & 15, p >> 4], dim=-1).reshape(*p.shape[:-1], 4, 8)
    out = torch.empty_like(u)
    out[..., ORDER] = u
    return (out.reshape(*p.shape[:-1], 32).float() - 8.0)


def _pool_of_keys(k):
    """[Hkv, pages, PAGE, D] fp32 -> the pages' bytes."""
    n, s = _quantise(k)
    data = _pack(n.view(*k.shape[:-1], 4, 32)).transpose(2, 3)                       # plane, key, 16
    return torch.cat([data.reshape(*k.shape[:2], -1), _codes(s).to(torch.uint8).reshape(*k.shape[:2], -1)], dim=-1)


def _pool_of_values(v):
    n, s = _quantise(v)
    data = _pack(n.transpose(2, 3).reshape(*v.shape[:2], D, 4, 32)).transpose(2, 3)   # plane, dim, 16
    codes = _codes(s.transpose(2, 3)).to(torch.uint8)
    return torch.cat([data.reshape(*v.shape[:2], -1), codes.reshape(*v.shape[:2], -1)], dim=-1)


def _keys_of(pages):
    """Bytes [.., PAGE_BYTES] of pages of keys -> [.., PAGE, D] fp32."""
    lead = pages.shape[:-1]
    n = _unpack(pages[..., :8192].reshape(*lead, 4, PAGE, 16)).transpose(-3, -2)      # key, plane, 32
    s = _scales(pages[..., 8192:].reshape(*lead, PAGE, 4))
    return (n * s[..., None]).reshape(*lead, PAGE, D)


def _values_of(pages):
    lead = pages.shape[:-1]
    n = _unpack(pages[..., :8192].reshape(*lead, 4, D, 16)).transpose(-3, -2).reshape(*lead, 4, GROUP, PAGE)
    s = _scales(pages[..., 8192:].reshape(*lead, 4, 1, PAGE))
    return (n * s).reshape(*lead, D, PAGE).transpose(-2, -1)


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _spread():
    """Keys have a few dims that are larger than the rest."""
    d = torch.arange(D, device="cuda")
    return torch.where(d % 37 == 5, 4.0, 1.0)


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
    s = {"case": case, "op": case["op"], "M": int(cu[-1]), "max_rows": max(rows), "Hq": case["Hq"], "Hkv": Hkv,
         "cu": torch.from_numpy(cu).cuda(), "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
         "table": torch.from_numpy(table).cuda()}
    s["kpool"] = torch.empty((Hkv, num_pages, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    s["vpool"] = torch.empty_like(s["kpool"])
    for h in range(Hkv):
        s["kpool"][h] = _pool_of_keys(_normal(g, (1, num_pages, PAGE, D), 1.0, torch.float32) * _spread())[0]
        s["vpool"][h] = _pool_of_values(_normal(g, (1, num_pages, PAGE, D), 0.5, torch.float32))[0]
    return s


def _turns(pos):
    ang = pos[:, None] * torch.tensor([THETA ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64,
                                      device="cuda")
    return torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        M, Hq, Hkv = case["rows"], case["Hq"], case["Hkv"]
        s = {"case": case, "op": "norm", "M": M, "Hq": Hq, "Hkv": Hkv}
        pos = torch.arange(M, device="cuda") + random.Random(seed).randint(0, 30000)
    else:
        s = _batch(case, seed, g, 5)
        M, Hq, Hkv = s["M"], s["Hq"], s["Hkv"]
        pos = _row_positions(s)[1]
    if case["op"] == "attention":
        # queries as a norm and a trained scale leave them: logits of a few units
        s["q"] = _normal(g, (M, Hq * D), 1.5)
    elif case["op"] != "read":
        s["qkv"] = _normal(g, (M, (Hq + 2 * Hkv) * D))      # the fused projection's rows
        s["wq"] = (1.0 + _normal(g, (D,), 0.2, torch.float32)).to(torch.bfloat16)
        s["wk"] = (1.0 + _normal(g, (D,), 0.2, torch.float32)).to(torch.bfloat16)
        s["cs"] = _turns(pos.double()) if case["rotate"] else None
        s["qout"] = torch.empty((M, Hq * D), dtype=torch.bfloat16, device="cuda")
        s["kout"] = torch.empty((M, Hkv * D), dtype=torch.bfloat16, device="cuda")
    return s


def _row_positions(s):
    """(sequence, position) of each packed row."""
    r = torch.arange(s["M"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], r, right=True) - 1
    return b, s["ctx"][b] + r - s["cu"][b]


# --------------------------------------------------------------------------- one pass
def _sum_of_squares(x):
    """Over the last axis of 128, neighbours first: the order is part of the definition, as what is stored in 4 bits
    hangs on the last bit."""
    x = x * x
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0::2] + x[..., 1::2]


def _turned(x, heads, w, cs):
    """Rows of `heads` heads normed (w not None) and rotated (cs not None), [M, heads, D] fp32."""
    x = x.float().reshape(x.shape[0], heads, D)
    if w is not None:
        x = x * (1.0 / torch.sqrt(_sum_of_squares(x) * (1.0 / D) + EPS)) * w.float()
    if cs is not None:
        c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
        a, b = x[..., :D // 2], x[..., D // 2:]
        x = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    return x


def _plain_norm(s):
    q, k, _ = s["qkv"].split([s["Hq"] * D, s["Hkv"] * D, s["Hkv"] * D], dim=1)
    s["qout"].copy_(_turned(q, s["Hq"], s["wq"], s["cs"]).reshape(s["M"], -1))
    s["kout"].copy_(_turned(k, s["Hkv"], s["wk"], s["cs"]).reshape(s["M"], -1))
    return {"q": s["qout"], "k": s["kout"]}


def _plain_read(s):
    b, p = _row_positions(s)
    page, slot = s["table"][b, p // PAGE].long(), (p % PAGE).long()
    Hkv, M = s["Hkv"], s["M"]
    h = torch.arange(Hkv, device="cuda")[:, None]
    plane = torch.arange(4, device="cuda")
    # keys: 4 planes of 16 bytes
    kd = s["kpool"][:, :, :8192].view(Hkv, -1, 4, PAGE, 16)[h, page, :, slot]                  # [Hkv, M, 4, 16]
    ks = _scales(s["kpool"][:, :, 8192:].view(Hkv, -1, PAGE, 4)[h, page, slot])
    k = (_unpack(kd) * ks[..., None]).view(Hkv, M, D)
    # values: the nibble of each dim's word that belongs to the key
    byte, shift = _place(slot)
    vd = s["vpool"][:, :, :8192].view(Hkv, -1, 4, D, 16)[h, page, slot // 32, :, byte]         # [Hkv, M, D]
    vs = _scales(s["vpool"][:, :, 8192:].view(Hkv, -1, 4, PAGE)[h[..., None], page[:, None], plane, slot[:, None]])
    v = (((vd >> shift[:, None]) & 15).float() - 8.0).view(Hkv, M, 4, GROUP) * vs[..., None]
    turn = lambda x: x.reshape(Hkv, M, D).transpose(0, 1).reshape(M, Hkv * D).to(torch.bfloat16)  # noqa: E731
    return {"k": turn(k), "v": turn(v)}


def _place(slot):
    """Byte of a row's 16 and shift of a key's entry (key `slot` of its page)."""
    nibble = torch.tensor([ORDER.index(e) for e in range(8)], device="cuda")[slot % 8]
    return slot % 32 // 8 * 4 + nibble // 2, (nibble % 2 * 4).to(torch.uint8)


def _plain_append(s):
    M, Hq, Hkv = s["M"], s["Hq"], s["Hkv"]
    norm, rotate = s["case"]["norm"], s["case"]["rotate"]
    q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], dim=1)
    b, p = _row_positions(s)
    page, slot = s["table"][b, p // PAGE].long(), (p % PAGE).long()
    h = torch.arange(Hkv, device="cuda")[:, None]
    if norm or rotate:
        s["qout"].copy_(_turned(q, Hq, s["wq"] if norm else None, s["cs"]).reshape(M, -1))
    k = _turned(k, Hkv, s["wk"] if norm else None, s["cs"]).transpose(0, 1).contiguous()
    v = v.float().reshape(M, Hkv, D).transpose(0, 1).contiguous()
    kn, ks = _quantise(k)
    vn, vs = _quantise(v)
    s["kpool"][:, :, :8192].view(Hkv, -1, 4, PAGE, 16)[h, page, :, slot] = _pack(kn.view(Hkv, M, 4, 32))
    s["kpool"][:, :, 8192:].view(Hkv, -1, PAGE, 4)[h, page, slot] = _codes(ks).to(torch.uint8)
    # a byte holds two keys of a dim: what changes in each is added (whole numbers, modulo 256)
    byte, shift = _place(slot)
    data = s["vpool"][:, :, :8192].view(Hkv, -1, 4, D, 16)
    old = (data[h, page, slot // 32, :, byte] >> shift[:, None]) & 15
    d = torch.arange(D, device="cuda")
    at = (h[..., None], page[:, None], (slot // 32)[:, None], d, byte[:, None])
    data.index_put_(at, ((vn + 8).to(torch.uint8) - old) << shift[:, None], accumulate=True)
    plane = torch.arange(4, device="cuda")
    s["vpool"][:, :, 8192:].view(Hkv, -1, 4, PAGE)[h[..., None], page[:, None], plane, slot[:, None]] = _codes(vs).to(
        torch.uint8)
    out = _plain_read(s)
    if norm or rotate:
        out["q"] = s["qout"]
    return out


def _plain_attention(s):
    Hq, Hkv, B = s["Hq"], s["Hkv"], s["case"]["B"]
    G, R, L = Hq // Hkv, s["max_rows"], s["table"].shape[1] * PAGE
    k = _keys_of(s["kpool"][:, s["table"].long()]).view(Hkv, B, L, D)
    v = _values_of(s["vpool"][:, s["table"].long()]).reshape(Hkv, B, L, D)
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
        if s["op"] == "attention":
            if _ws is None:
                _ws = S.Workspace("cuda")
            return S.spec_chunk_attention_paged_q4(s["q"], s["cu"], s["ctx"], s["kpool"], s["vpool"], s["table"],
                                                   max_rows=s["max_rows"], ws=_ws)
        cache = (s["cu"], s["ctx"], s["kpool"], s["vpool"], s["table"]) if s["op"] != "norm" else ()
        if s["op"] == "read":
            k, v = S.spec_kv_read_paged_q4(*cache, s["M"])
            return {"k": k, "v": v}
        hq, hk = s["Hq"] * D, s["Hkv"] * D
        q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:]
        if s["op"] == "norm":
            S.spec_qk_norm_rope(q, k, s["wq"], s["wk"], EPS, cs=s["cs"], Qout=s["qout"], Kout=s["kout"])
            return {"q": s["qout"], "k": s["kout"]}
        norm = s["case"]["norm"]
        turned = norm or s["case"]["rotate"]
        S.spec_kv_append_paged_q4(k, v, *cache, cs=s["cs"], Q=q if turned else None, Qrot=s["qout"] if turned else None,
                                  wq=s["wq"] if norm else None, wk=s["wk"] if norm else None, eps=EPS)
        k, v = S.spec_kv_read_paged_q4(*cache, s["M"])
        return {"k": k, "v": v, "q": s["qout"]} if turned else {"k": k, "v": v}
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "read":
        return _plain_read(s)
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


# --------------------------------------------------------------------------- 64 bits
def _exact_page(raw, keys):
    """One page's bytes (numpy) -> [PAGE, D] in 64 bits, entry by entry of the format."""
    words = raw[:8192].copy().view("<u4").reshape(4, 128, 4)
    n = np.empty((128, 128))                                   # [row, 32 plane + entry]
    for e in range(8):
        nib = (words >> np.uint32(4 * ORDER.index(e))) & np.uint32(15)
        for w in range(4):
            n[:, np.arange(4) * 32 + 8 * w + e] = nib[:, :, w].T.astype(np.float64) - 8.0
    c = raw[8192:].astype(np.int64)
    s = np.ldexp(1.0 + (c & 7) / 8.0, ((c >> 3) - 20).astype(np.int32))
    if keys:
        return n * np.repeat(s.reshape(128, 4), 32, axis=1)
    return n.T * np.repeat(s.reshape(4, 128).T, 32, axis=1)


def _exact_cache(s, h, b, n, keys):
    """The first n keys (or values) of sequence b, kv head h, on the GPU in 64 bits."""
    pages = s["table"][b, :(n + PAGE - 1) // PAGE].long()
    raw = s["kpool" if keys else "vpool"][h, pages]
    lut = torch.arange(16, device="cuda", dtype=torch.float64) - 8
    words = raw[:, :8192].contiguous().view(torch.int32).view(-1, 4, 128, 4)
    x = torch.empty((len(pages), 128, 4, 4, 8), dtype=torch.float64, device="cuda")   # page, row, plane, word, entry
    for i, e in enumerate(ORDER):
        x[..., e] = lut[((words >> (4 * i)) & 15).long()].permute(0, 2, 1, 3)
    c = raw[:, 8192:].long()
    sc = (1.0 + (c & 7).double() / 8.0) * torch.exp2((c >> 3).double() - 20.0)
    x = x.reshape(len(pages), 128, 128)
    if keys:
        x = x * sc.view(-1, 128, 4).repeat_interleave(32, dim=2)
    else:
        x = x.transpose(1, 2) * sc.view(-1, 4, 128).transpose(1, 2).repeat_interleave(32, dim=2)
    return x.reshape(-1, D)[:n]


def _exact_store(x):
    """What values [.., D] in 64 bits become in the cache."""
    g = x.reshape(*x.shape[:-1], 4, 32)
    t = (g.abs().amax(dim=-1) / _seven(g)).clamp(2.0 ** -20, TOP)
    e = torch.floor(torch.log2(t))
    e = torch.where(torch.exp2(e) > t, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= t, e + 1, e)
    s = torch.round(t / torch.exp2(e) * 8) / 8 * torch.exp2(e)
    return (torch.round(g / s[..., None]).clamp(-7, 7) * s[..., None]).reshape(x.shape)


def _exact_turned(x, w, cs):
    if w is not None:
        x = x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w.double()
    if cs is not None:
        t = torch.complex(cs[..., 0].double(), cs[..., 1].double())[:, None]
        z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * t
        x = torch.cat([z.real, z.imag], dim=-1)
    return x


def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits."""
    s = prepare(case, seed)
    M, Hq, Hkv = s["M"], s["Hq"], s["Hkv"]
    flat = lambda x: x.reshape(M, -1)  # noqa: E731
    if case["op"] in ("norm", "append"):
        x = s["qkv"].double().view(M, Hq + 2 * Hkv, D)
        norm = case["op"] == "norm" or case["norm"]
        q = _exact_turned(x[:, :Hq], s["wq"] if norm else None, s["cs"])
        k = _exact_turned(x[:, Hq:Hq + Hkv], s["wk"] if norm else None, s["cs"])
        if case["op"] == "norm":
            return {"q": flat(q), "k": flat(k)}
        out = {"k": flat(_exact_store(k)), "v": flat(_exact_store(x[:, Hq + Hkv:]))}
        if norm or case["rotate"]:
            out["q"] = flat(q)
        return out
    rows, ctx = lengths(case)
    first = 0
    if case["op"] == "read":
        out = {"k": torch.empty((M, Hkv, D), dtype=torch.float64, device="cuda")}
        out["v"] = torch.empty_like(out["k"])
        for b in range(case["B"]):
            for h in range(Hkv):
                for name in ("k", "v"):
                    x = _exact_cache(s, h, b, ctx[b] + rows[b], name == "k")
                    out[name][first:first + rows[b], h] = x[ctx[b]:]
            first += rows[b]
        # (one page entry by entry from its bytes, apart from the above)
        page = int(s["table"][0, ctx[0] // PAGE])
        n = min(rows[0], PAGE - ctx[0] % PAGE)
        for name in ("k", "v"):
            ref = _exact_page(s[name + "pool"][0, page].cpu().numpy(), name == "k")[ctx[0] % PAGE:][:n]
            out[name][:n, 0] = torch.from_numpy(ref).cuda()
        return {n: flat(x) for n, x in out.items()}
    if work(case)["flops"] > 1.3e12:      # (64-bit products run at about a teraflop per second)
        return None
    G = Hq // Hkv
    out = torch.empty((M, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n = ctx[b] + rows[b]
        for h in range(Hkv):
            k, v = _exact_cache(s, h, b, n, True), _exact_cache(s, h, b, n, False)
            for j0 in range(0, rows[b], 1024):      # a block of rows at a time, over the keys it can see
                j1 = min(rows[b], j0 + 1024)
                m = ctx[b] + j1
                q = s["q"].view(M, Hq, D)[first + j0:first + j1, h * G:(h + 1) * G].double()
                x = torch.einsum("jgd,kd->jgk", q, k[:m]) / math.sqrt(D)
                late = torch.arange(m, device="cuda")[None, :] > torch.arange(ctx[b] + j0, m, device="cuda")[:, None]
                x.masked_fill_(late[:, None], float("-inf"))
                out[first + j0:first + j1, h * G:(h + 1) * G] = torch.einsum("jgk,kd->jgd", torch.softmax(x, -1), v[:m])
        first += rows[b]
    return out.reshape(M, Hq * D)
