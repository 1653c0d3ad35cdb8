"""Prompt side of the paged cache in fp64: the rotation table of positions with several axes, the append
of a chunk's rotated keys and values, and the attention of a chunk over the pages (test
infrastructure only).

"How Speculative Decoding Works (and When It Doesn't)", "Prefill and Decode": the prompt's tokens are
processed together before the first token is generated.  The cache layout is the library's:
pools [Hkv, num_pages, 128, D], key p of sequence b in row p % 128 of page table[b, p // 128].
"""
import numpy as np

PAGE = 128


def frequency_axes(sections, half: int, interleaved: bool) -> np.ndarray:
    """Position axis of each of the `half` frequencies."""
    n = len(sections)
    if not interleaved:
        return np.repeat(np.arange(n), sections)
    axes = np.zeros(half, np.int64)
    for a in range(1, n):
        axes[a:max(a, n * sections[a]):n] = a
    return axes


def rope_table_axes(pos, sections, D: int, theta: float, interleaved: bool) -> np.ndarray:
    """cs [M, D/2, 2]: cos and sin of pos[axis(i)] theta^(-2 i / D); pos [axes, M]."""
    ax = frequency_axes(sections, D // 2, interleaved)
    inv = float(theta) ** (-2.0 * np.arange(D // 2) / D)
    ang = np.asarray(pos, np.float64)[ax].T * inv
    return np.stack([np.cos(ang), np.sin(ang)], axis=-1)


def rotate(x, cs):
    """Rotate-half of x [M, heads, D] with cs [M, D/2, 2]; also the sum of the magnitudes of the two
    products of each element (what an fp32 evaluation's error scales with)."""
    h = x.shape[-1] // 2
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., :h], x[..., h:]
    out = np.concatenate([a * c - b * s, b * c + a * s], axis=-1)
    mag = np.concatenate([abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)], axis=-1)
    return out, mag


def kv_append(Knew, Vnew, cu_rows, ctx_len, Kpool, Vpool, table):
    """The pools with the rows Knew / Vnew [M, Hkv, D] (already rotated) in their places."""
    Kp, Vp = np.array(Kpool), np.array(Vpool)
    for b in range(len(cu_rows) - 1):
        for r in range(int(cu_rows[b]), int(cu_rows[b + 1])):
            p = int(ctx_len[b]) + r - int(cu_rows[b])
            page = int(table[b, p // PAGE])
            Kp[:, page, p % PAGE] = Knew[r]
            Vp[:, page, p % PAGE] = Vnew[r]
    return Kp, Vp


def chunk_attention(Q, cu_rows, ctx_len, Kpool, Vpool, table, scale: float):
    """(O, mag) [M, Hq, D]: the attention outputs, and the same weights applied to |v|."""
    Q = np.asarray(Q, np.float64)
    M, Hq, D = Q.shape
    Hkv = Kpool.shape[0]
    G = Hq // Hkv
    O, mag = np.zeros((M, Hq, D)), np.zeros((M, Hq, D))
    for b in range(len(cu_rows) - 1):
        r0, r1, ctx = int(cu_rows[b]), int(cu_rows[b + 1]), int(ctx_len[b])
        n = ctx + r1 - r0
        if r1 == r0:
            continue
        pages = table[b, :(n + PAGE - 1) // PAGE]
        late = np.arange(n)[None, :] > (ctx + np.arange(r1 - r0))[:, None]
        for g in range(Hkv):
            k = np.asarray(Kpool[g, pages], np.float64).reshape(-1, D)[:n]
            v = np.asarray(Vpool[g, pages], np.float64).reshape(-1, D)[:n]
            for h in range(g * G, (g + 1) * G):
                s = np.where(late, -np.inf, Q[r0:r1, h] @ k.T * scale)
                w = np.exp(s - s.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                O[r0:r1, h] = w @ v
                mag[r0:r1, h] = w @ abs(v)
    return O, mag
