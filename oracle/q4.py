"""The paged cache in 4 bits and the norms of queries and keys, in fp64 (test infrastructure only).

A value is a whole number n of -7 .. 7 times the scale of its 32 neighbouring dims; byte c of a scale stands for
(1 + (c & 7) / 8) 2^((c >> 3) - 20).  Pages are written entry by entry from the format's description: 4 planes
of 128 rows of 16 bytes, then 512 scales; keys have a row per key (plane: 32 dims), values a row per dim (plane: 32
keys); a row's word of 4 bytes holds n + 8 of its entries 0, 2, 4, 6, 1, 3, 5, 7 from the low bits up.
"""
import numpy as np

PAGE, D, GROUP, PAGE_BYTES = 128, 128, 32, 8704
ORDER = (0, 2, 4, 6, 1, 3, 5, 7)
TOP = 3840.0


def scale_of(code) -> np.ndarray:
    c = np.asarray(code, np.int64)
    return (1.0 + (c & 7) / 8.0) * np.exp2((c >> 3) - 20.0)


SCALES = scale_of(np.arange(256))        # ascending


def scale_codes(t) -> np.ndarray:
    """The nearest scale to each t (clamped to the scales' range), halves to the even code."""
    t = np.clip(np.asarray(t, np.float64), SCALES[0], SCALES[-1])
    hi = np.clip(np.searchsorted(SCALES, t), 1, 255)
    lo = hi - 1
    below, above = t - SCALES[lo], SCALES[hi] - t
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantise(x):
    """(n [.., D] int, codes [.., D / 32] int) of x [.., D]; NaN becomes 0."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    mag = np.where(np.isnan(g), 0.0, abs(g))
    code = scale_codes(mag.max(axis=-1) / 7.0)
    with np.errstate(invalid="ignore"):
        n = np.clip(np.rint(np.where(np.isnan(g), 0.0, g) / scale_of(code)[..., None]), -7, 7)
    return n.astype(np.int64).reshape(x.shape), code


def dequantise(n, code) -> np.ndarray:
    g = np.asarray(n, np.float64).reshape(*n.shape[:-1], n.shape[-1] // GROUP, GROUP)
    return (g * scale_of(code)[..., None]).reshape(n.shape)


def _place(row: int, entry: int):
    """(byte of the page, shift) of entry `entry` (0 .. 127) of a row."""
    plane, e = divmod(entry, 32)
    nibble = ORDER.index(e % 8)
    return plane * 2048 + row * 16 + e // 8 * 4 + nibble // 2, nibble % 2 * 4


def put(page: np.ndarray, slot: int, n, code, keys: bool) -> None:
    """Writes key `slot`'s 128 whole numbers and 4 scale codes into a page (uint8 [PAGE_BYTES])."""
    for d in range(D):
        at, shift = _place(slot, d) if keys else _place(d, slot)
        page[at] = (int(page[at]) & ~(15 << shift)) | (int(n[d]) + 8) << shift
    for g in range(4):
        page[8192 + (4 * slot + g if keys else 128 * g + slot)] = code[g]


def unpack(page: np.ndarray, keys: bool) -> np.ndarray:
    """Values [PAGE, D] of pages [.., PAGE_BYTES] (any bytes)."""
    page = np.asarray(page, np.uint8)
    lead = page.shape[:-1]
    at = np.empty((128, 128), np.int64)
    shift = np.empty((128, 128), np.uint8)
    for r in range(128):
        for e in range(128):
            at[r, e], shift[r, e] = _place(r, e)
    n = ((page[..., at] >> shift) & 15).astype(np.float64) - 8.0           # [.., row, entry]
    s = scale_of(page[..., 8192:])
    if keys:
        return n * np.repeat(s.reshape(*lead, 128, 4), GROUP, axis=-1)
    return np.swapaxes(n, -1, -2) * np.repeat(np.swapaxes(s.reshape(*lead, 4, 128), -1, -2), GROUP, axis=-1)


def append(n, code, cu_rows, ctx_len, pool, table, keys: bool) -> np.ndarray:
    """The pool [Hkv, num_pages, PAGE_BYTES] with rows n [M, Hkv, D], code [M, Hkv, 4] in their places."""
    pool = np.array(pool)
    for b in range(len(cu_rows) - 1):
        for r in range(int(cu_rows[b]), int(cu_rows[b + 1])):
            p = int(ctx_len[b]) + r - int(cu_rows[b])
            for g in range(pool.shape[0]):
                put(pool[g, int(table[b, p // PAGE])], p % PAGE, n[r, g], code[r, g], keys)
    return pool


def read(pool, cu_rows, ctx_len, table, keys: bool, M: int) -> np.ndarray:
    """Rows [M, Hkv, D] that the append's cu_rows and ctx_len name (0 elsewhere)."""
    values = unpack(pool, keys)
    out = np.zeros((M, pool.shape[0], D))
    for b in range(len(cu_rows) - 1):
        for r in range(int(cu_rows[b]), int(cu_rows[b + 1])):
            p = int(ctx_len[b]) + r - int(cu_rows[b])
            out[r] = values[:, int(table[b, p // PAGE]), p % PAGE]
    return out


def norm(x, w, eps: float) -> np.ndarray:
    """RMSNorm over the last axis."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
