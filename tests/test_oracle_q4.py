"""CPU pins of the oracle of the cache in 4 bits: values worked out by hand, borders, pages entry by entry, round trips."""
import numpy as np
import pytest

from oracle import ops, prompt, q4


def test_scales():
    assert q4.SCALES[0] == 2.0 ** -20 and q4.SCALES[-1] == 3840.0 and np.all(np.diff(q4.SCALES) > 0)
    assert q4.scale_of(20 * 8) == 1.0 and q4.scale_of(20 * 8 + 3) == 1.375 and q4.scale_of(19 * 8 + 7) == 0.9375
    assert np.array_equal(q4.scale_codes(q4.SCALES), np.arange(256))


@pytest.mark.parametrize("t,code", [
    (1.0625, 160), (1.1875, 162), (1.0626, 161), (1.0624, 160), (1.9375, 168), (0.96875, 160), (0.0, 0), (1e-9, 0),
    (2.0 ** -20 * 1.0625, 0), (3840.0, 255), (5000.0, 255), (np.inf, 255),
])
def test_scale_rounds_to_the_nearest_halves_to_even(t, code):
    assert q4.scale_codes(t) == code


def test_quantise_by_hand():
    x = np.zeros(128)
    x[:5] = [7.0, -3.5, 0.5, 1.5, -0.51]        # scale 1: halves to even
    x[32:35] = [14.4, -14.4, 1.0]               # 14.4 / 7 = 2.057 -> scale 2
    x[64:67] = [np.inf, -np.inf, 1e9]           # saturates
    x[96:99] = [np.nan, 7e-9, -7.0 * 2.0 ** -20]
    n, c = q4.quantise(x)
    assert c.tolist() == [160, 168, 255, 0]
    assert n[:5].tolist() == [7, -4, 0, 2, -1] and n[32:35].tolist() == [7, -7, 0]
    assert n[64:67].tolist() == [7, -7, 7] and n[96:99].tolist() == [0, 0, -7]
    assert abs(n).max() <= 7


def test_error_is_half_a_scale():
    x = np.random.default_rng(0).standard_normal((200, 128)) * np.exp2(np.random.default_rng(1).integers(-12, 8, (200, 1)))
    n, c = q4.quantise(x)
    s = np.repeat(q4.scale_of(c), 32, axis=-1)
    # the largest of a group is at most 7 (1 + 1/17) scales (a scale is off by half of its 1/8 .. 1/15 step at most)
    assert np.all(abs(q4.dequantise(n, c) - x) <= 0.5 * s * (1 + 1e-12)) and np.all(abs(x) <= 7.5 * s)


def test_values_of_the_cache_are_bf16():
    n = np.tile(np.arange(-7, 9), 8)
    for c in range(256):
        v = q4.dequantise(n, np.full(4, c)).astype(np.float32)
        assert np.all((v.view(np.uint32) & 0xFFFF) == 0)


def test_page_bytes_by_hand():
    """Key 37: dims 32 .. 39 are its second plane's first word; value 37 is entry 5 of a dim's first word of plane 1."""
    page = np.zeros(8704, np.uint8)
    n = np.zeros(128, int)
    n[32:40] = [-7, -6, -5, -4, 1, 2, 3, 7]
    q4.put(page, 37, n, [1, 2, 3, 4], True)
    word = int.from_bytes(page[2048 + 37 * 16:2048 + 37 * 16 + 4].tobytes(), "little")
    assert [(word >> 4 * i) & 15 for i in range(8)] == [1, 3, 9, 11, 2, 4, 10, 15]
    assert page[8192 + 148:8192 + 152].tolist() == [1, 2, 3, 4]
    page = np.full(8704, 0xFF, np.uint8)
    q4.put(page, 37, n, [1, 2, 3, 4], False)
    for d, e in ((32, -7), (39, 7), (0, 0)):
        word = int.from_bytes(page[2048 + d * 16:2048 + d * 16 + 4].tobytes(), "little")
        assert word == 0xFFFFFFFF & ~(15 << 24) | (e + 8) << 24           # entry 5: nibble 6
    assert [int(page[8192 + 128 * g + 37]) for g in range(4)] == [1, 2, 3, 4]


@pytest.mark.parametrize("keys", [True, False])
def test_pages_round_trip(keys):
    rng = np.random.default_rng(3)
    n, c = rng.integers(-7, 8, (128, 128)), rng.integers(0, 256, (128, 4))
    page = rng.integers(0, 256, 8704).astype(np.uint8)
    for k in rng.permutation(128):
        q4.put(page, k, n[k], c[k], keys)
    assert np.array_equal(q4.unpack(page, keys), q4.dequantise(n, c))


def test_append_and_read_are_mirrors_and_touch_nothing_else():
    rng = np.random.default_rng(4)
    rows, ctx, Hkv = [3, 0, 140], [126, 50, 5], 2
    cu = np.concatenate([[0], np.cumsum(rows)])
    table = np.array([[4, 1], [0, 0], [3, 2]])
    for keys in (True, False):
        pool = rng.integers(0, 256, (Hkv, 6, 8704)).astype(np.uint8)
        before = q4.unpack(pool, keys)
        n, c = rng.integers(-7, 8, (143, Hkv, 128)), rng.integers(0, 256, (143, Hkv, 4))
        after = q4.append(n, c, cu, ctx, pool, table, keys)
        assert np.array_equal(q4.read(after, cu, ctx, table, keys, 143), q4.dequantise(n, c))
        ref = prompt.kv_append(q4.dequantise(n, c), q4.dequantise(n, c), cu, ctx, before, before, table)[0]
        assert np.array_equal(q4.unpack(after, keys), ref)


def test_norm_is_the_rows_norm():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((6, 3, 128)), rng.standard_normal(128)
    assert np.allclose(q4.norm(x, w, 1e-6), ops.rmsnorm(x.reshape(18, 128), w, 1e-6).reshape(6, 3, 128), rtol=0, atol=1e-12)
