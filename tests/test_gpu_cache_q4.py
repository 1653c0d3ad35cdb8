"""GPU parity of the cache in 4 bits (append, read) and of the norms of queries and keys with the fp64 oracle."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, prompt as oprompt, q4

from gpu_util import bf16_dev, bits_of, dev, f64_of_bf16

pytestmark = pytest.mark.gpu
PAGE, D, BYTES = 128, 128, 8704
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24


class Cache:
    """Ragged batch over a paged cache whose pages hold random bytes."""

    def __init__(self, seed, rows, ctx, Hkv, Hq=0, pad=0, extra=2, spare=1, std=1.0):
        rng = np.random.default_rng(seed)
        self.rows, self.ctx = np.asarray(rows, np.int32), np.asarray(ctx, np.int32)
        self.B, self.Hq, self.Hkv = len(rows), Hq, Hkv
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.M = int(self.cu[-1])
        self.Mp = self.M + pad
        need = [(c + n + PAGE - 1) // PAGE if n else 0 for c, n in zip(ctx, rows)]
        self.num_pages = sum(need) + extra
        perm = rng.permutation(self.num_pages)
        self.table = np.full((self.B, max(max(need), 1) + spare), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.kp, self.vp = rng.integers(0, 256, (2, Hkv, self.num_pages, BYTES)).astype(np.uint8)
        width = (Hq + 2 * Hkv) * D
        self.qkv = synth.normal_bf16_bits(seed + 1, (self.Mp, width + 8), std)      # rows apart by more than they are wide
        self.qkv[self.M:] = 0x7FC0
        x = obf.decode(self.qkv[:self.M, :width]).reshape(self.M, Hq + 2 * Hkv, D)
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def dev(self):
        return dev(self.cu), dev(self.ctx), dev(self.kp), dev(self.vp), dev(self.table)

    def parts(self):
        x = bf16_dev(self.qkv)
        hq, hk = self.Hq * D, self.Hkv * D
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:hq + 2 * hk]

    def append(self, x, pool, keys):
        n, c = q4.quantise(x)
        return q4.append(n, c, self.cu, self.ctx, pool, self.table, keys)


BATCHES = [
    ([1], [0], 1), ([1, 1, 1, 1, 1], [7, 8, 127, 128, 255], 2), ([3, 0, 17, 9], [5, 400, 126, 0], 8), ([300], [0], 4),
    ([8, 16, 1], [8, 120, 131], 3), ([7], [121], 5), ([130, 2], [3, 63], 2), ([0, 0, 2, 0], [9, 1, 1, 3], 2),
]


@pytest.mark.parametrize("rows,ctx,Hkv", BATCHES)
def test_append_as_they_are(lib, rows, ctx, Hkv):
    """Keys and values without a norm or a rotation: the pools, to the byte, everything else in them untouched."""
    c = Cache(10, rows, ctx, Hkv, pad=3)
    cu, cx, kp, vp, table = c.dev()
    _, k, v = c.parts()
    assert lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table) is None
    lib.spec_device_status()
    assert np.array_equal(kp.cpu().numpy(), c.append(c.k, c.kp, True))
    assert np.array_equal(vp.cpu().numpy(), c.append(c.v, c.vp, False))


def test_append_many_sequences(lib):
    """More sequences than lanes (places are searched in steps of 32), some of them empty."""
    rng = np.random.default_rng(3)
    rows, ctx = rng.integers(0, 4, 150).tolist(), rng.integers(0, 200, 150).tolist()
    c = Cache(11, rows, ctx, 1)
    cu, cx, kp, vp, table = c.dev()
    _, k, v = c.parts()
    lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table)
    lib.spec_device_status()
    assert np.array_equal(kp.cpu().numpy(), c.append(c.k, c.kp, True))
    assert np.array_equal(vp.cpu().numpy(), c.append(c.v, c.vp, False))


def test_append_many_rows(lib):
    """Enough rows for the shape with small CTAs."""
    c = Cache(12, [900, 1, 1199], [77, 500, 0], 2)
    cu, cx, kp, vp, table = c.dev()
    _, k, v = c.parts()
    lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table)
    lib.spec_device_status()
    assert np.array_equal(kp.cpu().numpy(), c.append(c.k, c.kp, True))
    assert np.array_equal(vp.cpu().numpy(), c.append(c.v, c.vp, False))


def test_append_many_rows_and_heads(lib):
    """Enough of both for values in blocks of 32 keys: sequences that end inside a block, rows of other chunks beside them,
    infinities, NaN and values past the scales here and there."""
    c = Cache(14, [333, 40, 427], [77, 500, 5], 64)
    rng = np.random.default_rng(15)
    at = rng.integers(0, c.M, 200), rng.integers(0, 2 * 64 * D, 200)
    c.qkv[at] = rng.choice(np.array([0x7F80, 0xFF80, 0x7FC0, 0x46D2, 0xC6D3, 0x7F7F, 0x0001], np.uint16), 200)
    x = obf.decode(c.qkv[:, :2 * 64 * D]).reshape(c.M, 128, D)
    c.k, c.v = x[:, :64], x[:, 64:]
    cu, cx, kp, vp, table = c.dev()
    _, k, v = c.parts()
    lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table)
    lib.spec_device_status()
    assert np.array_equal(kp.cpu().numpy(), c.append(c.k, c.kp, True))
    assert np.array_equal(vp.cpu().numpy(), c.append(c.v, c.vp, False))


def test_append_every_bf16(lib):
    """Every bf16 bit pattern, infinities and NaN among them, and borders of the scales and of the whole numbers."""
    bits = np.random.default_rng(5).permutation(np.arange(65536).astype(np.uint16))
    # groups of one magnitude (ties of a seventh), and of halves of a power of two
    ties = np.tile(np.arange(0x3F80, 0x4080, dtype=np.uint16)[:, None], (1, 128))
    ties[:, 1::2] = synth.f32_to_bf16_bits((np.arange(64) / 8 - 4).astype(np.float32))[None]
    k = np.concatenate([bits.reshape(512, 128), ties])
    M = len(k)
    c = Cache(13, [M], [0], 1)
    c.qkv[:, :128], c.qkv[:, 128:256] = k, k[::-1]
    cu, cx, kp, vp, table = c.dev()
    _, kd, vd = c.parts()
    lib.spec_kv_append_paged_q4(kd, vd, cu, cx, kp, vp, table)
    lib.spec_device_status()
    x = obf.decode(k)[:, None]
    assert np.array_equal(kp.cpu().numpy(), c.append(x, c.kp, True))
    assert np.array_equal(vp.cpu().numpy(), c.append(x[::-1], c.vp, False))
    back = lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, M)[0]
    assert torch.isfinite(back.float()).all()


def turned(c, x, w, cs):
    """Oracle of a norm and a rotation (either may be None), and what fp32's roundings of it are relative to."""
    y = x if w is None else q4.norm(x, w, 1e-6)
    return (y, abs(y)) if cs is None else oprompt.rotate(y, cs)


# fp32's part of an error, relative to the terms: squares (1 half step) summed in 7 levels, the mean exact, eps, root and
# reciprocal (halving what came before: (1 + 7 + 1) / 2 + 2), two products, and with a rotation a product and a sum
F32 = (9 / 2 + 2 + 2 + 2) * HALF_F32


def table_of(c, positions=True):
    pos = np.concatenate([c.ctx[b] + np.arange(c.rows[b]) for b in range(c.B)]) if positions else np.arange(c.M)
    cs = np.zeros((c.Mp, 64, 2), np.float32)
    cs[:c.M] = oprompt.rope_table_axes(pos[None], [64], D, 1e6, False)
    return cs


def assert_stored(page_values, codes_of, y, mag):
    """What the cache stands for against y: the scale that a maximum within fp32's error of the exact one gives, and the
    nearest whole number to a value within it."""
    tol = F32 * (1 + 1e-3)
    g = lambda a: a.reshape(*a.shape[:-1], 4, 32)
    top, slack = g(abs(y)).max(-1), g(mag).max(-1) * tol
    lo, hi = (q4.scale_codes((top + e) / 7 * (1 + np.sign(e) * 2 * HALF_F32)) for e in (-slack, slack))
    assert np.all((codes_of >= lo) & (codes_of <= hi))
    s = q4.scale_of(codes_of)[..., None]
    assert np.all(abs(g(page_values) - g(y)) <= 0.5 * s * (1 + 4 * HALF_F32) + g(mag) * tol)


def codes(pool, c, keys):
    """Scale codes [M, Hkv, 4] of the batch's rows."""
    out = np.empty((c.M, c.Hkv, 4), np.int64)
    s = pool[:, :, 8192:].reshape(c.Hkv, c.num_pages, *((128, 4) if keys else (4, 128)))
    for b in range(c.B):
        for r in range(c.cu[b], c.cu[b + 1]):
            p = c.ctx[b] + r - c.cu[b]
            pg = s[:, c.table[b, p // PAGE]]
            out[r] = pg[:, p % PAGE] if keys else pg[:, :, p % PAGE]
    return out


@pytest.mark.parametrize("with_norm", [True, False])
@pytest.mark.parametrize("with_cs", [True, False])
@pytest.mark.parametrize("rows,ctx,Hq,Hkv", [
    ([1, 5, 0, 30], [0, 126, 3, 999], 32, 8), ([2], [8191], 5, 1), ([4, 3], [12, 1], 28, 4), ([1700], [60], 4, 2),
    ([3], [77], 7, 7), ([2, 2], [5, 40], 16, 1),
])
def test_append_normed_and_rotated(lib, rows, ctx, Hq, Hkv, with_cs, with_norm):
    c = Cache(20, rows, ctx, Hkv, Hq, pad=2, std=1.7)
    cu, cx, kp, vp, table = c.dev()
    q, k, v = c.parts()
    wq, wk = (synth.f32_to_bf16_bits((1 + 0.3 * np.random.default_rng(s).standard_normal(D)).astype(np.float32)) for s in (1, 2))
    cs = table_of(c)
    Qrot = torch.full((c.Mp, Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    turn = with_cs or with_norm
    out = lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table, cs=dev(cs) if with_cs else None, Q=q if turn else None,
                                      Qrot=Qrot if turn else None, wq=bf16_dev(wq) if with_norm else None,
                                      wk=bf16_dev(wk) if with_norm else None)
    lib.spec_device_status()
    assert np.array_equal(vp.cpu().numpy(), c.append(c.v, c.vp, False))
    w = (obf.decode(wq), obf.decode(wk)) if with_norm else (None, None)
    table64 = cs[:c.M].astype(np.float64) if with_cs else None
    yk, mk = turned(c, c.k, w[1], table64)
    got = kp.cpu().numpy()
    assert_stored(q4.read(got, c.cu, c.ctx, c.table, True, c.M), codes(got, c, True), yk, mk)
    if turn:
        assert out is Qrot
        yq, mq = turned(c, c.q, w[0], table64)
        qr = f64_of_bf16(Qrot)
        assert np.all(qr[c.M:] == 7.0), "padding rows written"
        err = abs(qr[:c.M].reshape(yq.shape) - yq)
        assert np.all(err <= HALF_BF16 * abs(yq) + (1 + HALF_BF16) * F32 * mq)
    # in place gives the same
    if turn:
        lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table, cs=dev(cs) if with_cs else None, Q=q,
                                    wq=bf16_dev(wq) if with_norm else None, wk=bf16_dev(wk) if with_norm else None)
        assert torch.equal(q[:c.M], Qrot[:c.M]) and np.array_equal(kp.cpu().numpy(), got)


def test_a_rows_bytes_do_not_depend_on_its_chunk(lib):
    """A prompt in one chunk, in chunks of odd sizes and token by token: the same pools, to the byte."""
    n, Hq, Hkv = 150, 8, 2
    c = Cache(30, [n], [0], Hkv, Hq)
    cu, cx, kp, vp, table = c.dev()
    q, k, v = c.parts()
    w = bf16_dev(synth.normal_bf16_bits(4, (D,), 1.0))
    cs = dev(table_of(c))
    q0 = q.clone()

    def run(sizes):
        kp2, vp2, qr = kp.clone(), vp.clone(), q0.clone()
        at = 0
        for m in sizes:
            i = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            x = torch.tensor([at], dtype=torch.int32, device="cuda")
            lib.spec_kv_append_paged_q4(k[at:at + m], v[at:at + m], i, x, kp2, vp2, table, cs=cs[at:at + m],
                                        Q=q0[at:at + m], Qrot=qr[at:at + m], wq=w, wk=w)
            at += m
        assert at == n
        return kp2, vp2, qr
    whole = run([n])
    for sizes in ([1] * n, [3, 64, 1, 82], [149, 1]):
        for x, y in zip(run(sizes), whole):
            assert torch.equal(x, y)
    # ... and the norm alone gives the queries of the append
    qn, _ = lib.spec_qk_norm_rope(q0, None, w, None, cs=cs, Qout=torch.empty_like(q0))
    assert torch.equal(qn, whole[2])


@pytest.mark.parametrize("rows,first,Hkv", BATCHES + [([5000], [130], 1), ([32, 31, 33], [96, 1, 31], 2)])
def test_read(lib, rows, first, Hkv):
    """Any bytes in the pools; rows of the outputs that no sequence has stay as they were."""
    c = Cache(40, rows, first, Hkv, pad=4)
    cu, cx, kp, vp, table = c.dev()
    outs = [torch.full((c.Mp, Hkv * D + 16), 7.0, dtype=torch.bfloat16, device="cuda")[:, :Hkv * D] for _ in range(2)]
    lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, c.Mp, Kout=outs[0], Vout=outs[1])
    lib.spec_device_status()
    for out, pool, keys in ((outs[0], c.kp, True), (outs[1], c.vp, False)):
        got = f64_of_bf16(out)
        assert np.all(got[c.M:] == 7.0)
        ref = q4.read(pool, c.cu, c.ctx, c.table, keys, c.M)
        assert np.array_equal(got[:c.M].reshape(ref.shape), ref)
    assert np.array_equal(kp.cpu().numpy(), c.kp) and np.array_equal(vp.cpu().numpy(), c.vp)
    K, V = lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, c.M)
    assert torch.equal(K, outs[0][:c.M]) and torch.equal(V, outs[1][:c.M])


def test_read_into_a_bf16_cache(lib):
    """What is read goes to the pages of a bf16 cache as it is."""
    c = Cache(41, [140, 3], [0, 0], 2)
    cu, cx, kp, vp, table = c.dev()
    K, V = lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, c.M)
    kb, vb = torch.zeros((2, 2, c.num_pages, PAGE, D), dtype=torch.bfloat16, device="cuda")
    lib.spec_kv_append_paged(K, V, cu, cx, kb, vb, table)
    lib.spec_device_status()
    values = q4.unpack(c.kp, True)
    for b, n in ((0, 140), (1, 3)):
        for t in range((n + PAGE - 1) // PAGE):
            m = min(PAGE, n - t * PAGE)
            got = f64_of_bf16(kb[:, c.table[b, t], :m])
            assert np.array_equal(got, values[:, c.table[b, t], :m])


@pytest.mark.parametrize("M,Hq,Hkv", [(1, 32, 8), (9, 5, 1), (300, 16, 8), (1600, 7, 3), (4, 0, 2), (4, 3, 0)])
@pytest.mark.parametrize("with_cs", [True, False])
def test_qk_norm_rope(lib, M, Hq, Hkv, with_cs):
    c = Cache(50, [M], [33], max(Hkv, 1), Hq, std=2.5)
    q, k, _ = c.parts()
    wq, wk = (synth.normal_bf16_bits(s, (D,), 1.0) for s in (6, 7))
    cs = table_of(c)
    Q, K = (q if Hq else None), (k if Hkv else None)
    Qo, Ko = (None if x is None else torch.empty_like(x.contiguous()) for x in (Q, K))
    lib.spec_qk_norm_rope(Q, K, bf16_dev(wq) if Hq else None, bf16_dev(wk) if Hkv else None, cs=dev(cs) if with_cs else None,
                          Qout=Qo, Kout=Ko)
    lib.spec_device_status()
    t = cs.astype(np.float64) if with_cs else None
    for out, x, w in ((Qo, c.q, wq), (Ko, c.k, wk)):
        if out is None:
            continue
        y, mag = turned(c, x, obf.decode(w), t)
        err = abs(f64_of_bf16(out).reshape(y.shape) - y)
        assert np.all(err <= HALF_BF16 * abs(y) + (1 + HALF_BF16) * F32 * mag)
    a, b = lib.spec_qk_norm_rope(Q, K, bf16_dev(wq) if Hq else None, bf16_dev(wk) if Hkv else None,
                                 cs=dev(cs) if with_cs else None)          # in place
    assert (a is Q and b is K) and all(x is None or torch.equal(x, y) for x, y in ((Q, Qo), (K, Ko)))


def test_qk_norm_rope_of_zeros_and_tiny_rows(lib):
    x = torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda")
    x[1], x[2, 5] = 1e-20, float("nan")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    out, _ = lib.spec_qk_norm_rope(x, None, w, None, eps=1e-6, Qout=torch.empty_like(x))
    assert torch.all(out[0] == 0) and torch.all(out[1].float().sub(1e-17).abs() < 1e-19) and torch.isnan(out[2]).all()


@pytest.mark.parametrize("what", ["append", "read"])
def test_bad_batches_and_pages(lib, what):
    """A sequence past its table or outside the rows is skipped, a page that does not exist left out; the others are served."""
    c = Cache(60, [3, 3, 3], [0, 0, 0], 1, spare=0)
    cu, cx, kp, vp, table = c.dev()
    _, k, v = c.parts()

    def call(cu, cx, table):
        kp2, vp2 = kp.clone(), vp.clone()
        outs = [torch.full((9, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        if what == "append":
            lib.spec_kv_append_paged_q4(k, v, cu, cx, kp2, vp2, table)
        else:
            lib.spec_kv_read_paged_q4(cu, cx, kp2, vp2, table, 9, Kout=outs[0], Vout=outs[1])
        code, site = lib.spec_device_status_code()
        assert code == lib.SPEC_EINVAL and site in ((0x8F1, 0x8F2) if what == "append" else (0x9F1, 0x9F2)), hex(site)
        return (kp2, vp2) if what == "append" else outs

    def expect(seqs):
        if what == "append":
            out = []
            for x, pool, keys in ((c.k, c.kp, True), (c.v, c.vp, False)):
                n, code = q4.quantise(x)
                for b in seqs:
                    pool = q4.append(n[3 * b:3 * b + 3], code[3 * b:3 * b + 3], [0, 3], [0], pool, c.table[b:b + 1], keys)
                out.append(pool)
            return out
        out = []
        for pool, keys in ((c.kp, True), (c.vp, False)):
            ref = np.full((9, 128), 7.0)
            for b in seqs:
                ref[3 * b:3 * b + 3] = q4.read(pool, [0, 3], [0], c.table[b:b + 1], keys, 3)[:, 0]
            out.append(ref)
        return out

    def check(got, seqs):
        for g, r in zip(got, expect(seqs)):
            assert np.array_equal(g.cpu().numpy() if what == "append" else f64_of_bf16(g), r)
    far = cx.clone(); far[1] = 126
    check(call(cu, far, table), [0, 2])
    neg = cx.clone(); neg[2] = -1
    check(call(cu, neg, table), [0, 1])
    for bad in (-1, c.num_pages, 1 << 30):
        t = table.clone(); t[0, 0] = bad
        check(call(cu, cx, t), [1, 2])
    out = cu.clone(); out[3] = 10
    check(call(out, cx, table), [0, 1])


def test_pools_past_2_31_bytes(lib):
    """Pages whose offsets pass 32 bits."""
    pages = 260000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 5 GB")
    kp, vp = (lib.q4_pool(1, pages) for _ in range(2))
    table = torch.tensor([[pages - 1], [246724]], dtype=torch.int32, device="cuda")     # (246724 * 8704: just past 2^31)
    c = Cache(70, [5, 4], [100, 3], 1)
    cu, cx, *_ = c.dev()
    _, k, v = c.parts()
    for pool in (kp, vp):
        pool[0, pages - 1] = pool[0, 246724] = pool[0, 0] = 0
    lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table)
    K, V = lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, 9)
    lib.spec_device_status()
    for got, x in ((K, c.k), (V, c.v)):
        assert np.array_equal(f64_of_bf16(got).reshape(9, 1, D), q4.dequantise(*q4.quantise(x)))
    assert not kp[0, 0].any() and not vp[0, 0].any()


def test_captured_and_on_another_stream(lib):
    """A captured append, read and norm replayed on new inputs; the same calls on another stream than the current one."""
    c = Cache(80, [5, 40], [3, 100], 2, 8)
    cu, cx, kp, vp, table = c.dev()
    q, k, v = c.parts()
    w = bf16_dev(synth.normal_bf16_bits(4, (D,), 1.0))
    cs = dev(table_of(c))
    qr, kn = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    outs = [torch.empty_like(kn) for _ in range(2)]

    def calls(stream=None):
        lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table, cs=cs, Q=q, Qrot=qr, wq=w, wk=w, stream=stream)
        lib.spec_kv_read_paged_q4(cu, cx, kp, vp, table, c.M, Kout=outs[0], Vout=outs[1], stream=stream)
        lib.spec_qk_norm_rope(None, k, None, w, cs=cs, Kout=kn, stream=stream)
    everything = (kp, vp, qr, kn, *outs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls(side)
    side.synchronize()
    first = [t.clone() for t in everything]
    calls()
    assert all(torch.equal(a, b) for a, b in zip(first, everything))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    k.mul_(0.5); v.add_(1.0); cx.add_(1)
    graph.replay()
    got = [t.clone() for t in everything]
    calls()
    assert all(torch.equal(a, b) for a, b in zip(got, everything))
    assert not torch.equal(got[5], first[5])
    lib.spec_device_status()
