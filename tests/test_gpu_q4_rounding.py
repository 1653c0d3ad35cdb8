"""GPU: norm, rotation and quantisation against the same operations in fp32, each rounded once and in the order that the
header gives, bit by bit; and a row's bytes whatever the chunk that it came in."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, q4

from gpu_util import bf16_dev, bits_of, dev
from test_gpu_cache_q4 import Cache, codes, table_of

pytestmark = pytest.mark.gpu
D = 128
F = np.float32


def turned32(x, w, cs, eps=1e-6):
    """Norm (w not None) and rotation (cs not None) of [M, heads, D] in fp32.  (NumPy rounds every operation by itself.)"""
    x = x.astype(F)
    if w is not None:
        s = x * x
        while s.shape[-1] > 1:                               # neighbours first
            s = s[..., 0::2] + s[..., 1::2]
        x = x * (F(1) / np.sqrt(s * F(1 / D) + F(eps))) * w.astype(F)
    if cs is not None:
        c, s = cs[:, None, :, 0], cs[:, None, :, 1]
        a, b = x[..., :D // 2], x[..., D // 2:]
        x = np.concatenate([a * c - b * s, b * c + a * s], axis=-1)
    assert x.dtype == F
    return x


def stored32(x):
    """(whole numbers, scale codes) of fp32 values, quotients rounded to fp32."""
    g = x.reshape(*x.shape[:-1], 4, 32)
    code = q4.scale_codes(abs(g).max(-1) / F(7))
    n = np.clip(np.rint(g / q4.scale_of(code).astype(F)[..., None]), -7, 7)
    return n.reshape(x.shape), code


def weights():
    return [synth.f32_to_bf16_bits((1 + 0.3 * np.random.default_rng(s).standard_normal(D)).astype(F)) for s in (1, 2)]


# few rows and many (above 4 for each SM), values in blocks of 8 keys and of 32
SHAPES = [([1, 5, 0, 30], [0, 126, 3, 999], 32, 8), ([350, 3], [60, 5], 8, 4), ([1700, 20], [60, 7], 16, 4), ([1700], [60], 4, 32)]


@pytest.mark.parametrize("with_norm,with_cs", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("rows,ctx,Hq,Hkv", SHAPES)
def test_append_bit_by_bit(lib, rows, ctx, Hq, Hkv, with_norm, with_cs):
    c = Cache(20, rows, ctx, Hkv, Hq, pad=2, std=1.7)
    cu, cx, kp, vp, table = c.dev()
    q, k, v = c.parts()
    wq, wk = weights()
    cs = table_of(c)
    Qrot = torch.empty((c.Mp, Hq * D), dtype=torch.bfloat16, device="cuda")
    lib.spec_kv_append_paged_q4(k, v, cu, cx, kp, vp, table, cs=dev(cs) if with_cs else None, Q=q, Qrot=Qrot,
                                wq=bf16_dev(wq) if with_norm else None, wk=bf16_dev(wk) if with_norm else None)
    lib.spec_device_status()
    turns = cs[:c.M] if with_cs else None
    yq, yk = (turned32(x, obf.decode(w) if with_norm else None, turns) for x, w in ((c.q, wq), (c.k, wk)))
    assert np.array_equal(bits_of(Qrot[:c.M]).reshape(yq.shape), synth.f32_to_bf16_bits(yq).reshape(yq.shape))
    pool = kp.cpu().numpy()
    n, code = stored32(yk)
    assert np.array_equal(codes(pool, c, True), code)
    assert np.array_equal(q4.read(pool, c.cu, c.ctx, c.table, True, c.M), q4.dequantise(n, code))


@pytest.mark.parametrize("M,Hq,Hkv", [(9, 32, 8), (500, 16, 8), (1600, 32, 3)])
@pytest.mark.parametrize("with_cs", [True, False])
def test_norm_bit_by_bit(lib, M, Hq, Hkv, with_cs):
    c = Cache(50, [M], [33], Hkv, Hq, std=2.5)
    q, k, _ = c.parts()
    w = weights()
    cs = table_of(c)
    outs = lib.spec_qk_norm_rope(q, k, bf16_dev(w[0]), bf16_dev(w[1]), cs=dev(cs) if with_cs else None,
                                 Qout=torch.empty_like(q.contiguous()), Kout=torch.empty_like(k.contiguous()))
    lib.spec_device_status()
    for out, x, wb in zip(outs, (c.q, c.k), w):
        y = turned32(x, obf.decode(wb), cs[:M] if with_cs else None)
        assert np.array_equal(bits_of(out).reshape(y.shape), synth.f32_to_bf16_bits(y).reshape(y.shape))


@pytest.mark.parametrize("Hq,Hkv", [(16, 4), (2, 32)])
def test_chunks_of_every_launch_shape(lib, Hq, Hkv):
    """A prompt in one chunk of many rows and in chunks of few and many: the same pools and queries, to the byte."""
    n = 1700
    c = Cache(31, [n], [0], Hkv, Hq)
    cu, cx, kp, vp, table = c.dev()
    q, k, v = c.parts()
    w = bf16_dev(weights()[0])
    cs = dev(table_of(c))

    def run(sizes):
        kp2, vp2, qr = kp.clone(), vp.clone(), torch.empty_like(q.contiguous())
        at = 0
        for m in sizes:
            i = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            x = torch.tensor([at], dtype=torch.int32, device="cuda")
            lib.spec_kv_append_paged_q4(k[at:at + m], v[at:at + m], i, x, kp2, vp2, table, cs=cs[at:at + m],
                                        Q=q[at:at + m], Qrot=qr[at:at + m], wq=w, wk=w)
            at += m
        assert at == n
        return kp2, vp2, qr
    whole = run([n])
    for sizes in ([401, 1, 599, 37, 662], [1019, 681], [100] * 17):
        for x, y in zip(run(sizes), whole):
            assert torch.equal(x, y)
    # ... and the norm alone, of many rows and of few, gives the queries of the append
    for m in (n, 300):
        qn, _ = lib.spec_qk_norm_rope(q[:m], None, w, None, cs=cs[:m], Qout=torch.empty_like(q[:m].contiguous()))
        assert torch.equal(qn, whole[2][:m])
    lib.spec_device_status()
