"""The engine with norms of queries and keys, and over a paged cache in 4 bits: prompts in chunks, then verify passes on the
same pages, against the oracle's single pass over the whole sequences."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, ops as oops, stack as ostack

from gpu_util import STACK_PROB_BOUND, assert_close_chain, bf16_dev, bits_of, chain_floor, dev, f64_of_bf16
from test_gpu_glue_stack import _tiny_stack
from test_gpu_prefill import Paged, run_chunks

pytestmark = pytest.mark.gpu
PAGE = 128
LENGTHS, GAMMAS = [200, 131, 7], [3, 0, 4]
TOTAL = [n + g + 1 for n, g in zip(LENGTHS, GAMMAS)]
CUTS = [(0, 0, 0), (129, 1, 0), (129, 130, 6), (200, 131, 7)]


def stack_with_norms(L, seed, norms=True):
    dims, od, osw, gsw = _tiny_stack(L, seed)
    for li in range(L if norms else 0):
        for name in ("q_norm", "k_norm"):
            rng = np.random.default_rng([seed, li, len(name), name == "q_norm"])
            w = synth.f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(128)).astype(np.float32))
            setattr(osw.layers[li], name, w)
            setattr(gsw.layers[li], name, bf16_dev(w))
    return dims, od, osw, gsw


class Paged4(Paged):
    """The same pages in 4 bits, full of 0xff bytes."""

    def __init__(self, lib, dims, lengths, seed=3):
        super().__init__(dims, lengths, seed)
        n = self.k[0].shape[1]
        self.k, self.v = ([lib.q4_pool(dims.Hkv, n).fill_(255) for _ in range(dims.layers)] for _ in range(2))

    def read(self, lib, li, lengths):
        """Keys and values [rows, Hkv, 128] of the sequences from the start."""
        cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        zero = dev(np.zeros(len(lengths), np.int32))
        out = lib.spec_kv_read_paged_q4(dev(cu), zero, self.k[li], self.v[li], self.table, int(cu[-1]))
        return [f64_of_bf16(t).reshape(cu[-1], -1, 128) for t in out]


def whole(osw, od, x_bits, lengths, stored=None):
    cu = np.concatenate([[0], np.cumsum(lengths)])
    zeros = [np.zeros((len(lengths), od.Hkv, max(lengths), 128)) for _ in range(od.layers)]
    x, lg, _, _ = ostack.verify_pass(obf.decode(np.concatenate(x_bits)), osw, od, cu, [0] * len(lengths), zeros, zeros,
                                     stored=stored)
    return [x[cu[b]:cu[b + 1]] for b in range(len(lengths))], [lg[cu[b]:cu[b + 1]] for b in range(len(lengths))]


def prompt_then_verify(lib, eng, dims, x_bits):
    """Hidden rows of the prompts and of the verify pass behind them, per sequence, and both passes' probabilities."""
    hidden, P = run_chunks(eng, x_bits, CUTS, lib, temperature=1.0)
    P = P.cpu().numpy().astype(np.float64)
    cu = np.concatenate([[0], np.cumsum([g + 1 for g in GAMMAS])]).astype(np.int32)
    x0 = bf16_dev(np.concatenate([x[n:] for x, n in zip(x_bits, LENGTHS)]))
    Pv = eng.verify_pass(x0, dev(cu), dev(np.array(LENGTHS, np.int32)), 1.0)
    lib.spec_device_status()
    x = f64_of_bf16(eng.x[:cu[-1]])
    return [np.concatenate([h, x[cu[b]:cu[b + 1]]]) for b, h in enumerate(hidden)], P, Pv.cpu().numpy().astype(np.float64)


def check(got, P, Pv, ref_x, ref_lg, L, what):
    for b in range(3):
        assert_close_chain(got[b], ref_x[b], L, f"{what}: sequence {b}")
        p = oops.target_probs(ref_lg[b][LENGTHS[b] - 1:LENGTHS[b]], 1.0)[0]
        assert abs(P[b] - p).max() < STACK_PROB_BOUND
    lg = np.concatenate([x[n:] for x, n in zip(ref_lg, LENGTHS)])
    assert abs(Pv - oops.target_probs(lg, 1.0)).max() < STACK_PROB_BOUND


@pytest.mark.parametrize("L,fold", [(1, True), (2, False)])
def test_norms_of_queries_and_keys(lib, L, fold):
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = stack_with_norms(L, 130 + L)
    x_bits = [synth.normal_bf16_bits(90 + b, (TOTAL[b], dims.d), 1.0) for b in range(3)]
    cache = Paged(dims, TOTAL)
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=400, max_rows=5, fold_norms=fold, block_table=cache.table)
    check(*prompt_then_verify(lib, eng, dims, x_bits), *whole(osw, od, x_bits, TOTAL), L, "norms, pages")


def test_norms_over_a_contiguous_cache(lib):
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = stack_with_norms(1, 133)
    batch = synth.RaggedBatch([3, 0, 5], [40, 9, 0], cap=160)
    kc, vc = (synth.normal_bf16_bits(s, (batch.B, dims.Hkv, batch.cap, 128), 1.0) for s in (200, 300))
    x0 = synth.normal_bf16_bits(7, (batch.M, dims.d), 1.0)
    eng = E.VerifyEngine(dims, gsw, [bf16_dev(kc)], [bf16_dev(vc)], max_M=batch.M, max_rows=batch.max_rows)
    P = eng.verify_pass(bf16_dev(x0), dev(batch.cu_rows), dev(batch.ctx_len), 1.0)
    lib.spec_device_status()
    xr, lg, _, _ = ostack.verify_pass(obf.decode(x0), osw, od, batch.cu_rows, batch.ctx_len, [obf.decode(kc)], [obf.decode(vc)])
    assert_close_chain(f64_of_bf16(eng.x[:batch.M]), xr, 1, "norms, contiguous")
    assert abs(P.cpu().numpy().astype(np.float64) - oops.target_probs(lg, 1.0)).max() < STACK_PROB_BOUND


@pytest.mark.parametrize("L,norms,fold,max_rows", [(1, True, True, 5), (1, False, True, 5), (2, True, False, 5), (1, True, True, 40)])
def test_cache_in_4_bits(lib, L, norms, fold, max_rows):
    """The oracle attends the keys and values that the cache reads back; they are the oracle's own to half a scale and what
    separates two chains of the arithmetic."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = stack_with_norms(L, 140 + L, norms)
    x_bits = [synth.normal_bf16_bits(90 + b, (TOTAL[b], dims.d), 1.0) for b in range(3)]
    cache = Paged4(lib, dims, TOTAL)
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=400, max_rows=max_rows, fold_norms=fold, block_table=cache.table)
    got = prompt_then_verify(lib, eng, dims, x_bits)

    def hook(li):
        held = cache.read(lib, li, TOTAL)

        def stored(k, v):
            for mine, his in ((k, held[0]), (v, held[1])):
                g = lambda t: abs(t).reshape(len(t), od.Hkv, 4, 32).max(-1, keepdims=True).repeat(32, -1).reshape(t.shape)
                scale = np.maximum(g(mine), g(his)) / 7 * (1 + 1 / 16)
                rms = np.sqrt((mine ** 2).mean())
                assert np.all(abs(his - mine) <= scale / 2 + 2e-2 * abs(mine) + chain_floor(L) * rms)
            return held
        return stored
    check(*got, *whole(osw, od, x_bits, TOTAL, [hook(li) for li in range(L)]), L, "4 bits")


def test_captured_round_over_4_bits(lib):
    """A round captured over a cache in 4 bits gives, after other inputs are written into its buffers, what the eager round
    gives on them, cache included."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = stack_with_norms(2, 149)
    dims.rope_sections = (24, 20, 20)
    lengths = [140, 20]
    cache = Paged4(lib, dims, [n + 8 for n in lengths])
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=160, max_rows=6, block_table=cache.table)
    run_chunks(eng, [synth.normal_bf16_bits(99 + b, (lengths[b], dims.d), 1.0) for b in range(2)], [(0, 0), (140, 20)], lib)

    def inputs(seed, rows, ctx, shift):
        rng = np.random.default_rng(seed)
        q = rng.dirichlet(np.full(dims.V, 0.5), size=sum(rows) - 2).astype(np.float32)
        drafts = np.array([int(rng.integers(dims.V)) for _ in q], np.int32)
        pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, rows)])
        return (bf16_dev(synth.normal_bf16_bits(seed, (sum(rows), dims.d), 1.0)),
                dev(np.array([0, rows[0], sum(rows)], np.int32)), dev(np.array(ctx, np.int32)), dev(q), dev(drafts),
                dev(synth.uniforms_f32(seed + 1, sum(rows)))), dev(np.stack([pos + shift, pos, pos + 2 * shift]).astype(np.int32))

    bufs, pos = inputs(5, [3, 5], lengths, 0)
    out = tuple(torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, 8, 2))
    replay = eng.capture_round(*bufs, 0.8, out, positions=pos)
    before = [t.clone() for t in (*eng.kc, *eng.vc)]
    other, other_pos = inputs(6, [6, 2], [137, 19], 11)
    want = [t.cpu() for t in eng.verify_round(*other, 0.8, positions=other_pos)]
    written = [t.clone() for t in (*eng.kc, *eng.vc)]
    assert any(not torch.equal(a, b) for a, b in zip(before, written))
    for t, old in zip((*eng.kc, *eng.vc), before):
        t.copy_(old)
    for buf, new in zip((*bufs, pos), (*other, other_pos)):
        buf.copy_(new)
    replay()
    lib.spec_device_status()
    assert all(torch.equal(o.cpu(), w) for o, w in zip(out, want))
    assert all(torch.equal(t, w) for t, w in zip((*eng.kc, *eng.vc), written))


def test_draft_engine_over_4_bits(lib):
    """Drafts behind a prompt in a cache in 4 bits: q's rows are what a verify pass over the drafted tokens gives (both read
    the same bytes; their kernels sum in other orders)."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = stack_with_norms(1, 153)
    B, gamma, lengths = 2, 3, [140, 20]
    cache = Paged4(lib, dims, [n + gamma for n in lengths])
    g = E.DraftEngine(dims, gsw, cache.k, cache.v, B, gamma, block_table=cache.table, max_M=160)
    x_bits = [synth.normal_bf16_bits(97 + b, (lengths[b], dims.d), 1.0) for b in range(B)]
    run_chunks(g.eng, x_bits, [(0, 0), (140, 20)], lib)
    tok, ctx = dev(np.array([5, 9], np.int32)), dev(np.array(lengths, np.int32))
    U = dev(synth.uniforms_f32(4, gamma * B).reshape(gamma, B))
    Q = torch.zeros((B * gamma, dims.V), device="cuda")
    drafts = torch.zeros(B * gamma, dtype=torch.int32, device="cuda")
    g.draft(tok, ctx, U, 1.0, Q, drafts)
    held = [t.clone() for t in (cache.k[0], cache.v[0])]
    rows = torch.stack([torch.cat([tok[b:b + 1], drafts[b * gamma:(b + 1) * gamma - 1]]) for b in range(B)]).view(-1)
    x0 = lib.spec_embed(rows.contiguous(), g.table)
    v = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=B * gamma, max_rows=gamma, fold_norms=False, block_table=cache.table)
    P = v.verify_pass(x0, dev(np.array([0, gamma, 2 * gamma], np.int32)), ctx, 1.0)
    lib.spec_device_status()
    assert (P - Q).abs().max().item() < STACK_PROB_BOUND
    # the verify pass wrote the rows' keys and values again: the same to a step of a few entries
    assert all((a != b).float().mean().item() < 0.01 for a, b in zip(held, (cache.k[0], cache.v[0])))


def test_refusals(lib):
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, _, _, gsw = stack_with_norms(2, 157)
    pool = [lib.q4_pool(dims.Hkv, 2) for _ in range(2)]
    with pytest.raises(ValueError, match="paged"):
        E.VerifyEngine(dims, gsw, pool, pool, max_M=4, max_rows=1)
    gsw.layers[1].k_norm = None
    with pytest.raises(ValueError, match="every layer"):
        E.VerifyEngine(dims, gsw, pool, pool, max_M=4, max_rows=1, block_table=dev(np.zeros((1, 1), np.int32)))
