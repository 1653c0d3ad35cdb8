"""The engine's prompts over a paged cache: chunks of uneven length, then verify passes on the same pages,
against the oracle's single pass over the whole sequences."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, ops as oops, stack as ostack

from gpu_util import STACK_PROB_BOUND, assert_close_chain, bf16_dev, bits_of, dev, f64_of_bf16
from test_gpu_glue_stack import _tiny_stack

pytestmark = pytest.mark.gpu
PAGE = 128


class Paged:
    """Per-layer pools full of NaN and a block table in a random order."""

    def __init__(self, dims, lengths, seed=3):
        need = [(n + PAGE - 1) // PAGE for n in lengths]
        perm = np.random.default_rng(seed).permutation(sum(need) + 2)
        self.table_h = np.full((len(lengths), max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table_h[b, :n] = perm[at:at + n]
            at += n
        pool = lambda: torch.full((dims.Hkv, sum(need) + 2, PAGE, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.k, self.v = [pool() for _ in range(dims.layers)], [pool() for _ in range(dims.layers)]
        self.table = dev(self.table_h)


def whole(osw, od, x_bits, lengths):
    """The oracle's one pass over the sequences from position 0: hidden rows, logits per sequence."""
    cu = np.concatenate([[0], np.cumsum(lengths)])
    zeros = [np.zeros((len(lengths), od.Hkv, max(lengths), 128)) for _ in range(od.layers)]
    x, lg, _, _ = ostack.verify_pass(obf.decode(np.concatenate(x_bits)), osw, od, cu, [0] * len(lengths), zeros, zeros)
    return [x[cu[b]:cu[b + 1]] for b in range(len(lengths))], [lg[cu[b]:cu[b + 1]] for b in range(len(lengths))]


def run_chunks(eng, x_bits, cuts, lib, temperature=None, positions=None):
    """Runs the cuts' chunks through eng.prefill; the hidden rows per sequence (and the last P)."""
    out, P = [[] for _ in x_bits], None
    for at, to in zip(cuts[:-1], cuts[1:]):
        rows = [t - a for a, t in zip(at, to)]
        cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        x0 = bf16_dev(np.concatenate([x[a:t] for x, a, t in zip(x_bits, at, to)]))
        pos = None if positions is None else positions(at, to)
        r = eng.prefill(x0, dev(cu), dev(np.array(at, np.int32)), temperature=temperature, positions=pos)
        x, P = r if temperature is not None else (r, None)
        x = f64_of_bf16(x)
        for b in range(len(x_bits)):
            out[b].append(x[cu[b]:cu[b + 1]])
    lib.spec_device_status()
    return [np.concatenate(o) for o in out], P


@pytest.mark.parametrize("L,fold,fused", [(1, True, True), (2, True, True), (2, False, False)])
def test_prompt_then_verify(lib, L, fold, fused):
    """Three sequences' prompts in uneven chunks (one of them brings nothing at times), then a verify pass."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(L, 70 + L)
    lengths, gammas = [200, 131, 7], [3, 0, 4]
    total = [n + g + 1 for n, g in zip(lengths, gammas)]
    x_bits = [synth.normal_bf16_bits(90 + b, (total[b], dims.d), 1.0) for b in range(3)]
    cache = Paged(dims, total)
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=400, max_rows=5, fold_norms=fold, fused_rope=fused,
                         block_table=cache.table)
    cuts = [(0, 0, 0), (129, 1, 0), (129, 130, 6), (200, 131, 7)]
    hidden, P = run_chunks(eng, x_bits, cuts, lib, temperature=1.0)
    ref_x, ref_lg = whole(osw, od, x_bits, total)
    for b in range(3):
        assert_close_chain(hidden[b], ref_x[b][:lengths[b]], L, f"prompt rows of sequence {b}")
        # the next token's probabilities behind the prompt
        p = P[b].cpu().numpy().astype(np.float64)
        assert abs(p - oops.target_probs(ref_lg[b][lengths[b] - 1:lengths[b]], 1.0)[0]).max() < STACK_PROB_BOUND
    cu = np.concatenate([[0], np.cumsum([g + 1 for g in gammas])]).astype(np.int32)
    x0 = bf16_dev(np.concatenate([x[n:] for x, n in zip(x_bits, lengths)]))
    P = eng.verify_pass(x0, dev(cu), dev(np.array(lengths, np.int32)), 1.0)
    lib.spec_device_status()
    ref = np.concatenate([x[n:] for x, n in zip(ref_x, lengths)])
    assert_close_chain(f64_of_bf16(eng.x[:cu[-1]]), ref, L, "verify rows behind the prompts")
    lg = np.concatenate([x[n:] for x, n in zip(ref_lg, lengths)])
    assert abs(P.cpu().numpy().astype(np.float64) - oops.target_probs(lg, 1.0)).max() < STACK_PROB_BOUND


def test_prefill_captured(lib):
    """One graph of a chunk of up to 64 rows, replayed for the chunks of the prompts."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 87)
    lengths = [150, 41]
    x_bits = [synth.normal_bf16_bits(89 + b, (lengths[b], dims.d), 1.0) for b in range(2)]
    cache = Paged(dims, lengths)
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=64, max_rows=1, block_table=cache.table)
    x0 = torch.zeros((64, dims.d), dtype=torch.bfloat16, device="cuda")
    cu, ctx = dev(np.array([0, 0, 0], np.int32)), dev(np.zeros(2, np.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eng.prefill(x0, cu, ctx, temperature=1.0)            # (all rows padding)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        x, P = eng.prefill(x0, cu, ctx, temperature=1.0)
    ref_x, ref_lg = whole(osw, od, x_bits, lengths)
    for at, to in zip([(0, 0), (40, 20), (100, 20)], [(40, 20), (100, 20), (150, 34)]):
        rows = [t - a for a, t in zip(at, to)]
        cu.copy_(dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)))
        ctx.copy_(dev(np.array(at, np.int32)))
        x0[:sum(rows)] = bf16_dev(np.concatenate([xb[a:t] for xb, a, t in zip(x_bits, at, to)]))
        graph.replay()
        lib.spec_device_status()
        got, probs = f64_of_bf16(x), P.cpu().numpy().astype(np.float64)
        r0 = 0
        for b in range(2):
            assert_close_chain(got[r0:r0 + rows[b]], ref_x[b][at[b]:to[b]], 1, f"replayed chunk at {at}, sequence {b}")
            r0 += rows[b]
            if rows[b]:
                assert abs(probs[b] - oops.target_probs(ref_lg[b][to[b] - 1:to[b]], 1.0)[0]).max() < STACK_PROB_BOUND


def test_positions_of_several_axes(lib):
    """Text's positions on three axes are its one position; attention only sees differences, so positions that are
    all 5000 further on give the same rows."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 81)
    dims.rope_sections, dims.rope_interleaved = (24, 20, 20), True
    lengths = [150, 40]
    x_bits = [synth.normal_bf16_bits(95 + b, (lengths[b], dims.d), 1.0) for b in range(2)]
    ref_x, _ = whole(osw, od, x_bits, lengths)
    for shift in (0, 5000):
        cache = Paged(dims, lengths)
        eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=200, max_rows=1, block_table=cache.table)

        def positions(at, to):
            pos = np.concatenate([np.arange(a, t) for a, t in zip(at, to)]) + shift
            return dev(np.stack([pos] * 3).astype(np.int32))
        hidden, _ = run_chunks(eng, x_bits, [(0, 0), (100, 1), (150, 40)], lib, positions=positions)
        for b in range(2):
            assert_close_chain(hidden[b], ref_x[b], 1, f"shift {shift}, sequence {b}")


def test_captured_round_with_positions(lib):
    """A round captured over pages and positions on three axes: after other tokens, lengths and positions are written
    into its buffers a replay gives what the eager round gives on them."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(2, 89)
    dims.rope_sections = (24, 20, 20)
    lengths = [140, 20]
    cache = Paged(dims, [n + 8 for n in lengths])
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
    other, other_pos = inputs(6, [6, 2], [137, 19], 11)
    want = [t.cpu() for t in eng.verify_round(*other, 0.8, positions=other_pos)]
    written = [bits_of(k) for k in eng.kc]
    for buf, new in zip((*bufs, pos), (*other, other_pos)):
        buf.copy_(new)
    replay()
    lib.spec_device_status()
    assert all(torch.equal(o.cpu(), w) for o, w in zip(out, want))
    assert all(np.array_equal(bits_of(k), w) for k, w in zip(eng.kc, written))
    # the positions count: the same round at the plain ones writes other keys
    eng.verify_round(*other, 0.8)
    lib.spec_device_status()
    assert any(not np.array_equal(bits_of(k), w) for k, w in zip(eng.kc, written))


def test_draft_engine_over_pages(lib):
    """The draft phase on a paged cache that a prompt filled: the same drafts and q as on a contiguous cache with the
    same keys (one row per sequence takes the same key tiles in the same order)."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 83)
    B, gamma, lengths = 2, 3, [140, 20]
    cache = Paged(dims, [n + gamma for n in lengths])
    g = E.DraftEngine(dims, gsw, cache.k, cache.v, B, gamma, block_table=cache.table, max_M=160)
    x_bits = [synth.normal_bf16_bits(97 + b, (lengths[b], dims.d), 1.0) for b in range(B)]
    run_chunks(g.eng, x_bits, [(0, 0), (140, 20)], lib)
    kc = torch.zeros((B, dims.Hkv, 2 * PAGE, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    for b in range(B):
        for t in range((lengths[b] + gamma + PAGE - 1) // PAGE):
            n = min(PAGE, lengths[b] - t * PAGE)
            kc[b, :, t * PAGE:t * PAGE + n] = cache.k[0][:, cache.table_h[b, t], :n]
            vc[b, :, t * PAGE:t * PAGE + n] = cache.v[0][:, cache.table_h[b, t], :n]
    c = E.DraftEngine(dims, gsw, [kc], [vc], B, gamma)
    tok, ctx = dev(np.array([5, 9], np.int32)), dev(np.array(lengths, np.int32))
    U = dev(synth.uniforms_f32(4, gamma * B).reshape(gamma, B))
    res = []
    for e in (g, c):
        Q = torch.zeros((B * gamma, dims.V), device="cuda")
        drafts = torch.zeros(B * gamma, dtype=torch.int32, device="cuda")
        e.draft(tok, ctx, U, 1.0, Q, drafts)
        lib.spec_device_status()
        res.append((Q, drafts))
    assert torch.equal(res[0][1], res[1][1]) and torch.equal(res[0][0], res[1][0])


def test_prefill_refusals(lib):
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, _, _, gsw = _tiny_stack(1, 85)
    x = torch.zeros((2, dims.d), dtype=torch.bfloat16, device="cuda")
    cu, ctx = dev(np.array([0, 2], np.int32)), dev(np.zeros(1, np.int32))
    kc = [torch.zeros((1, dims.Hkv, 8, 128), dtype=torch.bfloat16, device="cuda")]
    eng = E.VerifyEngine(dims, gsw, kc, [kc[0].clone()], max_M=4, max_rows=2)
    with pytest.raises(ValueError):
        eng.prefill(x, cu, ctx)                                  # contiguous cache
    cache = Paged(dims, [8])
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=1, max_rows=1, block_table=cache.table)
    with pytest.raises(ValueError):
        eng.prefill(x, cu, ctx)                                  # more rows than the engine was sized for


def test_prefill_with_a_sequence_outside_the_rows(lib):
    """cu_rows past the chunk's rows: the status word says so, no index leaves the buffers, and the sequence that
    is in them gets its rows and its probabilities."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 91)
    lengths = [5, 4, 3]
    x_bits = [synth.normal_bf16_bits(101 + b, (lengths[b], dims.d), 1.0) for b in range(3)]
    cache = Paged(dims, lengths)
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=16, max_rows=1, block_table=cache.table)
    x0 = bf16_dev(np.concatenate(x_bits)[:7])
    ref_x, ref_lg = whole(osw, od, x_bits, lengths)
    for ends in ([5, 9, 12], [5, 1 << 30, 1 << 30], [5, 9, 1 << 30]):
        x, P = eng.prefill(x0, dev(np.array([0] + ends, np.int32)), dev(np.zeros(3, np.int32)), temperature=1.0)
        rc, _ = lib.spec_device_status_code()
        assert rc == lib.SPEC_EINVAL, ends
        assert_close_chain(f64_of_bf16(x)[:5], ref_x[0], 1, f"rows of the sequence in bounds, {ends}")
        p = P[0].cpu().numpy().astype(np.float64)
        assert abs(p - oops.target_probs(ref_lg[0][-1:], 1.0)[0]).max() < STACK_PROB_BOUND
        lib.spec_device_status()


def test_prefill_of_no_rows(lib):
    """A chunk to which no sequence brings a row, with and without the probabilities; and probabilities without an LM
    head are refused before anything runs."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, _, _, gsw = _tiny_stack(1, 93)
    cache = Paged(dims, [8, 8])
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=4, max_rows=1, block_table=cache.table)
    x0 = torch.empty((0, dims.d), dtype=torch.bfloat16, device="cuda")
    none, ctx = dev(np.zeros(3, np.int32)), dev(np.array([3, 0], np.int32))
    before = [bits_of(k) for k in cache.k]
    assert eng.prefill(x0, none, ctx).shape == (0, dims.d)
    x, P = eng.prefill(x0, none, ctx, temperature=1.0)
    lib.spec_device_status()
    assert x.shape == (0, dims.d) and P.shape == (2, dims.V)
    assert all(np.array_equal(bits_of(k), b) for k, b in zip(cache.k, before))
    gsw.w_lm = None
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=4, max_rows=1, block_table=cache.table)
    launched = lib.launch_count()
    with pytest.raises(ValueError):
        eng.prefill(x0.new_zeros((2, dims.d)), dev(np.array([0, 2, 2], np.int32)), ctx, temperature=1.0)
    assert lib.launch_count() == launched


def grid_positions(n, lead):
    """[3, n]: text, then a grid of patches 7 wide (one time, rows and columns apart), behind `lead` tokens."""
    i = np.arange(n)
    j = np.clip(i - lead, 0, None)
    grid = np.stack([0 * j, j // 7, j % 7]) + lead
    return np.where(i < lead, i, grid)


@pytest.mark.parametrize("interleaved", [True, False])
def test_draft_behind_a_prompt_with_positions(lib, interleaved):
    """Drafts behind prompts whose positions differ between the axes and from the token's index: hidden rows and q are
    those of one pass over the whole sequences at the given positions (the token's index would be off by 30 and
    10 times the bounds)."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 97)
    for d in (dims, od):
        d.rope_sections, d.rope_interleaved = (24, 20, 20), interleaved
    B, gamma, lengths = 2, 3, [140, 20]
    cache = Paged(dims, [n + gamma for n in lengths])
    g = E.DraftEngine(dims, gsw, cache.k, cache.v, B, gamma, block_table=cache.table, max_M=160)
    pos = [grid_positions(n, 5 + b) for b, n in enumerate(lengths)]
    x_bits = [synth.normal_bf16_bits(300 + b, (lengths[b], dims.d), 1.0) for b in range(B)]
    run_chunks(g.eng, x_bits, [(0, 0), (90, 1), (140, 20)], lib, positions=lambda at, to: dev(
        np.concatenate([p[:, a:t] for p, a, t in zip(pos, at, to)], axis=1).astype(np.int32)))
    tok, ctx = np.array([5, 9], np.int32), dev(np.array(lengths, np.int32))
    first = np.stack([np.full(3, p.max() + 1) for p in pos], axis=1).astype(np.int32)       # [3, B]
    Q = torch.zeros((B * gamma, dims.V), device="cuda")
    drafts = torch.zeros(B * gamma, dtype=torch.int32, device="cuda")
    U = dev(synth.uniforms_f32(4, gamma * B).reshape(gamma, B))
    g.draft(dev(tok), ctx, U, 1.0, Q, drafts, positions=dev(first))
    lib.spec_device_status()
    hidden, q, d = f64_of_bf16(g.eng.x[:B]), Q.cpu().numpy().astype(np.float64), drafts.cpu().numpy().reshape(B, gamma)
    table = obf.decode(osw.w_lm)
    for b in range(B):
        n = lengths[b] + gamma
        fed = table[[tok[b], *d[b, :-1]]]
        at = np.concatenate([pos[b], first[:, b:b + 1] + np.arange(gamma)], axis=1)
        zeros = [np.zeros((1, dims.Hkv, n, 128))]
        x, lg, _, _ = ostack.verify_pass(np.concatenate([obf.decode(x_bits[b]), fed]), osw, od, [0, n], [0], zeros, zeros,
                                         positions=at)
        assert_close_chain(hidden[b:b + 1], x[-1:], 1, f"last drafted row of sequence {b}")
        assert abs(q[b * gamma:(b + 1) * gamma] - oops.target_probs(lg[-gamma:], 1.0)).max() < STACK_PROB_BOUND
    with pytest.raises(ValueError):
        g.draft(dev(tok), ctx, U, 1.0, Q, drafts, positions=dev(first[:1]))


@pytest.mark.parametrize("interleaved", [True, False])
def test_unequal_axes_against_the_oracle(lib, interleaved):
    """Prompt and verify rows at positions that differ between the axes: the oracle's pass at the same positions (with two
    axes exchanged rows are off by 29 times the bound and more)."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(2, 103)
    for d in (dims, od):
        d.rope_sections, d.rope_interleaved = (24, 20, 20), interleaved
    lengths, new = [140, 20], [3, 5]
    pos = [grid_positions(n + m, 5 + b) for b, (n, m) in enumerate(zip(lengths, new))]
    x_bits = [synth.normal_bf16_bits(310 + b, (p.shape[1], dims.d), 1.0) for b, p in enumerate(pos)]
    cache = Paged(dims, [p.shape[1] for p in pos])
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=160, max_rows=5, block_table=cache.table)

    def packed(at, to):
        return dev(np.concatenate([p[:, a:t] for p, a, t in zip(pos, at, to)], axis=1).astype(np.int32))
    got, _ = run_chunks(eng, x_bits, [(0, 0), (77, 3), (140, 20)], lib, positions=packed)
    total = [n + m for n, m in zip(lengths, new)]
    x0 = bf16_dev(np.concatenate([x[n:] for x, n in zip(x_bits, lengths)]))
    P = eng.verify_pass(x0, dev(np.array([0, 3, 8], np.int32)), dev(np.array(lengths, np.int32)), 1.0,
                        positions=packed(lengths, total))
    lib.spec_device_status()
    probs, verified = P.cpu().numpy().astype(np.float64), np.split(f64_of_bf16(eng.x[:8]), [3])
    for b in range(2):
        zeros = [np.zeros((1, dims.Hkv, total[b], 128))] * 2
        x, lg, _, _ = ostack.verify_pass(obf.decode(x_bits[b]), osw, od, [0, total[b]], [0], zeros, zeros, positions=pos[b])
        assert_close_chain(got[b], x[:lengths[b]], 2, f"prompt rows of sequence {b}")
        assert_close_chain(verified[b], x[lengths[b]:], 2, f"verify rows of sequence {b}")
        rows = slice(0, 3) if b == 0 else slice(3, 8)
        assert abs(probs[rows] - oops.target_probs(lg[lengths[b]:], 1.0)).max() < STACK_PROB_BOUND


def test_more_slots_than_chunk_rows(lib):
    """40 slots and chunks of 8 rows at most: the LM head runs on a row per slot in the engine's own buffers (captured
    rounds keep their pointers), and the probabilities of the slots with rows are the oracle's."""
    from speculative_decoding_verify_05_gb300 import engine as E
    dims, od, osw, gsw = _tiny_stack(1, 107)
    lengths = [0] * 40
    lengths[0], lengths[17], lengths[39] = 3, 4, 1
    x_bits = [synth.normal_bf16_bits(320 + b, (n, dims.d), 1.0) for b, n in enumerate(lengths)]
    cache = Paged(dims, [max(n, 1) for n in lengths])
    eng = E.VerifyEngine(dims, gsw, cache.k, cache.v, max_M=8, max_rows=1, block_table=cache.table)
    buf, size = eng.ws.buf.data_ptr(), eng.ws.buf.numel()
    _, P = run_chunks(eng, x_bits, [[0] * 40, lengths], lib, temperature=1.0)
    assert P.data_ptr() == eng.P.data_ptr() and P.shape == (40, dims.V)
    assert (eng.ws.buf.data_ptr(), eng.ws.buf.numel()) == (buf, size)
    assert size >= lib.spec_lmhead_workspace_bytes(40, dims.d, dims.V)
    for b in (0, 17, 39):
        _, lg = whole(osw, od, [x_bits[b]], [lengths[b]])
        assert abs(P[b].cpu().numpy().astype(np.float64) - oops.target_probs(lg[0][-1:], 1.0)[0]).max() < STACK_PROB_BOUND
