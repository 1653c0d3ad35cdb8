"""GPU parity of the attention over a paged cache in 4 bits with the fp64 oracle, in both of its forms: any rows, and few
rows per sequence (max_rows given)."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, prompt as oprompt, q4

from gpu_util import bf16_dev, bits_of, dev, f64_of_bf16
from test_gpu_prompt import HALF_BF16, assert_attended

pytestmark = pytest.mark.gpu
PAGE, D, BYTES = 128, 128, 8704


def codes_for(rng, shape, size=1.0):
    """Scale codes of groups whose values are about `size` in rms."""
    return q4.scale_codes(size / 4.3 * np.exp2(rng.uniform(-0.7, 0.7, shape))).astype(np.uint8)


class Case:
    """Ragged batch over a paged cache in 4 bits: random pages, any bytes in every unused row and page."""

    def __init__(self, seed, rows, ctx, Hq, Hkv, q_std=1.0, pad=0, extra=3, spare=0):
        rng = np.random.default_rng(seed)
        self.rows, self.ctx = np.asarray(rows, np.int32), np.asarray(ctx, np.int32)
        self.B, self.Hq, self.Hkv = len(rows), Hq, Hkv
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.M = int(self.cu[-1])
        self.Mp = self.M + pad
        self.need = need = [max(0, int(c + n + PAGE - 1) // PAGE) for c, n in zip(ctx, rows)]
        self.max_pages = max(max(need), 1) + spare
        self.num_pages = sum(need) + extra
        perm = rng.permutation(self.num_pages)
        self.table = np.full((self.B, self.max_pages), -7, np.int32)      # ids that do not exist past the last page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (Hkv, self.num_pages)
        self.used = np.zeros((self.num_pages, PAGE), bool)
        for b in range(self.B):
            n = int(ctx[b] + rows[b]) if rows[b] else 0
            for t in range((n + PAGE - 1) // PAGE):
                self.used[self.table[b, t], :min(PAGE, n - t * PAGE)] = True
        self.kp, self.vp = (np.concatenate([rng.integers(0, 256, (*shape, 8192)).astype(np.uint8),
                                            codes_for(rng, (*shape, 512))], axis=-1) for _ in range(2))
        # scales of unused keys: anything, the largest among them
        free = ~self.used
        wild = rng.choice([0, 255, 130], (*shape, PAGE, 4)).astype(np.uint8)
        ks = self.kp[:, :, 8192:].reshape(*shape, PAGE, 4)
        vs = self.vp[:, :, 8192:].reshape(*shape, 4, PAGE)
        ks[:, free] = wild[:, free]
        np.swapaxes(vs, 2, 3)[:, free] = wild[:, free]
        self.q = synth.normal_bf16_bits(seed + 3, (self.Mp, Hq * D), q_std)
        if pad:
            self.q[self.M:] = 0x7FC0

    def dev(self):
        return dev(self.cu), dev(self.ctx), dev(self.kp), dev(self.vp), dev(self.table)

    def set_values(self, k=None, v=None):
        """Pools from values [Hkv, num_pages, PAGE, D] as the cache stores them."""
        for pool, x, keys in ((self.kp, k, True), (self.vp, v, False)):
            if x is None:
                continue
            n, c = q4.quantise(x)
            for h in range(self.Hkv):
                for p in range(self.num_pages):
                    for s in range(PAGE):
                        q4.put(pool[h, p], s, n[h, p, s], c[h, p, s], keys)

    def oracle(self, scale):
        kp, vp = (np.where(self.used[None, :, :, None], q4.unpack(x, keys), 0.0)
                  for x, keys in ((self.kp, True), (self.vp, False)))
        q = obf.decode(self.q[:self.M]).reshape(self.M, self.Hq, D)
        return oprompt.chunk_attention(q, self.cu, self.ctx, kp, vp, self.table, scale)


def run(lib, c, few, scale=None, ws=None, O=None):
    cu, ctx, kp, vp, table = c.dev()
    O = lib.spec_chunk_attention_paged_q4(bf16_dev(c.q), cu, ctx, kp, vp, table, scale=scale, ws=ws, O=O,
                                          max_rows=max(1, int(c.rows.max())) if few else None)
    lib.spec_device_status()
    assert np.array_equal(kp.cpu().numpy(), c.kp) and np.array_equal(vp.cpu().numpy(), c.vp)     # reads only
    return O


def check(lib, c, what, few, scale=None, ws=None):
    O = torch.full((c.Mp, c.Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    run(lib, c, few, scale, ws, O)
    ref, mag = c.oracle(1.0 / np.sqrt(D) if scale is None else scale)
    got = f64_of_bf16(O)
    assert np.all(got[c.M:] == 7.0), f"{what}: padding rows written"
    assert_attended(got[:c.M].reshape(ref.shape), ref, mag, what)
    return O


both = pytest.mark.parametrize("few", [False, True], ids=["any", "few"])


# --------------------------------------------------------------------------- shapes
@both
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (16, 8), (4, 4), (5, 1), (16, 1), (28, 4)])
@pytest.mark.parametrize("rows,ctx", [
    ([1], [0]), ([2, 1, 4], [126, 0, 1000]), ([1, 0, 3, 0], [127, 5, 128, 9]), ([4, 4], [255, 2047])])
def test_few_rows(lib, Hq, Hkv, rows, ctx, few):
    check(lib, Case(1, rows, ctx, Hq, Hkv, pad=2), "few rows", few)


@both
@pytest.mark.parametrize("Hq,Hkv,rows,ctx", [
    (64, 1, [1, 1], [300, 4]), (64, 2, [2], [130]), (40, 8, [12, 3], [0, 4000]), (4, 4, [64, 1, 33], [0, 700, 129]),
    (33, 1, [1], [77]), (21, 7, [21, 2], [500, 11]), (8, 8, [16], [112]), (32, 8, [16] * 3, [1, 111, 112])])
def test_rows_up_to_64_per_kv_head(lib, Hq, Hkv, rows, ctx, few):
    check(lib, Case(2, rows, ctx, Hq, Hkv, pad=1), "up to 64 rows", few)


@pytest.mark.parametrize("Hq,Hkv,rows,ctx", [
    (32, 8, [300], [0]), (16, 8, [129, 5, 64], [200, 0, 1]), (4, 4, [500, 1], [3, 900]), (128, 1, [3, 1], [130, 0]),
    (65, 1, [1, 2], [40, 300]), (28, 4, [40, 41, 42], [0, 128, 90]), (8, 2, [1200], [77])])
@pytest.mark.parametrize("grid", [0, 5])
def test_chunks(lib, Hq, Hkv, rows, ctx, grid):
    lib.spec_set_option("persistent_grid", grid)
    try:
        check(lib, Case(3, rows, ctx, Hq, Hkv, pad=2), "chunks", False)
    finally:
        lib.spec_set_option("persistent_grid", 0)


@both
@pytest.mark.parametrize("rows,ctx", [([3], [20000]), ([1, 1], [9000, 3]), ([1] * 5, [0, 0, 6000, 1, 4095])])
def test_long_contexts(lib, rows, ctx, few):
    check(lib, Case(4, rows, ctx, 8, 2), "long", few)


@both
def test_many_sequences(lib, few):
    """More sequences than lanes, some of them empty."""
    rng = np.random.default_rng(5)
    check(lib, Case(5, rng.integers(0, 5, 200).tolist(), rng.integers(0, 300, 200).tolist(), 8, 2, pad=3), "many", few)


@both
def test_empty_sequences_are_not_looked_at(lib, few):
    c = Case(6, [0, 2, 0, 1], [5, 40, 1, 130], 8, 2)
    c.ctx[0], c.ctx[2] = -5, 2 ** 31 - 1
    check(lib, c, "empty", few)
    c = Case(7, [0, 0], [0, 0], 8, 2, pad=4)
    check(lib, c, "nobody", few)


@both
@pytest.mark.parametrize("grid", [1, 3, 37, 600])
def test_grids(lib, grid, few):
    """Fewer and more CTAs than the chip holds: sequences in many pieces, sharers that run after one another."""
    lib.spec_set_option("persistent_grid", grid)
    try:
        check(lib, Case(8, [5, 1, 0, 7, 8], [0, 4000, 9, 130, 9000], 16, 2), f"grid {grid}", few)
    finally:
        lib.spec_set_option("persistent_grid", 0)


# --------------------------------------------------------------------------- scores and values
@both
@pytest.mark.parametrize("kind", ["peaked", "zero", "rising", "falling", "deep"])
def test_scores(lib, kind, few):
    c = Case(9, [6, 4, 1], [400, 126, 3000], 8, 2, q_std={"peaked": 30.0, "zero": 0.0}.get(kind, 1.0))
    if kind in ("rising", "falling", "deep"):
        sign = {"rising": 1, "falling": -1, "deep": -1}[kind]
        c.kp[:, :, :8192] = 0x11 * (8 + 7 * sign)                    # every whole number 7 or -7
        for b in range(3):
            for t in range(c.need[b]):
                c.kp[:, c.table[b, t], 8192:] = q4.scale_codes(4.0 * (t + 1 if kind != "deep" else c.need[b] - t) / 7)
        c.q[:] = synth.f32_to_bf16_bits(np.full(1, 1.0, np.float32))[0]
    check(lib, c, kind, few)


@both
@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0])
def test_scales(lib, scale, few):
    check(lib, Case(10, [5, 1], [10, 300], 8, 2), f"scale {scale}", few, scale=scale)


@both
@pytest.mark.parametrize("code", [0, 90, 255])
def test_sizes_of_values(lib, code, few):
    """The smallest and the largest values that the cache holds."""
    c = Case(11, [6, 2], [300, 2000], 8, 2, q_std=3.0)
    c.vp[:, :, 8192:] = code
    check(lib, c, f"values of scale {code}", few)


@both
def test_a_single_key_is_its_value(lib, few):
    """First tokens: one weight of 1, so the output is the stored value as it is, whatever the score."""
    c = Case(12, [1] * 9, [0] * 9, 8, 2, q_std=3.0)
    got = f64_of_bf16(run(lib, c, few)).reshape(9, 2, 4, D)
    v = q4.unpack(c.vp, False)
    want = np.stack([v[:, c.table[b, 0], 0] for b in range(9)])
    assert np.array_equal(got, np.broadcast_to(want[:, :, None], got.shape))


@both
def test_non_finite_queries_stay_in_their_rows(lib, few):
    """A NaN or an infinity in a query head reaches its own output only."""
    c = Case(13, [4, 2], [200, 900], 8, 2)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    c.q[1, 3 * D + 5], c.q[4, 7] = 0x7FC0, 0x7F80
    got = f64_of_bf16(run(lib, c, few)).reshape(ref.shape)
    clean = np.ones((c.M, 8), bool)
    clean[1, 3] = clean[4, 0] = False
    assert_attended(got[clean], ref[clean], mag[clean], "the other rows")
    assert np.isnan(got[1, 3]).all()


# --------------------------------------------------------------------------- use
@both
def test_strided_and_odd_buffers(lib, few):
    """Leading dimensions wider than the rows, outputs on odd 16-byte boundaries."""
    c = Case(14, [5, 3], [200, 0], 8, 2)
    cu, ctx, kp, vp, table = c.dev()
    Qw = torch.full((c.M, 8 * D + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    Qw[:, 8:8 + 8 * D] = bf16_dev(c.q)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    for at, width in ((16, 24), (8, 24)):
        Ow = torch.full((c.M, 8 * D + width), 5.0, dtype=torch.bfloat16, device="cuda")
        lib.spec_chunk_attention_paged_q4(Qw[:, 8:8 + 8 * D], cu, ctx, kp, vp, table, O=Ow[:, at:at + 8 * D],
                                          max_rows=5 if few else None)
        lib.spec_device_status()
        assert_attended(f64_of_bf16(Ow[:, at:at + 8 * D]).reshape(ref.shape), ref, mag, "strided")
        assert torch.all(Ow[:, :at] == 5.0) and torch.all(Ow[:, at + 8 * D:] == 5.0)


@both
def test_shared_prefix_pages(lib, few):
    c = Case(15, [6, 7], [256, 256], 8, 2)
    c.table[1, :2] = c.table[0, :2]
    check(lib, c, "shared pages", few)


def test_deterministic_on_one_workspace(lib):
    """The same bits on every call of one workspace, with other shapes and the other form in between."""
    ws = lib.Workspace("cuda")
    cases = [(Case(16, [7, 1], [3000, 5000], 32, 8), True), (Case(17, [400, 9], [0, 2500], 16, 8), False),
             (Case(18, [1], [30000], 8, 2), True), (Case(18, [1], [30000], 8, 2), False)]
    first = [bits_of(run(lib, c, few, ws=ws)) for c, few in cases]
    for _ in range(2):
        for (c, few), want in list(zip(cases, first))[::-1]:
            assert np.array_equal(bits_of(run(lib, c, few, ws=ws)), want)


@pytest.mark.parametrize("grid", [0, 600])
@pytest.mark.parametrize("Hq,Hkv,rows,ctx", [
    (4, 1, [1], [30000]), (8, 1, [2], [40000]), (48, 1, [1], [50000]), (16, 1, [3, 1], [20000, 25000]), (12, 2, [3], [9000])])
def test_items_of_many_pieces(lib, Hq, Hkv, rows, ctx, grid):
    """Few rows over a context that more than 32 slots share."""
    lib.spec_set_option("persistent_grid", grid)
    try:
        check(lib, Case(29, rows, ctx, Hq, Hkv), (rows, ctx, grid), True)
    finally:
        lib.spec_set_option("persistent_grid", 0)


@both
def test_a_page_twice_in_one_sequence(lib, few):
    """A table may name a page more than once: attention only reads."""
    c = Case(25, [5, 3], [800, 300], 8, 2)
    c.table[0, 4] = c.table[0, 1]
    c.table[1, 0] = c.table[1, 1] = c.table[0, 2]
    check(lib, c, "a page twice", few)


def test_two_graphs_in_turn_on_one_workspace(lib):
    """Both forms captured on one workspace, replayed in turn on one stream, and an eager call between them."""
    cases = [(Case(26, [7, 1], [3000, 5000], 32, 8), True), (Case(27, [300, 9], [0, 2500], 16, 8), False),
             (Case(28, [1, 2], [20000, 0], 8, 2), True)]
    ws = lib.Workspace("cuda", max(lib.spec_chunk_attention_q4_workspace_bytes(c.B, c.M, c.M, c.Hq, c.Hkv, D, c.max_pages)
                                   for c, _ in cases))
    held, graphs = [], []
    for c, few in cases:
        args = (bf16_dev(c.q), *c.dev())
        O = torch.zeros((c.M, c.Hq * D), dtype=torch.bfloat16, device="cuda")
        held.append((args, O))

        def call():
            lib.spec_chunk_attention_paged_q4(*args, O=O, ws=ws, max_rows=int(c.rows.max()) if few else None)
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    want = [bits_of(O) for _, O in held]
    for (c, _), (_, O) in zip(cases, held):
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, "before capture")
        O.fill_(3.0)
    for _ in range(4):
        for g in graphs:
            g.replay()
        lib.spec_chunk_attention_paged_q4(*held[0][0], O=held[0][1], ws=ws, max_rows=7)
    lib.spec_device_status()
    for w, (_, O) in zip(want, held):
        assert np.array_equal(bits_of(O), w)


@both
def test_bad_input_is_flagged(lib, few):
    c = Case(19, [5, 7, 3], [130, 40, 0], 8, 2, spare=1)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    for what in ("page", "length", "negative", "rows", "more rows"):
        cu, ctx, kp, vp, table = c.dev()
        most = 8 if few else c.M
        if what == "page":
            table[1, 0] = c.num_pages + 5
        elif what == "length":
            ctx[1] = c.max_pages * PAGE - 5
        elif what == "negative":
            ctx[1] = -3
        elif what == "rows":
            cu[3] = c.M + 1
        else:
            most = 6
        O = torch.full((c.M, 8 * D), 9.0, dtype=torch.bfloat16, device="cuda")
        lib.spec_chunk_attention_paged_q4(bf16_dev(c.q), cu, ctx, kp, vp, table, O=O, max_rows=most)
        rc, _ = lib.spec_device_status_code()
        assert rc == lib.SPEC_EINVAL, what
        lib.spec_device_status()
        got = f64_of_bf16(O).reshape(ref.shape)
        bad = 2 if what == "rows" else 1
        for b in range(3):
            sl = slice(c.cu[b], c.cu[b + 1])
            if b != bad:
                assert_attended(got[sl], ref[sl], mag[sl], f"{what}: sequence {b}")
            elif what != "page":
                assert np.all(got[sl] == 9.0), what


@both
def test_captured_and_replayed_with_other_lengths(lib, few):
    """One graph, replayed after the lengths, the table, the pools and the queries changed on the device."""
    big = Case(20, [4, 9, 1], [0, 1000, 9000], 8, 2)
    other = Case(21, [1, 7, 3], [8000, 0, 200], 8, 2)
    mp, npg = max(big.max_pages, other.max_pages), max(big.num_pages, other.num_pages)
    cu, ctx = dev(big.cu), dev(big.ctx)
    table = torch.zeros((3, mp), dtype=torch.int32, device="cuda")
    kp = torch.zeros((2, npg, BYTES), dtype=torch.uint8, device="cuda")
    vp, q = torch.zeros_like(kp), torch.zeros((14, 8 * D), dtype=torch.bfloat16, device="cuda")
    O = torch.zeros_like(q)
    most = 9 if few else 14
    ws = lib.Workspace("cuda", lib.spec_chunk_attention_q4_workspace_bytes(3, 14, most, 8, 2, D, mp))

    def load(c):
        cu.copy_(dev(c.cu)); ctx.copy_(dev(c.ctx)); table[:, :c.max_pages] = dev(c.table)
        kp[:, :c.num_pages] = dev(c.kp); vp[:, :c.num_pages] = dev(c.vp); q[:c.M] = bf16_dev(c.q)

    def call():
        lib.spec_chunk_attention_paged_q4(q, cu, ctx, kp, vp, table, O=O, ws=ws, max_rows=most)
    load(big)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in (other, big, other):
        load(c)
        O.fill_(4.0)
        graph.replay()
        lib.spec_device_status()
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        got = f64_of_bf16(O)
        assert_attended(got[:c.M].reshape(ref.shape), ref, mag, "replay")
        assert np.all(got[c.M:] == 4.0)


@both
def test_on_two_streams_at_once_with_workspaces_of_their_own(lib, few):
    cases = [Case(22, [6], [3000], 8, 2), Case(23, [2, 1], [0, 2000], 8, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(bf16_dev(c.q), *c.dev()) for c in cases]
    outs = [[torch.zeros((c.M, 8 * D), dtype=torch.bfloat16, device="cuda") for _ in range(6)] for c in cases]
    torch.cuda.synchronize()
    wss = [lib.Workspace("cuda") for _ in cases]
    for i in range(6):
        for c, a, w, o, s in zip(cases, args, wss, outs, streams):
            lib.spec_chunk_attention_paged_q4(*a, O=o[i], ws=w if i % 2 else None, stream=s,
                                              max_rows=int(c.rows.max()) if few else None)
    torch.cuda.synchronize()
    lib.spec_device_status()
    for c, out in zip(cases, outs):
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        for o in out:
            assert_attended(f64_of_bf16(o).reshape(ref.shape), ref, mag, "two streams")


@both
def test_pages_past_2_31_bytes(lib, few):
    pages = 260000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 5 GB")
    c = Case(24, [5, 4], [100, 300], 4, 1, extra=0)
    kp, vp = (lib.q4_pool(1, pages) for _ in range(2))
    far = np.array([pages - 1, 246724, 246723, 3, 250000], np.int64)[:c.num_pages]
    for pool, src in ((kp, c.kp), (vp, c.vp)):
        pool[:, torch.from_numpy(far).cuda()] = dev(src)
    table = np.where(c.table >= 0, far[np.maximum(c.table, 0)], 0).astype(np.int32)
    O = lib.spec_chunk_attention_paged_q4(bf16_dev(c.q), dev(c.cu), dev(c.ctx), kp, vp, dev(table),
                                          max_rows=5 if few else None)
    lib.spec_device_status()
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, "far pages")


def test_binding_refuses_wrong_tensors(lib):
    c = Case(25, [2], [0], 4, 2)
    cu, ctx, kp, vp, table = c.dev()
    q = bf16_dev(c.q)
    call = lib.spec_chunk_attention_paged_q4
    for bad in (lambda: call(q.float(), cu, ctx, kp, vp, table), lambda: call(q, cu, ctx, kp.view(torch.int8), vp, table),
                lambda: call(q, cu.long(), ctx, kp, vp, table)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: call(q[:, :100], cu, ctx, kp, vp, table), lambda: call(q, cu, ctx, kp[:, :, :8192], vp, table),
                lambda: call(q, cu, ctx, kp[:, :1], vp, table), lambda: call(q, cu, ctx[:0], kp, vp, table),
                lambda: call(q, cu, ctx, kp, vp, table, O=q[:1]), lambda: call(q, cu, ctx, kp[:, ::2], vp[:, ::2], table)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.SpecError):
        call(q, cu, ctx, kp, vp, table, max_rows=0)


# --------------------------------------------------------------------------- together
@both
def test_prompt_then_rounds(lib, few):
    """Two prompts appended (normed, rotated, quantised) and attended in uneven chunks, then rounds of a few rows of which
    not all are kept, as a verify loop does: every output is attention over what the cache reads back."""
    Hq, Hkv = 8, 2
    hq, hk = Hq * D, Hkv * D
    rng = np.random.default_rng(26)
    table = dev(rng.permutation(9)[:8].reshape(2, 4).astype(np.int32))
    kp, vp = (lib.q4_pool(Hkv, 9) for _ in range(2))
    kp.fill_(255); vp.fill_(255)
    wq, wk = (bf16_dev(synth.f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))) for _ in range(2))
    ws = lib.Workspace("cuda")
    ctx = np.zeros(2, np.int32)
    for rows, keep in (([200, 1], [200, 1]), ([0, 150], [0, 150]), ([5, 3], [2, 3]), ([1, 5], [1, 1]), ([4, 4], [4, 1])):
        M = sum(rows)
        cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        x = bf16_dev(synth.normal_bf16_bits(int(ctx.sum()) + 7, (M, hq + 2 * hk), 1.5))
        cs = lib.spec_rope_table(dev(cu), dev(ctx), M, D, 1e6)
        q = lib.spec_kv_append_paged_q4(x[:, hq:hq + hk], x[:, hq + hk:], dev(cu), dev(ctx), kp, vp, table, cs=cs, Q=x[:, :hq],
                                        wq=wq, wk=wk)
        O = lib.spec_chunk_attention_paged_q4(q, dev(cu), dev(ctx), kp, vp, table, ws=ws,
                                              max_rows=max(rows) if few else None)
        lib.spec_device_status()
        n = ctx + np.array(rows)
        call = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        K, V = (f64_of_bf16(t).reshape(-1, Hkv, D) for t in
                lib.spec_kv_read_paged_q4(dev(call), dev(np.zeros(2, np.int32)), kp, vp, table, int(n.sum())))
        pools = np.zeros((2, Hkv, 8, PAGE, D))
        one = np.arange(8).reshape(2, 4)
        kk, vv = oprompt.kv_append(K, V, call, [0, 0], *pools, one)
        ref, mag = oprompt.chunk_attention(f64_of_bf16(q).reshape(M, Hq, D), cu, ctx, kk, vv, one, 1.0 / np.sqrt(D))
        assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, f"rows {rows}")
        ctx = (ctx + np.array(keep)).astype(np.int32)
