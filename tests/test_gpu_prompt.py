"""GPU parity of the prompt-side operators (rotation table of several axes, rotated append to the paged
cache, attention of a chunk over it) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import synth
from oracle import bf16 as obf, ops as oops, prompt as oprompt

from gpu_util import bf16_dev, bits_of, dev, f64_of_bf16

pytestmark = pytest.mark.gpu
PAGE, D = 128, 128
HALF_BF16 = 2.0 ** -8       # half a bf16 step, relative to the value
HALF_F32 = 2.0 ** -24

# Table: one rounding of a cosine or sine (<= 1) by a function good to 2 units in the last place (2 half
# steps of 2^-24 each), the rounded reduced angle (<= pi/4, half a step of it), the turn truncated to
# 32 bits, and the fp64 frequency on both sides (2^-52 of the whole angle).
def table_tol(max_angle):
    return (1 + 2 * 2 + np.pi / 4) * HALF_F32 + 2 * np.pi * 2.0 ** -32 + max_angle * 2.0 ** -51


def assert_rotated(got, ref, mag, what):
    """Two fp32 products, their sum (three half steps of the summed magnitudes), one bf16 rounding."""
    bound = HALF_BF16 * abs(ref) + (1 + HALF_BF16) * 3 * HALF_F32 * mag
    bad = abs(got - ref) > bound
    assert np.all(np.isfinite(got)) and not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance"


def assert_attended(got, ref, mag, what):
    """One bf16 rounding of the output; the weights' bf16 rounding, of each term that is summed; 2^-10 of
    the terms for what stays in 32 bits (scores of 128 products, the exponential, two sums)."""
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bound = HALF_BF16 * abs(ref) + (HALF_BF16 + 2.0 ** -10) * mag
    err = abs(got - ref)
    bad = err > bound
    if bad.any():
        i = np.unravel_index(np.argmax(err - bound), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of tolerance; worst at {i}: got {got[i]!r} "
                             f"ref {ref[i]!r} magnitude {mag[i]!r}")


class Case:
    """Ragged batch over a paged cache: random pages, noise in every unused row and page."""

    def __init__(self, seed, rows, ctx, Hq, Hkv, q_std=1.0, pad=0, extra=3, spare=0, poison=False):
        rng = np.random.default_rng(seed)
        self.rows, self.ctx = np.asarray(rows, np.int32), np.asarray(ctx, np.int32)
        self.B, self.Hq, self.Hkv = len(rows), Hq, Hkv
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.M = int(self.cu[-1])
        self.Mp = self.M + pad
        need = [max(0, int(c + n + PAGE - 1) // PAGE) for c, n in zip(ctx, rows)]
        self.need, self.max_pages = need, max(max(need), 1) + spare
        self.num_pages = sum(need) + extra
        perm = rng.permutation(self.num_pages)
        # entries past a sequence's last page hold ids that do not exist
        self.table = np.full((self.B, self.max_pages), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.kp = synth.normal_bf16_bits(seed + 1, (Hkv, self.num_pages, PAGE, D), 1.0)
        self.vp = synth.normal_bf16_bits(seed + 2, (Hkv, self.num_pages, PAGE, D), 1.0)
        self.used = np.zeros((self.num_pages, PAGE), bool)
        for b in range(self.B):
            n = int(ctx[b] + rows[b]) if rows[b] else 0
            for t in range((n + PAGE - 1) // PAGE):
                self.used[self.table[b, t], :min(PAGE, n - t * PAGE)] = True
        if poison:           # whatever no sequence's keys occupy: NaN and infinities
            nan = np.where(rng.random((Hkv, self.num_pages, PAGE, D)) < 0.5, 0x7FC0, 0x7F80).astype(np.uint16)
            self.kp = np.where(self.used[None, :, :, None], self.kp, nan)
            self.vp = np.where(self.used[None, :, :, None], self.vp, nan)
        self.q = synth.normal_bf16_bits(seed + 3, (self.Mp, Hq * D), q_std)
        if pad:
            self.q[self.M:] = 0x7FC0

    def dev(self):
        return (dev(self.cu), dev(self.ctx), bf16_dev(self.kp).clone(), bf16_dev(self.vp).clone(), dev(self.table))

    def oracle(self, scale):
        kp, vp = (np.where(self.used[None, :, :, None], obf.decode(x), 0.0) for x in (self.kp, self.vp))
        q = obf.decode(self.q[:self.M]).reshape(self.M, self.Hq, D)
        return oprompt.chunk_attention(q, self.cu, self.ctx, kp, vp, self.table, scale)


def run_attention(lib, c, scale=None, ws=None, O=None):
    cu, ctx, kp, vp, table = c.dev()
    O = lib.spec_chunk_attention_paged(bf16_dev(c.q), cu, ctx, kp, vp, table, scale=scale, ws=ws, O=O)
    lib.spec_device_status()
    assert np.array_equal(bits_of(kp), c.kp) and np.array_equal(bits_of(vp), c.vp)     # reads only
    return O


def check_attention(lib, c, what, scale=None, ws=None):
    O = torch.full((c.Mp, c.Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    run_attention(lib, c, scale, ws, O)
    ref, mag = c.oracle(1.0 / np.sqrt(D) if scale is None else scale)
    got = f64_of_bf16(O)
    assert np.all(got[c.M:] == 7.0), f"{what}: padding rows written"
    assert_attended(got[:c.M].reshape(ref.shape), ref, mag, what)
    return O


# --------------------------------------------------------------------------- rotation table
@pytest.mark.parametrize("M,sections,D_,il", [
    (1, [64], 128, False), (77, [16, 24, 24], 128, False), (301, [24, 20, 20], 128, True), (5, [0, 64], 128, False),
    (33, [22, 21, 21], 128, True), (9, [3], 6, False), (40, [1, 2, 3, 4, 5, 6, 7, 8], 72, False),
    (130, [44, 42, 42], 256, True), (3, [64, 0, 0], 128, True), (7, [1], 2, True),
])
def test_table_axes(lib, M, sections, D_, il):
    rng = np.random.default_rng(M)
    pos = rng.integers(-5, 200000, (len(sections), M)).astype(np.int32)
    pos[0, 0] = 0
    wide = torch.full((len(sections), M + 3), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :M] = dev(pos)
    cs = lib.spec_rope_table_axes(wide[:, :M], sections, D_, 1e6, interleaved=il)
    ref = oprompt.rope_table_axes(pos, sections, D_, 1e6, il)
    err = abs(cs.cpu().numpy().astype(np.float64) - ref)
    assert err.max() <= table_tol(2e5), err.max()


def test_table_axes_far_positions_and_theta(lib):
    """Positions to the ends of 32 bits; theta below one (frequencies above one turn per position)."""
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789, -1]], np.int32)
    for theta in (1e4, 1.0, 0.25):
        cs = lib.spec_rope_table_axes(dev(pos), [4], 8, theta).cpu().numpy().astype(np.float64)
        top = 2.0 ** 31 * max(1.0, float(theta) ** -0.75)
        # (the fp64 angle itself is good to 2^-53 of the angle only)
        assert abs(cs - oprompt.rope_table_axes(pos, [4], 8, theta, False)).max() <= table_tol(top)


def test_table_axes_equals_plain_table_on_text(lib):
    batch = synth.RaggedBatch([4, 0, 10], [8190, 0, 333])
    plain = lib.spec_rope_table(dev(batch.cu_rows), dev(batch.ctx_len), batch.M, 128, 1e6)
    pos = np.concatenate([batch.ctx_len[b] + np.arange(batch.gammas[b] + 1) for b in range(batch.B)]).astype(np.int32)
    axes = lib.spec_rope_table_axes(dev(np.stack([pos] * 3)), [16, 24, 24], 128, 1e6)
    assert (plain - axes).abs().max().item() <= 2 * table_tol(8200)


# --------------------------------------------------------------------------- append
APPEND = [
    ([1], [0], 32, 8), ([1, 1, 1], [127, 128, 300], 32, 8), ([300, 0, 1, 129], [100, 50, 255, 0], 16, 8),
    ([40], [88], 5, 1), ([2, 3], [0, 126], 28, 4), ([0, 0, 7], [0, 0, 121], 3, 3), ([5] * 40, list(range(100, 140)), 8, 2),
    ([900, 0, 1, 640], [100, 5, 300, 0], 28, 4), ([1, 1600], [7, 50], 5, 1),
]


@pytest.mark.parametrize("rows,ctx,Hq,Hkv", APPEND)
@pytest.mark.parametrize("mode", ["out", "inplace", "kv", "copy"])
def test_append(lib, rows, ctx, Hq, Hkv, mode):
    """Rotated queries into another buffer, in place, none, and keys that are rotated already."""
    c = Case(11, rows, ctx, Hq, Hkv, pad=3, poison=True)
    hq, hk = Hq * D, Hkv * D
    x_bits = synth.normal_bf16_bits(5, (c.Mp, hq + 2 * hk), 1.0)
    x_bits[c.M:] = 0x7FC0                                   # padding
    x = bf16_dev(x_bits).clone()
    cs_h = np.random.default_rng(3).uniform(-1, 1, (c.Mp, 64, 2)).astype(np.float32)
    cu, ctx_d, kp, vp, table = c.dev()
    rotate = mode != "copy"
    q = x[:, :hq] if mode in ("out", "inplace") else None
    qrot = torch.full((c.Mp, hq + 8), 3.0, dtype=torch.bfloat16, device="cuda") if mode == "out" else None
    got_q = lib.spec_kv_append_paged(x[:, hq:hq + hk], x[:, hq + hk:], cu, ctx_d, kp, vp, table,
                                     cs=dev(cs_h) if rotate else None, Q=q,
                                     Qrot=qrot[:, :hq] if mode == "out" else None)
    lib.spec_device_status()
    dec = obf.decode(x_bits[:c.M])
    k = dec[:, hq:hq + hk].reshape(c.M, Hkv, D)
    v = dec[:, hq + hk:].reshape(c.M, Hkv, D)
    cs64 = cs_h[:c.M].astype(np.float64)
    k_ref, k_mag = oprompt.rotate(k, cs64) if rotate else (k, 0 * k)
    kp_b, vp_b = bits_of(kp), bits_of(vp)
    hit = np.zeros((c.num_pages, PAGE), bool)
    for b in range(c.B):
        for j in range(rows[b]):
            p, r = ctx[b] + j, c.cu[b] + j
            page = c.table[b, p // PAGE]
            hit[page, p % PAGE] = True
            assert np.array_equal(vp_b[:, page, p % PAGE], x_bits[r, hq + hk:].reshape(Hkv, D))
            got = obf.decode(kp_b[:, page, p % PAGE])
            assert_rotated(got, k_ref[r], k_mag[r], "append keys")
    # every other row of the pools is as it was
    assert np.array_equal(kp_b[:, ~hit], c.kp[:, ~hit]) and np.array_equal(vp_b[:, ~hit], c.vp[:, ~hit])
    if q is not None:
        ref, mag = oprompt.rotate(dec[:, :hq].reshape(c.M, Hq, D), cs64)
        g = f64_of_bf16(got_q[:c.M]).reshape(ref.shape)
        assert_rotated(g, ref, mag, "append queries")
        if mode == "out":
            assert torch.all(qrot[c.M:] == 3.0) and torch.all(qrot[:, hq:] == 3.0)
    if mode != "inplace":
        assert np.array_equal(bits_of(x), x_bits)
    else:
        assert np.array_equal(bits_of(x)[:, hq:], x_bits[:, hq:]) and np.array_equal(bits_of(x)[c.M:], x_bits[c.M:])


def test_append_bad_pages_and_lengths_are_flagged(lib):
    """A page id that does not exist: that row is not written.  A sequence past the table, and one past
    the buffers' rows: skipped whole.  The others go on."""
    c = Case(21, [2, 3, 4], [127, 300, 10], 8, 2, spare=1)
    hk = 2 * D
    kv = bf16_dev(synth.normal_bf16_bits(6, (c.M, 2 * hk), 1.0))
    for what in ("page", "length", "negative", "rows"):
        table, ctx, cu = c.table.copy(), c.ctx.copy(), c.cu.copy()
        if what == "page":
            table[0, 1] = c.num_pages                       # the second row of sequence 0
        elif what == "length":
            ctx[1] = c.max_pages * PAGE - 2
        elif what == "negative":
            ctx[1] = -1
        else:
            cu[3] = c.M + 1
        kp, vp = bf16_dev(c.kp).clone(), bf16_dev(c.vp).clone()
        lib.spec_kv_append_paged(kv[:, :hk], kv[:, hk:], dev(cu), dev(ctx), kp, vp, dev(table))
        rc, _ = lib.spec_device_status_code()
        assert rc == lib.SPEC_EINVAL
        ref_k = c.kp.copy()
        bits = bits_of(kv)
        for b in range(3):
            if (b == 1 and what in ("length", "negative")) or (b == 2 and what == "rows"):
                continue
            for j in range(c.rows[b]):
                p = c.ctx[b] + j
                if what == "page" and b == 0 and p >= PAGE:
                    continue
                ref_k[:, c.table[b, p // PAGE], p % PAGE] = bits[c.cu[b] + j, :hk].reshape(2, D)
        assert np.array_equal(bits_of(kp), ref_k), what
        lib.spec_device_status()


# --------------------------------------------------------------------------- chunk attention
HEADS = [(32, 8), (16, 8), (4, 4), (28, 4), (5, 1), (16, 1), (12, 4)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("rows,ctx", [
    ([1], [0]), ([1, 1, 1, 1], [0, 127, 128, 511]), ([127], [0]), ([128], [0]), ([129], [0]), ([64], [64]),
    ([33, 0, 1, 200, 5], [0, 50, 1000, 127, 128]), ([300], [85]),
])
def test_attention(lib, Hq, Hkv, rows, ctx):
    check_attention(lib, Case(31, rows, ctx, Hq, Hkv, pad=2, spare=1, poison=True), f"{Hq}/{Hkv} {rows} {ctx}")


@pytest.mark.parametrize("Hq,Hkv,rows,ctx", [
    (128, 1, [3, 1], [200, 0]), (100, 1, [5], [130]), (65, 1, [9, 2], [0, 300]), (33, 1, [20], [100]),
    (2, 2, [700], [0]), (1, 1, [513, 1], [3, 4]), (64, 2, [17, 40], [250, 1]),
])
def test_attention_odd_groups(lib, Hq, Hkv, rows, ctx):
    check_attention(lib, Case(32, rows, ctx, Hq, Hkv, poison=True), f"{Hq}/{Hkv}")


@pytest.mark.parametrize("rows,ctx", [([3], [20000]), ([1, 1], [9000, 3]), ([70, 1, 1], [4000, 7000, 129]),
                                      ([1], [33000]), ([65], [6000])])
def test_attention_long_contexts(lib, rows, ctx):
    """Few rows behind long contexts: one sequence's keys are shared between many blocks."""
    check_attention(lib, Case(33, rows, ctx, 8, 2, poison=True), f"{rows} at {ctx}")


def test_attention_one_item_for_all(lib):
    """One row tile over a long cache: shares longer than an even cut's, most CTAs without any."""
    check_attention(lib, Case(66, [9], [40100], 5, 1, poison=True), "one item")


def test_attention_many_sequences(lib):
    rng = np.random.default_rng(4)
    rows = [int(x) for x in rng.integers(0, 4, 700)]
    ctx = [int(x) for x in rng.integers(0, 160, 700)]
    check_attention(lib, Case(34, rows, ctx, 4, 1, poison=True), "700 sequences")


def test_empty_sequences_are_not_looked_at(lib):
    """Slots without rows whose lengths (and pages) mean nothing."""
    c = Case(67, [0, 3, 0, 40, 0], [0, 130, 0, 7, 0], 8, 2)
    c.ctx[[0, 2, 4]] = [-5, 1 << 30, 128 * c.max_pages + 1]
    check_attention(lib, c, "empty sequences")
    cu, ctx, kp, vp, table = c.dev()
    kv = bf16_dev(synth.normal_bf16_bits(68, (c.M, 4 * D), 1.0))
    lib.spec_kv_append_paged(kv[:, :2 * D], kv[:, 2 * D:], cu, ctx, kp, vp, table)
    lib.spec_device_status()


def test_attention_padded_batch(lib):
    """Hundreds of slots without rows between the sequences that have some."""
    rows = [0] * 900
    rows[3], rows[4], rows[500], rows[897] = 1, 70, 2, 1
    ctx = [(11 * b) % 300 for b in range(900)]
    ctx[3], ctx[897] = 2000, 1000
    check_attention(lib, Case(65, rows, ctx, 8, 2, poison=True), "padded batch")


def test_attention_all_sequences_empty(lib):
    check_attention(lib, Case(35, [0, 0], [5, 0], 4, 1, pad=4), "no rows")


@pytest.mark.parametrize("q_std,rising", [(30.0, False), (1.0, True), (0.0, False)])
def test_attention_extreme_scores(lib, q_std, rising):
    """Peaked rows; scores that rise by far more than 2^8 from tile to tile (every tile raises the maximum);
    equal scores."""
    c = Case(36, [90, 2], [400, 777], 8, 2, q_std=q_std)
    if rising:
        for b in range(2):
            for t in range(c.need[b]):
                c.kp[:, c.table[b, t]] = synth.f32_to_bf16_bits(np.full(1, 4.0 * (t + 1), np.float32))[0]
        c.q[:] = synth.f32_to_bf16_bits(np.full(1, 1.0, np.float32))[0]
    check_attention(lib, c, f"q_std {q_std} rising {rising}")


@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0])
def test_attention_scales(lib, scale):
    check_attention(lib, Case(37, [50, 1], [10, 300], 8, 2), f"scale {scale}", scale=scale)


def test_attention_strided_buffers(lib):
    c = Case(38, [50, 3], [200, 0], 8, 2)
    cu, ctx, kp, vp, table = c.dev()
    Qw = torch.full((c.M, 8 * D + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    Qw[:, 8:8 + 8 * D] = bf16_dev(c.q)
    Ow = torch.full((c.M, 8 * D + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    lib.spec_chunk_attention_paged(Qw[:, 8:8 + 8 * D], cu, ctx, kp, vp, table, O=Ow[:, 16:16 + 8 * D])
    lib.spec_device_status()
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    assert_attended(f64_of_bf16(Ow[:, 16:16 + 8 * D]).reshape(ref.shape), ref, mag, "strided")
    assert torch.all(Ow[:, :16] == 5.0) and torch.all(Ow[:, 16 + 8 * D:] == 5.0)


def test_attention_shared_prefix_pages(lib):
    """Two sequences read the same pages for their common prefix."""
    c = Case(39, [10, 20], [256, 256], 8, 2)
    c.table[1, :2] = c.table[0, :2]
    check_attention(lib, c, "shared pages")


def test_attention_is_deterministic_and_reuses_its_workspace(lib):
    """The same bits on every call of one workspace, with other shapes in between."""
    ws = lib.Workspace("cuda")
    a, b = Case(40, [70, 1], [3000, 5000], 32, 8), Case(41, [400, 9], [0, 2500], 16, 8)
    first = [bits_of(run_attention(lib, x, ws=ws)) for x in (a, b)]
    for _ in range(2):
        for x, want in ((b, first[1]), (a, first[0])):
            assert np.array_equal(bits_of(run_attention(lib, x, ws=ws)), want)


def test_attention_bad_input_is_flagged(lib):
    c = Case(42, [5, 200, 3], [130, 40, 0], 8, 2, spare=1)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    for what in ("page", "length", "negative", "rows"):
        cu, ctx, kp, vp, table = c.dev()
        if what == "page":
            table[1, 0] = c.num_pages + 5
        elif what == "length":
            ctx[1] = c.max_pages * PAGE - 100
        elif what == "negative":
            ctx[1] = -3
        else:
            cu[3] = c.M + 1
        O = torch.full((c.M, 8 * D), 9.0, dtype=torch.bfloat16, device="cuda")
        lib.spec_chunk_attention_paged(bf16_dev(c.q), cu, ctx, kp, vp, table, O=O)
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


def test_attention_captured_and_replayed_with_other_lengths(lib):
    """One graph, replayed after the lengths, the table and the queries changed on the device."""
    big = Case(43, [40, 300, 1], [0, 100, 900], 8, 2, spare=0)
    other = Case(44, [1, 7, 333], [1000, 0, 200], 8, 2)
    mp, npg = max(big.max_pages, other.max_pages), max(big.num_pages, other.num_pages)
    cu, ctx = dev(big.cu), dev(big.ctx)
    table = torch.zeros((3, mp), dtype=torch.int32, device="cuda")
    kp = torch.zeros((2, npg, PAGE, D), dtype=torch.bfloat16, device="cuda")
    vp, q = torch.zeros_like(kp), torch.zeros((341, 8 * D), dtype=torch.bfloat16, device="cuda")
    O = torch.zeros_like(q)
    ws = lib.Workspace("cuda", lib.spec_chunk_attention_workspace_bytes(3, 341, 8, 2, D, mp))

    def load(c):
        cu.copy_(dev(c.cu)); ctx.copy_(dev(c.ctx)); table[:, :c.max_pages] = dev(c.table)
        kp[:, :c.num_pages] = bf16_dev(c.kp); vp[:, :c.num_pages] = bf16_dev(c.vp); q[:c.M] = bf16_dev(c.q)

    load(big)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, O=O, ws=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, O=O, ws=ws)
    for c in (other, big, other):
        load(c)
        O.fill_(4.0)
        graph.replay()
        lib.spec_device_status()
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        got = f64_of_bf16(O)
        assert_attended(got[:c.M].reshape(ref.shape), ref, mag, "replay")
        assert np.all(got[c.M:] == 4.0)


def test_attention_on_two_streams_at_once(lib):
    """Calls that overlap on two streams, each with its own workspace."""
    cases = [Case(45, [60], [3000], 8, 2), Case(46, [200, 1], [0, 2000], 8, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(bf16_dev(c.q), *c.dev()) for c in cases]
    wss = [lib.Workspace("cuda", lib.spec_chunk_attention_workspace_bytes(c.B, c.M, 8, 2, D, c.max_pages)) for c in cases]
    outs = [[torch.zeros((c.M, 8 * D), dtype=torch.bfloat16, device="cuda") for _ in range(6)] for c in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for a, w, o, s in zip(args, wss, outs, streams):
            lib.spec_chunk_attention_paged(a[0], a[1], a[2], a[3], a[4], a[5], O=o[i], ws=w, stream=s)
    torch.cuda.synchronize()
    lib.spec_device_status()
    for c, out in zip(cases, outs):
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        for o in out:
            assert_attended(f64_of_bf16(o).reshape(ref.shape), ref, mag, "two streams")


def test_binding_refuses_wrong_tensors(lib):
    c = Case(47, [2], [0], 4, 2)
    cu, ctx, kp, vp, table = c.dev()
    q = bf16_dev(c.q)
    with pytest.raises(TypeError):
        lib.spec_chunk_attention_paged(q.float(), cu, ctx, kp, vp, table)
    with pytest.raises(ValueError):
        lib.spec_chunk_attention_paged(q[:, :100], cu, ctx, kp, vp, table)
    with pytest.raises(ValueError):
        lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table[:, :0].repeat(2, 1))
    with pytest.raises(ValueError):
        lib.spec_kv_append_paged(q[:, :D], q[:, :D], cu, ctx, kp, vp, table)
    with pytest.raises(lib.SpecError):
        lib.spec_kv_append_paged(q[:, :2 * D], q[:, :2 * D], cu, ctx, kp, vp, table, Q=q)     # no table
    with pytest.raises(ValueError):
        lib.spec_rope_table_axes(torch.zeros((2, 3), dtype=torch.int32, device="cuda"), [64], 128)


@pytest.mark.parametrize("falling", [True, False])
def test_attention_scores_far_below_zero(lib, falling):
    """Every score far below 0 (no weight near 1 until the row's reference is taken), falling or rising from tile to
    tile; rows of one item that see a tile that others do not."""
    c = Case(60, [90, 4, 1], [400, 126, 3000], 8, 2)
    for b in range(3):
        for t in range(c.need[b]):
            k = -4.0 * (t + 1 if falling else c.need[b] - t)
            c.kp[:, c.table[b, t]] = synth.f32_to_bf16_bits(np.full(1, k, np.float32))[0]
    c.q[:] = synth.f32_to_bf16_bits(np.full(1, 1.0, np.float32))[0]
    check_attention(lib, c, f"falling {falling}")


def test_attention_of_a_single_key_is_its_value(lib):
    """First tokens: one weight, whatever the score (the weight enters the product as bf16, so it has to be 1)."""
    c = Case(64, [1] * 9, [0] * 9, 8, 2, q_std=3.0)
    got = bits_of(run_attention(lib, c)).reshape(9, 2, 4, D)
    want = np.stack([c.vp[:, c.table[b, 0], 0] for b in range(9)])
    assert np.array_equal(got, np.broadcast_to(want[:, :, None], got.shape))


@pytest.mark.parametrize("size", [1e25, 1e-15])
def test_attention_values_far_from_one(lib, size):
    c = Case(61, [130, 2], [300, 2000], 8, 2, q_std=6.0)
    c.vp = synth.f32_to_bf16_bits((obf.decode(c.vp) * size).astype(np.float32))
    check_attention(lib, c, f"values of {size}")


@pytest.mark.parametrize("rows,ctx,Hq,Hkv", [
    ([500] * 8, [0] * 8, 8, 2), ([130, 0] * 16, [(37 * b) % 500 for b in range(32)], 4, 4), ([2048], [0], 16, 8),
    ([1, 600, 257, 256, 255], [255, 0, 128, 127, 130], 28, 4), ([700], [1], 16, 1),
    ([130, 1, 0, 77] * 12, [(53 * b) % 300 for b in range(48)], 8, 2), ([90] * 33, [0] * 33, 8, 2),
    (list(range(10, 202, 3)), [200 - 3 * b for b in range(64)], 5, 1)])
def test_attention_many_items(lib, rows, ctx, Hq, Hkv):
    """Prompts whose items outnumber the CTAs, with equal and unequal lengths; and on a few CTAs."""
    c = Case(63, rows, ctx, Hq, Hkv, poison=True, pad=2)
    check_attention(lib, c, "many items")
    lib.spec_set_option("persistent_grid", 5)
    try:
        check_attention(lib, c, "many items on 5 CTAs")
    finally:
        lib.spec_set_option("persistent_grid", 0)


@pytest.mark.parametrize("grid", [1, 3, 37, 600])
def test_attention_grids(lib, grid):
    """Fewer and more CTAs than the chip holds: whole items, items in hundreds of pieces, sharers that run after
    one another."""
    lib.spec_set_option("persistent_grid", grid)
    try:
        check_attention(lib, Case(62, [300, 1, 0, 7, 61], [0, 4000, 9, 130, 9000], 8, 2, poison=True), f"grid {grid}")
    finally:
        lib.spec_set_option("persistent_grid", 0)


# --------------------------------------------------------------------------- together
def test_prompt_in_chunks_then_verify(lib):
    """Two sequences' prompts in three uneven chunks through table, append and chunk attention, then a verify
    call on the same pages: every output is that of attention over the whole prompt."""
    Hq, Hkv, n = 8, 2, [301, 170]
    hq, hk = Hq * D, Hkv * D
    rng = np.random.default_rng(8)
    table = rng.permutation(7)[:6].reshape(2, 3).astype(np.int32)
    kp = torch.full((Hkv, 7, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    x_bits = [synth.normal_bf16_bits(50 + b, (n[b], hq + 2 * hk), 1.0) for b in range(2)]
    cuts = [(0, 0), (1, 128), (200, 129), (297, 166)]
    ws = lib.Workspace("cuda")
    got = [[], []]
    for i in range(3):
        at, to = cuts[i], cuts[i + 1]
        rows = [to[b] - at[b] for b in range(2)]
        cu, ctx = np.array([0, rows[0], sum(rows)], np.int32), np.array(at, np.int32)
        x = bf16_dev(np.concatenate([x_bits[b][at[b]:to[b]] for b in range(2)])).clone()
        pos = np.concatenate([np.arange(at[b], to[b]) for b in range(2)]).astype(np.int32)
        cs = lib.spec_rope_table_axes(dev(np.stack([pos] * 3)), [24, 20, 20], D, 1e6, interleaved=True)
        q = lib.spec_kv_append_paged(x[:, hq:hq + hk], x[:, hq + hk:], dev(cu), dev(ctx), kp, vp, dev(table), cs=cs,
                                     Q=x[:, :hq])
        O = f64_of_bf16(lib.spec_chunk_attention_paged(q, dev(cu), dev(ctx), kp, vp, dev(table), ws=ws))
        got[0].append(O[:rows[0]])
        got[1].append(O[rows[0]:])
    # the last rows of both as a verify block, rotated by spec_rope
    rows = [n[b] - cuts[3][b] for b in range(2)]
    cu, ctx = np.array([0, rows[0], sum(rows)], np.int32), np.array(cuts[3], np.int32)
    x = bf16_dev(np.concatenate([x_bits[b][cuts[3][b]:] for b in range(2)])).clone()
    lib.spec_rope(x[:, :hq], x[:, hq:hq + hk], dev(cu), dev(ctx), D, 1e6)
    O = f64_of_bf16(lib.spec_verify_attention_paged(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], dev(cu), dev(ctx), kp,
                                                    vp, dev(table), max(rows)))
    got[0].append(O[:rows[0]])
    got[1].append(O[rows[0]:])
    lib.spec_device_status()
    for b in range(2):
        x = obf.decode(x_bits[b])
        pos = np.arange(n[b])
        q, k = (obf.round_to_bf16(oops.rope(t.reshape(n[b], -1, D), pos, 1e6)) for t in (x[:, :hq], x[:, hq:hq + hk]))
        v = x[:, hq + hk:].reshape(n[b], Hkv, D)
        z = np.zeros((Hkv, 3, PAGE, D))
        cu1, one = np.array([0, n[b]]), np.array([[0, 1, 2]])
        kk, vv = oprompt.kv_append(k, v, cu1, [0], z, z, one)
        ref, mag = oprompt.chunk_attention(q, cu1, [0], kk, vv, one, 1.0 / np.sqrt(D))
        # q and k rounded to bf16 from an fp32 rotation may land one step from the fp64 rotation's: a step of
        # either moves a score by up to 2^-7 of its products' magnitude sum, so the weights are held to
        # 2^-4 here and the attention's own tests hold them to theirs
        g = np.concatenate(got[b]).reshape(ref.shape)
        assert np.all(abs(g - ref) <= HALF_BF16 * abs(ref) + 2.0 ** -4 * mag)


# --------------------------------------------------------------------------- the weights' reference
def test_attention_largest_weight_is_not_rounded(lib):
    """Rows of 8 to 128 keys: the largest weight enters the product exactly, so what is left are the output's rounding
    and the other weights'.  A rounding to bf16 of values spread over the octaves errs by a uniform
    +-2^-8 / m for a mantissa m, 1 <= m < 2, of density 1 / (m ln 2): its mean square is (2^-7)^2 / 12 * (3/8) / ln 2.
    The errors are independent and their squares add up; a tenth above the sum is far outside what 150000
    outputs can deviate by (the largest weight's rounding would add half of it)."""
    c = Case(70, [1] * 150, [7 + (37 * b) % 121 for b in range(150)], 8, 2, q_std=2.0)
    got = f64_of_bf16(run_attention(lib, c)).reshape(c.M, 8, D)
    ref, _ = c.oracle(1.0 / np.sqrt(D))
    step2 = 2.0 ** -14 / 12 * 0.375 / np.log(2)
    q = obf.decode(c.q).reshape(c.M, 2, 4, D)
    others = 0.0
    for b in range(c.B):
        page, n = c.table[b, 0], c.ctx[b] + 1
        k, v = (obf.decode(x[:, page, :n]) for x in (c.kp, c.vp))
        s = np.einsum("ghd,gkd->ghk", q[b], k) / np.sqrt(D)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        np.put_along_axis(w, w.argmax(-1)[..., None], 0.0, -1)
        others += np.einsum("ghk,gkd->", w ** 2, v ** 2)
    assert ((got - ref) ** 2).sum() <= 1.1 * step2 * ((ref ** 2).sum() + others)


@pytest.mark.parametrize("size", [1e-30, 1e-25, 1.0])
def test_attention_scores_below_zero_with_small_values(lib, size):
    """Scores about -28 (2^-41 as a weight relative to 0) and values down to 1e-30: their products must not leave fp32."""
    c = Case(71, [130, 2, 1, 40], [0, 500, 2000, 90], 8, 2)
    c.kp[:] = synth.f32_to_bf16_bits((obf.decode(c.kp) * 0.1 - 2.5).astype(np.float32))
    c.q[:] = synth.f32_to_bf16_bits(np.full(1, 1.0, np.float32))[0]
    c.vp = synth.f32_to_bf16_bits((obf.decode(c.vp) * size).astype(np.float32))
    check_attention(lib, c, f"values of {size}")


@pytest.mark.parametrize("Hq,Hkv,block", [(8, 2, 64), (4, 4, 256), (12, 4, 84)])
@pytest.mark.parametrize("what", ["K nan", "K inf", "V nan", "V inf"])
def test_attention_reach_of_a_non_finite_new_key(lib, Hq, Hkv, block, what):
    """A NaN or infinity in one dim of a new key: in K it is seen by the rows that see the key, in V by them and the
    earlier rows of the block of rows, in this dim of this kv head only.  Everything else is as without it."""
    rows, ctx, at, dim = 3 * block + 5, 100, 2 * block - 3, 21
    c = Case(72, [rows, 9], [ctx, 40], Hq, Hkv)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    pool = c.kp if what[0] == "K" else c.vp
    pool[0, c.table[0, (ctx + at) // PAGE], (ctx + at) % PAGE, dim] = 0x7FC0 if what.endswith("nan") else 0x7F80
    got = f64_of_bf16(run_attention(lib, c)).reshape(ref.shape)
    clean = np.ones(ref.shape, bool)
    heads = slice(0, Hq // Hkv)
    if what[0] == "K":          # (an infinite score may be -inf: no weight, and nothing to see)
        clean[at:rows, heads] = False
        if what == "K nan":
            assert np.all(np.isnan(got[at:rows, heads]))
    else:
        clean[block:rows, heads, dim] = False
        assert not np.any(np.isfinite(got[at:rows, heads, dim]))
    assert_attended(got[clean], ref[clean], mag[clean], what)


@pytest.mark.parametrize("cu,good", [
    ([0, 2, 5, 9], 2), ([0, 2, 1 << 30, 1 << 30], 1), ([0, 5, 5, 6], 1), ([-4, 0, 2, 5], 0), ([0, 5, 3, 3], 1),
    ([0] * 300 + [2, 5, 9], 301)])
@pytest.mark.parametrize("rotate", [True, False])
def test_append_flags_every_sequence_out_of_bounds(lib, cu, good, rotate):
    """Five rows, and sequences that leave them: the status word is set whether or not one of the rows is theirs, the
    sequences before the first bad one get theirs, and a batch in bounds leaves the word alone."""
    B, M = len(cu) - 1, 5
    bits = synth.normal_bf16_bits(73, (M, 4 * D), 1.0)
    kv, ctx = bf16_dev(bits), dev(np.full(B, 7, np.int32))
    table = dev(np.arange(B, dtype=np.int32)[:, None].copy())
    cs = torch.zeros((M, 64, 2), device="cuda")
    cs[..., 0] = 1.0                                        # (a rotation by 0)

    def append(cu):
        kp, vp = (torch.zeros((2, B, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.spec_kv_append_paged(kv[:, :2 * D], kv[:, 2 * D:], dev(np.array(cu, np.int32)), ctx, kp, vp, table,
                                 cs=cs if rotate else None)
        rc, _ = lib.spec_device_status_code()
        lib.spec_device_status()
        return rc, bits_of(kp)

    rc, kp = append(cu)
    assert rc == lib.SPEC_EINVAL
    want = np.zeros_like(kp)
    for b in range(good):
        for j in range(cu[b + 1] - cu[b]):
            want[:, b, 7 + j] = bits[cu[b] + j, :2 * D].reshape(2, D)
    if cu[0] >= 0 and cu == sorted(cu):
        assert np.array_equal(kp, want)
    rc, _ = append([min(max(c, 0), M) for c in sorted(cu)])
    assert rc == lib.SPEC_OK


def test_table_of_the_most_rows(lib):
    """2^31 - 1 rows of a table with one frequency: the last ones (and none behind them) are written."""
    M = 2 ** 31 - 1
    pos = torch.zeros((1, M), dtype=torch.int32, device="cuda")
    pos[0, -100:] = torch.arange(100, dtype=torch.int32, device="cuda")
    buf = torch.full((M + 9, 1, 2), 5.0, device="cuda")
    lib.spec_rope_table_axes(pos, [1], 2, cs=buf[:M])
    lib.spec_device_status()
    ref = oprompt.rope_table_axes(np.arange(100)[None], [1], 2, 1e6, False)
    assert abs(buf[M - 100:M].cpu().numpy() - ref).max() <= table_tol(100)
    assert bool((buf[M:] == 5.0).all()) and bool((buf[:1000, 0, 0] == 1.0).all())
    sample = buf[:M - 100:12345, 0]
    assert bool((sample[:, 0] == 1.0).all()) and bool((sample[:, 1] == 0.0).all())
    del pos, buf, sample
    torch.cuda.empty_cache()


def test_binding_refuses_what_does_not_fit_32_bits(lib):
    """Leading dimensions above 2^31 - 1 are refused, not cut off: cut, the first would be 1024."""
    c = Case(74, [2], [0], 8, 2)
    cu, ctx, kp, vp, table = c.dev()
    far = torch.empty((1 << 32) + 2048, dtype=torch.bfloat16, device="cuda").as_strided((2, 8 * D), ((1 << 32) + 8 * D, 1))
    near = bf16_dev(c.q)
    with pytest.raises(ValueError, match="leading dimension"):
        lib.spec_chunk_attention_paged(far, cu, ctx, kp, vp, table)
    with pytest.raises(ValueError, match="leading dimension"):
        lib.spec_chunk_attention_paged(near, cu, ctx, kp, vp, table, O=far)
    with pytest.raises(ValueError, match="leading dimension"):
        lib.spec_kv_append_paged(far[:, :2 * D], far[:, 2 * D:4 * D], cu, ctx, kp, vp, table)
    with pytest.raises(ValueError, match="leading dimension"):
        lib.spec_verify_linear(far, torch.zeros((128, 8 * D), dtype=torch.bfloat16, device="cuda"))
    del far
    wide = torch.empty((1, 1 << 31), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="leading dimension"):
        lib.spec_rope_table_axes(wide, [1], 2)
    del wide
    torch.cuda.empty_cache()


def test_pools_past_32_bits(lib):
    """Pages whose elements lie past 2^31 of a pool (and past 2^32 bytes): append and attention of a few rows."""
    pages, Hkv, rows = 70000, 2, 150
    kp, vp = (torch.zeros((Hkv, pages, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.array([[69999, 69000], [3, 66001]], np.int32)
    bits = synth.normal_bf16_bits(75, (2 * rows, (4 + 2 * Hkv) * D), 1.0)
    x = bf16_dev(bits)
    q, k, v = x[:, :4 * D], x[:, 4 * D:6 * D], x[:, 6 * D:]
    cu, ctx = dev(np.array([0, rows, 2 * rows], np.int32)), dev(np.zeros(2, np.int32))
    lib.spec_kv_append_paged(k, v, cu, ctx, kp, vp, dev(table))
    O = lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, dev(table))
    lib.spec_device_status()
    dec = obf.decode(bits)
    pool = np.zeros((2, Hkv, 4, PAGE, D))
    small = np.array([[0, 1], [2, 3]])
    kv = [dec[:, a:a + 2 * D].reshape(-1, Hkv, D) for a in (4 * D, 6 * D)]
    kk, vv = oprompt.kv_append(*kv, [0, rows, 2 * rows], [0, 0], *pool, small)
    for got, want in ((kp, kk), (vp, vv)):
        assert np.array_equal(f64_of_bf16(got[:, torch.from_numpy(table.reshape(-1)).long().cuda()]), want)
    ref, mag = oprompt.chunk_attention(dec[:, :4 * D].reshape(-1, 4, D), [0, rows, 2 * rows], [0, 0], kk, vv, small,
                                       1.0 / np.sqrt(D))
    assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, "pages past 32 bits")
    del kp, vp
    torch.cuda.empty_cache()


def test_two_graphs_on_one_workspace(lib):
    """Two captured calls of other shapes on one workspace, replayed in turn on one stream."""
    cases = [Case(76, [3, 40], [9000, 700], 8, 2), Case(77, [300, 1, 0], [0, 5000, 4], 16, 8)]
    ws = lib.Workspace("cuda")
    graphs = []
    for c in cases:
        args = (bf16_dev(c.q), *c.dev())
        O = torch.zeros((c.M, c.Hq * D), dtype=torch.bfloat16, device="cuda")
        lib.spec_chunk_attention_paged(*args, O=O, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.spec_chunk_attention_paged(*args, O=O, ws=ws)
        graphs.append((c, args, O, graph))
    for _ in range(3):
        for _, _, O, graph in graphs:
            O.fill_(4.0)
            graph.replay()
        for c, _, O, _ in graphs:
            ref, mag = c.oracle(1.0 / np.sqrt(D))
            assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, "replayed in turn")
    lib.spec_device_status()
