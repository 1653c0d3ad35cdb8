"""Calls on a stream that is not the current one, with workspaces and outputs that the call makes itself: the
current stream is kept busy, so that whatever was left to it would come too late."""
import numpy as np
import pytest
import torch

from oracle import bf16 as obf, ops as oops

import synth
from gpu_util import assert_close_rel, bf16_dev, f64_of_bf16
from test_gpu_prompt import D, Case, assert_attended

pytestmark = pytest.mark.gpu
BUSY = 200_000_000       # cycles: a tenth of a second


def dirty(nbytes):
    """Leaves a block of 0xff bytes of this size with the allocator, on the current stream."""
    torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("own", ["none", "grown", "made"])
def test_chunk_attention_clears_its_workspace_on_its_stream(lib, own):
    """Keys shared between CTAs (the counters have to start at 0): no workspace given, an empty one that the call grows,
    one of the right size made on the current stream just before."""
    c = Case(80, [3, 40], [9000, 3000], 8, 2)
    cu, ctx, kp, vp, table = c.dev()
    q = bf16_dev(c.q)
    O = torch.zeros((c.M, 8 * D), dtype=torch.bfloat16, device="cuda")
    need = lib.spec_chunk_attention_workspace_bytes(c.B, c.M, 8, 2, D, c.max_pages)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dirty(need)
    dirty(need)
    ref, mag = c.oracle(1.0 / np.sqrt(D))
    torch.cuda._sleep(BUSY)
    ws = {"none": lambda: None, "grown": lambda: lib.Workspace("cuda"), "made": lambda: lib.Workspace("cuda", need)}[own]()
    for _ in range(2):
        lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, O=O, ws=ws, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        got = f64_of_bf16(O)
    lib.spec_device_status(side)
    assert_attended(got.reshape(ref.shape), ref, mag, own)


def test_split_product_clears_its_workspace_on_its_stream(lib):
    """The same for a product of the verify stack with its sums split over CTAs."""
    M, N, K = 5, 1024, 4096
    x, w = synth.normal_bf16_bits(81, (M, K), 1.0), synth.normal_bf16_bits(82, (N, K), 0.02)
    X, W = bf16_dev(x), bf16_dev(w)
    Y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    need = max(lib.spec_linear_workspace_bytes(M, N, K), 1)
    with torch.cuda.stream(side):
        dirty(need)
    dirty(need)
    torch.cuda._sleep(BUSY)
    lib.spec_verify_linear(X, W, Y=Y, ws=lib.Workspace("cuda"), stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        got = f64_of_bf16(Y)
    lib.spec_device_status(side)
    assert_close_rel(got, oops.linear(obf.decode(x), obf.decode(w)), "product on another stream")


def test_workspace_grown_while_calls_run(lib):
    """A workspace that grows between two calls on one stream: the block that the first still uses goes to nobody."""
    a, b = Case(83, [60], [20000], 8, 2), Case(84, [5, 9], [300, 4000], 8, 2)
    args = [(bf16_dev(c.q), *c.dev()) for c in (a, b)]
    need = lib.spec_chunk_attention_workspace_bytes(1, 60, 8, 2, D, a.max_pages)
    side = torch.cuda.Stream()
    ws = lib.Workspace("cuda", need)
    outs = [torch.zeros((c.M, 8 * D), dtype=torch.bfloat16, device="cuda") for c in (a, b)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    q, cu, ctx, kp, vp, table = args[0]
    lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, O=outs[0], ws=ws, stream=side)
    ws.ensure(need + (1 << 20), stream=side)
    torch.full((need,), 255, dtype=torch.uint8, device="cuda")       # (would land in the old block)
    torch.cuda.current_stream().synchronize()
    q, cu, ctx, kp, vp, table = args[1]
    lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, O=outs[1], ws=ws, stream=side)
    torch.cuda.synchronize()
    lib.spec_device_status(side)
    for c, O in zip((a, b), outs):
        ref, mag = c.oracle(1.0 / np.sqrt(D))
        assert_attended(f64_of_bf16(O).reshape(ref.shape), ref, mag, "grown workspace")


@pytest.mark.parametrize("call", ["attention", "product", "table", "sampler"])
def test_outputs_made_for_another_stream(lib, call):
    """The current stream is about to write a block that it has already given back: an output of a call on another stream
    must not lie in it.  And an output given up while that call still runs goes to nobody."""
    side = torch.cuda.Stream()
    if call == "attention":
        c = Case(85, [2000], [0], 8, 2)
        cu, ctx, kp, vp, table = c.dev()
        q, ws = bf16_dev(c.q), lib.Workspace("cuda", lib.spec_chunk_attention_workspace_bytes(1, 2000, 8, 2, D, c.max_pages))
        run = lambda **k: lib.spec_chunk_attention_paged(q, cu, ctx, kp, vp, table, ws=ws, **k)
    elif call == "product":
        x, w = (bf16_dev(synth.normal_bf16_bits(86 + i, (n, 1024), 1.0)) for i, n in enumerate((300, 2048)))
        ws = lib.Workspace("cuda", max(lib.spec_linear_workspace_bytes(300, 2048, 1024), 1))
        run = lambda **k: lib.spec_verify_linear(x, w, ws=ws, **k)
    elif call == "table":
        pos = torch.arange(3 * 5000, dtype=torch.int32, device="cuda").view(3, 5000)
        run = lambda **k: lib.spec_rope_table_axes(pos, [16, 24, 24], 128, **k)
    else:
        P = torch.rand((4000, 512), device="cuda")
        P, U = P / P.sum(dim=1, keepdim=True), torch.rand(4000, device="cuda")
        run = lambda **k: lib.spec_sample_rows(P, U, **k)
    want = run()
    torch.cuda.synchronize()
    nbytes = want.numel() * want.element_size()
    old = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(BUSY)
    old.fill_(255)
    del old
    got = run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # given up at once: a block of the same size, filled on the current stream, stays as it was filled
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    run(stream=side)
    fresh = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    lib.spec_device_status(side)
    assert bool((fresh == 7).all())
